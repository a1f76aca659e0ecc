// Beam search: the best continuations of each group of beams over the
// vocabulary, and the recurrent states moved to the rows that continue them.
//
//   lse_r = log sum_t exp x_rt,  score(k, t) = s_k + x_kt - lse_k
//
// An ended beam offers one candidate, the end token, at its own score; every other
// candidate of it has -inf.  So has every candidate of a row without a finite lse (all
// masked, a NaN, +inf) or of a beam whose score is not finite.  The best M of a group
// in the order (score descending, beam, logit descending, token).
#include "gdr_device.h"
#include "gdr_generation.h"
#include "gdr_launch.h"

namespace gdr {

namespace {

typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRoom = 1024;                           // candidates that a chunk may add before it is sifted first
constexpr int kList = kMostSelected * 32 + kMostSelected;  // what sifting can leave, and the best so far

// Whole numbers that order as the values do (+0 and -0 alike, as x + 0 makes them).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t order_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | ((uint64_t)1 << 63));
}
// A candidate of a row: larger is better, no two alike, none is 0.
__device__ __forceinline__ uint64_t key_of(float x, int t) { return ((uint64_t)order_of(x) << 32) | (0xffffffffu - (uint32_t)t); }
__device__ __forceinline__ int token_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

// The workgroup's keys list[0 .. n - 1] (no two alike): the best `m` of them to best[],
// in order; 0 behind the last.
__device__ __forceinline__ void sort_best(const uint64_t* list, int n, uint64_t* best, int m) {
    for (int i = threadIdx.x; i < m; i += kThreads) best[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t mine = list[i];
        int before = 0;
        for (int j0 = 0; j0 < n; j0 += 8) {           // eight reads at a time
            uint64_t other[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) other[u] = list[min(j0 + u, n - 1)];
#pragma unroll
            for (int u = 0; u < 8; ++u) before += (int)(j0 + u < n) & (int)(other[u] > mine);
        }
        if (before < m) best[before] = mine;
    }
    __syncthreads();
}

// The values that four words hold, and the word of two bf16 values (one fp32 value) of a
// tensor, absent ones as -inf.
template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    static constexpr int N = 8;
    __device__ static __forceinline__ float value(uint4v u, int i) {
        return __uint_as_float(i % 2 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    }
    __device__ static __forceinline__ void put(uint4v& u, int i, bool there, const uint16_t* at) {
        const uint32_t v = there ? *at : 0xff80u;
        u[i / 2] = i % 2 ? (u[i / 2] & 0xffffu) | v << 16 : (u[i / 2] & 0xffff0000u) | v;
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ float value(uint4v u, int i) { return __uint_as_float(u[i]); }
    __device__ static __forceinline__ void put(uint4v& u, int i, bool there, const float* at) {
        u[i] = there ? __float_as_uint(*at) : 0xff800000u;
    }
};

}  // namespace

// One run of a row's logits: its maximum, its sum of exp2((x - max) log2 e), and its best M.
// The run is read once, 256 x 32 values (bf16; 256 x 16 in fp32) at a time, 16 bytes a load,
// a chunk ahead of the work on it; a row may start anywhere (its vectors are those of the
// tensor's aligned memory).
//
// A bound, some M values of the run that are at least as large, keeps the candidates few:
// first the M-th of the largest values of 64 runs of the first chunk, later the M-th best so
// far, which is made anew when enough candidates have been collected.  A value that
// equals the bound from a later chunk has a higher token and does not pass.  Where more
// values pass than there is room for (rising logits, many equal ones) the chunk is
// sifted by the threads' own largest keys: M values reach the M-th of them, and at most 32
// of each of M threads.
//
// 64 x 8 beams over 131,072 bf16 values: 44 us, 2.9 TB/s, vector instructions 65% of the cycles (an
// exponential and five more a value; those of the values that pass, and of their neighbours, as many
// again); the rest are the runs' starts and ends.
constexpr int kEnough = 256;                          // collected candidates that are worth a new bound

template <typename T>
__global__ __launch_bounds__(kThreads, 4) void beam_rows(BeamParams p, int per) {
    constexpr int VE = Vec<T>::N, U = 4, E = VE * U;  // values of a vector; vectors and values of a thread's chunk
    __shared__ uint64_t s_list[kList];
    __shared__ uint64_t s_best[kMostSelected];
    __shared__ uint64_t s_top[kThreads];
    __shared__ uint32_t s_run[64];                    // largest values of runs of four threads
    __shared__ uint64_t s_bound;
    __shared__ int s_n;
    __shared__ float s_ms[2 * kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, seg = blockIdx.x, r = blockIdx.y, M = p.M;
    if (p.ended && p.ended[r]) return;                // what it offers does not depend on its logits

    const T* row = (const T*)p.logits + (long long)r * p.stride;
    const int shift = (int)(((uintptr_t)row & 15u) / sizeof(T));     // values before the row in its first vector
    const uint4v* base = reinterpret_cast<const uint4v*>(row - shift);
    const int vecs = (p.V + shift + VE - 1) / VE;
    const int v0 = min(seg * per, vecs), v1 = min(v0 + per, vecs);

    float m = -INFINITY, sum = 0.f;
    uint64_t bound = 0;                               // keys have to be larger
    int kept = 0, listed = 0;                         // in s_best, in s_list
    if (tid == 0) s_n = 0;

    // vectors v of the run, whose values are all the row's; the others are read value by
    // value, -inf where there is none
    auto whole = [&](int v) { return v < v1 && v * VE >= shift && v * VE - shift + VE <= p.V; };
    auto partly = [&](int v) {
        const int t = v * VE - shift;
        uint4v w;
#pragma unroll
        for (int j = 0; j < VE; ++j) Vec<T>::put(w, j, v < v1 && t + j >= 0 && t + j < p.V, row + t + j);
        return w;
    };
    constexpr int kChunk = U * kThreads;
    auto inside = [&](int c) { return c + kChunk <= v1 && c * VE >= shift && (c + kChunk) * VE - shift <= p.V; };
    uint4v cur[U], ahead[U];
    auto load = [&](int c) {
        if (inside(c)) {
#pragma unroll
            for (int u = 0; u < U; ++u) ahead[u] = base[c + u * kThreads + tid];
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ahead[u] = uint4v{0, 0, 0, 0};
                if (whole(c + u * kThreads + tid)) ahead[u] = base[c + u * kThreads + tid];
            }
        }
    };
    // f(key) of each of this thread's values of chunk c, read again (few chunks need it)
    auto each_key = [&](int c, auto f) {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            const int v = c + u * kThreads + tid;
            const uint4v w = whole(v) ? base[v] : partly(v);
            const int t = v * VE - shift;
#pragma unroll 1
            for (int j = 0; j < VE; ++j) {
                float y = Vec<T>::value(w, 0);
#pragma unroll
                for (int i = 1; i < VE; ++i) y = j == i ? Vec<T>::value(w, i) : y;
                if (v < v1 && t + j >= 0 && t + j < p.V) f(key_of(y, t + j));
            }
        }
    };
    // the best of list and s_best to s_best
    auto merge = [&](int n) {
        if (tid < kept) s_list[n + tid] = s_best[tid];
        __syncthreads();
        sort_best(s_list, n + kept, s_best, M);
        kept = min(n + kept, M);
        if (kept == M) bound = s_best[M - 1];
    };

    auto value = [&](int i) { return Vec<T>::value(cur[i / VE], i % VE); };
    if (v0 < v1) load(v0);
    for (int c = v0; c < v1; c += kChunk) {
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = ahead[u];
        if (!inside(c)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (!whole(c + u * kThreads + tid)) cur[u] = partly(c + u * kThreads + tid);
        }
        if (c + kChunk < v1) load(c + kChunk);
        float tops[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tops[u] = value(u * VE);
#pragma unroll
            for (int j = 1; j < VE; ++j) tops[u] = fmaxf(tops[u], value(u * VE + j));
        }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        if (top > m) {
            sum *= __builtin_amdgcn_exp2f((m - top) * kLog2e);
            m = top;
        }
        const float at = m == -INFINITY ? 0.f : m;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) part[i % 4] += __builtin_amdgcn_exp2f((value(i) - at) * kLog2e);
        sum += (part[0] + part[1]) + (part[2] + part[3]);

        // the M-th largest of 64 runs' largest values, as the smallest key of that value less one
        auto of_runs = [&]() {
            const uint32_t mine = order_of(top);      // (a thread without values has the least: -inf's)
            uint32_t both = max(mine, (uint32_t)__shfl_xor((int)mine, 1, 64));
            both = max(both, (uint32_t)__shfl_xor((int)both, 2, 64));
            if ((tid & 3) == 0) s_run[tid >> 2] = both;
            __syncthreads();
            const uint32_t run = s_run[lane];
            int before = 0;
            for (int j = 0; j < 64; ++j) {
                const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)run, j);
                before += other > run || (other == run && j < lane);
            }
            const uint64_t which = __ballot(before == M - 1);
            const uint32_t least = (uint32_t)__builtin_amdgcn_readlane((int)run, __builtin_ctzll(which));
            return (uint64_t)least << 32;
        };
        if (c == v0) bound = of_runs();
        // (as floats, one comparison a value: few waves have none that passes, and most of their
        // values do not; keys are made of those that do)
        const float least = value_of((uint32_t)(bound >> 32));
        if (!(top < least)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (!(tops[u] < least)) {
                    const int v = c + u * kThreads + tid, t = v < v1 ? v * VE - shift : p.V;
#pragma unroll
                    for (int j = 0; j < VE; ++j) {
                        float y = value(u * VE + j);
                        if (y < least) continue;
                        asm volatile("" : "+v"(y));   // (keys made where they are needed, not 32 of them ahead)
                        const uint64_t k = key_of(y, t + j);
                        if (k > bound && (unsigned)(t + j) < (unsigned)p.V) {
                            const int to = atomicAdd(&s_n, 1);
                            if (to < kRoom) s_list[to] = k;
                        }
                    }
                }
        }
        lds_barrier();
        int n = s_n;
        if (n > kRoom) {
            // what was listed goes into the best first; then those of the chunk that also
            // reach the M-th of the threads' largest keys
            if (c == v0) bound = 0;
            __syncthreads();
            if (listed > 0) merge(listed);
            listed = 0;
            uint64_t mine = 0;
            each_key(c, [&](uint64_t k) { if (k > bound && k > mine) mine = k; });
            s_top[tid] = mine;
            if (tid == 0) { s_bound = 1; s_n = 0; }   // (fewer than M threads have one: all count)
            __syncthreads();
            int before = 0;
            for (int j = 0; j < kThreads; ++j) before += s_top[j] > mine;
            if (mine && before == M - 1) s_bound = mine;
            __syncthreads();
            const uint64_t sift = s_bound;
            each_key(c, [&](uint64_t k) { if (k > bound && k >= sift) s_list[atomicAdd(&s_n, 1)] = k; });
            __syncthreads();
            n = s_n;
            if (sift - 1 > bound) bound = sift - 1;
        }
        listed = n;
        if (listed > kEnough) {
            merge(listed);
            listed = 0;
            if (tid == 0) s_n = 0;
        }
        lds_barrier();                                // s_n is read, and set, before the next chunk counts on
    }
    if (listed > 0) merge(listed);

    // the workgroup's maximum and sum
    for (int o = 32; o > 0; o >>= 1) {
        const float m2 = __shfl_xor(m, o, 64), s2 = __shfl_xor(sum, o, 64), both = fmaxf(m, m2), at = both == -INFINITY ? 0.f : both;
        sum = sum * __builtin_amdgcn_exp2f((m - at) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - at) * kLog2e);
        m = both;
    }
    if (lane == 0) { s_ms[2 * (tid >> 6)] = m; s_ms[2 * (tid >> 6) + 1] = sum; }
    __syncthreads();
    const long long out = (long long)r * p.segs + seg;
    if (tid == 0) {
        float all = -INFINITY, s = 0.f;
        for (int w = 0; w < kThreads / 64; ++w) all = fmaxf(all, s_ms[2 * w]);
        const float at = all == -INFINITY ? 0.f : all;
        for (int w = 0; w < kThreads / 64; ++w) s += s_ms[2 * w + 1] * __builtin_amdgcn_exp2f((s_ms[2 * w] - at) * kLog2e);
        p.part[2 * out] = all;
        p.part[2 * out + 1] = s;
    }
    if (tid < M) p.best[out * M + tid] = tid < kept ? s_best[tid] : 0;
}

// One workgroup of a group: its rows' sums joined in 64 bits, then the best M of the runs'
// best by score.  As in the rows: the M-th best of the runs' first ones is a bound, which
// few others reach.  All it reads comes by two loads, one after the other (27 us with the
// candidates read one by one, for 64 groups of 8 beams; so 8.9).
namespace {
// Candidates in LDS: the score, ordered (0: none), and what decides between equal ones: the
// lower beam, the higher logit, the lower token, as one number.
struct Candidates {
    uint64_t* score;
    uint64_t* tie;
};
__device__ __forceinline__ uint64_t tie_of(int beam, uint64_t key) {
    return ((uint64_t)(kMostBeams - 1 - beam) << 58) | (key >> 32 << 26) | (kMostTokens - 1 - (uint32_t)token_of(key));
}
__device__ __forceinline__ int beam_of(uint64_t tie) { return kMostBeams - 1 - (int)(tie >> 58); }
// Candidates of a list of n that come before number i of it.
__device__ __forceinline__ int before_in(const Candidates& c, int n, int i) {
    const uint64_t score = c.score[i];
    const uint64_t tie = c.tie[i];
    int before = 0;
    for (int j0 = 0; j0 < n; j0 += 8) {               // eight reads at a time, none in a branch
        uint64_t s[8];
        uint64_t t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) { s[u] = c.score[min(j0 + u, n - 1)]; t[u] = c.tie[min(j0 + u, n - 1)]; }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            before += (int)(j0 + u < n) & ((int)(s[u] > score) | ((int)(s[u] == score) & (int)(t[u] > tie)));
    }
    return before;
}
constexpr int kMostRuns = 128;                        // of a group (beam_segments)
constexpr int kCandidate = 8 + 8;
__device__ __forceinline__ Candidates candidates_at(char* at, int n) {
    Candidates c;
    c.score = reinterpret_cast<uint64_t*>(at);
    c.tie = reinterpret_cast<uint64_t*>(at + 8 * n);
    return c;
}
inline unsigned join_lds(int M, int runs) { return (unsigned)((2 * M * M + runs) * kCandidate + 4 * M); }
}  // namespace

__global__ __launch_bounds__(kThreads) void beam_join(BeamParams p) {
    __shared__ double s_lse[kMostBeams];              // lse; NaN: the row offers nothing but -inf
    __shared__ float s_score[kMostBeams];
    __shared__ uint8_t s_ended[kMostBeams];
    __shared__ int s_n;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, g = blockIdx.x, K = p.K, M = p.M, S = p.segs, runs = K * S;
    // of at most M runs, M each; and the same again
    const Candidates list = candidates_at(smem, M * M), other = candidates_at(smem + M * M * kCandidate, M * M);
    char* behind = smem + 2 * M * M * kCandidate;
    const Candidates first = candidates_at(behind, runs);                // the runs' first ones
    float2* sums = reinterpret_cast<float2*>(behind);                    // [runs] before that: maxima and sums
    int* passed = reinterpret_cast<int*>(behind + runs * kCandidate);      // [M] the runs that reach the bound
    const double inf = INFINITY;

    // the runs' sums and first keys, the beams' scores
    static_assert(kMostRuns <= kThreads, "a run a thread");
    uint64_t first_key = 0;
    {
        const float base = tid < K ? p.scores[g * K + tid] : 0.f;
        const bool over = tid < K && p.ended && p.ended[g * K + tid];
        if (tid < runs) {
            const float2 ms = *reinterpret_cast<const float2*>(p.part + 2 * ((long long)g * runs + tid));
            first_key = p.best[((long long)g * runs + tid) * M];
            sums[tid] = ms;
        }
        if (tid < K) { s_score[tid] = base; s_ended[tid] = over; }
        if (tid == 0) s_n = 0;
    }
    __syncthreads();
    for (int k0 = 0; k0 < K; k0 += kThreads / 16) {                // 16 lanes a row
        const int k = k0 + (tid >> 4), part = tid & 15;
        const bool live = k < K;
        float m = -INFINITY;
        bool bad = live && !(s_score[k] - s_score[k] == 0.f);
        double sum = 0.0;
        const bool over = !live || s_ended[k];
        if (!over)
            for (int s = part; s < S; s += 16) {
                bad = bad || !(sums[k * S + s].y < INFINITY);
                m = fmaxf(m, sums[k * S + s].x);
            }
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        if (!over)
            for (int s = part; s < S; s += 16)
                if (sums[k * S + s].x > -INFINITY) sum += (double)sums[k * S + s].y * exp((double)sums[k * S + s].x - (double)m);
        for (int o = 8; o > 0; o >>= 1) {
            sum += __shfl_xor(sum, o, 64);
            bad = bad | (__shfl_xor((int)bad, o, 64) != 0);
        }
        if (!over) bad = bad || !(m > -INFINITY) || !(m < INFINITY);
        if (live && part == 0) s_lse[k] = bad ? NAN : over ? 0.0 : (double)m + log(sum);
    }
    __syncthreads();

    // candidate j of run s of beam k, whose key is read already: its score (0: there is
    // none) and key
    auto candidate = [&](int k, int s, int j, uint64_t& key) {
        const double lse = s_lse[k];
        if (lse != lse || s_ended[k]) {
            // (an ended beam's end token, then) the first tokens, all at -inf
            int t = j;
            bool at_score = false;
            if (lse == lse) {
                at_score = j == 0;
                t = at_score ? p.end_token : j - 1 + (j - 1 >= p.end_token ? 1 : 0);
            }
            key = (at_score ? 1ull << 32 : 0ull) | (0xffffffffu - (uint32_t)t);
            return s == 0 && t < p.V ? order_of(at_score ? (double)s_score[k] : -inf) : (uint64_t)0;
        }
        return key != 0 ? order_of((double)s_score[k] + (double)value_of((uint32_t)(key >> 32)) - lse) : (uint64_t)0;
    };
    // the runs whose first candidate is among the best M of all first ones
    int lists = runs;
    if (runs > M) {
        if (tid < runs) {
            first.score[tid] = candidate(tid / S, tid % S, 0, first_key);
            first.tie[tid] = tie_of(tid / S, first_key);
        }
        __syncthreads();
        if (tid < runs && first.score[tid] && before_in(first, runs, tid) < M) passed[atomicAdd(&s_n, 1)] = tid;
        __syncthreads();
        lists = s_n;
    }
    for (int i = tid; i < lists * M; i += kThreads) {
        const int run = runs > M ? passed[i / M] : i / M, j = i % M;
        uint64_t key = p.best[((long long)g * runs + run) * M + j];
        const uint64_t score = candidate(run / S, run % S, j, key);
        list.score[i] = score;
        list.tie[i] = score ? tie_of(run / S, key) : 0;
    }
    __syncthreads();
    // the lists, each in order, merged two by two: a candidate's place is its own and the
    // number of the other list's that are better, found by halving
    uint64_t* from_score = list.score;
    uint64_t* from_tie = list.tie;
    uint64_t* to_score = other.score;
    uint64_t* to_tie = other.tie;
    int left = lists;
    for (; left > 1; left = (left + 1) / 2) {
        for (int i = tid; i < left * M; i += kThreads) {
            const int l = i / M, j = i % M, o = l ^ 1;
            const uint64_t score = from_score[i];
            const uint64_t tie = from_tie[i];
            int z = 0;
            if (o < left) {
                int end = M;                          // better ones of list o: 0 .. z - 1
                while (z < end) {
                    const int mid = (z + end) / 2;
                    const uint64_t s = from_score[o * M + mid];
                    if (s > score || (s == score && from_tie[o * M + mid] > tie)) z = mid + 1;
                    else end = mid;
                }
            }
            // (what is no candidate has score 0 and stands last, in either list: once)
            if (j + z < M && (score || o >= left || l < o)) {
                to_score[(l / 2) * M + j + z] = score;
                to_tie[(l / 2) * M + j + z] = tie;
            }
        }
        __syncthreads();
        uint64_t* x = from_score; from_score = to_score; to_score = x;
        x = from_tie; from_tie = to_tie; to_tie = x;
    }
    if (tid >= 64) return;

    // where each goes: in order, or the first continuation of a beam in the beam's own row
    // and the others in the rows left, both in order (one wave, a lane each)
    const uint64_t one = from_tie[min(lane, M - 1)];
    const int beam = beam_of(one);
    int slot = lane;
    if (p.flags & GDR_KEEP_SLOTS) {
        uint64_t taken = 0, again = 0;
        for (int i = 0; i < M; ++i) {
            const uint64_t bit = 1ull << __builtin_amdgcn_readlane(beam, i);
            if (taken & bit) again |= 1ull << i;
            taken |= bit;
        }
        slot = beam;
        if (again >> lane & 1) {
            uint64_t left = ~taken;
            for (int i = __popcll(again & ((1ull << lane) - 1)); i > 0; --i) left &= left - 1;
            slot = __builtin_ctzll(left);
        }
    }
    if (lane < M) {
        const long long at = (long long)g * M + slot;
        const int t = (int)(kMostTokens - 1 - ((uint32_t)one & (kMostTokens - 1)));
        const uint32_t value = (uint32_t)(one >> 26);            // the logit, ordered; an ended beam's: 1 for its end token
        const double lse = s_lse[beam];
        float score = -INFINITY;
        if (lse == lse) {
            if (s_ended[beam]) score = value ? s_score[beam] : -INFINITY;
            else score = (float)((double)s_score[beam] + (double)value_of(value) - lse);
        }
        p.tokens[at] = t;
        p.rows[at] = g * K + beam;
        p.scores_out[at] = score;
        p.ended_out[at] = s_ended[beam] || t == p.end_token;
    }
}

int beam_segments(int G, int K, int V) {
    // Enough workgroups for every compute unit where there are few rows (twice as many and half
    // as many take 64 x 8 beams over 131,072 tokens from 53.7 us a call to 58 and 70.5); a run of
    // 8,192 values at the least, a bf16 chunk (4 beams over 131,072: 19.0; of 2,048, 20.8, and 28 with
    // up to 256 runs); and no more runs of a group than the join has soon ranked (4 beams over
    // 2,000,000: 36.2; of up to 256 runs 34.9, but one row there 28.6 for 21.3; of up to 64, 46.8 and 19.8).
    const long long rows = (long long)G * K;
    long long s = (1024 + rows - 1) / rows;
    const long long most = ((long long)V + 8191) / 8192;
    if (s > most) s = most;
    if (s > kMostRuns / K) s = kMostRuns / K;
    return s < 1 ? 1 : (int)s;
}

hipError_t launch_beam_select(const BeamParams& p, hipStream_t st) {
    const bool wide = (p.flags & GDR_ACT_F32) != 0;
    const int VE = wide ? 4 : 8;
    // vectors of a run: a row's, and one more where it does not start at one
    const int per = ((p.V + VE - 1) / VE + 1 + p.segs - 1) / p.segs;
    const dim3 grid((unsigned)p.segs, (unsigned)(p.G * p.K)), block(kThreads);
    if (wide) hipLaunchKernelGGL(beam_rows<float>, grid, block, 0, st, p, per);
    else hipLaunchKernelGGL(beam_rows<uint16_t>, grid, block, 0, st, p, per);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    static std::atomic<unsigned long long> done{0};
    e = ensure_dyn_lds(reinterpret_cast<const void*>(&beam_join), (int)join_lds(kMostSelected, kMostRuns), done);
    if (e != hipSuccess) return e;
    const unsigned lds = join_lds(p.M, p.K * p.segs);
    hipLaunchKernelGGL(beam_join, dim3((unsigned)p.G), block, lds, st, p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// states
// ---------------------------------------------------------------------------
//
// In place: a thread holds 16 bytes of every row of its group (8 of more than 32, for the
// registers), so that a row may be another's source and itself be replaced.  Rows that keep their own state cost nothing,
// which is most of them where the beams that live on stay in their rows.  HBM bounds it: 64 groups
// of 4 rows of 2 MiB, 40% of them replaced, 76 us, 5.2 TB/s (85 with branches in the loads).
namespace {
template <int KT, typename V>
__global__ __launch_bounds__(kThreads) void reorder_kernel(ReorderParams p, int blocks, int groups) {
    long long b = blockIdx.x;
    const long long column = (b % blocks) * kThreads + threadIdx.x;
    b /= blocks;
    const int g = (int)(b % groups), layer = (int)(b / groups);
    if (column * (long long)sizeof(V) >= p.row_bytes) return;
    uint8_t* at = p.state + ((long long)layer * p.N + (long long)g * p.K) * p.row_bytes + column * sizeof(V);
    const int* parent = p.parent + (long long)g * p.K;
    // a row that stays is read as one that moves, whose bytes are at hand: loads without
    // a branch, all in flight together
    int moved = -1;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        const int from = k < p.K ? parent[k] - g * p.K : k;
        if (from != k && (unsigned)from < (unsigned)p.K) moved = from;
    }
    if (moved < 0) return;
    V x[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        const int from = k < p.K ? parent[k] - g * p.K : k;
        x[k] = *reinterpret_cast<const V*>(at + (from != k && (unsigned)from < (unsigned)p.K ? from : moved) * p.row_bytes);
    }
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        const int from = k < p.K ? parent[k] - g * p.K : k;
        if (from != k && (unsigned)from < (unsigned)p.K) *reinterpret_cast<V*>(at + k * p.row_bytes) = x[k];
    }
}
int reorder_blocks(int K, long long row_bytes) {
    const long long per = (long long)kThreads * (K > 32 ? 8 : 16);
    return (int)((row_bytes + per - 1) / per);
}
}  // namespace

long long state_reorder_workgroups(int layers, int N, int K, long long row_bytes) {
    const long long per = (long long)kThreads * (K > 32 ? 8 : 16), blocks = (row_bytes + per - 1) / per;
    return blocks > (1LL << 31) ? 1LL << 31 : blocks * layers * (N / K);
}

hipError_t launch_state_reorder(const ReorderParams& p, hipStream_t st) {
    const int blocks = reorder_blocks(p.K, p.row_bytes), groups = p.N / p.K;
    const dim3 grid((unsigned)state_reorder_workgroups(p.layers, p.N, p.K, p.row_bytes)), block(kThreads);
    if (p.K <= 4) hipLaunchKernelGGL((reorder_kernel<4, uint4v>), grid, block, 0, st, p, blocks, groups);
    else if (p.K <= 8) hipLaunchKernelGGL((reorder_kernel<8, uint4v>), grid, block, 0, st, p, blocks, groups);
    else if (p.K <= 16) hipLaunchKernelGGL((reorder_kernel<16, uint4v>), grid, block, 0, st, p, blocks, groups);
    else if (p.K <= 32) hipLaunchKernelGGL((reorder_kernel<32, uint4v>), grid, block, 0, st, p, blocks, groups);
    else hipLaunchKernelGGL((reorder_kernel<64, uint2v>), grid, block, 0, st, p, blocks, groups);
    return hipGetLastError();
}

}  // namespace gdr
