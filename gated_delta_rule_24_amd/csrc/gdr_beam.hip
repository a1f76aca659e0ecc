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
__device__ __forceinline__ unsigned long long order_of(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u ^ ((unsigned long long)((long long)u >> 63) | (1ull << 63));
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
        for (int j = 0; j < n; ++j) before += list[j] > mine;
        if (before < m) best[before] = mine;
    }
    __syncthreads();
}

template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void open(const uint4& u, float* x) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) { x[2 * j] = __uint_as_float(w[j] << 16); x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u); }
    }
    __device__ static __forceinline__ float one(uint16_t v) { return bf16_to_f32(v); }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void open(const uint4& u, float* x) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    __device__ static __forceinline__ float one(float v) { return v; }
};

}  // namespace

// One run of a row's logits: its maximum, its sum of exp2((x - max) log2 e), and its best M.
// The run is read once, 256 x 32 values (bf16; 256 x 16 in fp32) at a time, 16 bytes a load;
// a row may start anywhere (its vectors are those of the tensor's aligned memory).
//
// The best so far give a bound that later values have to pass (strictly: an equal one has
// a higher token).  Few do, so a chunk's own work is the sum; those that pass are
// collected and sorted in.  Where more than kRoom would be collected, the first chunk and
// rising logits, the M-th largest of the threads' own largest values is a second bound:
// at least M values reach it, and at most 32 of each of M threads.
template <typename T>
__global__ __launch_bounds__(kThreads) void beam_rows(BeamParams p, long long per) {
    constexpr int VE = Vec<T>::N, U = 4, E = VE * U;  // values of a vector; vectors and values of a thread's chunk
    __shared__ uint64_t s_list[kList];
    __shared__ uint64_t s_best[kMostSelected];
    __shared__ uint64_t s_top[kThreads];
    __shared__ uint64_t s_bound;
    __shared__ int s_n[2];
    __shared__ float s_ms[2 * kThreads / 64];
    const int tid = threadIdx.x, seg = blockIdx.x, r = blockIdx.y, M = p.M;
    if (p.ended && p.ended[r]) return;                // what it offers does not depend on its logits

    const T* row = (const T*)p.logits + (long long)r * p.stride;
    const int shift = (int)(((uintptr_t)row & 15u) / sizeof(T));     // values before the row in its first vector
    const T* base = row - shift;
    const long long vecs = ((long long)p.V + shift + VE - 1) / VE;
    const long long v0 = seg * per, v1 = v0 + per < vecs ? v0 + per : vecs;

    float m = -INFINITY, sum = 0.f;
    uint64_t bound = 0;                               // the M-th best so far
    if (tid < kMostSelected) s_best[tid] = 0;
    int slot = 0;
    if (tid < 2) s_n[tid] = 0;
    __syncthreads();

    float x[E];
    for (long long c = v0; c < v1; c += U * kThreads) {
        // absent values are -inf in the sum and are no candidates
        uint32_t there = 0;
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long v = c + u * kThreads + tid, t = v * VE - shift;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (v < v1 && t >= 0 && t + VE <= p.V) raw[u] = *reinterpret_cast<const uint4*>(base + v * VE);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long v = c + u * kThreads + tid, t = v * VE - shift;
            if (v < v1 && t >= 0 && t + VE <= p.V) {
                Vec<T>::open(raw[u], x + u * VE);
                there |= ((1u << VE) - 1) << (u * VE);
            } else {
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    x[u * VE + j] = -INFINITY;
                    if (v < v1 && t + j >= 0 && t + j < p.V) {
                        x[u * VE + j] = Vec<T>::one(row[t + j]);
                        there |= 1u << (u * VE + j);
                    }
                }
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < E; ++i) top = fmaxf(top, x[i]);
        if (top > m) {
            sum *= __builtin_amdgcn_exp2f((m - top) * kLog2e);
            m = top;
        }
        const float at = m == -INFINITY ? 0.f : m;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) part[i % 4] += __builtin_amdgcn_exp2f((x[i] - at) * kLog2e);
        sum += (part[0] + part[1]) + (part[2] + part[3]);

        // those that pass the bound
        int* count = &s_n[slot];
        auto token = [&](int i) { return (int)((c + (i / VE) * kThreads + tid) * VE - shift) + i % VE; };
        auto passes = [&](int i, uint64_t b) { return (there >> i & 1) && key_of(x[i], token(i)) > b; };
        if (there && key_of(top, 0) > bound) {        // (token 0 has the largest key of a value)
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (passes(i, bound)) {
                    const int to = atomicAdd(count, 1);
                    if (to < kRoom) s_list[to] = key_of(x[i], token(i));
                }
        }
        __syncthreads();
        int n = *count;
        slot ^= 1;
        if (tid == 0) s_n[slot] = 0;                  // (the next chunk's counter)
        if (n > kRoom) {
            uint64_t mine = 0;
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (passes(i, bound)) { const uint64_t k = key_of(x[i], token(i)); mine = k > mine ? k : mine; }
            s_top[tid] = mine;
            if (tid == 0) s_bound = 1;                // fewer than M threads have one: all count
            __syncthreads();
            int before = 0;
            for (int j = 0; j < kThreads; ++j) before += s_top[j] > mine;
            if (mine && before == M - 1) s_bound = mine;
            if (tid == 0) *count = 0;
            __syncthreads();
            const uint64_t sift = s_bound;
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (passes(i, bound)) {
                    const uint64_t k = key_of(x[i], token(i));
                    if (k >= sift) s_list[atomicAdd(count, 1)] = k;
                }
            __syncthreads();
            n = *count;
        }
        if (n > 0) {
            // beside the best so far
            if (tid < M && s_best[tid]) s_list[n + tid] = s_best[tid];
            int kept = 0;
            for (int j = 0; j < M; ++j) kept += s_best[j] != 0;
            __syncthreads();
            sort_best(s_list, n + kept, s_best, M);
            bound = s_best[M - 1];
        }
        __syncthreads();
    }

    // the workgroup's maximum and sum
    for (int o = 32; o > 0; o >>= 1) {
        const float m2 = __shfl_xor(m, o, 64), s2 = __shfl_xor(sum, o, 64), both = fmaxf(m, m2), at = both == -INFINITY ? 0.f : both;
        sum = sum * __builtin_amdgcn_exp2f((m - at) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - at) * kLog2e);
        m = both;
    }
    if ((tid & 63) == 0) { s_ms[2 * (tid >> 6)] = m; s_ms[2 * (tid >> 6) + 1] = sum; }
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
    if (tid < M) p.best[out * M + tid] = s_best[tid];
}

// One workgroup of a group: its rows' sums joined in 64 bits, then the best M of the runs'
// best by score.  As in the rows: the M-th best of the runs' first ones is a bound that
// leaves few.
namespace {
struct Candidate {
    unsigned long long score;   // ordered; 0: none
    uint64_t key;
    int beam;
};
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b) {
    if (a.score != b.score) return a.score > b.score;
    if (a.beam != b.beam) return a.beam < b.beam;
    return a.key > b.key;
}
}  // namespace

__global__ __launch_bounds__(kThreads) void beam_join(BeamParams p) {
    __shared__ double s_lse[kMostBeams];              // lse; NaN: the row offers nothing but -inf
    __shared__ uint8_t s_ended[kMostBeams];
    extern __shared__ __attribute__((aligned(16))) char smem[];
    Candidate* list = reinterpret_cast<Candidate*>(smem);          // [M * M]: of at most M runs
    __shared__ Candidate s_best[kMostSelected], s_bound;
    __shared__ int s_n, s_slot[kMostSelected];
    const int tid = threadIdx.x, g = blockIdx.x, K = p.K, M = p.M, S = p.segs;
    const double inf = INFINITY;

    for (int k = tid >> 6; k < K; k += kThreads / 64) {            // a wave a row
        const int r = g * K + k, lane = tid & 63;
        const bool over = p.ended && p.ended[r];
        float m = -INFINITY;
        bool bad = false;
        double sum = 0.0;
        if (!over) {
            for (int s = lane; s < S; s += 64) {
                const float2 ms = *reinterpret_cast<const float2*>(p.part + 2 * ((long long)r * S + s));
                bad = bad || !(ms.y < INFINITY);
                m = fmaxf(m, ms.x);
            }
            for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
            for (int s = lane; s < S; s += 64) {
                const float2 ms = *reinterpret_cast<const float2*>(p.part + 2 * ((long long)r * S + s));
                if (ms.x > -INFINITY) sum += (double)ms.y * exp((double)ms.x - (double)m);
            }
            for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
            bad = __any(bad) || !(m > -INFINITY) || !(m < INFINITY);
        }
        const float base = p.scores[r];
        if (!(base - base == 0.f)) bad = true;
        if (lane == 0) {
            s_lse[k] = bad ? NAN : over ? 0.0 : (double)m + log(sum);
            s_ended[k] = over;
        }
    }
    if (tid == 0) s_n = 0;
    __syncthreads();

    // candidate j of run s of beam k, if there is one
    auto candidate = [&](int k, int s, int j, Candidate& c) {
        const int r = g * K + k;
        const double lse = s_lse[k];
        c.beam = k;
        if (lse != lse || s_ended[k]) {
            // (an ended beam's end token, then) the first tokens, all at -inf
            int t = j;
            bool first = false;
            if (lse == lse) {
                first = j == 0;
                t = first ? p.end_token : j - 1 + (j - 1 >= p.end_token ? 1 : 0);
            }
            c.score = order_of(first ? (double)p.scores[r] : -inf);
            c.key = (first ? 1ull << 32 : 0ull) | (0xffffffffu - (uint32_t)t);
            return s == 0 && t < p.V;
        }
        c.key = p.best[((long long)r * S + s) * M + j];
        c.score = order_of((double)p.scores[r] + (double)value_of((uint32_t)(c.key >> 32)) - lse);
        return c.key != 0;
    };
    // bound: the M-th best of the runs' first candidates
    const int runs = K * S;
    if (tid == 0) s_bound = Candidate{0, 0, INT_MAX};
    __syncthreads();
    if (runs > M)
        for (int i = tid; i < runs; i += kThreads) {
            Candidate mine, c;
            if (!candidate(i / S, i % S, 0, mine)) continue;
            int before = 0;
            for (int j = 0; j < runs && before < M; ++j)
                if (candidate(j / S, j % S, 0, c) && better(c, mine)) ++before;
            if (before == M - 1) s_bound = mine;
        }
    __syncthreads();
    const Candidate bound = s_bound;
    for (int i = tid; i < runs; i += kThreads)
        for (int j = 0; j < M; ++j) {
            Candidate c;
            if (!candidate(i / S, i % S, j, c) || better(bound, c)) break;    // (a run is in order)
            list[atomicAdd(&s_n, 1)] = c;
        }
    __syncthreads();
    const int n = s_n;
    for (int i = tid; i < n; i += kThreads) {
        const Candidate mine = list[i];
        int before = 0;
        for (int j = 0; j < n && before < M; ++j) before += better(list[j], mine);
        if (before < M) s_best[before] = mine;
    }
    __syncthreads();

    // where each goes: in order, or the first continuation of a beam in the beam's own row
    // and the others in the rows left, both in order
    if (tid < M) {
        int slot = tid;
        if (p.flags & GDR_KEEP_SLOTS) {
            const int beam = s_best[tid].beam;
            bool first = true;
            int others = 0;                           // later continuations before this one
            for (int i = 0; i < tid; ++i) {
                bool f = true;
                for (int j = 0; j < i; ++j) f = f && s_best[j].beam != s_best[i].beam;
                others += !f;
                first = first && s_best[i].beam != beam;
            }
            slot = beam;
            if (!first)
                for (slot = 0; slot < K; ++slot) {
                    bool taken = false;
                    for (int i = 0; i < M; ++i) taken = taken || s_best[i].beam == slot;
                    if (!taken && others-- == 0) break;
                }
        }
        s_slot[tid] = slot;
    }
    __syncthreads();
    if (tid < M) {
        const Candidate c = s_best[tid];
        const long long at = (long long)g * M + s_slot[tid];
        const int r = g * K + c.beam, t = token_of(c.key);
        const double lse = s_lse[c.beam];
        float score = -INFINITY;
        if (lse == lse) {
            if (s_ended[c.beam]) score = c.key >> 32 ? p.scores[r] : -INFINITY;
            else score = (float)((double)p.scores[r] + (double)value_of((uint32_t)(c.key >> 32)) - lse);
        }
        p.tokens[at] = t;
        p.rows[at] = r;
        p.scores_out[at] = score;
        p.ended_out[at] = s_ended[c.beam] || t == p.end_token;
    }
}

int beam_segments(int G, int K, int V) {
    // Enough workgroups for every compute unit where there are few rows; a run of 2,048
    // values at the least.
    const long long rows = (long long)G * K;
    long long s = (1024 + rows - 1) / rows;
    const long long most = ((long long)V + 2047) / 2048;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

hipError_t launch_beam_select(const BeamParams& p, hipStream_t st) {
    const bool wide = (p.flags & GDR_ACT_F32) != 0;
    const int VE = wide ? 4 : 8;
    // vectors of a run: a row's, and one more where it does not start at one
    long long per = ((p.V + VE - 1) / VE + 1 + p.segs - 1) / p.segs;
    const dim3 grid((unsigned)p.segs, (unsigned)(p.G * p.K)), block(kThreads);
    if (wide) hipLaunchKernelGGL(beam_rows<float>, grid, block, 0, st, p, per);
    else hipLaunchKernelGGL(beam_rows<uint16_t>, grid, block, 0, st, p, per);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    static std::atomic<unsigned long long> done{0};
    e = ensure_dyn_lds(reinterpret_cast<const void*>(&beam_join), kMostSelected * kMostSelected * (int)sizeof(Candidate), done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(beam_join, dim3((unsigned)p.G), block, (unsigned)(p.M * p.M * sizeof(Candidate)), st, p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// states
// ---------------------------------------------------------------------------
//
// In place: a thread holds 16 bytes of every row of its group, so that a row may be
// another's source and itself be replaced.  Rows that keep their own state cost nothing,
// which is most of them where the beams that live on stay in their rows.
namespace {
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
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
