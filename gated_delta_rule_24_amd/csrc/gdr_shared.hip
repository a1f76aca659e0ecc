// Attention of one query token per sequence over the paged 8-bit cache, where groups
// of sequences share their first pages (samples and beams of one prompt, a common
// system prompt).
//
//   o = sum_j p_j v_j / sum_j p_j, p_j = exp2(s_j - m), s_j = scale log2(e) q.k_j
//
// over the last `window` of a sequence's cached tokens (all: window 0).  A softmax over
// the shared pages and one over a sequence's own join as partial results do: each keeps
// its maximum m, its sum of exp2(s - m) and its unnormalised output.  So the
// shared pages are read once for the rows (a sequence's query heads on a key head) of
// the whole group, as further columns of the products that one sequence's heads
// already share in gdr_attn_decode.
#include <type_traits>

#include "gdr_device.h"
#include "gdr_attn.h"
#include "gdr_attn_tile.h"
#include "gdr_generation.h"
#include "gdr_kv_tile.h"
#include "gdr_launch.h"

namespace gdr {

namespace {

constexpr int kPage = 64;
constexpr int kWaves = 4;

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// first and one past the last cached token that a sequence's query sees
__device__ __forceinline__ void seen_range(const SharedParams& p, int n, int& lo, int& hi) {
    const long long room = (long long)p.max_pages * kPage;
    const int len = p.cache_len[n];
    hi = len < 0 ? 0 : (int)(len > room ? room : len);
    lo = (p.window > 0 && len > p.window) ? min(len - p.window, hi) : 0;
}

// What the plan makes of group g (see attn_shared_plan_kernel).
struct Group {
    int first, rows;            // its first sequence; rows: its (sequence, query head) pairs on a key head
    int pg0, pg1;               // the shared pages that some row of it sees
    int tiles;                  // workgroups that its rows take
    int slots;                  // runs of pages; 0: nothing shared
    int base;                   // its first item: item base + (slot * Hkv + kh) * tiles + tile
    int shared;                 // pages that it shares, seen or not
};
static_assert(sizeof(Group) == 32, "read as two 16-byte loads");

// Which group sequence n is in, or -1; and the one that is read as.
__device__ __forceinline__ Group group_of(const SharedParams& p, int g) {
    const int4* at = reinterpret_cast<const int4*>(p.plan_groups) + 2 * (size_t)g;
    const int4 x = at[0], y = at[1];
    return Group{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

__device__ __forceinline__ void store_out(const SharedParams& p, size_t idx, float x) {
    if (p.flags & GDR_OUT_BF16) reinterpret_cast<uint16_t*>(p.o)[idx] = f32_to_bf16(x);
    else reinterpret_cast<float*>(p.o)[idx] = x;
}

// e4m3 bytes that are NaN (0x7f, 0xff), as 0x80 in their places
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }


// Which run of the pages pg0 .. pg1 - 1 is number i of `splits`: a page for each of
// the waves that take them in turn, at least.
__device__ __forceinline__ void run_of(int& pg0, int& pg1, int i, int splits) {
    if (pg1 <= pg0) { pg1 = pg0; return; }
    const int per = max((pg1 - pg0 + splits - 1) / splits, kWaves);
    const long long begin = pg0 + (long long)i * per;
    pg0 = begin < pg1 ? (int)begin : pg1;
    pg1 = min(pg0 + per, pg1);
}

// Joins what the waves from, from + step, .. (n of them) hold in LDS for the same `rows`
// rows, each relative to its own maximum; `put` gets four channels of a row at a time, with
// the row's maximum and sum.
template <int D, typename O, typename ML, typename F>
__device__ __forceinline__ void join_waves(const O& o, const ML& ml, int from, int step, int n, int rows, int thread, int threads, F put) {
    for (int idx = thread; idx < rows * (D / 4); idx += threads) {
        const int c = idx / (D / 4), ch = 4 * (idx % (D / 4));
        float top = -INFINITY;
        for (int y = 0; y < n; ++y) top = fmaxf(top, ml[from + y * step][c][0]);
        const float at = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4v x = {0.f, 0.f, 0.f, 0.f};
        for (int y = 0; y < n; ++y) {
            const float f = __builtin_amdgcn_exp2f(ml[from + y * step][c][0] - at);
            sum += ml[from + y * step][c][1] * f;
            x += *reinterpret_cast<const float4v*>(&o[from + y * step][c][ch]) * f;
        }
        put(c, ch, x, make_float2(top, sum));
    }
}

}  // namespace

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------
//
// One workgroup looks at the groups and deals out their shared pages, as the host does
// not know them: a run has the same number of pages in every group, so that long
// prefixes take more workgroups than short ones and all end together; as many
// pages as keep the items (run, key head, tile of rows) within the workgroups that
// can be at work at once.
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long plan_sum(long long x, long long* s) {
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    long long sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) sum += s[w];
    return sum;
}

__global__ __launch_bounds__(kPlanThreads) void attn_shared_plan_kernel(SharedParams p) {
    __shared__ long long s_sum[kPlanThreads / 64];
    __shared__ int s_most, s_end;                     // pages of the longest prefix; items that have a group
    const int tid = threadIdx.x, lane = tid & 63, rep = p.Hq / p.Hkv, width = 32 * p.across;
    Group* groups = reinterpret_cast<Group*>(p.plan_groups);
    for (int n = tid; n < p.N; n += kPlanThreads) p.plan_group_of[n] = -1;
    if (tid == 0) { s_most = 0; s_end = INT_MAX; }
    __syncthreads();
    // a wave a group
    for (int g = tid >> 6; g < p.groups; g += kPlanThreads / 64) {
        const int first = clampi(p.group_start[g], 0, p.N), end = clampi(p.group_start[g + 1], first, p.N);
        const int shared = clampi(p.shared_pages[g], 0, p.max_pages);
        int lo = INT_MAX, hi = 0;
        for (int n = first + lane; n < end; n += 64) {
            int a, b;
            seen_range(p, n, a, b);
            if (a < b) { lo = min(lo, a); hi = max(hi, b); }
            p.plan_group_of[n] = g;
        }
        for (int o = 32; o > 0; o >>= 1) { lo = min(lo, __shfl_xor(lo, o, 64)); hi = max(hi, __shfl_xor(hi, o, 64)); }
        Group x;
        x.first = first;
        x.rows = (end - first) * rep;
        x.pg0 = lo / kPage;
        x.pg1 = min((int)(((long long)hi + kPage - 1) / kPage), shared);
        if (x.pg0 >= x.pg1) x.pg0 = x.pg1 = 0;
        x.tiles = (int)(((long long)x.rows + width - 1) / width);
        x.slots = x.base = 0;
        x.shared = shared;
        if (lane == 0) {
            groups[g] = x;
            atomicMax(&s_most, x.pg1 - x.pg0);
        }
    }
    __syncthreads();                                  // (one workgroup: what it wrote, it reads)
    __threadfence_block();
    // pages of a run
    long long all = 0;
    for (int g = tid; g < p.groups; g += kPlanThreads) all += (long long)groups[g].tiles * (groups[g].pg1 - groups[g].pg0);
    all = plan_sum(all, s_sum) * p.Hkv;
    const int most = s_most, least = 2 * kWaves / p.across;
    int per = (int)min((all + p.items - 1) / p.items, (long long)INT_MAX);
    per = max(per, least);
    while (per < most) {
        long long items = 0;
        for (int g = tid; g < p.groups; g += kPlanThreads)
            items += (long long)groups[g].tiles * ((groups[g].pg1 - groups[g].pg0 + per - 1) / per);
        if (plan_sum(items, s_sum) * p.Hkv <= p.items) break;
        per += (per + 15) / 16;
    }
    // each group's items behind those of the groups before it
    long long before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += kPlanThreads) {
        const int g = g0 + tid;
        long long mine = 0;
        int slots = 0;
        if (g < p.groups) {
            slots = (groups[g].pg1 - groups[g].pg0 + per - 1) / per;
            mine = (long long)slots * groups[g].tiles * p.Hkv;
        }
        long long run = mine;
        for (int o = 1; o < 64; o <<= 1) {
            const long long y = __shfl_up(run, o, 64);
            if (lane >= o) run += y;
        }
        __syncthreads();
        if (lane == 63) s_sum[tid >> 6] = run;
        __syncthreads();
        long long base = before;
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w < (tid >> 6)) base += s_sum[w];
            before += s_sum[w];
        }
        base += run - mine;
        if (g < p.groups) {
            // (bounds that overlap may want more than there are: from there on nothing is shared)
            const bool fits = base + mine <= p.items;
            if (!fits) atomicMin(&s_end, (int)min(base, (long long)p.items));
            groups[g].slots = fits ? slots : 0;
            groups[g].base = fits ? (int)base : 0;
        }
    }
    __syncthreads();
    for (int g = tid >> 6; g < p.groups; g += kPlanThreads / 64) {
        const int base = groups[g].base, items = groups[g].slots * groups[g].tiles * p.Hkv;
        for (int i = lane; i < items; i += 64) p.plan_items[base + i] = g;
    }
    if (tid == 0) {
        p.plan_head[0] = (int)min(before, (long long)s_end);
        p.plan_head[1] = per;
    }
}

// ---------------------------------------------------------------------------
// the shared pages
// ---------------------------------------------------------------------------
//
// A wave has 32 rows of a group on a key head (row r being query head r % rep of sequence
// first + r / rep), as the columns of 32 x 32 products:
//   S^T[key][row] = K Q^T, O^T[channel][row] += V^T W^T.
// Row m of S^T stands for key 16 (m / 4 % 2) + 4 (m / 8) + m % 4 of 32, which leaves lane half
// h with the keys 16 h .. 16 h + 15: those of its 16-byte reads of values, a channel each.
//
// ACROSS waves of a workgroup have different rows and share their pages, the teams of
// them take pages in turn.  Pages come through a ring in LDS of R pages a team, as they
// lie in memory, by direct loads R - 1 pages ahead (no registers, 1 KiB an instruction;
// read straight to registers in the operands' order, 16 bytes a lane from 32 rows, the same
// walk took 3 times as long).  A key's row keeps its 16-byte units u at u ^ f(row), so that
// the 16 rows of a read phase land on 16 different places of the banks' 256 bytes.
//
// A weight is exp2(s - m).  For the product with v it is taken times 2^b, b = 15 +
// log2 v_scale + m - wm, wm the running maximum of s + log2 v_scale, so that it has
// its f16 bits whatever the pages' scales: as the sum of two f16 values (22 bits) for
// fp32 results, as one (11 bits) for bf16 ones, whose own rounding is 8 times that.  The
// sum takes the same exponentials, times 2^-b once a page; where |b| is large (a page of
// zeros has a scale of 2^-96) it has its own.
template <int D, int ACROSS>
struct __attribute__((aligned(256))) SharedSmem {
    static constexpr int TEAMS = kWaves / ACROSS;
    static constexpr int R = ACROSS == 4 ? 4 : 2;
    union {
        uint8_t ring[TEAMS][R][2 * kPage * D];        // keys [64][D], then values [4][D][16]
        struct {
            float o[kWaves][32][D + 4];
            float ml[kWaves][32][2];
        };
    };
};

// A page's loads by one wave of the team that shares it: 16-byte direct loads, a KiB of
// keys or values each.
template <int D, int ACROSS>
struct PageLoader {
    static constexpr int KI = kPage * D / 1024, N = 2 * KI / ACROSS;      // loads of a side; of a wave
    int off;                                          // lane's source inside a KiB of keys, before the instruction's flip
    int lane16;

    __device__ __forceinline__ explicit PageLoader(int lane) {
        constexpr int CH = D / 16;
        const int f = D == 128 ? (lane >> 4) & 3 : (lane >> 4) & 1;
        off = (lane / CH) * D + 16 * ((lane % CH) ^ f);
        lane16 = 16 * lane;
    }
    template <int I> __device__ __forceinline__ void issue(uint64_t k, uint64_t v, uint32_t to, int first) const {
        if constexpr (I < N) {
            // (a wave's loads are all of one side where two or four waves share a page)
            const int i = first + I;
            const bool keys = ACROSS == 1 ? I < KI : first < KI;
            const int flip = D == 128 ? ((i >> 1) & 1) << 6 : (i & 1) << 5;
            attn::direct_load16<0>((keys ? off ^ flip : lane16) + 1024 * (keys ? i : i - KI), keys ? k : v, to + 1024 * i);
            issue<I + 1>(k, v, to, first);
        }
    }
};

template <int N> __device__ __forceinline__ void wait_loads_but() {
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));     // vmcnt(N)
}

template <int D, int PARTS, int ACROSS>
__global__ __launch_bounds__(64 * kWaves, ACROSS == 1 ? 1 : 2) void attn_shared_kernel(SharedParams p) {
    constexpr int KL = D / 32;                        // 16-byte reads of a key's row by a lane
    constexpr int DB = D / 32;                        // 32-channel tiles of the output
    typedef SharedSmem<D, ACROSS> Smem;
    constexpr int R = Smem::R, TEAMS = Smem::TEAMS;
    extern __shared__ __attribute__((aligned(256))) char smem[];
    Smem& sm = *reinterpret_cast<Smem*>(smem);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5, rep = p.Hq / p.Hkv;

    // consecutive workgroups go round the 8 XCDs: each of these takes a run of items, the
    // tiles that share pages one after the other
    const int items = p.plan_head[0], each = (items + 7) / 8;
    const int item = (blockIdx.x % 8) * each + blockIdx.x / 8;
    if ((int)(blockIdx.x / 8) >= each || item >= items) return;
    const Group x = group_of(p, p.plan_items[item]);
    const int per = p.plan_head[1];
    int w = item - x.base;
    const int tile = w % x.tiles; w /= x.tiles;
    const int kh = w % p.Hkv, slot = w / p.Hkv;
    const int row0 = 32 * ACROSS * tile, rows = min(32 * ACROSS, x.rows - row0);
    const int wr = wave % ACROSS, team = wave / ACROSS;
    const int pg0 = x.pg0 + slot * per, pg1 = min(pg0 + per, x.pg1);
    const int turns = (pg1 - pg0 + TEAMS - 1) / TEAMS;                    // of every team
    const int n = max(0, (pg1 - pg0 - team + TEAMS - 1) / TEAMS);         // pages of this one

    // this lane's row: its query (channels 32 s + 16 h .. + 15) and the keys it sees
    const int mine = 32 * wr + col;
    const bool live = mine < rows;
    const int seq = x.first + (row0 + mine) / rep, head = kh * rep + (row0 + mine) % rep;
    bf8v qf[KL][2];
#pragma unroll
    for (int s = 0; s < KL; ++s)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (live) u = *reinterpret_cast<const uint4*>((const uint16_t*)p.q + ((size_t)seq * p.Hq + head) * D + 32 * s + 16 * h + 8 * f);
            qf[s][f] = __builtin_bit_cast(bf8v, u);
        }
    int lo = 0, hi = 0, lo_most = 0, hi_least = INT_MAX, lo_least = INT_MAX, hi_most = 0;
    if (live) {
        seen_range(p, seq, lo, hi);
        lo_most = lo_least = lo;
        hi_least = hi_most = hi;
    }
    for (int o = 16; o > 0; o >>= 1) {
        lo_most = max(lo_most, __shfl_xor(lo_most, o, 64));
        hi_least = min(hi_least, __shfl_xor(hi_least, o, 64));
        lo_least = min(lo_least, __shfl_xor(lo_least, o, 64));
        hi_most = max(hi_most, __shfl_xor(hi_most, o, 64));
    }
    lo_most = __builtin_amdgcn_readfirstlane(lo_most);
    hi_least = __builtin_amdgcn_readfirstlane(hi_least);

    // the team's pages k0 .. k0 + 63, one a lane: place (-1: absent) and scales
    const int* entries = p.block_table + (size_t)x.first * p.max_pages + pg0 + team;
    int e_page;
    float e_ks, e_vs;
    auto look_up = [&](int k0) {
        const int k = k0 + lane;
        const int e = k < n ? entries[k * TEAMS] : -1;
        e_page = (unsigned)e < (unsigned)p.n_pages ? e : -1;
        const size_t ph = (size_t)max(e_page, 0) * p.Hkv + kh;
        e_ks = p.k_scale[ph];
        e_vs = p.v_scale[ph];
    };
    const PageLoader<D, ACROSS> loader(lane);
    const uint32_t ring = attn::lds_address(sm.ring[team][0]);
    constexpr uint32_t kBytes = 2 * kPage * D;
    // (an absent page is read as the first one: its bytes are masked)
    auto load_page = [&](int k) {
        const int pg = __builtin_amdgcn_readlane(e_page, k & 63);
        const size_t at = ((size_t)max(pg, 0) * p.Hkv + kh) * (kPage * D);
        loader.template issue<0>((uint64_t)p.k_cache + at, (uint64_t)p.v_cache + at, ring + (k % R) * kBytes, wr * loader.N);
    };

    float16v o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    float m = -INFINITY, l = 0.f, wm = -INFINITY;     // maximum and sum of the scores; maximum of the weights
    const float to2 = p.scale * 1.4426950408889634f;
    uint32_t k_at, v_at;                              // this lane's reads: of keys, to flip by 32 s; of values
    {
        const int tok = 16 * ((col >> 2) & 1) + 4 * (col >> 3) + (col & 3);
        const int f = D == 128 ? ((tok >> 1) & 3) | ((tok >> 4) & 1) << 2 : ((tok >> 2) & 1) | ((tok >> 4) & 1) << 1;
        k_at = tok * D + 16 * (h ^ f);
        v_at = kPage * D + (h * D + col) * 16;
    }
    typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
    auto read16 = [](uint32_t at) { return *(const __attribute__((address_space(3))) uint4v*)(uintptr_t)at; };

    look_up(0);
    int old_page = 0;                                 // of the 64 pages before, while some of them are still to come
    float old_ks = 0.f, old_vs = 0.f;
    for (int k = 0; k < R - 1; ++k)
        if (k < n) load_page(k);
    for (int k = 0; k < turns; ++k) {
        const int ahead = k + R - 1;
        if (ahead < n) wait_loads_but<(R - 2) * PageLoader<D, ACROSS>::N>();
        else attn::wait_loads();
        if (ACROSS > 1) lds_barrier();
        // the ring's place of page k - 1 is free: its reads are done
        if (ahead < n) {
            if ((ahead & 63) == 0) {
                old_page = e_page;
                old_ks = e_ks;
                old_vs = e_vs;
                look_up(ahead);
            }
            if (ACROSS == 1) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            load_page(ahead);
        }
        if (k >= n || 32 * wr >= rows) continue;      // no page, or no rows
        const bool before = (min(ahead, n - 1) >> 6) != (k >> 6);
        const int page = __builtin_amdgcn_readlane(before ? old_page : e_page, k & 63);
        const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(before ? old_ks : e_ks), k & 63));
        const float vs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(before ? old_vs : e_vs), k & 63));
        const int at0 = (pg0 + team + k * TEAMS) * kPage;
        const bool absent = page < 0;
        const uint32_t ring_k = ring + (k % R) * kBytes + k_at, ring_v = ring + (k % R) * kBytes + v_at;

        float by = ks * to2;                          // a score is st times this
        float16v st[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int j = 0; j < 16; ++j) st[b][j] = 0.f;
#pragma unroll
            for (int s = 0; s < KL; ++s) {
                const uint4v u = read16((ring_k ^ (32 * s)) + 32 * b * D);
                st[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(u.x, u.y), qf[s][0], st[b], 0, 0, 0);
                st[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(u.z, u.w), qf[s][1], st[b], 0, 0, 0);
            }
        }
        const bool edge = absent || at0 < lo_most || at0 + kPage > hi_least;
        if (edge || !(by >= 0.f)) {
            // (negative scales turn the order of the scores; masked ones stay -inf whatever the scale)
            asm volatile("");
#pragma unroll
            for (int b = 0; b < 2; ++b) st[b] *= by;
            by = 1.f;
        }
        if (edge) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = at0 + 32 * b + 16 * h + i;
                    if (absent || j < lo || j >= hi) st[b][i] = -INFINITY;
                }
        }

        float top = st[0][0];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, st[b][i]);
        top = max_across32(top);
        const bool none = !(top > -INFINITY);         // (the scale of a page that a row does not see does not reach it)
        top = none ? -INFINITY : top * by;
        const float log_vs = __builtin_amdgcn_logf(vs);   // base 2
        const float wt = none ? wm : fmaxf(wm, top + log_vs);
        top = fmaxf(top, m);
        if (__any(top > m || wt > wm)) {
            asm volatile("");
            l *= top > m ? __builtin_amdgcn_exp2f(m - top) : 1.f;      // 0 from -inf
            const float fade = wt > wm ? __builtin_amdgcn_exp2f(wm - wt) : 1.f;
            m = top;
            wm = wt;
#pragma unroll
            for (int i = 0; i < DB; ++i) o[i] *= fade;
        }
        const float at = m == -INFINITY ? 0.f : m, wat = wm == -INFINITY ? 0.f : wm;
        const float up = none ? 0.f : log_vs - wat + 15.f;      // a weight's exponent over its score's
        const float b2 = up + at;
        half8 w_hi[2][2], w_lo[2][2];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(st[b][i], by, up));
                sum[b] += w;
                const _Float16 a = (_Float16)w;
                w_hi[b][i / 8][i % 8] = a;
                if (PARTS == 2) w_lo[b][i / 8][i % 8] = (_Float16)(w - (float)a);
            }
        if (!__any(!none && !(fabsf(b2) <= 60.f))) {
            l += (sum[0] + sum[1]) * (none ? 0.f : __builtin_amdgcn_exp2f(-b2));
        } else {
            float y = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    y += __builtin_amdgcn_exp2f(__builtin_fmaf(st[b][i], by, -at));
                    asm volatile("" : "+v"(y));       // (one after the other: no registers for it)
                }
            l += y;
        }

        // values, and what remains of them in a page that some row sees in part: masked keys
        // count nothing, whatever their bytes.  Those of keys that no row sees become 0; a
        // NaN among those that some row does not see (its 0 would carry it over) becomes 0
        // as well, and is put into the rows that see it by the product of its place with
        // what they see.
        auto products = [&](auto in_part) {
            constexpr bool EDGE = decltype(in_part)::value;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t keep[4];
                half8 sees[2];
                if constexpr (EDGE) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = at0 + 32 * b + 16 * h + i;
                        if (i % 4 == 0) keep[i / 4] = 0;
                        if (!absent && j >= lo_least && j < hi_most) keep[i / 4] |= 0xffu << (8 * (i % 4));
                        sees[i / 8][i % 8] = (_Float16)(!absent && j >= lo && j < hi ? 1.f : 0.f);
                    }
                }
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    uint4v u = read16(ring_v + (2 * b * D + 32 * i) * 16);
                    if constexpr (EDGE) {
                        uint32_t x[4] = {u.x & keep[0], u.y & keep[1], u.z & keep[2], u.w & keep[3]}, one[4], nan = 0;
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t whole = (nan_bytes(x[t]) >> 7) * 0xffu;
                            nan |= whole;
                            x[t] &= ~whole;
                            one[t] = whole & 0x38383838u;
                        }
                        u = uint4v{x[0], x[1], x[2], x[3]};
                        if (__any(nan != 0)) {
                            float16v hit;
#pragma unroll
                            for (int j = 0; j < 16; ++j) hit[j] = 0.f;
                            hit = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_f16(one[0], one[1]), sees[0], hit, 0, 0, 0);
                            hit = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_f16(one[2], one[3]), sees[1], hit, 0, 0, 0);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (hit[j] > 0.f) o[i][j] = NAN;
                        }
                    }
                    const half8 v0 = e4m3x8_to_f16(u.x, u.y), v1 = e4m3x8_to_f16(u.z, u.w);
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, w_hi[b][0], o[i], 0, 0, 0);
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w_hi[b][1], o[i], 0, 0, 0);
                    if (PARTS == 2) {
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, w_lo[b][0], o[i], 0, 0, 0);
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w_lo[b][1], o[i], 0, 0, 0);
                    }
                }
            }
        };
        if (edge) products(std::true_type{});
        else products(std::false_type{});
    }

    // the waves that had the same rows join, in LDS: no load into it is left, and no read of the ring
    attn::wait_loads();
    lds_barrier();
    l = sum_across32(l);
    if (h == 0) { sm.ml[wave][col][0] = m; sm.ml[wave][col][1] = l; }
    const float down = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm - m - 15.f);   // to the scores' maximum
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4v y;
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = o[i][4 * j + k] * down;
            *reinterpret_cast<float4v*>(&sm.o[wave][col][32 * i + 8 * j + 4 * h]) = y;
        }
    lds_barrier();
    // all their lanes together; item's row 32 wr + c
    const size_t part = (size_t)item * (32 * ACROSS) + 32 * wr;
    join_waves<D>(sm.o, sm.ml, wr, ACROSS, TEAMS, min(32, rows - 32 * wr), team * 64 + lane, TEAMS * 64, [&](int c, int ch, float4v y, float2 ml) {
        *reinterpret_cast<float4v*>(&p.part_o[(part + c) * D + ch]) = y;
        if (ch == 0) *reinterpret_cast<float2*>(&p.part_ml[(part + c) * 2]) = ml;
    });
}

// ---------------------------------------------------------------------------
// a sequence's own pages, and the join
// ---------------------------------------------------------------------------
//
// Up to 16 of a sequence's query heads on a key head are the columns of 16 x 16
// products, the waves take pages in turn (as attn_decode_kernel has them).  Where one
// workgroup has all of the pages it joins the shared ones' partial results as well and
// writes the output; where there are few sequences their pages are dealt to several, and
// a kernel behind this one joins.
template <int D> struct __attribute__((aligned(16))) OwnSmem {
    float o[kWaves][16][D + 4];
    float ml[kWaves][16][2];
};

// where the partial result of run `slot` of group x's pages is for a sequence's query head
__device__ __forceinline__ size_t part_of(const SharedParams& p, const Group& x, int slot, int kh, int row) {
    const int width = 32 * p.across;
    return (size_t)(x.base + (slot * p.Hkv + kh) * x.tiles + row / width) * width + row % width;
}

template <int D, int PARTS>
__global__ __launch_bounds__(64 * kWaves) void attn_own_kernel(SharedParams p) {
    constexpr int KS = D / 64;                        // 64-channel steps of a key row
    constexpr int VT = D / 16;                        // 16-channel tiles of the output
    __shared__ OwnSmem<D> sm;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const int rep = p.Hq / p.Hkv, sets = (rep + 15) / 16;
    int w = blockIdx.x;
    const int qg = w % sets; w /= sets;
    const int kh = w % p.Hkv; w /= p.Hkv;
    const int n = w, i = blockIdx.y;
    const int q0 = kh * rep + 16 * qg, nq = min(16, rep - 16 * qg);
    int lo, hi;
    seen_range(p, n, lo, hi);
    const int gi = p.plan_group_of[n];
    Group x = {0, 0, 0, 0, 0, 0, 0, 0};
    if (gi >= 0) x = group_of(p, gi);
    int pg0 = max(lo / kPage, x.shared), pg1 = (int)(((long long)hi + kPage - 1) / kPage);
    if (p.own_splits > 1) run_of(pg0, pg1, i, p.own_splits);

    // queries: column col, channels 64 s + 16 g + 8 half ..
    bf8v qf[KS][2];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (col < nq)
                u = *reinterpret_cast<const uint4*>((const uint16_t*)p.q + ((size_t)n * p.Hq + q0 + col) * D + 64 * s + 16 * g + 8 * hf);
            qf[s][hf] = __builtin_bit_cast(bf8v, u);
        }
    float4v o[VT];
#pragma unroll
    for (int j = 0; j < VT; ++j) o[j] = float4v{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f, wm = -INFINITY;
    const float to2 = p.scale * 1.4426950408889634f;
    const int krow = 16 * (col >> 2) + (col & 3);     // key of tile 0's row `col`

    for (int pg = pg0 + wave; pg < pg1; pg += kWaves) {
        int page = p.block_table[(size_t)n * p.max_pages + pg];
        const int at0 = pg * kPage;
        const bool absent = (unsigned)page >= (unsigned)p.n_pages;
        if (absent) page = 0;
        const size_t ph = (size_t)page * p.Hkv + kh;
        const uint8_t* kp = p.k_cache + ph * (kPage * D);
        const uint8_t* vp = p.v_cache + ph * (kPage * D);
        uint4 kk[4][KS], vv[VT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                kk[t][s] = *reinterpret_cast<const uint4*>(kp + (krow + 4 * t) * D + 64 * s + 16 * g);
#pragma unroll
        for (int j = 0; j < VT; ++j)
            vv[j] = *reinterpret_cast<const uint4*>(vp + (size_t)(g * D + 16 * j + col) * 16);
        const float ks = p.k_scale[ph] * to2, vs = absent ? -INFINITY : __builtin_amdgcn_logf(p.v_scale[ph]);   // base 2

        float4v sc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            sc[t] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3x8_to_bf16(kk[t][s].x, kk[t][s].y), qf[s][0], sc[t], 0, 0, 0);
                sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3x8_to_bf16(kk[t][s].z, kk[t][s].w), qf[s][1], sc[t], 0, 0, 0);
            }
            sc[t] *= ks;
        }
        if (absent || at0 < lo || at0 + kPage > hi) {
            // the first and last pages: masked keys count nothing, whatever their bytes
            uint32_t keep[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                keep[t] = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = at0 + 16 * g + 4 * t + k;
                    const bool in = !absent && j >= lo && j < hi;
                    if (!in) sc[t][k] = -INFINITY;
                    else keep[t] |= 0xffu << (8 * k);
                }
            }
#pragma unroll
            for (int j = 0; j < VT; ++j) {
                vv[j].x &= keep[0]; vv[j].y &= keep[1]; vv[j].z &= keep[2]; vv[j].w &= keep[3];
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, sc[t][k]);
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = max_across32(top);
        const float wt = fmaxf(wm, top + vs);
        top = fmaxf(top, m);
        const float at = top == -INFINITY ? 0.f : top, wat = wt == -INFINITY ? 0.f : wt;
        l *= __builtin_amdgcn_exp2f(m - at);          // 0 from -inf
        const float fade = __builtin_amdgcn_exp2f(wm - wat), up = vs - wat + 15.f;
        m = top;
        wm = wt;
#pragma unroll
        for (int j = 0; j < VT; ++j) o[j] *= fade;
        half8 w_hi[2], w_lo[2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                l += __builtin_amdgcn_exp2f(sc[t][k] - at);
                const float x = __builtin_amdgcn_exp2f(sc[t][k] + up);
                const _Float16 a = (_Float16)x;
                w_hi[t >> 1][(t & 1) * 4 + k] = a;
                if (PARTS == 2) w_lo[t >> 1][(t & 1) * 4 + k] = (_Float16)(x - (float)a);
            }
#pragma unroll
        for (int j = 0; j < VT; ++j) {
            const half8 v0 = e4m3x8_to_f16(vv[j].x, vv[j].y), v1 = e4m3x8_to_f16(vv[j].z, vv[j].w);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w_hi[0], o[j], 0, 0, 0);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w_hi[1], o[j], 0, 0, 0);
            if (PARTS == 2) {
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w_lo[0], o[j], 0, 0, 0);
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w_lo[1], o[j], 0, 0, 0);
            }
        }
    }

    l += __shfl_xor(l, 16, 64);
    l = sum_across32(l);
    if (g == 0) { sm.ml[wave][col][0] = m; sm.ml[wave][col][1] = l; }
    const float down = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm - m - 15.f);   // to the scores' maximum
#pragma unroll
    for (int j = 0; j < VT; ++j)
        *reinterpret_cast<float4v*>(&sm.o[wave][col][16 * j + 4 * g]) = o[j] * down;
    __syncthreads();
    const size_t heads = (size_t)p.N * p.Hq;
    join_waves<D>(sm.o, sm.ml, 0, 1, kWaves, nq, wave * 64 + lane, kWaves * 64, [&](int c, int ch, float4v y, float2 ml) {
        const size_t head = (size_t)n * p.Hq + q0 + c;
        if (p.own_splits > 1) {
            *reinterpret_cast<float4v*>(&p.own_o[(i * heads + head) * D + ch]) = y;
            if (ch == 0) *reinterpret_cast<float2*>(&p.own_ml[(i * heads + head) * 2]) = ml;
            return;
        }
        const int row = (n - x.first) * rep + 16 * qg + c;
        float top = ml.x;
        for (int s = 0; s < x.slots; ++s) top = fmaxf(top, p.part_ml[2 * part_of(p, x, s, kh, row)]);
        const float at = top == -INFINITY ? 0.f : top, f0 = __builtin_amdgcn_exp2f(ml.x - at);
        float sum = ml.y * f0;
        y *= f0;
        for (int s = 0; s < x.slots; ++s) {
            const size_t from = part_of(p, x, s, kh, row);
            const float2 other = *reinterpret_cast<const float2*>(&p.part_ml[2 * from]);
            const float f = __builtin_amdgcn_exp2f(other.x - at);
            sum += other.y * f;
            y += *reinterpret_cast<const float4v*>(&p.part_o[from * D + ch]) * f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = top == -INFINITY && !(y[k] != y[k]) ? 0.f : y[k] / sum;
        if (p.flags & GDR_OUT_BF16)
            *reinterpret_cast<uint2*>((uint16_t*)p.o + head * D + ch) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        else
            *reinterpret_cast<float4v*>((float*)p.o + head * D + ch) = y;
    });
}

// Joins a head's partial results: one workgroup per head; its lanes read the maxima
// and sums side by side, then 1024 / D groups of them the outputs.
template <int D>
__global__ __launch_bounds__(256) void attn_shared_join(SharedParams p) {
    constexpr int GROUPS = 1024 / D;                  // D / 4 lanes each, four channels a lane
    __shared__ float s_x[GROUPS][D], s_ml[8], s_sum;
    const size_t head = blockIdx.x, heads = (size_t)p.N * p.Hq;
    const int tid = threadIdx.x, gi = tid / (D / 4), ch = 4 * (tid % (D / 4));
    const int n = (int)(head / p.Hq), hq = (int)(head % p.Hq), rep = p.Hq / p.Hkv;
    const int in = p.plan_group_of[n];
    Group x = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in >= 0) x = group_of(p, in);
    const int row = (n - x.first) * rep + hq % rep, slots = x.slots + p.own_splits;
    auto ml_at = [&](int s) {
        return s < x.slots ? &p.part_ml[2 * part_of(p, x, s, hq / rep, row)] : &p.own_ml[((s - x.slots) * heads + head) * 2];
    };
    auto o_at = [&](int s) {
        return s < x.slots ? &p.part_o[part_of(p, x, s, hq / rep, row) * D] : &p.own_o[((s - x.slots) * heads + head) * D];
    };
    float top = -INFINITY, sum = 0.f;
    for (int s = tid; s < slots; s += 256) {
        const float2 ml = *reinterpret_cast<const float2*>(ml_at(s));
        const float both = fmaxf(top, ml.x);
        if (both != -INFINITY) sum = sum * __builtin_amdgcn_exp2f(top - both) + ml.y * __builtin_amdgcn_exp2f(ml.x - both);
        else sum += ml.y;                             // 0, or NaN where every score is
        top = both;
    }
    for (int o = 32; o > 0; o >>= 1) {
        const float t2 = __shfl_xor(top, o, 64), s2 = __shfl_xor(sum, o, 64), both = fmaxf(top, t2);
        sum = both == -INFINITY ? sum + s2
                                : sum * __builtin_amdgcn_exp2f(top - both) + s2 * __builtin_amdgcn_exp2f(t2 - both);
        top = both;
    }
    if ((tid & 63) == 0) { s_ml[2 * (tid >> 6)] = top; s_ml[2 * (tid >> 6) + 1] = sum; }
    __syncthreads();
    top = fmaxf(fmaxf(s_ml[0], s_ml[2]), fmaxf(s_ml[4], s_ml[6]));
    const float at = top == -INFINITY ? 0.f : top;
    if (tid == 0) {
        float all = 0.f;
        for (int w = 0; w < 4; ++w)
            all += top == -INFINITY ? s_ml[2 * w + 1] : s_ml[2 * w + 1] * __builtin_amdgcn_exp2f(s_ml[2 * w] - at);
        s_sum = all;
    }
    float4v y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = gi; s < slots; s += GROUPS)
        y += *reinterpret_cast<const float4v*>(o_at(s) + ch) * __builtin_amdgcn_exp2f(*ml_at(s) - at);
    *reinterpret_cast<float4v*>(&s_x[gi][ch]) = y;
    __syncthreads();
    if (tid < D) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) z += s_x[i][tid];
        store_out(p, head * D + tid, top == -INFINITY && !(z != z) ? 0.f : z / s_sum);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

SharedPlan attn_shared_plan(int N, int groups, int Hq, int Hkv, int d, int max_pages, int window) {
    SharedPlan x;
    const int rep = Hq / Hkv;
    const long long rows = (long long)N * rep;        // of a key head
    const long long each = (rows + groups - 1) / groups;
    x.across = each > 64 ? 4 : each > 32 ? 2 : 1;
    const int width = 32 * x.across;
    // at most: every group's last tile has one row
    const long long some = groups < N ? groups : N;
    const long long tiles = (rows + some * (width - 1)) / width;
    // items that are at work at once; more only where there are more tiles than that
    const long long fill = x.across == 1 ? 256 : 512;
    x.items = tiles * Hkv > fill ? tiles * Hkv : fill;
    x.own_items = (long long)N * Hkv * ((rep + 15) / 16);
    int pages = max_pages;
    if (window > 0 && window / kPage + 2 < pages) pages = window / kPage + 2;
    long long s = (512 + x.own_items - 1) / x.own_items;
    const long long most = (pages + kWaves - 1) / kWaves;
    if (s > most) s = most;
    x.own_splits = s < 1 ? 1 : (int)s;
    // the workspace: plan, then partial results
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t y = at; at += up(bytes); return y; };
    x.at_head = take(16);
    x.at_groups = take(sizeof(Group) * (size_t)groups);
    x.at_group_of = take(4 * (size_t)N);
    x.at_items = take(4 * (size_t)x.items);
    x.at_part_o = take(4 * (size_t)x.items * width * d);
    x.at_part_ml = take(8 * (size_t)x.items * width);
    const size_t own = x.own_splits > 1 ? (size_t)x.own_splits * N * Hq : 0;
    x.at_own_o = take(4 * own * d);
    x.at_own_ml = take(8 * own);
    x.bytes = at;
    return x;
}

long long attn_shared_workgroups(const SharedPlan& x, long long heads) {
    const long long most = x.items > x.own_items ? x.items : x.own_items;
    return x.own_splits > 1 && heads > most ? heads : most;
}

template <int D, int PARTS, int ACROSS> static hipError_t launch_shared(const SharedParams& p, hipStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const int lds = (int)sizeof(SharedSmem<D, ACROSS>);
    const hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_shared_kernel<D, PARTS, ACROSS>), lds, done);
    if (e != hipSuccess) return e;
    // (the items of the 8 XCDs' runs: up to 7 more numbers than items)
    hipLaunchKernelGGL((attn_shared_kernel<D, PARTS, ACROSS>), dim3((unsigned)((p.items + 7) / 8 * 8)), dim3(64 * kWaves), lds, st, p);
    return hipGetLastError();
}

template <int D, int PARTS> static hipError_t launch_d(const SharedParams& p, const SharedPlan& x, hipStream_t st) {
    hipError_t e = p.across == 4 ? launch_shared<D, PARTS, 4>(p, st)
                 : p.across == 2 ? launch_shared<D, PARTS, 2>(p, st) : launch_shared<D, PARTS, 1>(p, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_own_kernel<D, PARTS>), dim3((unsigned)x.own_items, (unsigned)p.own_splits), dim3(64 * kWaves), 0, st, p);
    e = hipGetLastError();
    if (e != hipSuccess || p.own_splits == 1) return e;
    hipLaunchKernelGGL(attn_shared_join<D>, dim3((unsigned)((long long)p.N * p.Hq)), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_attn_shared(const SharedParams& p, const SharedPlan& x, hipStream_t st) {
    hipLaunchKernelGGL(attn_shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool one = (p.flags & GDR_OUT_BF16) != 0;
    if (p.d == 64) return one ? launch_d<64, 1>(p, x, st) : launch_d<64, 2>(p, x, st);
    return one ? launch_d<128, 1>(p, x, st) : launch_d<128, 2>(p, x, st);
}

}  // namespace gdr
