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
// Weights reach 2^(kTop + kLag) = 2^15 at most: f16 has room for that.
constexpr float kLag = 3.f, kTop = 12.f;

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

// bits i of 0 .. 31: key `base` + 32 (i / 16) + i % 16 is one of lo .. hi - 1
__device__ __forceinline__ uint32_t seen_bits(int base, int lo, int hi) {
    uint32_t bits = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int from = clampi(lo - base - 32 * b, 0, 16), to = clampi(hi - base - 32 * b, 0, 16);
        bits |= (((1u << to) - 1) & ~((1u << from) - 1)) << (16 * b);
    }
    return bits;
}
// bytes 0xff where the four bits from i on are set
__device__ __forceinline__ uint32_t bytes_of(uint32_t bits, int i) { return (((bits >> i) & 15u) * 0x00204081u & 0x01010101u) * 0xffu; }

// e4m3 bytes that are NaN (0x7f, 0xff), as 0x80 in their places
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }


// Which run of the pages pg0 .. pg1 - 1 is number i of `splits`; two pages at least, as the
// second is loaded beside the first one's work.
__device__ __forceinline__ void run_of(int& pg0, int& pg1, int i, int splits) {
    if (pg1 <= pg0) { pg1 = pg0; return; }
    const int per = max((pg1 - pg0 + splits - 1) / splits, 2);
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

struct PlanGroup {
    int first, shared, lo, hi;  // first sequence; pages; first and one past the last token that some sequence sees
    int base;
};

__global__ __launch_bounds__(kPlanThreads) void attn_shared_plan_kernel(SharedParams p) {
    extern __shared__ __attribute__((aligned(256))) char smem[];
    PlanGroup* s = reinterpret_cast<PlanGroup*>(smem);       // [groups + 1]
    __shared__ int s_per, s_items;
    const int tid = threadIdx.x, lane = tid & 63, rep = p.Hq / p.Hkv, G = p.groups;
    for (int g = tid; g <= G; g += kPlanThreads)
        s[g] = PlanGroup{clampi(p.group_start[g], 0, p.N), g < G ? clampi(p.shared_pages[g], 0, p.max_pages) : 0, INT_MAX, 0, 0};
    __syncthreads();
    for (int n = tid; n < p.N; n += kPlanThreads) {
        int a, b;
        seen_range(p, n, a, b);
        int g = 0, z = G - 1;                         // the last start at or before n
        while (g < z) {
            const int mid = (g + z + 1) / 2;
            if (s[mid].first <= n) g = mid;
            else z = mid - 1;
        }
        const bool in = n >= s[g].first && n < s[g + 1].first;
        p.plan_group_of[n] = in ? g : -1;
        if (in && a < b) {
            atomicMin(&s[g].lo, a);
            atomicMax(&s[g].hi, b);
        }
    }
    __syncthreads();
    // one wave: a run's pages, and where each group's items start
    auto tiles_of = [&](int g) {
        const long long rows = (long long)max(s[g + 1].first - s[g].first, 0) * rep;
        return (int)((rows + p.width - 1) / p.width);
    };
    auto first_page = [&](int g) { return s[g].lo / kPage; };
    auto pages_of = [&](int g) { return max(0, min((int)(((long long)s[g].hi + kPage - 1) / kPage), s[g].shared) - first_page(g)); };
    if (tid < 64) {
        auto sum_of = [&](auto f) {
            long long x = 0;
            for (int g = lane; g < G; g += 64) x += f(g);
            for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
            return x;
        };
        int most = 0;
        for (int g = lane; g < G; g += 64) most = max(most, pages_of(g));
        for (int o = 32; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o, 64));
        const long long room = p.items / p.Hkv;       // (tile, run) pairs of a key head
        const long long all = sum_of([&](int g) { return (long long)tiles_of(g) * pages_of(g); });
        int per = max((int)min((all + room - 1) / max(room, 1LL), (long long)INT_MAX / 2), 2 * kWaves);   // two pages a wave
        while (per < most && sum_of([&](int g) { return (long long)tiles_of(g) * ((pages_of(g) + per - 1) / per); }) > room)
            per += (per + 15) / 16;
        long long before = 0;
        int end = INT_MAX;
        for (int g0 = 0; g0 < G; g0 += 64) {
            const int g = g0 + lane;
            const long long mine = g < G ? (long long)tiles_of(g) * ((pages_of(g) + per - 1) / per) * p.Hkv : 0;
            long long run = mine;
            for (int o = 1; o < 64; o <<= 1) {
                const long long y = __shfl_up(run, o, 64);
                if (lane >= o) run += y;
            }
            const long long base = before + run - mine;
            // (bounds that overlap may want more than there are: from there on nothing is shared)
            const bool fits = base + mine <= p.items;
            if (g < G) s[g].base = fits ? (int)base : -1;
            if (!fits) end = min(end, (int)min(base, (long long)p.items));
            before += __shfl(run, 63, 64);
        }
        for (int o = 32; o > 0; o >>= 1) end = min(end, __shfl_xor(end, o, 64));
        if (lane == 0) { s_per = per; s_items = (int)min(before, (long long)end); }
    }
    __syncthreads();
    const int per = s_per;
    Group* groups = reinterpret_cast<Group*>(p.plan_groups);
    for (int g = tid; g < G; g += kPlanThreads) {
        Group x;
        x.first = s[g].first;
        x.rows = max(s[g + 1].first - s[g].first, 0) * rep;
        x.pg0 = pages_of(g) > 0 ? first_page(g) : 0;
        x.pg1 = x.pg0 + pages_of(g);
        x.tiles = tiles_of(g);
        x.slots = s[g].base < 0 ? 0 : (pages_of(g) + per - 1) / per;
        x.base = max(s[g].base, 0);
        x.shared = s[g].shared;
        groups[g] = x;
    }
    for (int i = tid; i < s_items; i += kPlanThreads) {      // the last group that starts at or before item i
        int g = 0, z = G - 1;
        while (g < z) {
            const int mid = (g + z + 1) / 2;
            if (s[mid].base >= 0 && s[mid].base <= i) g = mid;
            else z = mid - 1;
        }
        p.plan_items[i] = g;
    }
    if (tid == 0) {
        p.plan_head[0] = s_items;
        p.plan_head[1] = per;
    }
}

// ---------------------------------------------------------------------------
// the shared pages
// ---------------------------------------------------------------------------
//
// Rows of a group on a key head (row r being query head r % rep of sequence
// first + r / rep), as the columns of 32 x 32 products:
//   S^T[key][row] = K Q^T, O^T[channel][row] += V^T W^T.
// Row m of S^T stands for key 16 (m / 4 % 2) + 4 (m / 8) + m % 4 of 32, which leaves lane half
// h with the keys 16 h .. 16 h + 15: those of its 16-byte reads of values, a channel each.
//
// A wave has 64 rows (32 where groups are smaller): what a page costs beside its products,
// its bytes' conversion above all, is then shared by as many.  The waves of a workgroup
// have the same rows and take pages in turn, each for itself: with waves that shared
// a page and waited for each other at every one, 1,024 rows on 512 pages took 215 us for
// 181.  Pages come through two places in LDS a wave, as they lie in memory, by direct loads a
// page ahead (no registers, 1 KiB an instruction): read straight to registers in the
// operands' order, 16 bytes a lane from 32 rows, the same walk took 265.
//
// A weight is exp2(s - m).  For the product with v it is taken times 2^b, b = 12 +
// log2 v_scale + m - wm, wm the running maximum of s + log2 v_scale, so that it has
// its f16 bits whatever the pages' scales: as the sum of two f16 values (22 bits) for
// fp32 results, as one (11 bits) for bf16 ones, whose own rounding is 8 times that.  The
// sum takes the same exponentials, times 2^-b once a page; where |b| is large (a page of
// zeros has a scale of 2^-96) it has its own.
template <int D>
struct __attribute__((aligned(256))) SharedSmem {
    union {
        uint8_t ring[kWaves][2][2 * kPage * D];       // keys [64][D], then values [4][D][16]
        struct {
            float o[kWaves][32][D + 4];
            float ml[kWaves][32][2];
        };
    };
};

// A page into LDS by a wave: 16-byte direct loads, a KiB of keys or values each.  A key's
// row keeps its 16-byte units u at u ^ f(row), so that the 16 rows that a phase of the
// operand's reads takes land on 16 different places of the banks' 256 bytes: rows
// 4 a + b and 16 + 4 a + b of 32 x 32 products (a in two following ones, b < 4), or
// 16 a + b of 16 x 16 products (OWN; a, b < 4), + 4 t.
template <int D, bool OWN> __device__ __forceinline__ constexpr int key_flip(int row) {
    if (OWN) return D == 128 ? ((row >> 1) & 1) | ((row >> 4) & 3) << 1 : (row >> 4) & 3;
    return D == 128 ? ((row >> 1) & 3) | ((row >> 4) & 1) << 2 : ((row >> 2) & 1) | ((row >> 4) & 1) << 1;
}
template <int D, bool OWN>
struct PageLoader {
    static constexpr int N = kPage * D / 1024;        // loads of a side
    static constexpr int ROWS = 1024 / D;             // keys of one
    int off;                                          // a lane's place in a KiB of keys, before the instruction's flip
    int lane16;

    __device__ __forceinline__ explicit PageLoader(int lane) {
        constexpr int CH = D / 16;
        off = (lane / CH) * D + 16 * ((lane % CH) ^ key_flip<D, OWN>(lane / CH));
        lane16 = 16 * lane;
    }
    // (the flip of a row is that of its place in the KiB xor that of the KiB's first row)
    template <int I = 0> __device__ __forceinline__ void keys(uint64_t from, uint32_t to) const {
        attn::direct_load16<1024 * I>((off ^ (16 * key_flip<D, OWN>(ROWS * I))) + 1024 * I, from, to);
        if constexpr (I + 1 < N) keys<I + 1>(from, to);
    }
    template <int I = 0> __device__ __forceinline__ void values(uint64_t from, uint32_t to) const {
        attn::direct_load16<1024 * I>(lane16 + 1024 * I, from, to);
        if constexpr (I + 1 < N) values<I + 1>(from, to);
    }
};

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4v read16(uint32_t at) { return *(const __attribute__((address_space(3))) uint4v*)(uintptr_t)at; }

template <int D, int PARTS, int NB>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_shared_kernel(SharedParams p) {
    constexpr int KL = D / 32;                        // 16-byte reads of a key's row by a lane
    constexpr int DB = D / 32;                        // 32-channel tiles of the output
    constexpr int kRows = 32 * NB;                    // of the workgroup: its waves have the same ones
    extern __shared__ __attribute__((aligned(256))) char smem[];
    SharedSmem<D>& sm = *reinterpret_cast<SharedSmem<D>*>(smem);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5, rep = p.Hq / p.Hkv;

    // consecutive workgroups go round the 8 XCDs: each of these takes a run of items, the
    // tiles that share pages one after the other
    const int items = p.plan_head[0], each = (items + 7) / 8;
    const int item = (blockIdx.x % 8) * each + blockIdx.x / 8;
    if ((int)(blockIdx.x / 8) >= each || item >= items) return;
    const Group x = group_of(p, p.plan_items[item]);
    const int per = p.plan_head[1];
    int rest = item - x.base;
    const int tile = rest % x.tiles; rest /= x.tiles;
    const int kh = rest % p.Hkv, slot = rest / p.Hkv;
    const int row0 = kRows * tile, rows = min(kRows, x.rows - row0);
    const int pg0 = x.pg0 + slot * per, pg1 = min(pg0 + per, x.pg1);
    const int n = max(0, (pg1 - pg0 - wave + kWaves - 1) / kWaves);      // pages of this wave

    // this wave's pages k0 .. k0 + 63, one a lane: place (-1: absent) and scales
    const int* entries = p.block_table + (size_t)x.first * p.max_pages + pg0 + wave;
    int e_page;
    float e_ks, e_vs;
    auto look_up = [&](int k0) {
        const int k = k0 + lane;
        const int e = k < n ? entries[k * kWaves] : -1;
        e_page = (unsigned)e < (unsigned)p.n_pages ? e : -1;
        const size_t ph = (size_t)max(e_page, 0) * p.Hkv + kh;
        e_ks = p.k_scale[ph];
        e_vs = p.v_scale[ph];
    };
    const PageLoader<D, false> loader(lane);
    const uint32_t ring = attn::lds_address(sm.ring[wave][0]);
    constexpr uint32_t kSide = kPage * D;
    // (an absent page is read as the first one: its bytes are masked)
    auto load = [&](int k) {
        const int pg = __builtin_amdgcn_readlane(e_page, k & 63);
        const size_t at = ((size_t)max(pg, 0) * p.Hkv + kh) * kSide;
        const uint32_t to = ring + (k & 1) * (2 * kSide);
        loader.keys((uint64_t)p.k_cache + at, to);
        loader.values((uint64_t)p.v_cache + at, to + kSide);
    };
    look_up(0);
    if (n > 0) load(0);

    // this lane's rows: their queries (channels 32 s + 16 h .. + 15) and the keys they see
    bf8v qf[NB][KL][2];
    int lo[NB], hi[NB], lo_most = 0, hi_least = INT_MAX, lo_least = INT_MAX, hi_most = 0;
#pragma unroll
    for (int c = 0; c < NB; ++c) {
        const int mine = 32 * c + col;
        const bool live = mine < rows;
        const int seq = x.first + (row0 + mine) / rep, head = kh * rep + (row0 + mine) % rep;
#pragma unroll
        for (int s = 0; s < KL; ++s)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live)
                    u = *reinterpret_cast<const uint4*>((const uint16_t*)p.q + ((size_t)seq * p.Hq + head) * D + 32 * s + 16 * h + 8 * f);
                qf[c][s][f] = __builtin_bit_cast(bf8v, u);
            }
        lo[c] = hi[c] = 0;
        if (live) {
            seen_range(p, seq, lo[c], hi[c]);
            lo_most = max(lo_most, lo[c]);
            lo_least = min(lo_least, lo[c]);
            hi_least = min(hi_least, hi[c]);
            hi_most = max(hi_most, hi[c]);
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        lo_most = max(lo_most, __shfl_xor(lo_most, o, 64));
        hi_least = min(hi_least, __shfl_xor(hi_least, o, 64));
        lo_least = min(lo_least, __shfl_xor(lo_least, o, 64));
        hi_most = max(hi_most, __shfl_xor(hi_most, o, 64));
    }
    lo_most = __builtin_amdgcn_readfirstlane(lo_most);
    hi_least = __builtin_amdgcn_readfirstlane(hi_least);

    float16v o[NB][DB];
    float m[NB], l[NB], wm[NB];                       // maximum and sum of the scores; maximum of the weights
#pragma unroll
    for (int c = 0; c < NB; ++c) {
        m[c] = -INFINITY; l[c] = 0.f; wm[c] = -INFINITY;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[c][i][j] = 0.f;
    }
    const float to2 = p.scale * 1.4426950408889634f;
    uint32_t k_at, v_at;                              // this lane's reads: of keys, to flip by 32 s; of values
    {
        const int tok = 16 * ((col >> 2) & 1) + 4 * (col >> 3) + (col & 3);
        k_at = tok * D + 16 * (h ^ key_flip<D, false>(tok));
        v_at = kPage * D + (h * D + col) * 16;
    }

    uint32_t nans = 0;                                // some value that not every row sees is NaN
    for (int k = 0; k < n; ++k) {
        const int page = __builtin_amdgcn_readlane(e_page, k & 63);
        const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_ks), k & 63));
        const float vs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_vs), k & 63));
        const int at0 = (pg0 + wave + k * kWaves) * kPage;
        const bool absent = page < 0;
        const uint32_t ring_k = ring + (k & 1) * (2 * kSide) + k_at, ring_v = ring + (k & 1) * (2 * kSide) + v_at;
        // this page is there, and the place of the one before it is free: its reads are done
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        if (k + 1 < n) {
            if (((k + 1) & 63) == 0) look_up(k + 1);
            load(k + 1);
        }

        uint4v kr[2][KL];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int s = 0; s < KL; ++s) kr[b][s] = read16((ring_k ^ (32 * s)) + 32 * b * D);
        float16v st[NB][2];
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j) st[c][b][j] = 0.f;
#pragma unroll
        for (int s = 0; s < KL; ++s)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const bf8v k0 = e4m3x8_to_bf16(kr[b][s].x, kr[b][s].y), k1 = e4m3x8_to_bf16(kr[b][s].z, kr[b][s].w);
#pragma unroll
                for (int c = 0; c < NB; ++c) st[c][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k0, qf[c][s][0], st[c][b], 0, 0, 0);
#pragma unroll
                for (int c = 0; c < NB; ++c) st[c][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k1, qf[c][s][1], st[c][b], 0, 0, 0);
            }
        uint4v vr[2][DB];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < DB; ++i) vr[b][i] = read16(ring_v + (2 * b * D + 32 * i) * 16);

        float by = ks * to2;                          // a score is st times this
        const bool edge = absent || at0 < lo_most || at0 + kPage > hi_least;
        if (edge || !(by >= 0.f)) {
            // (negative scales turn the order of the scores; masked ones stay -inf whatever the scale)
            asm volatile("");
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    st[c][b] *= by;
                    if (edge) {
                        const uint32_t sees = absent ? 0 : seen_bits(at0 + 16 * h, lo[c], hi[c]);
#pragma unroll
                        for (int i = 0; i < 16; ++i) st[c][b][i] = sees >> (16 * b + i) & 1 ? st[c][b][i] : -INFINITY;
                    }
                }
            by = 1.f;
            if (edge) {
                // some row sees the page in part: values of keys that no row sees count as 0,
                // and so do NaNs, which the 0 of a row that does not see them would carry
                // over: the rows that see them get them at the end
                const uint32_t some = absent ? 0 : seen_bits(at0 + 16 * h, lo_least, hi_most);
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t keep = bytes_of(some, 16 * b + 4 * t);
#pragma unroll
                        for (int i = 0; i < DB; ++i) {
                            uint32_t y = vr[b][i][t] & keep;
                            const uint32_t whole = (nan_bytes(y) >> 7) * 0xffu;
                            nans |= whole;
                            vr[b][i][t] = y & ~whole;
                        }
                    }
            }
        }

        // The maxima are followed when they are more than 2^kLag ahead, each row's by itself
        // (the roundings of a row do not depend on keys that only its neighbours see): in
        // most pages some row of 32 has a new one, and o would be scaled anew.
        const float log_vs = __builtin_amdgcn_logf(vs);   // base 2
        float top[NB];
        bool none[NB], ahead_m[NB], ahead_w[NB], any = false;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            top[c] = st[c][0][0];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top[c] = fmaxf(top[c], st[c][b][i]);
            top[c] = max_across32(top[c]);
            none[c] = !(top[c] > -INFINITY);          // (the scale of a page that a row does not see does not reach it)
            top[c] = none[c] ? -INFINITY : top[c] * by;
            ahead_m[c] = top[c] > m[c] + kLag;
            ahead_w[c] = !none[c] && top[c] + log_vs > wm[c] + kLag;
            any = any || ahead_m[c] || ahead_w[c];
        }
        if (__any(any)) {
            asm volatile("");
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                const float fade = ahead_w[c] ? __builtin_amdgcn_exp2f(wm[c] - (top[c] + log_vs)) : 1.f;
                l[c] *= ahead_m[c] ? __builtin_amdgcn_exp2f(m[c] - top[c]) : 1.f;      // 0 from -inf
                m[c] = ahead_m[c] ? top[c] : m[c];
                wm[c] = ahead_w[c] ? top[c] + log_vs : wm[c];
#pragma unroll
                for (int i = 0; i < DB; ++i) o[c][i] *= fade;
            }
        }
        float up[NB], share[NB];                      // a weight's exponent over its score's; its part in the sum
        bool far = false;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            const float at = m[c] == -INFINITY ? 0.f : m[c], wat = wm[c] == -INFINITY ? 0.f : wm[c];
            up[c] = none[c] ? 0.f : log_vs - wat + kTop;
            share[c] = none[c] ? 0.f : __builtin_amdgcn_exp2f(-(up[c] + at));
            far = far || (!none[c] && !(fabsf(up[c] + at) <= 60.f));
        }
        if (__any(far)) {
            // the sum's own exponentials
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                const float at = m[c] == -INFINITY ? 0.f : m[c];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        l[c] += __builtin_amdgcn_exp2f(__builtin_fmaf(st[c][b][i], by, -at));
                        asm volatile("" : "+v"(l[c]));    // (one after the other: no registers for it)
                    }
                share[c] = 0.f;
            }
        }

        half8 w_hi[NB][2], w_lo[NB][2];
        auto weights = [&](int c, int b) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(st[c][b][i], by, up[c]));
                sum[i & 1] += w;
                const _Float16 a = (_Float16)w;
                w_hi[c][i / 8][i % 8] = a;
                if (PARTS == 2) w_lo[c][i / 8][i % 8] = (_Float16)(w - (float)a);
            }
            l[c] += (sum[0] + sum[1]) * share[c];
        };
        auto product = [&](int i, half8 v0, half8 v1) {
#pragma unroll
            for (int c = 0; c < NB; ++c) o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, w_hi[c][0], o[c][i], 0, 0, 0);
#pragma unroll
            for (int c = 0; c < NB; ++c) o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w_hi[c][1], o[c][i], 0, 0, 0);
            if (PARTS == 2) {
#pragma unroll
                for (int c = 0; c < NB; ++c) o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, w_lo[c][0], o[c][i], 0, 0, 0);
#pragma unroll
                for (int c = 0; c < NB; ++c) o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w_lo[c][1], o[c][i], 0, 0, 0);
            }
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int c = 0; c < NB; ++c) weights(c, b);
#pragma unroll
            for (int i = 0; i < DB; ++i)
                product(i, e4m3x8_to_f16(vr[b][i].x, vr[b][i].y), e4m3x8_to_f16(vr[b][i].z, vr[b][i].w));
        }
    }

    // the waves that had the same rows join, in LDS, 32 rows at a time: no load into it is
    // left, and no read of the ring
    attn::wait_loads();
#pragma unroll
    for (int c = 0; c < NB; ++c) {
        lds_barrier();
        l[c] = sum_across32(l[c]);
        if (h == 0) { sm.ml[wave][col][0] = m[c]; sm.ml[wave][col][1] = l[c]; }
        const float down = m[c] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm[c] - m[c] - kTop);   // to the scores' maximum
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4v y;
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = o[c][i][4 * j + k] * down;
                *reinterpret_cast<float4v*>(&sm.o[wave][col][32 * i + 8 * j + 4 * h]) = y;
            }
        lds_barrier();
        // all their lanes together
        const size_t part = (size_t)item * kRows + 32 * c;
        join_waves<D>(sm.o, sm.ml, 0, 1, kWaves, min(32, rows - 32 * c), wave * 64 + lane, kWaves * 64, [&](int r, int ch, float4v y, float2 ml) {
            *reinterpret_cast<float4v*>(&p.part_o[(part + r) * D + ch]) = y;
            if (ch == 0) *reinterpret_cast<float2*>(&p.part_ml[(part + r) * 2]) = ml;
        });
    }
    if (!__syncthreads_or(nans != 0)) return;
    // NaNs among values that not every row sees: into the rows that see them, one by one
    __threadfence_block();
    for (int pg = pg0; pg < pg1; ++pg) {
        const int page = p.block_table[(size_t)x.first * p.max_pages + pg];
        if ((unsigned)page >= (unsigned)p.n_pages) continue;
        const uint8_t* values = p.v_cache + ((size_t)page * p.Hkv + kh) * (kPage * D);
        for (int i = threadIdx.x; i < kPage * D; i += 64 * kWaves) {
            if ((values[i] & 0x7f) != 0x7f) continue;
            const int j = pg * kPage + 16 * (i / (16 * D)) + i % 16, ch = i / 16 % D;
            for (int r = 0; r < rows; ++r) {
                int a, b;
                seen_range(p, x.first + (row0 + r) / rep, a, b);
                if (j >= a && j < b) p.part_o[((size_t)item * kRows + r) * D + ch] = NAN;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// a sequence's own pages, and the join
// ---------------------------------------------------------------------------
//
// Up to 16 of a sequence's query heads on a key head are the columns of 16 x 16
// products (as attn_decode_kernel has them).  A wave has all of the pages of one, or a run of
// them where there are few sequences, and loads each page while it works on the one before:
// a few pages a sequence are too few to be dealt to four waves, whose starts and joins
// took as long as the pages.  Where a wave
// has all pages it joins the shared ones' partial results as well and writes the output;
// else a kernel behind this one does.

// where the partial result of run `slot` of group x's pages is for a sequence's query head
__device__ __forceinline__ size_t part_of(const SharedParams& p, const Group& x, int slot, int kh, int row) {
    return (size_t)(x.base + (slot * p.Hkv + kh) * x.tiles + row / p.width) * p.width + row % p.width;
}

template <int D, int PARTS>
__global__ __launch_bounds__(64) void attn_own_kernel(SharedParams p) {
    constexpr int KS = D / 64;                        // 64-channel steps of a key row
    constexpr int VT = D / 16;                        // 16-channel tiles of the output
    __shared__ __attribute__((aligned(256))) uint8_t s_ring[2][2 * kPage * D];       // keys [64][D], then values [4][D][16]
    const int lane = threadIdx.x;
    const int col = lane & 15, g = lane >> 4;
    const int rep = p.Hq / p.Hkv, sets = (rep + 15) / 16;
    int w = blockIdx.x;
    const int qg = w % sets; w /= sets;
    const int kh = w % p.Hkv; w /= p.Hkv;
    const int n = w % p.N, run = w / p.N;
    const int q0 = kh * rep + 16 * qg, nq = min(16, rep - 16 * qg);
    const int gi = p.plan_group_of[n];
    int lo, hi;
    seen_range(p, n, lo, hi);
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
    Group x = {0, 0, 0, 0, 0, 0, 0, 0};
    if (gi >= 0) x = group_of(p, gi);
    int pg0 = max(lo / kPage, x.shared), pg1 = (int)(((long long)hi + kPage - 1) / kPage);
    run_of(pg0, pg1, run, p.own_splits);
    pg0 = __builtin_amdgcn_readfirstlane(pg0);
    pg1 = __builtin_amdgcn_readfirstlane(pg1);
    const int count = pg1 - pg0;

    // pages k0 .. k0 + 63 of the run, one a lane: place (-1: absent) and scales
    const int* entries = p.block_table + (size_t)n * p.max_pages + pg0;
    int e_page;
    float e_ks, e_vs;
    auto look_up = [&](int k0) {
        const int e = k0 + lane < count ? entries[k0 + lane] : -1;
        e_page = (unsigned)e < (unsigned)p.n_pages ? e : -1;
        const size_t ph = (size_t)max(e_page, 0) * p.Hkv + kh;
        e_ks = p.k_scale[ph];
        e_vs = p.v_scale[ph];
    };
    const PageLoader<D, true> loader(lane);
    const uint32_t ring = attn::lds_address(s_ring[0]);
    constexpr uint32_t kSide = kPage * D;
    auto load = [&](int k) {                          // (an absent page is read as the first one)
        const size_t at = ((size_t)max(__builtin_amdgcn_readlane(e_page, k & 63), 0) * p.Hkv + kh) * kSide;
        const uint32_t to = ring + (k & 1) * (2 * kSide);
        loader.keys((uint64_t)p.k_cache + at, to);
        loader.values((uint64_t)p.v_cache + at, to + kSide);
    };
    if (count > 0) {
        look_up(0);
        load(0);
    }
    const int krow = 16 * (col >> 2) + (col & 3);     // key of tile 0's row `col`; its flip is that of the others, + 4 t, too
    const uint32_t k_at = krow * D + 16 * (g ^ key_flip<D, true>(krow)), v_at = kSide + (g * D + col) * 16;

    float4v o[VT];
#pragma unroll
    for (int j = 0; j < VT; ++j) o[j] = float4v{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f, wm = -INFINITY;
    const float to2 = p.scale * 1.4426950408889634f;
    for (int k = 0; k < count; ++k) {
        const int page = __builtin_amdgcn_readlane(e_page, k & 63);
        const float k_scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_ks), k & 63));
        const float v_scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_vs), k & 63));
        // this page is there, and the place of the one before it is free: its reads are done
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        if (k + 1 < count) {
            if (((k + 1) & 63) == 0) look_up(k + 1);
            load(k + 1);
        }
        const uint32_t at_k = ring + (k & 1) * (2 * kSide) + k_at, at_v = ring + (k & 1) * (2 * kSide) + v_at;
        const int at0 = (pg0 + k) * kPage;
        const bool absent = page < 0;
        const float ks = k_scale * to2, vs = absent ? -INFINITY : __builtin_amdgcn_logf(v_scale);   // base 2
        uint4v vv[VT];
        float4v sc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            sc[t] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint4v u = read16((at_k ^ (64 * s)) + 4 * t * D);
                sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3x8_to_bf16(u.x, u.y), qf[s][0], sc[t], 0, 0, 0);
                sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3x8_to_bf16(u.z, u.w), qf[s][1], sc[t], 0, 0, 0);
            }
            sc[t] *= ks;
        }
#pragma unroll
        for (int j = 0; j < VT; ++j) vv[j] = read16(at_v + 256 * j);
        if (absent || at0 < lo || at0 + kPage > hi) {
            // the first and last pages: masked keys count nothing, whatever their bytes
            uint32_t keep[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                keep[t] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = at0 + 16 * g + 4 * t + i;
                    const bool in = !absent && j >= lo && j < hi;
                    if (!in) sc[t][i] = -INFINITY;
                    else keep[t] |= 0xffu << (8 * i);
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
            for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[t][i]);
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
            for (int i = 0; i < 4; ++i) {
                l += __builtin_amdgcn_exp2f(sc[t][i] - at);
                const float z = __builtin_amdgcn_exp2f(sc[t][i] + up);
                const _Float16 a = (_Float16)z;
                w_hi[t >> 1][(t & 1) * 4 + i] = a;
                if (PARTS == 2) w_lo[t >> 1][(t & 1) * 4 + i] = (_Float16)(z - (float)a);
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

    // a lane has channels 16 j + 4 g .. + 3 of column col
    l += __shfl_xor(l, 16, 64);
    l = sum_across32(l);
    const float down = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm - m - 15.f);   // to the scores' maximum
#pragma unroll
    for (int j = 0; j < VT; ++j) o[j] *= down;
    if (col >= nq) return;
    const size_t head = (size_t)n * p.Hq + q0 + col, heads = (size_t)p.N * p.Hq;
    if (p.own_splits > 1) {
        // (nothing in the run: the join does not read the output)
        if (count > 0)
#pragma unroll
            for (int j = 0; j < VT; ++j) *reinterpret_cast<float4v*>(&p.own_o[(run * heads + head) * D + 16 * j + 4 * g]) = o[j];
        if (g == 0) *reinterpret_cast<float2*>(&p.own_ml[(run * heads + head) * 2]) = make_float2(m, l);
        return;
    }
    const int row = (n - x.first) * rep + 16 * qg + col;
    float top = m;
    for (int s = 0; s < x.slots; ++s) top = fmaxf(top, p.part_ml[2 * part_of(p, x, s, kh, row)]);
    const float at = top == -INFINITY ? 0.f : top;
    {
        const float f = __builtin_amdgcn_exp2f(m - at);
        l *= f;
#pragma unroll
        for (int j = 0; j < VT; ++j) o[j] *= f;
    }
    for (int s = 0; s < x.slots; ++s) {
        const size_t from = part_of(p, x, s, kh, row);
        const float2 ml = *reinterpret_cast<const float2*>(&p.part_ml[2 * from]);
        const float f = __builtin_amdgcn_exp2f(ml.x - at);
        l += ml.y * f;
#pragma unroll
        for (int j = 0; j < VT; ++j) o[j] += *reinterpret_cast<const float4v*>(&p.part_o[from * D + 16 * j + 4 * g]) * f;
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int j = 0; j < VT; ++j) {
        float4v y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = l == 0.f && !(o[j][i] != o[j][i]) ? 0.f : o[j][i] * inv;   // l = 0: nothing seen
        if (p.flags & GDR_OUT_BF16)
            *reinterpret_cast<uint2*>((uint16_t*)p.o + head * D + 16 * j + 4 * g) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        else
            *reinterpret_cast<float4v*>((float*)p.o + head * D + 16 * j + 4 * g) = y;
    }
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
    for (int s = gi; s < slots; s += GROUPS) {
        const float2 ml = *reinterpret_cast<const float2*>(ml_at(s));
        if (s >= x.slots && ml.x == -INFINITY && ml.y == 0.f) continue;      // an empty run: not written
        y += *reinterpret_cast<const float4v*>(o_at(s) + ch) * __builtin_amdgcn_exp2f(ml.x - at);
    }
    *reinterpret_cast<float4v*>(&s_x[gi][ch]) = y;
    __syncthreads();
    if (tid < D) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) z += s_x[i][tid];
        store_out(p, head * D + tid, s_sum == 0.f && !(z != z) ? 0.f : z / s_sum);      // (0: nothing seen)
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
    x.width = each > 32 ? 64 : 32;
    // at most: every group's last tile has one row
    const long long some = groups < N ? groups : N;
    const long long tiles = (rows + some * (x.width - 1)) / x.width;
    // items: as many workgroups as the compute units' LDS holds; more only where there are
    // more tiles than that
    const long long fill = d == 64 ? 512 : 256;
    x.items = tiles * Hkv > fill ? tiles * Hkv : fill;
    x.own_items = (long long)N * Hkv * ((rep + 15) / 16);
    int pages = max_pages;
    if (window > 0 && window / kPage + 2 < pages) pages = window / kPage + 2;
    // about two waves a SIMD
    long long s = (2048 + x.own_items / 2) / x.own_items;
    const long long most = (pages + 1) / 2;
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
    x.at_part_o = take(4 * (size_t)x.items * x.width * d);
    x.at_part_ml = take(8 * (size_t)x.items * x.width);
    const size_t own = x.own_splits > 1 ? (size_t)x.own_splits * N * Hq : 0;
    x.at_own_o = take(4 * own * d);
    x.at_own_ml = take(8 * own);
    x.bytes = at;
    return x;
}

long long attn_shared_workgroups(const SharedPlan& x, long long heads) {
    const long long own = x.own_items * x.own_splits, most = x.items > own ? x.items : own;
    return x.own_splits > 1 && heads > most ? heads : most;
}

template <int D, int PARTS, int NB> static hipError_t launch_shared(const SharedParams& p, hipStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const int lds = (int)sizeof(SharedSmem<D>);
    const hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_shared_kernel<D, PARTS, NB>), lds, done);
    if (e != hipSuccess) return e;
    // (the items of the 8 XCDs' runs: up to 7 more numbers than items)
    hipLaunchKernelGGL((attn_shared_kernel<D, PARTS, NB>), dim3((unsigned)((p.items + 7) / 8 * 8)), dim3(64 * kWaves), lds, st, p);
    return hipGetLastError();
}

template <int D, int PARTS> static hipError_t launch_d(const SharedParams& p, const SharedPlan& x, hipStream_t st) {
    hipError_t e = p.width == 64 ? launch_shared<D, PARTS, 2>(p, st) : launch_shared<D, PARTS, 1>(p, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_own_kernel<D, PARTS>), dim3((unsigned)(x.own_items * p.own_splits)), dim3(64), 0,
                       st, p);
    e = hipGetLastError();
    if (e != hipSuccess || p.own_splits == 1) return e;
    hipLaunchKernelGGL(attn_shared_join<D>, dim3((unsigned)((long long)p.N * p.Hq)), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_attn_shared(const SharedParams& p, const SharedPlan& x, hipStream_t st) {
    static std::atomic<unsigned long long> done{0};
    hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_shared_plan_kernel), (kMostGroups + 1) * (int)sizeof(PlanGroup), done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attn_shared_plan_kernel, dim3(1), dim3(kPlanThreads), (unsigned)((p.groups + 1) * sizeof(PlanGroup)), st, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool one = (p.flags & GDR_OUT_BF16) != 0;
    if (p.d == 64) return one ? launch_d<64, 1>(p, x, st) : launch_d<64, 2>(p, x, st);
    return one ? launch_d<128, 1>(p, x, st) : launch_d<128, 2>(p, x, st);
}

}  // namespace gdr
