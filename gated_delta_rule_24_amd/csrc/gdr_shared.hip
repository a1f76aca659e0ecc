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

// a / b of numbers from 0 on; 64-bit divisions take some hundred instructions
__device__ __forceinline__ long long div_of(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}
// tiles of `width` (32 or 64) that these rows take
__device__ __forceinline__ int tiles_of_rows(const SharedParams& p, long long rows) {
    const int shift = p.width == 64 ? 6 : 5;
    return (int)((rows + (1 << shift) - 1) >> shift);
}

// What the plan makes of group g (see attn_shared_plan_kernel).  Unit kh * tiles + tile of it
// is `width` of its rows on a key head, over all its shared pages.
struct Group {
    int first, rows;            // its first sequence; rows: its (sequence, query head) pairs on a key head
    int pg0, pages;             // the shared pages that some row of it sees; 0: nothing shared
    int unit0;                  // its first unit's number
    int shared;                 // pages that it shares, seen or not
    long long pos0;             // the place of its first unit's pages in the line of all
};
static_assert(sizeof(Group) == 32, "read as two 16-byte loads");

__device__ __forceinline__ Group group_at(const void* groups, int g) {
    const int4* at = reinterpret_cast<const int4*>(groups) + 2 * (size_t)g;
    const int4 x = at[0], y = at[1];
    return Group{x.x, x.y, x.z, x.w, y.x, y.y, (long long)((uint64_t)(uint32_t)y.z | (uint64_t)(uint32_t)y.w << 32)};
}
struct PlanHead {
    int workgroups;
    int whole;                  // units are stretched to whole runs
    long long per;              // pages of a workgroup
};
__device__ __forceinline__ PlanHead plan_head(const SharedParams& p) { return *reinterpret_cast<const PlanHead*>(p.plan_head); }

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


// A sequence's own pages: begin .. end - 1, in runs of `per` (own_splits at the most; a short
// sequence has fewer, as a wave's start and end cost some pages' time).
constexpr int kOwnRun = 4;
struct OwnPages {
    int begin, end, per;
};
__device__ __forceinline__ OwnPages own_pages_of(const SharedParams& p, int n, int shared, int& lo, int& hi) {
    seen_range(p, n, lo, hi);
    OwnPages x;
    x.begin = max(lo / kPage, shared);
    x.end = max(x.begin, (int)(((long long)hi + kPage - 1) / kPage));
    x.per = max((int)(((uint32_t)(x.end - x.begin) + (uint32_t)p.own_splits - 1) / (uint32_t)p.own_splits), kOwnRun);
    return x;
}

// Joins what the workgroup's waves hold in LDS for the same `rows` rows, each relative to
// its own maximum; `put` gets four channels of a row at a time, with the row's maximum and sum.
template <int D, typename O, typename ML, typename F>
__device__ __forceinline__ void join_waves(const O& o, const ML& ml, int rows, F put) {
    for (int idx = threadIdx.x; idx < rows * (D / 4); idx += 64 * kWaves) {
        const int c = idx / (D / 4), ch = 4 * (idx % (D / 4));
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < kWaves; ++y) top = fmaxf(top, ml[y][c][0]);
        const float at = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4v x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
            const float f = __builtin_amdgcn_exp2f(ml[y][c][0] - at);
            sum += ml[y][c][1] * f;
            x += *reinterpret_cast<const float4v*>(&o[y][c][ch]) * f;
        }
        put(c, ch, x, make_float2(top, sum));
    }
}

}  // namespace

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------
//
// One workgroup looks at the groups, as the host does not know them, and lays the pages of all
// units end to end: each of as many workgroups as can be at work at once takes a run of the same
// length of that line, over the ends of units, so that all end together.  (With whole runs of each
// unit's pages, as many as fit, 3 groups of 340 rows on 256 pages keep 144 of 256
// workgroups: 119 us for the shared pages, over the ends 101, when a weight had one f16 part.)  Where
// whole runs of units are little longer they are taken: a unit's start and end cost some pages' time
// (16 groups of 4 39.3 us a call, never 40.6; 255 sequences behind 3 prompts 174 either way).
constexpr int kPlanThreads = 1024;
constexpr int kLonger = 8;                            // pages that a unit's start and end are worth

struct PlanGroup {
    int first, shared, lo, hi;  // first sequence; pages; first and one past the last token that some sequence sees
    int unit0;
    long long pos0;
};
// runs of `per` that a unit's pages take
__device__ __forceinline__ int runs_of(int pages, long long per) {
    return pages <= per ? 1 : (int)(((uint32_t)pages + (uint32_t)per - 1) / (uint32_t)per);
}
// Workgroups that the pages of all units are dealt to: two a compute unit only where each has many
// (64 rows a wave: 128 rows on 512 pages 49 us a call, with two 57; 256 on 125 39 and 44; 512 on 256 79
// and 78; 1,024 on 512 240 and 220).
constexpr int kShort = 64;
__device__ __forceinline__ int workgroups_for(const SharedParams& p, long long all) {
    return p.workgroups > 256 && all < (long long)p.workgroups * kShort ? 256 : p.workgroups;
}
// the pages that some sequence sees of a group's shared ones, whose tokens lo .. hi - 1 some see
__device__ __forceinline__ int pages_seen(int lo, int hi, int shared) {
    return max(0, min((int)(((long long)hi + kPage - 1) / kPage), shared) - lo / kPage);
}
__device__ __forceinline__ Group planned(int first, int rows, int pages, int lo, int shared, int unit0, long long pos0) {
    return Group{first, rows, pages > 0 ? lo / kPage : 0, pages, unit0, shared, pos0};
}

__global__ __launch_bounds__(kPlanThreads) void attn_shared_plan_kernel(SharedParams p) {
    extern __shared__ __attribute__((aligned(256))) char smem[];
    PlanGroup* s = reinterpret_cast<PlanGroup*>(smem);       // [groups + 1]
    __shared__ long long s_per;
    __shared__ int s_workgroups, s_whole, s_fits[kPlanThreads / 64];
    static_assert(kPlanThreads / 64 > kLonger, "a wave for each length");
    const int tid = threadIdx.x, lane = tid & 63, rep = p.Hq / p.Hkv, G = p.groups;
    int a0 = 0, b0 = 0;                               // of the first sequence it looks at: asked for before the groups
    if (tid < p.N) seen_range(p, tid, a0, b0);
    auto group_of = [&](int n) {                      // or -1
        int g = 0, z = G - 1;                         // the last start at or before n
        while (g < z) {
            const int mid = (g + z + 1) / 2;
            if (s[mid].first <= n) g = mid;
            else z = mid - 1;
        }
        return n >= s[g].first && n < s[g + 1].first ? g : -1;
    };
    for (int g = tid; g <= G; g += kPlanThreads)
        s[g] = PlanGroup{clampi(p.group_start[g], 0, p.N), g < G ? clampi(p.shared_pages[g], 0, p.max_pages) : 0, INT_MAX, 0, 0, 0};
    __syncthreads();
    // (bounds that fall are held where they were: no sequence is in two groups)
    if (tid < 64) {
        int top = 0;
        for (int g0 = 0; g0 <= G; g0 += 64) {
            int first = max(top, g0 + lane <= G ? s[g0 + lane].first : 0);
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(first, o, 64);
                if (lane >= o) first = max(first, y);
            }
            if (g0 + lane <= G) s[g0 + lane].first = first;
            top = __shfl(first, 63, 64);
        }
    }
    __syncthreads();
    for (int n = tid; n < p.N; n += kPlanThreads) {
        int a = a0, b = b0;
        if (n != tid) seen_range(p, n, a, b);
        const int g = group_of(n);
        if (g >= 0 && a < b) {
            atomicMin(&s[g].lo, a);
            atomicMax(&s[g].hi, b);
        }
    }
    __syncthreads();
    // one wave: where each group's units and pages start
    auto tiles_of = [&](int g) {
        return tiles_of_rows(p, (long long)(s[g + 1].first - s[g].first) * rep);
    };
    auto pages_of = [&](int g) { return pages_seen(s[g].lo, s[g].hi, s[g].shared); };
    auto sum_of = [&](auto f) {
        long long x = 0;
        for (int g = lane; g < G; g += 64) x += (long long)tiles_of(g) * p.Hkv * f(pages_of(g));
        for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
        return x;
    };
    // two pages a wave, as the second's keys are loaded beside the first one's work
    const long long all = sum_of([](int pages) { return (long long)pages; });
    const int workgroups = workgroups_for(p, all);
    long long per = max(div_of(all + workgroups - 1, workgroups), 2LL * kWaves);
    // a unit's start and end are worth some pages: whole runs of a unit where they are little
    // longer (each wave looks at another length)
    {
        const long long longer = per + (tid >> 6);
        const bool fits = sum_of([&](int pages) { return pages > 0 ? runs_of(pages, longer) : 0; }) <= workgroups;
        if (lane == 0) s_fits[tid >> 6] = fits;
    }
    __syncthreads();
    if (tid < 64) {
        bool whole = false;
        for (int i = 0; i <= kLonger && !whole; ++i)
            if (s_fits[i]) {
                whole = true;
                per += i;
            }
        long long units = 0, pos = 0;                 // of the groups before
        for (int g0 = 0; g0 < G; g0 += 64) {
            const int g = g0 + lane;
            const int pages = g < G ? pages_of(g) : 0;
            const long long u = pages > 0 ? (long long)tiles_of(g) * p.Hkv : 0;
            const long long mine = whole ? u * (runs_of(pages, per) * per) : u * pages;
            long long run = u, at = mine;
            for (int o = 1; o < 64; o <<= 1) {
                const long long y = __shfl_up(run, o, 64), z = __shfl_up(at, o, 64);
                if (lane >= o) { run += y; at += z; }
            }
            if (g < G) {
                s[g].unit0 = (int)(units + run - u);
                s[g].pos0 = pos + at - mine;
            }
            units += __shfl(run, 63, 64);
            pos += __shfl(at, 63, 64);
        }
        if (lane == 0) {
            s_per = per;
            s_whole = whole;
            s_workgroups = (int)div_of(pos + per - 1, per);
        }
    }
    __syncthreads();
    auto group = [&](int g) {
        return planned(s[g].first, (s[g + 1].first - s[g].first) * rep, pages_of(g), s[g].lo, s[g].shared, s[g].unit0, s[g].pos0);
    };
    for (int g = tid; g < G; g += kPlanThreads) reinterpret_cast<Group*>(p.plan_groups)[g] = group(g);
    // (each sequence its group's, so that nobody has to look up which one that is)
    for (int n = tid; n < p.N; n += kPlanThreads) {
        const int g = group_of(n);
        reinterpret_cast<Group*>(p.plan_sequences)[n] = g >= 0 ? group(g) : Group{0, 0, 0, 0, 0, 0, 0};
    }
    for (int w = tid; w < s_workgroups; w += kPlanThreads) { // the last group that starts at or before this one's run
        int g = 0, z = G - 1;
        while (g < z) {
            const int mid = (g + z + 1) / 2;
            if (s[mid].pos0 <= w * s_per) g = mid;
            else z = mid - 1;
        }
        p.plan_items[w] = g;
    }
    if (tid == 0) {
        PlanHead* head = reinterpret_cast<PlanHead*>(p.plan_head);
        head->workgroups = s_workgroups;
        head->whole = s_whole;
        head->per = s_per;
    }
}

// The same in each workgroup for itself, a group a lane, where there are few groups and
// sequences: a plan kernel takes 5.5 to 9 us before the others start.  (4 sequences behind 300
// tokens 17.5 us a call, with a plan kernel 19.5; 16 groups of 4 39 to 40.5 and 43; 64 of 16 52.5 and
// 57.  Not with 64 rows a wave: the registers of the products have no room left, and scratch
// memory in the pages' loop costs more than the plan.)
constexpr int kFewGroups = 64, kFewSequences = 1024;
struct LanePlan {
    PlanHead head;
    Group group;                // lane g's: group g
    int end;                    // one past the last group's last sequence
};
struct LaneScratch {
    int first[kFewGroups], lo[kFewGroups], hi[kFewGroups], fits[16];
};
// first sequence of lane g's group, as the plan kernel has it, and its end in `next`
__device__ __forceinline__ int lane_bounds(const SharedParams& p, int lane, int& next) {
    const int G = p.groups;
    int first = lane < G ? clampi(p.group_start[lane], 0, p.N) : 0, end = clampi(p.group_start[G], 0, p.N);
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(first, o, 64);
        if (lane >= o) first = max(first, y);
    }
    end = max(end, __shfl(first, 63, 64));
    next = __shfl_down(first, 1, 64);
    if (lane >= G - 1) next = end;
    return first;
}
template <int THREADS>
__device__ __forceinline__ LanePlan lane_plan(const SharedParams& p, char* smem) {
    LaneScratch& s = *reinterpret_cast<LaneScratch*>(smem);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));                     // (what follows from it is not kept between two plans)
    const int lane = tid & 63, rep = p.Hq / p.Hkv, G = p.groups;
    int next;
    const int shared = lane < G ? clampi(p.shared_pages[lane], 0, p.max_pages) : 0;
    const int first = lane_bounds(p, lane, next), end = __shfl(next, 63, 64);
    if (tid < 64) { s.first[lane] = first; s.lo[lane] = INT_MAX; s.hi[lane] = 0; }
    __syncthreads();
    for (int n = tid; n < p.N; n += THREADS) {
        int a, b;
        seen_range(p, n, a, b);
        int g = 0, z = G - 1;                         // the last start at or before n
        while (g < z) {
            const int mid = (g + z + 1) / 2;
            if (s.first[mid] <= n) g = mid;
            else z = mid - 1;
        }
        if (a < b && n >= s.first[g] && n < (g + 1 < G ? s.first[g + 1] : end)) {
            atomicMin(&s.lo[g], a);
            atomicMax(&s.hi[g], b);
        }
    }
    __syncthreads();
    const int lo = s.lo[lane], pages = lane < G ? pages_seen(lo, s.hi[lane], shared) : 0, rows = lane < G ? (next - first) * rep : 0;
    const int u = pages > 0 ? tiles_of_rows(p, rows) * p.Hkv : 0;
    long long all = (long long)u * pages;
    for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o, 64);
    const int workgroups = workgroups_for(p, all);
    long long per = max(div_of(all + workgroups - 1, workgroups), 2LL * kWaves);
    for (int i = tid >> 6; i <= kLonger; i += THREADS / 64) {
        int runs = pages > 0 ? (int)min((long long)u * runs_of(pages, per + i), 1LL << 20) : 0;
        for (int o = 32; o > 0; o >>= 1) runs += __shfl_xor(runs, o, 64);
        if (lane == 0) s.fits[i] = runs <= workgroups;
    }
    __syncthreads();
    bool whole = false;
    for (int i = 0; i <= kLonger && !whole; ++i)
        if (s.fits[i]) {
            whole = true;
            per += i;
        }
    const long long mine = whole ? u * (runs_of(pages, per) * per) : (long long)u * pages;
    long long at = mine;
    int run = u;
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(run, o, 64);
        const long long z = __shfl_up(at, o, 64);
        if (lane >= o) { run += y; at += z; }
    }
    LanePlan x;
    x.head.workgroups = (int)div_of(__shfl(at, 63, 64) + per - 1, per);
    x.head.whole = whole;
    x.head.per = per;
    x.group = planned(first, rows, pages, lo, shared, run - u, at - mine);
    x.end = end;
    __syncthreads();                                  // (the scratch is free)
    return x;
}
__device__ __forceinline__ Group group_of_lane(const Group& x, int g) {
    auto get = [&](int v) { return __builtin_amdgcn_readlane(v, g); };
    const uint32_t lo = (uint32_t)get((int)(uint32_t)x.pos0), hi = (uint32_t)get((int)(uint32_t)(x.pos0 >> 32));
    return Group{get(x.first), get(x.rows), get(x.pg0), get(x.pages), get(x.unit0), get(x.shared),
                 (long long)((uint64_t)lo | (uint64_t)hi << 32)};
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
// have the same rows and take pages in turn, each for itself (times here, but for the last, are
// of weights in one f16 part): with waves that shared a page and waited for each other at every
// one, 1,024 rows on 512 pages took 215 us for 181.  Pages come to a wave's place in LDS as they lie in memory, by direct loads (no
// registers, 1 KiB an instruction; read straight to registers in the operands'
// order, 16 bytes a lane from 32 rows, the same walk took 265): the next page's keys when
// this one's are read, its values when these are.  With one place and the queries in LDS,
// two waves of 256 registers are on a SIMD: 170 us, and with weights in two parts 220, of which
// the products' share at the matrix cores' peak is 82.  A page takes a wave 96 products of 32 cycles,
// and beside them the conversions of its bytes, 64 exponentials and those weights' conversions to two
// parts.  For 255 sequences behind 3 prompts a SIMD's vector instructions take 53% of the cycles and
// its products 36%, 89% together: neither is full, what bounds it is that they hardly overlap.  A
// page's score products all come first, then the maxima, then exponentials and value products, and
// two waves in the same phase have nothing for the other unit.
//
// Workgroups for sequences' own pages, which memory bounds, stand on the compute units beside
// these, two a unit: one kernel after the other took 101 and 75 us for 255 sequences
// behind 3 prompts, both together 128 (with one f16 part a weight).
//
// A weight is exp2(s - m).  For the product with v it is taken times 2^b, b = 12 +
// log2 v_scale + m - wm, wm the running maximum of s + log2 v_scale, so that it has
// its f16 bits whatever the pages' scales: as the sum of two f16 values, 22 bits, as
// gdr_attn_decode has it.  (As one, 11 bits, 255 sequences behind 3 prompts take 149 us for 174,
// but 9% of bf16 results are then another value than the fp32 ones rounded.)  The
// sum takes the same exponentials, times 2^-b once a page; where |b| is large (a page of
// zeros has a scale of 2^-96) it has its own.
template <int D, int NB>
struct __attribute__((aligned(256))) SharedSmem {
    union {
        struct {
            uint8_t page[kWaves][2 * kPage * D];      // keys [64][D], then values [4][D][16]
            uint4 q[NB * D / 16][64];                 // queries, operand by operand
        };
        struct {
            float o[kWaves][32][D + 4];
            float ml[kWaves][32][2];
            int nans[kWaves];
        };
    };
};
static_assert(sizeof(SharedSmem<128, 2>) <= 80 * 1024, "two workgroups' (and no LDS beside it)");

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
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint2v read8(uint32_t at) { return *(const __attribute__((address_space(3))) uint2v*)(uintptr_t)at; }
__device__ __forceinline__ uint4v read16(uint32_t at) { return *(const __attribute__((address_space(3))) uint4v*)(uintptr_t)at; }

// pages of the line that one of group x's units takes
__device__ __forceinline__ long long length_of(const PlanHead& head, const Group& x) {
    return head.whole ? div_of(x.pages + head.per - 1, head.per) * head.per : x.pages;
}

// all but the last N of this wave's loads have arrived
template <int N> __device__ __forceinline__ void wait_but() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// A sequence's own pages: up to 16 of its query heads on a key head are the columns of 16 x 16
// products (as attn_decode_kernel has them).  A wave has a run of the pages of one, and
// loads each page while it works on the one before: a few pages a sequence are too few
// to be dealt to four waves, whose starts and joins took as long as the pages.
template <int D, bool FEW>
__device__ __forceinline__ void own_pages(const SharedParams& p, int w, uint32_t place, int lane) {
    constexpr int KS = D / 64;                        // 64-channel steps of a key row
    constexpr int VT = D / 16;                        // 16-channel tiles of the output
    const int col = lane & 15, g = lane >> 4;
    const int rep = p.Hq / p.Hkv, sets = (rep + 15) / 16;
    const int qg = w % sets; w /= sets;
    const int kh = w % p.Hkv; w /= p.Hkv;
    const int n = w % p.N, run = w / p.N;
    const int q0 = kh * rep + 16 * qg, nq = min(16, rep - 16 * qg);
    int shared;
    if constexpr (FEW) {
        const int pages = lane < p.groups ? clampi(p.shared_pages[lane], 0, p.max_pages) : 0;
        int next;
        const int first = lane_bounds(p, lane, next);
        const uint64_t in = __ballot(lane < p.groups && first <= n && n < next);
        shared = in ? __builtin_amdgcn_readlane(pages, __builtin_ctzll(in)) : 0;
    } else {
        shared = group_at(p.plan_sequences, n).shared;
    }
    int lo, hi;
    const OwnPages mine = own_pages_of(p, n, shared, lo, hi);
    const long long begin = mine.begin + (long long)run * mine.per;
    if (begin >= mine.end) return;                    // (the join does not read it)
    const int pg0 = __builtin_amdgcn_readfirstlane((int)begin), pg1 = __builtin_amdgcn_readfirstlane(min((int)begin + mine.per, mine.end));
    const int count = pg1 - pg0;
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
    constexpr uint32_t kSide = kPage * D;
    // (an absent page is read as the first one)
    auto page_at = [&](int k) { return ((size_t)max(__builtin_amdgcn_readlane(e_page, k & 63), 0) * p.Hkv + kh) * kSide; };
    look_up(0);
    loader.keys((uint64_t)p.k_cache + page_at(0), place);
    loader.values((uint64_t)p.v_cache + page_at(0), place + kSide);
    const int krow = 16 * (col >> 2) + (col & 3);     // key of tile 0's row `col`; its flip is that of the others, + 4 t, too
    const uint32_t at_k = place + krow * D + 16 * (g ^ key_flip<D, true>(krow)), at_v = place + kSide + (g * D + col) * 16;

    float4v o[VT];
#pragma unroll
    for (int j = 0; j < VT; ++j) o[j] = float4v{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f, wm = -INFINITY;
    const float to2 = p.scale * 1.4426950408889634f;
    for (int k = 0; k < count; ++k) {
        const int page = __builtin_amdgcn_readlane(e_page, k & 63);
        const float k_scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_ks), k & 63));
        const float v_scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_vs), k & 63));
        // the keys are there: what was asked for behind them are values
        wait_but<PageLoader<D, true>::N>();
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
        // the keys are read: the next page's take their place, then the values'
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const bool more = k + 1 < count;
        if (more) {
            if (((k + 1) & 63) == 0) look_up(k + 1);
            loader.keys((uint64_t)p.k_cache + page_at(k + 1), place);
            wait_but<PageLoader<D, true>::N>();
        } else {
            wait_but<0>();
        }
#pragma unroll
        for (int j = 0; j < VT; ++j) vv[j] = read16(at_v + 256 * j);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (more) loader.values((uint64_t)p.v_cache + page_at(k + 1), place + kSide);
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
                w_lo[t >> 1][(t & 1) * 4 + i] = (_Float16)(z - (float)a);
            }
#pragma unroll
        for (int j = 0; j < VT; ++j) {
            const half8 v0 = e4m3x8_to_f16(vv[j].x, vv[j].y), v1 = e4m3x8_to_f16(vv[j].z, vv[j].w);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w_hi[0], o[j], 0, 0, 0);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w_hi[1], o[j], 0, 0, 0);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w_lo[0], o[j], 0, 0, 0);
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w_lo[1], o[j], 0, 0, 0);
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
#pragma unroll
    for (int j = 0; j < VT; ++j) *reinterpret_cast<float4v*>(&p.own_o[(run * heads + head) * D + 16 * j + 4 * g]) = o[j];
    if (g == 0) *reinterpret_cast<float2*>(&p.own_ml[(run * heads + head) * 2]) = make_float2(m, l);
}

template <int D, int NB, bool FEW>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_shared_kernel(SharedParams p) {
    constexpr int KL = D / 32;                        // 16-byte reads of a key's row by a lane
    constexpr int DB = D / 32;                        // 32-channel tiles of the output
    constexpr int kRows = 32 * NB;                    // of the workgroup: its waves have the same ones
    extern __shared__ __attribute__((aligned(256))) char smem[];
    SharedSmem<D, NB>& sm = *reinterpret_cast<SharedSmem<D, NB>*>(smem);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rep = p.Hq / p.Hkv;

    // a workgroup for shared pages for each of 256 compute units and one for own ones by turns,
    // as long as there are both (255 sequences behind 3 prompts 174 us; all of the first kind
    // before the others 175, and 163 for 147 when a weight had one f16 part; by turns of 8, as shader
    // engines are taken one after the other, half of them get all of the first kind: 216)
    constexpr int kTurn = 256 / 8;
    int number = blockIdx.x / 8;
    const int some = p.workgroups / 8, turns = min(some, (int)(gridDim.x / 8) - some) / kTurn;
    bool own = number / kTurn & 1;
    if (number < 2 * turns * kTurn) {
        number = number / (2 * kTurn) * kTurn + number % kTurn;
    } else {
        number -= turns * kTurn;
        own = number >= some;
        if (own) number -= some - turns * kTurn;
    }
    if (own) {
        const long long w = (long long)(8 * number + blockIdx.x % 8) * kWaves + wave;
        if (w < p.own_runs) own_pages<D, FEW>(p, (int)w, attn::lds_address(sm.page[wave]), threadIdx.x & 63);
        return;
    }
    // consecutive workgroups go round the 8 XCDs: each of these takes a run of them, the
    // tiles that share pages one after the other
    PlanHead head;
    int wg, group;
    Group x;
    if constexpr (FEW) {
        const LanePlan plan = lane_plan<64 * kWaves>(p, smem);
        head = plan.head;
        if (blockIdx.x == 0) {
            // for the join
            if (threadIdx.x == 0) *reinterpret_cast<PlanHead*>(p.plan_head) = head;
            for (int n0 = 0; n0 < p.N; n0 += 64 * kWaves) {
                const int n = n0 + threadIdx.x;
                int g = -1;
                for (int i = 0; i < p.groups; ++i) {
                    const int first = __builtin_amdgcn_readlane(plan.group.first, i);
                    const int end = i + 1 < p.groups ? __builtin_amdgcn_readlane(plan.group.first, i + 1) : plan.end;
                    if (n >= first && n < end) g = i;
                }
                auto get = [&](int v) { return __shfl(v, max(g, 0), 64); };
                const int pos_lo = get((int)(uint32_t)plan.group.pos0), pos_hi = get((int)(uint32_t)(plan.group.pos0 >> 32));
                const Group y = {get(plan.group.first), get(plan.group.rows), get(plan.group.pg0), get(plan.group.pages), get(plan.group.unit0),
                                 get(plan.group.shared), (long long)((uint64_t)(uint32_t)pos_lo | (uint64_t)(uint32_t)pos_hi << 32)};
                if (n < p.N) reinterpret_cast<Group*>(p.plan_sequences)[n] = g >= 0 ? y : Group{0, 0, 0, 0, 0, 0, 0};
            }
        }
        const int each = (head.workgroups + 7) / 8;
        wg = (blockIdx.x % 8) * each + number;
        if (number >= each || wg >= head.workgroups) return;
        // the last group that starts at or before this run: it has pages
        const int lane = threadIdx.x & 63;
        group = 63 - __builtin_clzll(__ballot(lane < p.groups && plan.group.pos0 <= wg * head.per));
        x = group_of_lane(plan.group, group);
    } else {
        head = plan_head(p);
        const int each = (head.workgroups + 7) / 8;
        wg = (blockIdx.x % 8) * each + number;
        if (number >= each || wg >= head.workgroups) return;
        group = p.plan_items[wg];
        x = group_at(p.plan_groups, group);
    }
    // the unit and its page that the run starts with, and the run's length
    long long left = head.per, length = length_of(head, x);
    int unit, page0;
    {
        const long long rel = wg * head.per - x.pos0;
        unit = (int)div_of(rel, length);
        page0 = (int)(rel - unit * length);
    }
    for (;;) {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));                    // (what follows from it is not kept over the units)
        const int col = lane & 31, h = lane >> 5;
        const int tiles = (x.rows + kRows - 1) / kRows, tile = unit % tiles, kh = __builtin_amdgcn_readfirstlane(unit / tiles);
        const int row0 = kRows * tile, rows = min(kRows, x.rows - row0);
        const int pg0 = __builtin_amdgcn_readfirstlane(x.pg0 + page0);
        const int pg1 = __builtin_amdgcn_readfirstlane((int)min((long long)pg0 + left, (long long)x.pg0 + x.pages));
        const size_t part0 = (size_t)(x.unit0 + unit + wg) * kRows;
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
        const uint32_t place = attn::lds_address(sm.page[wave]);
        constexpr uint32_t kSide = kPage * D;
        // (an absent page is read as the first one: its bytes are masked)
        auto page_at = [&](int k) { return ((size_t)max(__builtin_amdgcn_readlane(e_page, k & 63), 0) * p.Hkv + kh) * kSide; };
        look_up(0);
        if (n > 0) {
            const PageLoader<D, false> loader(lane);
            loader.keys((uint64_t)p.k_cache + page_at(0), place);
            loader.values((uint64_t)p.v_cache + page_at(0), place + kSide);
        }

        // this lane's rows: their queries (channels 32 s + 16 h .. + 15) and the keys they see
        int lo_most = 0, hi_least = INT_MAX, lo_least = INT_MAX, hi_most = 0;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            const int mine = 32 * c + col;
            const bool live = mine < rows;
            const int seq = x.first + (row0 + mine) / rep, head = kh * rep + (row0 + mine) % rep;
            for (int s = wave; s < 2 * KL; s += kWaves) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live)
                    u = *reinterpret_cast<const uint4*>((const uint16_t*)p.q + ((size_t)seq * p.Hq + head) * D + 32 * (s / 2) + 16 * h + 8 * (s % 2));
                sm.q[2 * KL * c + s][lane] = u;
            }
            if (live) {
                int lo, hi;
                seen_range(p, seq, lo, hi);
                lo_most = max(lo_most, lo);
                lo_least = min(lo_least, lo);
                hi_least = min(hi_least, hi);
                hi_most = max(hi_most, hi);
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
        lo_least = __builtin_amdgcn_readfirstlane(lo_least);
        hi_most = __builtin_amdgcn_readfirstlane(hi_most);

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
        // (the pages' loads go on)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

        uint32_t nans = 0;                                // some value that not every row sees is NaN
        for (int k = 0; k < n; ++k) {
            const int page = __builtin_amdgcn_readlane(e_page, k & 63);
            const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_ks), k & 63));
            const float vs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e_vs), k & 63));
            const int at0 = (pg0 + wave + k * kWaves) * kPage;
            const bool absent = page < 0;
            // A lane's places are made anew for each page: kept over the loop some of them would be
            // in scratch memory, and a wait for what is read from there is one for the page's
            // loads as well.
            int mine = lane;
            asm volatile("" : "+v"(mine));
            const PageLoader<D, false> loader(mine);
            const int tok = 16 * ((mine >> 2) & 1) + 4 * ((mine & 31) >> 3) + (mine & 3);
            const uint32_t k_at = place + tok * D + 16 * ((mine >> 5) ^ key_flip<D, false>(tok));   // its reads of keys, to flip by 32 s
            const uint32_t v_at = place + kSide + ((mine >> 5) * D + (mine & 31)) * 16, q_at = attn::lds_address(sm.q) + 16 * mine;
            // the keys are there: what was asked for behind them are values
            wait_but<PageLoader<D, false>::N>();
            float16v st[NB][2];
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 16; ++j) st[c][b][j] = 0.f;
#pragma unroll
            for (int s = 0; s < KL; ++s) {
                uint4v kr[2], qr[NB][2];
#pragma unroll
                for (int b = 0; b < 2; ++b) kr[b] = read16((k_at ^ (32 * s)) + 32 * b * D);
#pragma unroll
                for (int c = 0; c < NB; ++c)
#pragma unroll
                    for (int f = 0; f < 2; ++f) qr[c][f] = read16(q_at + 1024 * (2 * KL * c + 2 * s + f));
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bf8v k0 = e4m3x8_to_bf16(kr[b].x, kr[b].y), k1 = e4m3x8_to_bf16(kr[b].z, kr[b].w);
#pragma unroll
                    for (int c = 0; c < NB; ++c) st[c][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k0, __builtin_bit_cast(bf8v, qr[c][0]), st[c][b], 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < NB; ++c) st[c][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k1, __builtin_bit_cast(bf8v, qr[c][1]), st[c][b], 0, 0, 0);
                }
            }
            // the keys are read: the next page's take their place while these values are worked on
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (k + 1 < n) {
                if (((k + 1) & 63) == 0) look_up(k + 1);
                loader.keys((uint64_t)p.k_cache + page_at(k + 1), place);
            }
            // (the values are older than these, where there are any)
            auto wait_values = [&] {
                if (k + 1 < n) wait_but<PageLoader<D, false>::N>();
                else wait_but<0>();
            };

            float by = ks * to2;                          // a score is st times this
            const bool edge = absent || at0 < lo_most || at0 + kPage > hi_least;
            if (edge || !(by >= 0.f)) {
                // (negative scales turn the order of the scores; masked ones stay -inf whatever the scale)
                asm volatile("");
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    uint32_t sees = 0;                    // (looked up again: few pages are read in part)
                    if (edge && !absent && 32 * c + col < rows) {
                        int lo, hi;
                        seen_range(p, x.first + (row0 + 32 * c + col) / rep, lo, hi);
                        sees = seen_bits(at0 + 16 * h, lo, hi);
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        st[c][b] *= by;
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) st[c][b][i] = sees >> (16 * b + i) & 1 ? st[c][b][i] : -INFINITY;
                        }
                    }
                }
                by = 1.f;
                if (edge) {
                    // some row sees the page in part: values of keys that no row sees count as 0,
                    // and so do NaNs, which the 0 of a row that does not see them would carry
                    // over: the rows that see them get them at the end
                    // (in LDS: a lane writes what it will read)
                    const uint32_t some = absent ? 0 : seen_bits(at0 + 16 * h, lo_least, hi_most);
                    wait_values();
                    for (int i = 0; i < 2 * DB; ++i) {
                        const int b = i & 1;
                        const uint32_t at = v_at + (2 * b * D + 16 * (i & ~1)) * 16;
                        uint4v u = read16(at);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t y = u[t] & bytes_of(some, 16 * b + 4 * t);
                            const uint32_t whole = (nan_bytes(y) >> 7) * 0xffu;
                            nans |= whole;
                            u[t] = y & ~whole;
                        }
                        *(__attribute__((address_space(3))) uint4v*)(uintptr_t)at = u;
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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
            bool far[NB], some_far = false;
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                const float at = m[c] == -INFINITY ? 0.f : m[c], wat = wm[c] == -INFINITY ? 0.f : wm[c];
                up[c] = none[c] ? 0.f : log_vs - wat + kTop;
                share[c] = none[c] ? 0.f : __builtin_amdgcn_exp2f(-(up[c] + at));
                far[c] = !none[c] && !(fabsf(up[c] + at) <= 60.f);
                some_far = some_far || far[c];
            }
            if (__any(some_far)) {
                // the sum's own exponentials, for the rows that need them
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    const float at = m[c] == -INFINITY ? 0.f : m[c];
                    float sum = 0.f;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            sum += __builtin_amdgcn_exp2f(__builtin_fmaf(st[c][b][i], by, -at));
                            asm volatile("" : "+v"(sum));     // (one after the other: no registers for it)
                        }
                    l[c] += far[c] ? sum : 0.f;
                    share[c] = far[c] ? 0.f : share[c];
                }
            }

            wait_values();
            // (16 keys of the page at a time: the two parts of 32 keys' weights do not fit into the registers)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    half8 w_hi[NB], w_lo[NB];
#pragma unroll
                    for (int c = 0; c < NB; ++c) {
                        float sum[2] = {0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(st[c][b][8 * f + i], by, up[c]));
                            sum[i & 1] += w;
                            const _Float16 a = (_Float16)w;
                            w_hi[c][i] = a;
                            w_lo[c][i] = (_Float16)(w - (float)a);
                        }
                        l[c] += (sum[0] + sum[1]) * share[c];
                    }
#pragma unroll
                    for (int i = 0; i < DB; ++i) {
                        const uint2v u = read8(v_at + (2 * b * D + 32 * i) * 16 + 8 * f);
                        const half8 v = e4m3x8_to_f16(u.x, u.y);
#pragma unroll
                        for (int c = 0; c < NB; ++c) o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w_hi[c], o[c][i], 0, 0, 0);
#pragma unroll
                        for (int c = 0; c < NB; ++c) o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w_lo[c], o[c][i], 0, 0, 0);
                    }
                }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (k + 1 < n) loader.values((uint64_t)p.v_cache + page_at(k + 1), place + kSide);
        }

        // the waves that had the same rows join, in LDS, 32 rows at a time: no load into it is
        // left, and no read of the ring
        attn::wait_loads();
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            lds_barrier();
            l[c] = sum_across32(l[c]);
            if (h == 0) { sm.ml[wave][col][0] = m[c]; sm.ml[wave][col][1] = l[c]; }
            if (c == 0) sm.nans[wave] = __any(nans != 0);
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
            const size_t part = part0 + 32 * c;
            join_waves<D>(sm.o, sm.ml, min(32, rows - 32 * c), [&](int r, int ch, float4v y, float2 ml) {
                *reinterpret_cast<float4v*>(&p.part_o[(part + r) * D + ch]) = y;
                if (ch == 0) *reinterpret_cast<float2*>(&p.part_ml[(part + r) * 2]) = ml;
            });
        }
        int any_nans = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) any_nans |= sm.nans[w];
        __syncthreads();                                  // (LDS is free again, what was joined is written)
        if (any_nans) {
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
                        if (j >= a && j < b) p.part_o[(part0 + r) * D + ch] = NAN;
                    }
                }
            }
        }
        // the next unit
        left -= length - page0;
        if (left <= 0) return;
        page0 = 0;
        if (++unit == tiles * p.Hkv) {
            unit = 0;
            if constexpr (FEW) {
                // (made again: kept, the groups would take registers that the pages' products need)
                const LanePlan plan = lane_plan<64 * kWaves>(p, smem);
                int lane = threadIdx.x & 63;
                asm volatile("" : "+v"(lane));
                const uint64_t later = __ballot(lane < p.groups && lane > group && plan.group.pages > 0);
                if (later == 0) return;
                group = __builtin_ctzll(later);
                x = group_of_lane(plan.group, group);
            } else {
                do {
                    if (++group >= p.groups) return;
                    x = group_at(p.plan_groups, group);
                } while (x.pages == 0);
            }
            length = length_of(head, x);
        }
    }
}

// ---------------------------------------------------------------------------
// the join
// ---------------------------------------------------------------------------

// where the partial results of a row's shared pages are: those of a unit's pages, cut at the
// ends of the workgroups' runs, lie one after the other
struct Parts {
    size_t first;
    int n;
};
__device__ __forceinline__ Parts parts_of(const SharedParams& p, const Group& x, int kh, int row) {
    if (x.pages == 0) return {0, 0};
    const PlanHead head = plan_head(p);
    const int unit = kh * tiles_of_rows(p, x.rows) + (row >> (p.width == 64 ? 6 : 5));
    const long long at = x.pos0 + unit * length_of(head, x);
    const long long w0 = div_of(at, head.per), w1 = div_of(at + x.pages - 1, head.per);
    return {(size_t)(x.unit0 + unit + w0) * p.width + (row & (p.width - 1)), (int)(w1 - w0) + 1};
}

// Joins a head's partial results: THREADS for a head, in 4 THREADS / D groups of lanes, four
// channels a lane; each takes every so many of the results with a running maximum, four at a
// time, maxima and outputs asked for together.
template <int D, int THREADS>
__global__ __launch_bounds__(THREADS) void attn_shared_join(SharedParams p) {
    constexpr int GROUPS = 4 * THREADS / D, kAtOnce = 4;
    __shared__ float s_x[GROUPS][D], s_ml[GROUPS][2];
    const size_t head = blockIdx.x, heads = (size_t)p.N * p.Hq;
    const int tid = threadIdx.x, gi = tid / (D / 4), ch = 4 * (tid % (D / 4));
    const int n = (int)(head / p.Hq), hq = (int)(head % p.Hq), rep = p.Hq / p.Hkv;
    const Group x = group_at(p.plan_sequences, n);
    const Parts parts = parts_of(p, x, hq / rep, (n - x.first) * rep + hq % rep);
    int lo, hi;
    const OwnPages own = own_pages_of(p, n, x.shared, lo, hi);
    const int slots = parts.n + (int)((uint32_t)(own.end - own.begin + own.per - 1) / (uint32_t)own.per);
    float top = -INFINITY, sum = 0.f;
    float4v y = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = gi; s0 < slots; s0 += kAtOnce * GROUPS) {
        float2 ml[kAtOnce];
        float4v part[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int s = min(s0 + i * GROUPS, slots - 1);
            const bool shared = s < parts.n;
            const size_t at = shared ? parts.first + s * (size_t)p.width : (s - parts.n) * heads + head;
            ml[i] = *reinterpret_cast<const float2*>((shared ? p.part_ml : p.own_ml) + 2 * at);
            part[i] = *reinterpret_cast<const float4v*>((shared ? p.part_o : p.own_o) + at * D + ch);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int s = s0 + i * GROUPS;
            if (s >= slots) continue;
            const float both = fmaxf(top, ml[i].x), at = both == -INFINITY ? 0.f : both;
            const float f = __builtin_amdgcn_exp2f(top - at), g = __builtin_amdgcn_exp2f(ml[i].x - at);
            sum = sum * f + ml[i].y * g;
            y = y * f + part[i] * g;
            top = both;
        }
    }
    *reinterpret_cast<float4v*>(&s_x[gi][ch]) = y;
    if (ch == 0) { s_ml[gi][0] = top; s_ml[gi][1] = sum; }
    __syncthreads();
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) top = fmaxf(top, s_ml[i][0]);
    const float at = top == -INFINITY ? 0.f : top;
    for (int c = tid; c < D; c += THREADS) {
        float z = 0.f, all = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const float f = __builtin_amdgcn_exp2f(s_ml[i][0] - at);
            z += s_x[i][c] * f;
            all += s_ml[i][1] * f;
        }
        store_out(p, head * D + c, all == 0.f && !(z != z) ? 0.f : z / all);            // (0: nothing seen)
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
    int pages = max_pages;
    if (window > 0 && window / kPage + 2 < pages) pages = window / kPage + 2;
    // Rows of a wave: 64 share what a page costs beside its products, 32 start and end sooner and
    // plan for themselves (not by the lengths, which the host does not know, nor by single groups).  160
    // rows on 256 pages 40 us a call, with 64 a wave 49; 256 on 125 32 and 39; on 256 47 and 51; 340 of
    // each of 3 groups 190 and 176; 512 on 256 81 and 79; 128 on 512 48 and 49, on 1,563 129 and 114.
    x.width = each > 256 || (each > 64 && pages > 1024) ? 64 : 32;
    // at most: every group's last tile has one row
    const long long some = groups < N ? groups : N;
    const long long tiles = (rows + some * (x.width - 1)) / x.width;
    x.units = tiles * Hkv;
    // Two workgroups a compute unit where 64 rows share a page's bytes and the products count
    // (1,024 rows on 512 pages: 220 us, with one 240); one where the bytes do and every cut
    // costs a start and an end (16 groups of 4 on 63 pages 39 to 40.5, with two 43.7; 32 rows on 512
    // pages 26.6 and 30.1).
    x.workgroups = x.width == 64 ? 512 : 256;
    x.few = x.width == 32 && groups <= kFewGroups && N <= kFewSequences;
    x.own_items = (long long)N * Hkv * ((rep + 15) / 16);
    // Four waves a SIMD, and those of short sequences end at once: 255 sequences of up to 2,000 own
    // tokens behind 3 prompts of up to 4,000 154 us a call (with one a SIMD 173), of up to 1,000
    // behind up to 16,384 174 (178), behind none 86 (88); 60 of up to 4,000 67 (67), 64 of 200 17.4 (17.7).
    long long s = (4096 + x.own_items / 2) / x.own_items;
    const long long most = (pages + kOwnRun - 1) / kOwnRun;
    if (s > most) s = most;
    x.own_splits = s < 1 ? 1 : (int)s;
    // the workspace: plan, then partial results
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t y = at; at += up(bytes); return y; };
    x.at_head = take(16);
    x.at_groups = take(sizeof(Group) * (size_t)groups);
    x.at_sequences = take(sizeof(Group) * (size_t)N);
    x.at_items = take(4 * (size_t)x.workgroups);
    x.at_part_o = take(4 * (size_t)(x.units + x.workgroups) * x.width * d);
    x.at_part_ml = take(8 * (size_t)(x.units + x.workgroups) * x.width);
    const size_t own = (size_t)x.own_splits * N * Hq;
    x.at_own_o = take(4 * own * d);
    x.at_own_ml = take(8 * own);
    x.bytes = at;
    return x;
}

// the most that is numbered in 32 bits: waves for own pages, units and their parts, heads
long long attn_shared_workgroups(const SharedPlan& x, long long heads) {
    long long most = x.own_items * x.own_splits + 8LL * kWaves * (x.workgroups + 1);
    if (x.units + x.workgroups > most) most = x.units + x.workgroups;
    return heads > most ? heads : most;
}

// One wave a head in the join where there are many, else four: 8,160 heads 9.1 us, with four 19.9;
// 2,048: 4.6 and 6.2; 1,024 of some 30 parts: 7.6 and 6.4; 256 of some 70: 9.6 and 5.1.
constexpr long long kHeadsOfWaves = 2048;
template <int D, int NB, bool FEW> static hipError_t launch_shared(const SharedParams& p, hipStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const int lds = (int)sizeof(SharedSmem<D, NB>);
    const hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_shared_kernel<D, NB, FEW>), lds, done);
    if (e != hipSuccess) return e;
    const long long own = (p.own_runs + 8 * kWaves - 1) / (8 * kWaves);
    hipLaunchKernelGGL((attn_shared_kernel<D, NB, FEW>), dim3((unsigned)(p.workgroups + 8 * own)), dim3(64 * kWaves), lds, st, p);
    return hipGetLastError();
}

template <int D> static hipError_t launch_d(const SharedParams& p, hipStream_t st) {
    hipError_t e;
    if (p.width == 64) e = launch_shared<D, 2, false>(p, st);
    else e = p.few ? launch_shared<D, 1, true>(p, st) : launch_shared<D, 1, false>(p, st);
    if (e != hipSuccess) return e;
    const long long heads = (long long)p.N * p.Hq;
    if (heads >= kHeadsOfWaves) hipLaunchKernelGGL((attn_shared_join<D, 64>), dim3((unsigned)heads), dim3(64), 0, st, p);
    else hipLaunchKernelGGL((attn_shared_join<D, 256>), dim3((unsigned)heads), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_attn_shared(const SharedParams& p, hipStream_t st) {
    if (!p.few) {
        static std::atomic<unsigned long long> done{0};
        hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_shared_plan_kernel), (kMostGroups + 1) * (int)sizeof(PlanGroup), done);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(attn_shared_plan_kernel, dim3(1), dim3(kPlanThreads), (unsigned)((p.groups + 1) * sizeof(PlanGroup)), st, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return p.d == 64 ? launch_d<64>(p, st) : launch_d<128>(p, st);
}

}  // namespace gdr
