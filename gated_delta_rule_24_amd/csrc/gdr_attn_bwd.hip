// Gradients of causal attention (gdr_attn_fwd.hip), the probabilities recomputed
// from the forward's log-sum-exps:
//   P_ij = exp(scale q_i.k_j - lse_i),  D_i = dO_i.o_i,  dS_ij = P_ij (dO_i.v_j - D_i)
//   dq_i = scale sum_j dS_ij k_j;  dk_j = scale sum_i dS_ij q_i;  dv_j = sum_i P_ij dO_i
// Two kernels, each the owner of what it sums, so that no atomics are needed and
// the result does not depend on the order of workgroups: the query-side one walks
// the keys of its queries (three products), the key-side one the queries of its
// keys and of every head that shares them (four products).  That recomputes the
// scores and dO v once more than a single kernel would: seven products for five.
#include <limits.h>

#include <type_traits>

#include "gdr_attn_tile.h"

namespace gdr {

using namespace attn;

namespace {

__device__ __forceinline__ void zero16(float16v& x) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.f;
}

// four consecutive channels of a gradient row
__device__ __forceinline__ void store4(uint16_t* at, const float16v& x, int j, float by) {
    *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16(x[4 * j] * by, x[4 * j + 1] * by),
                                               pack_bf16(x[4 * j + 2] * by, x[4 * j + 3] * by));
}

}  // namespace

// ---------------------------------------------------------------------------
// query side: dq, and D and the base-2 log-sum-exps for the key side
// ---------------------------------------------------------------------------

namespace {

constexpr int kQM = 128, kQN = 64, kQWaves = 4;

template <int D>
struct __attribute__((aligned(256))) DqSmem {
    uint16_t k[2][kQN * D];
    uint16_t v[2][kQN * D];
    int bound[kQM];
    int shared[3];
    int bad[kQWaves];
};

// The wave's 32 queries from the definition (see dot_row); lane r % 32 holds query
// r's key range, base-2 log-sum-exp and D.
template <int D>
__device__ __forceinline__ void queries_one_by_one(const AttnParams& p, long long head, const uint16_t* k, const uint16_t* v,
                                                   int first, int used, int lo32, int hi32, float lse32, float delta32, int lane) {
    const float to2 = p.scale * kLog2e;
    for (int r = 0; r < 32 && first + r < used; ++r) {
        const int lo = __builtin_amdgcn_readlane(lo32, r), hi = __builtin_amdgcn_readlane(hi32, r);
        const float lse2 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lse32), r));
        const float delta = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(delta32), r));
        const long long row = head + (long long)(first + r) * p.sq.t;
        const uint16_t* q = (const uint16_t*)p.q + row;
        const uint16_t* g = (const uint16_t*)p.dO + row;
        float acc[D / 64] = {};
        for (int j0 = lo; j0 < hi; j0 += 64) {
            float w = 0.f;
            if (j0 + lane < hi) {
                const long long j = (long long)(j0 + lane) * p.sk.t;
                w = __builtin_amdgcn_exp2f(dot_row<D>(q, k + j) * to2 - lse2) * (dot_row<D>(g, v + j) - delta);
            }
            add_rows<D>(acc, w, k + (long long)j0 * p.sk.t, p.sk.t, min(64, hi - j0), lane);
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            ((uint16_t*)p.dq)[row + lane + 64 * c] = f32_to_bf16(acc[c] * (hi - lo == 1 ? 0.f : p.scale));
    }
}

}  // namespace

template <int D>
__global__ __launch_bounds__(64 * kQWaves, 2) void attn_dq_kernel(AttnParams p, int tiles) {
    constexpr int KS = D / 16, DB = D / 32;
    extern __shared__ __attribute__((aligned(256))) char smem[];
    DqSmem<D>& sm = *reinterpret_cast<DqSmem<D>*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;

    int unit, tile;
    work_item(blockIdx.x, p.B * p.Hq, tiles, unit, tile);
    tile = tiles - 1 - tile;
    const int b = unit / p.Hq, hq = unit % p.Hq, hk = hq / (p.Hq / p.Hkv);
    const int r0 = tile * kQM, off = p.Tk - p.Tq;

    int used = p.Tq;
    if (p.cu_seqlens) {
        row_bounds<kQM, false>(p.cu_seqlens, p.nseq, p.Tq, r0, sm.bound, sm.shared, tid, 64 * kQWaves, used);
        if (r0 >= used) return;
    }
    const int row = r0 + 32 * wave + col, at = row + off;
    const bool live = row < used;
    int lo = p.cu_seqlens ? sm.bound[32 * wave + col] : 0, hi = live ? at + 1 : 0;
    if (p.window > 0 && at - p.window + 1 > lo) lo = at - p.window + 1;
    if (hi <= lo) { lo = 0; hi = 0; }
    const int last_row = min(r0 + kQM, used) - 1, end = last_row + off + 1;
    int begin = p.cu_seqlens ? sm.bound[0] : 0;
    int lo_most = p.cu_seqlens ? sm.bound[last_row - r0] : 0;
    if (p.window > 0) {
        begin = max(begin, r0 + off - p.window + 1);
        lo_most = max(lo_most, last_row + off - p.window + 1);
    }
    begin = max(begin, 0);
    const int hi_least = r0 + off + 1;

    const uint16_t* kp = (const uint16_t*)p.k + b * p.sk.b + hk * p.sk.h;
    const uint16_t* vp = (const uint16_t*)p.v + b * p.sk.b + hk * p.sk.h;
    const long long qrow = b * p.sq.b + hq * p.sq.h + (long long)min(row, p.Tq - 1) * p.sq.t;
    const long long stat = ((long long)b * p.Hq + hq) * p.Tq + min(row, p.Tq - 1);

    // two tiles a turn, so that every LDS address is a fixed register and a constant
    const ReadAt<D> kt = ReadAt<D>(lane).in(lds_address(sm.k[0]));
    const Stager<D, kQN, kQWaves, true> loads(p.sk.t, wave, lane);
    const int j_first = begin / kQN * kQN;
    const int n = end > begin ? (end - j_first + kQN - 1) / kQN : 0;
    uint64_t k_rows = loads.rows(kp, j_first), v_rows = loads.rows(vp, j_first);
    const uint64_t tile_bytes = (uint64_t)kQN * 2 * p.sk.t;
    const uint32_t k_lds = lds_address(sm.k[0]), v_lds = lds_address(sm.v[0]);
    if (n > 0) {
        loads.load(k_rows, j_first, p.Tk - 1, k_lds, lane);
        loads.load(v_rows, j_first, p.Tk - 1, v_lds, lane);
    }
    bf8v qf[KS], gf[KS];
    float delta = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.q + qrow + 16 * s + 8 * h));
        gf[s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.dO + qrow + 16 * s + 8 * h));
        const bf8v of = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.o + qrow + 16 * s + 8 * h));
#pragma unroll
        for (int j = 0; j < 8; ++j) delta += (float)gf[s][j] * (float)of[j];
    }
    delta = sum_across32(delta);
    // a row that saw nothing has lse -inf: +inf makes its weights exp2(-inf) = 0
    const bool sees_any = hi > lo;
    const float lse2 = sees_any ? p.lse[stat] * kLog2e : INFINITY;
    if (live && h == 0) {
        p.delta[stat] = sees_any ? delta : 0.f;
        p.delta[(long long)p.B * p.Hq * p.Tq + stat] = lse2;
    }

    float16v dq[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) zero16(dq[i]);
    const float to2 = p.scale * kLog2e;

    bool bad = false;
    int j0 = j_first;
    // one tile, in buffer BUF; false ends the walk
    auto tile_step = [&](auto buffer) {
        constexpr int BUF = decltype(buffer)::value, kTile = kQN * D * 2;
        constexpr int kKey = BUF * kTile, kVal = (int)(offsetof(DqSmem<D>, v) - offsetof(DqSmem<D>, k)) + BUF * kTile;
        wait_loads();
        lds_barrier();
        if (j0 + kQN < end) {
            k_rows += tile_bytes;
            v_rows += tile_bytes;
            loads.load(k_rows, j0 + kQN, p.Tk - 1, k_lds + (BUF ^ 1) * kTile, lane);
            loads.load(v_rows, j0 + kQN, p.Tk - 1, v_lds + (BUF ^ 1) * kTile, lane);
        }
        const bool edge = j0 < lo_most || j0 + kQN > hi_least;
        if (edge) {
            const bool mine = any_not_finite<D>(sm.k[BUF] + 16 * wave * D, lane);
            if (lane == 0) sm.bad[wave] = mine;
            lds_barrier();
            bad = (sm.bad[0] | sm.bad[1] | sm.bad[2] | sm.bad[3]) != 0;
            if (bad) return false;
        }
        if (!edge || __any(hi > j0 && lo < j0 + kQN)) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                float16v st, dp;
                zero16(st);
                zero16(dp);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    st = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kt.row_frag(32 * kb, s, kKey), qf[s], st, 0, 0, 0);
                    dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kt.row_frag(32 * kb, s, kVal), gf[s], dp, 0, 0, 0);
                }
                sched_reads_ahead<4, 2 * KS, 1>();
#pragma unroll
                for (int i = 0; i < 16; ++i) st[i] = __builtin_amdgcn_exp2f(st[i] * to2 - lse2) * (dp[i] - delta);
                if (edge) {
                    const int base = j0 + 32 * kb + 4 * h - lo;
                    const unsigned seen = (unsigned)(hi - lo);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if ((unsigned)(base + 8 * (i / 4) + i % 4) >= seen) st[i] = 0.f;
                }
                bf8v ds[2];
#pragma unroll
                for (int i = 0; i < 16; ++i) ds[i / 8][i % 8] = (__bf16)st[i];
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < DB; ++i)
                        dq[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kt.col_frag(32 * kb + 16 * s, i, kKey), ds[s], dq[i], 0, 0, 0);
                sched_reads_ahead<4, 2 * DB, 2>();
            }
        }
        j0 += kQN;
        return j0 < end;
    };
    if (n > 0)
        while (tile_step(std::integral_constant<int, 0>{}) && tile_step(std::integral_constant<int, 1>{})) {
        }
    if (bad) {
        wait_loads();                                 // no load into LDS outlives the wave
        const long long head = b * p.sq.b + hq * p.sq.h;
        queries_one_by_one<D>(p, head, kp, vp, r0 + 32 * wave, used, lo, hi, lse2, delta, lane);
        return;
    }
    if (live) {
        // the softmax over one key is constant: its gradient is 0, not a rounding error
        const float by = hi - lo == 1 ? 0.f : p.scale;
        uint16_t* out = (uint16_t*)p.dq + qrow;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) store4(out + 32 * i + 8 * j + 4 * h, dq[i], j, by);
    }
}

// ---------------------------------------------------------------------------
// key side: dk, dv
// ---------------------------------------------------------------------------

namespace {

constexpr int kKN = 128, kKM = 64, kKWaves = 4, kKB = 1;   // keys, queries a step, waves, 32-key blocks of a wave

template <int D> constexpr int kKeyLds = D == 128 && kKB == 1 ? 3 : 0;

template <int D>
struct __attribute__((aligned(256))) DkvSmem {
    uint16_t q[2][kKM * D];
    uint16_t g[2][kKM * D];
    float delta[2][kKM];
    float lse2[2][kKM];
    // key operands that do not fit the 256 registers beside the sums (d = 128): the
    // last kKeyLds of a key's D / 16
    uint4 key[kKWaves * kKB][kKeyLds<D> > 0 ? kKeyLds<D> : 1][64];
    int4 range[kKN];            // of each key: first query, one past the last, whether alone
    int bound[kKN];
    int shared[3];
    int bad[kKWaves];
};

static_assert(sizeof(DkvSmem<128>) <= 80 * 1024 && sizeof(DkvSmem<64>) <= 80 * 1024, "two workgroups on a compute unit");

// 32 keys from the definition (see dot_row); lane r % 32 holds key r's range of
// queries.
template <int D>
__device__ __forceinline__ void keys_one_by_one(const AttnParams& p, const uint16_t* k, const uint16_t* v, int b, int bh, int hk,
                                                int h0, int heads, int split, int first, int used, int lo32, int hi32,
                                                int alone32, int lane) {
    const float to2 = p.scale * kLog2e;
    const long long all = (long long)p.B * p.Hq * p.Tq, one = (long long)p.B * p.Hkv * p.Tk * D;
    for (int r = 0; r < 32 && first + r < used; ++r) {
        const int lo = __builtin_amdgcn_readlane(lo32, r), hi = __builtin_amdgcn_readlane(hi32, r);
        const float by = __builtin_amdgcn_readlane(alone32, r) ? 0.f : p.scale;
        const long long j = (long long)(first + r) * p.sk.t;
        float dk[D / 64] = {}, dv[D / 64] = {};
        for (int hq = h0; hq < h0 + heads; ++hq) {
            const long long head = b * p.sq.b + hq * p.sq.h, stat = ((long long)b * p.Hq + hq) * p.Tq;
            const uint16_t* q = (const uint16_t*)p.q + head;
            const uint16_t* g = (const uint16_t*)p.dO + head;
            for (int i0 = lo; i0 < hi; i0 += 64) {
                float x = 0.f, y = 0.f;
                if (i0 + lane < hi) {
                    const long long i = (long long)(i0 + lane) * p.sq.t;
                    x = __builtin_amdgcn_exp2f(dot_row<D>(q + i, k + j) * to2 - p.delta[all + stat + i0 + lane]);
                    y = x * (dot_row<D>(g + i, v + j) - p.delta[stat + i0 + lane]);
                }
                add_rows<D>(dv, x, g + (long long)i0 * p.sq.t, p.sq.t, min(64, hi - i0), lane);
                add_rows<D>(dk, y, q + (long long)i0 * p.sq.t, p.sq.t, min(64, hi - i0), lane);
            }
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            if (p.splits == 1) {
                const long long at = b * p.sk.b + hk * p.sk.h + j + lane + 64 * c;
                ((uint16_t*)p.dk)[at] = f32_to_bf16(dk[c] * by);
                ((uint16_t*)p.dv)[at] = f32_to_bf16(dv[c]);
            } else {
                float* at = p.part + split * one + ((long long)bh * p.Tk + first + r) * D + lane + 64 * c;
                at[0] = dk[c] * by;
                at[p.splits * one] = dv[c];
            }
        }
    }
}

}  // namespace

template <int D>
__global__ __launch_bounds__(64 * kKWaves, 2) void attn_dkv_kernel(AttnParams p, int tiles) {
    constexpr int KS = D / 16, DB = D / 32;
    extern __shared__ __attribute__((aligned(256))) char smem[];
    DkvSmem<D>& sm = *reinterpret_cast<DkvSmem<D>*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;

    int unit, tile;
    work_item(blockIdx.x, p.B * p.Hkv * p.splits, tiles, unit, tile);
    const int split = unit % p.splits, bh = unit / p.splits, b = bh / p.Hkv, hk = bh % p.Hkv;
    const int heads = p.Hq / p.Hkv / p.splits, h0 = hk * (p.Hq / p.Hkv) + split * heads;
    const int c0 = tile * kKN, off = p.Tk - p.Tq;

    int used = p.Tk, rows = p.Tq;
    if (p.cu_seqlens) {
        row_bounds<kKN, true>(p.cu_seqlens, p.nseq, p.Tk, c0, sm.bound, sm.shared, tid, 64 * kKWaves, used);
        if (c0 >= used) return;
        rows = used;
    }
    // the queries that see key j: places j .. j + window - 1, inside its sequence;
    // kept in LDS, for the steps that need them lane by lane
    int see_from = INT_MAX, see_to = 0, all_from = 0, all_to = INT_MAX;   // of the wave's keys: some row / every key
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb) {
        const int in = 32 * (kKB * wave + kb) + col, j = c0 + in;
        int lo = max(j - off, 0), hi = p.cu_seqlens ? min(sm.bound[in], rows) : rows;
        if (p.window > 0) hi = min(hi, j - off + p.window);
        if (j >= used || hi <= lo) { lo = 0; hi = 0; }
        // seen by one query that sees no other key: the window is one key, or the key is
        // all its sequence has.  The softmax over one key is constant, its gradient 0
        const bool first = j == 0 || (p.cu_seqlens && (in == 0 ? sm.shared[2] != 0 : sm.bound[in - 1] == j));
        const bool alone = p.window == 1 || (first && j >= off && hi - lo == 1);
        if (h == 0) sm.range[in] = make_int4(lo, hi, alone, 0);
        if (hi > lo) see_from = min(see_from, lo);
        see_to = max(see_to, hi);
        all_from = max(all_from, hi > lo ? lo : INT_MAX);
        all_to = min(all_to, hi);
    }
    for (int x = 32; x > 0; x >>= 1) {
        see_from = min(see_from, __shfl_xor(see_from, x, 64));
        see_to = max(see_to, __shfl_xor(see_to, x, 64));
        all_from = max(all_from, __shfl_xor(all_from, x, 64));
        all_to = min(all_to, __shfl_xor(all_to, x, 64));
    }
    see_from = __builtin_amdgcn_readfirstlane(see_from);
    see_to = __builtin_amdgcn_readfirstlane(see_to);
    all_from = __builtin_amdgcn_readfirstlane(all_from);
    all_to = __builtin_amdgcn_readfirstlane(all_to);
    const int last_key = min(c0 + kKN, used) - 1;
    const int begin = max(c0 - off, 0);
    int end = rows, hi_least = rows;
    if (p.cu_seqlens) { end = min(end, sm.bound[last_key - c0]); hi_least = min(hi_least, sm.bound[0]); }
    if (p.window > 0) {
        end = min(end, last_key - off + p.window);
        hi_least = min(hi_least, c0 - off + p.window);
    }
    const int lo_most = c0 + kKN <= used ? max(last_key - off, 0) : rows;   // a tile with dead keys is never whole

    const uint16_t* kp = (const uint16_t*)p.k + b * p.sk.b + hk * p.sk.h;
    const uint16_t* vp = (const uint16_t*)p.v + b * p.sk.b + hk * p.sk.h;
    constexpr int KR = KS - kKeyLds<D>;
    bf8v kf[kKB][KR], vf[kKB][KS];
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb) {
        const long long kr = (long long)min(c0 + 32 * (kKB * wave + kb) + col, p.Tk - 1) * p.sk.t + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint4 u = *reinterpret_cast<const uint4*>(kp + kr + 16 * s);
            if (s < KR) kf[kb][s < KR ? s : 0] = __builtin_bit_cast(bf8v, u);
            else sm.key[kKB * wave + kb][s < KR ? 0 : s - KR][lane] = u;
            vf[kb][s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>(vp + kr + 16 * s));
        }
    }
    float16v dk[kKB][DB], dv[kKB][DB];
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
        for (int i = 0; i < DB; ++i) { zero16(dk[kb][i]); zero16(dv[kb][i]); }
    const float to2 = p.scale * kLog2e;

    const ReadAt<D> at_lane(lane);
    const Stager<D, kKM, kKWaves, false> loads(p.sq.t, wave, lane);
    const int i_first = begin / kKM * kKM;
    const int n = end > begin ? (end - i_first + kKM - 1) / kKM * heads : 0;
    const long long all = (long long)p.B * p.Hq * p.Tq;
    const uint64_t step_bytes = (uint64_t)kKM * 2 * p.sq.t;

    // the step whose loads go out next: queries next_i .. of head next_h
    int next_h = h0, next_i = i_first;
    uint64_t q_rows = 0, g_rows = 0, stats = 0;
    auto fetch = [&](int buf) {
        if (next_i == i_first) {
            q_rows = loads.rows((const uint16_t*)p.q + b * p.sq.b + next_h * p.sq.h, i_first);
            g_rows = loads.rows((const uint16_t*)p.dO + b * p.sq.b + next_h * p.sq.h, i_first);
            stats = (uint64_t)(p.delta + (wave ? all : 0) + ((long long)b * p.Hq + next_h) * p.Tq + i_first);
        }
        loads.load(q_rows, next_i, p.Tq - 1, lds_address(sm.q[0]) + buf * kKM * D * 2, lane);
        loads.load(g_rows, next_i, p.Tq - 1, lds_address(sm.g[0]) + buf * kKM * D * 2, lane);
        if (wave < 2)
            direct_load4(4 * min(lane, p.Tq - 1 - next_i), stats, lds_address(wave ? sm.lse2[0] : sm.delta[0]) + buf * kKM * 4);
        q_rows += step_bytes;
        g_rows += step_bytes;
        stats += kKM * 4;
        next_i += kKM;
        if (next_i >= end) { next_i = i_first; ++next_h; }
    };
    if (n > 0) fetch(0);
    bool bad = false;
    int i0 = i_first - kKM;
    for (int it = 0; it < n; ++it) {
        const int buf = it & 1;
        i0 += kKM;
        if (i0 >= end) i0 = i_first;
        wait_loads();
        lds_barrier();
        if (it + 1 < n) fetch(buf ^ 1);
        const uint16_t* qt = sm.q[buf];
        const uint16_t* gt = sm.g[buf];
        const bool inner = i0 >= lo_most && i0 + kKM <= hi_least;
        if (!inner) {
            bool mine = false;
#pragma unroll
            for (int i = 0; i < kKM / 16 / kKWaves; ++i) {
                const int r = (kKM / kKWaves) * wave + 16 * i;
                mine = mine || any_not_finite<D>(qt + r * D, lane) || any_not_finite<D>(gt + r * D, lane);
            }
            // a masked pair's weight is 0, and so must be its product with dO v - D
            const float d = sm.delta[buf][lane], l2 = sm.lse2[buf][lane];
            mine = mine || __any(!(fabsf(d) < INFINITY) || !(l2 > -INFINITY));
            if (lane == 0) sm.bad[wave] = mine;
            lds_barrier();
            bad = false;
#pragma unroll
            for (int w = 0; w < kKWaves; ++w) bad = bad || sm.bad[w] != 0;
            if (bad) break;
        }
        const ReadAt<D> at = at_lane.fresh(lds_address(qt));
        constexpr int kG = offsetof(DkvSmem<D>, g) - offsetof(DkvSmem<D>, q);
#pragma unroll
        for (int ib = 0; ib < kKM / 32; ++ib) {
            const int ir = i0 + 32 * ib;
            if (ir >= see_to || ir + 32 <= see_from) continue;
            const bool whole = ir >= all_from && ir + 32 <= all_to;
            // the weights, and dv from them
            float16v st[kKB], dp[kKB];
#pragma unroll
            for (int kb = 0; kb < kKB; ++kb) zero16(st[kb]);
#pragma unroll
            for (int s = 0; s < KR; ++s) {
                const bf8v a = at.row_frag(32 * ib, s);
#pragma unroll
                for (int kb = 0; kb < kKB; ++kb) st[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, kf[kb][s], st[kb], 0, 0, 0);
            }
            sched_reads_ahead<2, KR, 1, kKB>();
            __builtin_amdgcn_sched_barrier(0);        // the registers are full: no reads for the next part yet
            if constexpr (KR < KS) {
#pragma unroll
                for (int s = KR; s < KS; ++s) {
                    const bf8v a = at.row_frag(32 * ib, s);
#pragma unroll
                    for (int kb = 0; kb < kKB; ++kb) {
                        const bf8v k = __builtin_bit_cast(bf8v, sm.key[kKB * wave + kb][s - KR][lane_now()]);
                        st[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, k, st[kb], 0, 0, 0);
                    }
                }
                sched_reads_ahead<2, KS - KR, 1 + kKB, kKB>();
                __builtin_amdgcn_sched_barrier(0);
            }
            if (!whole) {
#pragma unroll
                for (int kb = 0; kb < kKB; ++kb) {
                    const int here = lane_now();
                    const int2 see = *reinterpret_cast<const int2*>(&sm.range[32 * (kKB * wave + kb) + (here & 31)]);
                    const int from = ir + 4 * (here >> 5) - see.x;
                    const unsigned seen = (unsigned)(see.y - see.x);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if ((unsigned)(from + 8 * (i / 4) + i % 4) >= seen) st[kb][i] = -INFINITY;
                }
            }
            bf8v pf[kKB][2];
            const float* lse_at = &sm.lse2[buf][32 * ib + 4 * (lane_now() >> 5)];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
                const float4v l4 = *reinterpret_cast<const float4v*>(lse_at + 8 * q4);
#pragma unroll
                for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[kb][4 * q4 + i] = __builtin_amdgcn_exp2f(st[kb][4 * q4 + i] * to2 - l4[i]);
            }
#pragma unroll
            for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) pf[kb][i / 8][i % 8] = (__bf16)st[kb][i];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    const bf8v g = at.col_frag(32 * ib + 16 * s, i, kG);
#pragma unroll
                    for (int kb = 0; kb < kKB; ++kb) dv[kb][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(g, pf[kb][s], dv[kb][i], 0, 0, 0);
                }
            sched_reads_ahead<2, 2 * DB, 2, kKB>();
            __builtin_amdgcn_sched_barrier(0);
            // their gradients, and dk from them
#pragma unroll
            for (int kb = 0; kb < kKB; ++kb) zero16(dp[kb]);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bf8v g = at.row_frag(32 * ib, s, kG);
#pragma unroll
                for (int kb = 0; kb < kKB; ++kb) dp[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(g, vf[kb][s], dp[kb], 0, 0, 0);
            }
            sched_reads_ahead<2, KS, 1, kKB>();
            __builtin_amdgcn_sched_barrier(0);
            bf8v ds[kKB][2];
            const float* delta_at = &sm.delta[buf][32 * ib + 4 * (lane_now() >> 5)];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
                const float4v d4 = *reinterpret_cast<const float4v*>(delta_at + 8 * q4);
#pragma unroll
                for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dp[kb][4 * q4 + i] = st[kb][4 * q4 + i] * (dp[kb][4 * q4 + i] - d4[i]);
            }
#pragma unroll
            for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) ds[kb][i / 8][i % 8] = (__bf16)dp[kb][i];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < DB; ++i) {
                    const bf8v a = at.col_frag(32 * ib + 16 * s, i);
#pragma unroll
                    for (int kb = 0; kb < kKB; ++kb) dk[kb][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, ds[kb][s], dk[kb][i], 0, 0, 0);
                }
            sched_reads_ahead<2, 2 * DB, 2, kKB>();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (bad) {
        wait_loads();                                 // no load into LDS outlives the wave
#pragma unroll
        for (int kb = 0; kb < kKB; ++kb) {
            const int4 see = sm.range[32 * (kKB * wave + kb) + col];
            keys_one_by_one<D>(p, kp, vp, b, bh, hk, h0, heads, split, c0 + 32 * (kKB * wave + kb), used, see.x, see.y, see.z, lane);
        }
        return;
    }
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb) {
        const int key = c0 + 32 * (kKB * wave + kb) + col;
        if (key >= used) continue;
        const int4 see = sm.range[key - c0];
        const float by = see.z ? 0.f : p.scale;
        if (see.y <= see.x) {                         // no query sees it: 0, not its 0 * NaN
#pragma unroll
            for (int i = 0; i < DB; ++i) { zero16(dk[kb][i]); zero16(dv[kb][i]); }
        }
        if (p.splits == 1) {
            const long long at = b * p.sk.b + hk * p.sk.h + (long long)key * p.sk.t;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    store4((uint16_t*)p.dk + at + 32 * i + 8 * j + 4 * h, dk[kb][i], j, by);
                    store4((uint16_t*)p.dv + at + 32 * i + 8 * j + 4 * h, dv[kb][i], j, 1.f);
                }
        } else {
            const long long one = (long long)p.B * p.Hkv * p.Tk * D;
            float* at = p.part + split * one + ((long long)bh * p.Tk + key) * D;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4v x = {dk[kb][i][4 * j], dk[kb][i][4 * j + 1], dk[kb][i][4 * j + 2], dk[kb][i][4 * j + 3]};
                    const float4v y = {dv[kb][i][4 * j], dv[kb][i][4 * j + 1], dv[kb][i][4 * j + 2], dv[kb][i][4 * j + 3]};
                    *reinterpret_cast<float4v*>(at + 32 * i + 8 * j + 4 * h) = x * by;
                    *reinterpret_cast<float4v*>(at + p.splits * one + 32 * i + 8 * j + 4 * h) = y;
                }
        }
    }
}

// Sums the splits' partial dk and dv in their order; 8 channels a thread.
template <int D>
__global__ __launch_bounds__(256) void attn_dkv_sum(AttnParams p) {
    const long long one = (long long)p.B * p.Hkv * p.Tk * D;
    const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= one) return;
    const int c = (int)(at % D);
    const long long row = at / D, bh = row / p.Tk;
    const int t = (int)(row % p.Tk), b = (int)(bh / p.Hkv), hk = (int)(bh % p.Hkv);
    if (p.cu_seqlens && t >= p.cu_seqlens[p.nseq]) return;
    const long long to = b * p.sk.b + hk * p.sk.h + t * p.sk.t + c;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const float* src = p.part + side * p.splits * one + at;
        float4v x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < p.splits; ++s) {
            x += *reinterpret_cast<const float4v*>(src + s * one);
            y += *reinterpret_cast<const float4v*>(src + s * one + 4);
        }
        *reinterpret_cast<uint4*>((uint16_t*)(side ? p.dv : p.dk) + to) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    }
}

int attn_bwd_splits(int B, int Hq, int Hkv, int Tk) {
    const int G = Hq / Hkv;
    const long long base = (long long)B * Hkv * ((Tk + kKN - 1) / kKN);
    // the smallest divisor of the shared heads that gives every compute unit's two
    // workgroups something to do
    int s = 1;
    while (s < G && (base * s < 512 || G % s != 0)) ++s;
    while (G % s != 0) ++s;
    return s;
}

template <int D>
static hipError_t launch_bwd_d(const AttnParams& p, hipStream_t st) {
    static std::atomic<unsigned long long> done_q{0}, done_k{0};
    hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_dq_kernel<D>), (int)sizeof(DqSmem<D>), done_q);
    if (e != hipSuccess) return e;
    e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_dkv_kernel<D>), (int)sizeof(DkvSmem<D>), done_k);
    if (e != hipSuccess) return e;
    const int qt = (p.Tq + kQM - 1) / kQM, kt = (p.Tk + kKN - 1) / kKN;
    if (qt > 0) {
        hipLaunchKernelGGL((attn_dq_kernel<D>), dim3((unsigned)((long long)p.B * p.Hq * qt)), dim3(64 * kQWaves),
                           sizeof(DqSmem<D>), st, p, qt);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (kt == 0) return hipSuccess;
    hipLaunchKernelGGL((attn_dkv_kernel<D>), dim3((unsigned)((long long)p.B * p.Hkv * p.splits * kt)), dim3(64 * kKWaves),
                       sizeof(DkvSmem<D>), st, p, kt);
    e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const long long items = (long long)p.B * p.Hkv * p.Tk * D / 8;
    hipLaunchKernelGGL((attn_dkv_sum<D>), dim3((unsigned)((items + 255) / 256)), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnParams& p, hipStream_t st) {
    return p.d == 64 ? launch_bwd_d<64>(p, st) : launch_bwd_d<128>(p, st);
}

}  // namespace gdr
