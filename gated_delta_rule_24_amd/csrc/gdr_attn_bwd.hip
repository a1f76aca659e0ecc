// Gradients of causal attention (gdr_attn_fwd.hip), the probabilities recomputed
// from the forward's log-sum-exps:
//   P_ij = exp(scale q_i.k_j - lse_i),  D_i = dO_i.o_i,  dS_ij = P_ij (dO_i.v_j - D_i)
//   dq_i = scale sum_j dS_ij k_j;  dk_j = scale sum_i dS_ij q_i;  dv_j = sum_i P_ij dO_i
// Two kinds of workgroups, each the owner of what it sums, so that no atomics are
// needed and the result does not depend on their order: the query side walks the
// keys of its queries (three products), the key side the queries of its keys and of
// every head that shares them (four products).  That recomputes the scores and dO v
// once more than a single walk would: seven products for five.  Both kinds run in
// one kernel, the key side's first, after a small one that forms D: one tail
// instead of two, and short calls fill the chip with both.
//
// P and dS are rounded to bf16 for their products, as the forward's weights are and for
// the same reason.  dS's rounding is as large as that of the results: dq and dk are
// sqrt(2) times as far off as that alone (0.24% for 0.17%); its remainder as a second
// operand would be two products more.
//
// Bound by the matrix cores' share of the time (query side 55% of the cycles, key side
// 49%) and by power: on random data the clock falls from 2.4 to about 1.9 GHz (all
// inputs zero: 634 us for 819).  Measured, d = 128: 2 x 8,192 tokens, 16 heads, window
// 2,048 820 us, 734 TFLOP/s for the five products of a single walk and 1,030 for the
// seven; 2,047 tokens, 16 heads on 4, 88 us, 488 and 683, of which 6 form D and 7 sum
// the splits (bound by the steps that one workgroup takes after the other: 40 of 1.8 us
// on the key side, up to 32 of 1.9 on the query side).  A single walk would add dq into
// memory from every key tile: with atomics, whose order would change results, or with
// a partial dq for each of them.
#include <limits.h>

#include <type_traits>

#include "gdr_attn_tile.h"

namespace gdr {

using namespace attn;

// A weight times dO v - D, 0 where the weight is 0, as that of every masked pair is.
// dO v may have overflowed there (values near the type's largest are finite
// themselves), and 0 times infinity would reach the gradients of rows that do not see
// each other.  One instruction, as the plain product: the one for which 0 times
// anything is 0 (the intrinsic by its name, as there is no builtin for it).
__device__ float multiply_zero_wins(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float weighted(float weight, float x) { return multiply_zero_wins(weight, x); }

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

// D and the base-2 log-sum-exps of every query row: D / 8 lanes a row.  A row that
// saw nothing has lse -inf: +inf makes its weights exp2(-inf) = 0.
//
// dO.o carries o's rounding to bf16, up to 2^-8 of it.  Where few keys share the weight, dO v - D
// is a small difference of such numbers, and dq and dk come out many times as far off as
// their own roundings leave them.  So a row of at most kFew keys takes D = sum_j P_ij dO.v_j
// from the keys themselves, in fp32, in calls of every size; with more keys o is the
// smaller the more they are.  The rows behind a call's start that are such rows are one
// tile of 32 queries and 32 keys of each head, which the grid's first blocks take, a block
// a head (16 heads x 257 tokens 32.4 -> 34.1 us a call, 2,047 tokens 92.6 -> 92.9).  Where any
// row may be one (a window of at most kFew, packed sequences: p.few), the row's own lanes
// go over its keys, 8 at a time.
// (Where its weights do not sum to 1, o and lse are not what the forward made of these
// keys, infinities among them say; then o counts.)
constexpr int kFew = 32;

__device__ __forceinline__ float few_or_all(float direct, float whole, float all) {
    return fabsf(whole - 1.f) < 1e-4f && fabsf(direct) < INFINITY ? direct : all;
}

__device__ __forceinline__ void put_delta(const AttnParams& p, long long row, float delta, float lse) {
    p.delta[row] = lse == -INFINITY ? 0.f : delta;
    p.delta[(long long)p.B * p.Hq * p.Tq + row] = lse == -INFINITY ? INFINITY : lse * kLog2e;
}

// Queries first .. first + count - 1 of one head, which see keys 0 .. 31 or fewer: scores
// and dO v as one 32 x 32 product each (S^T[key][query], as the query side's), rows and keys
// past the last held at it.  The block's four waves take a quarter of the channels each, so
// that all of it is one trip to memory, and the first sums them.
struct __attribute__((aligned(16))) FirstRows {
    float4v st[3][4][64], dp[3][4][64];
    float all[3][64];
};

template <int D>
__device__ __forceinline__ void first_rows_delta(const AttnParams& p, FirstRows& sm, int b, int hq, int first, int count) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5, t = first + min(col, count - 1);
    const long long at = b * p.sq.b + hq * p.sq.h + t * p.sq.t + D / 4 * wave + 8 * h;
    const long long to = b * p.sk.b + hq / (p.Hq / p.Hkv) * p.sk.h + (long long)min(col, p.Tk - 1) * p.sk.t + D / 4 * wave + 8 * h;
    const long long row = ((long long)b * p.Hq + hq) * p.Tq + t;
    const float lse = p.lse[row];
    auto load = [](const void* x, long long i) { return __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)x + i)); };
    float16v st, dp;
    zero16(st);
    zero16(dp);
    float all = 0.f;
#pragma unroll
    for (int s = 0; s < D / 64; ++s) {
        const bf8v g = load(p.dO, at + 16 * s), x = load(p.o, at + 16 * s);
        st = __builtin_amdgcn_mfma_f32_32x32x16_bf16(load(p.k, to + 16 * s), load(p.q, at + 16 * s), st, 0, 0, 0);
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(load(p.v, to + 16 * s), g, dp, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) all += (float)x[j] * (float)g[j];
    }
    if (wave) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sm.st[wave - 1][i][lane] = float4v{st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]};
            sm.dp[wave - 1][i][lane] = float4v{dp[4 * i], dp[4 * i + 1], dp[4 * i + 2], dp[4 * i + 3]};
        }
        sm.all[wave - 1][lane] = all;
    }
    __syncthreads();
    if (wave) return;
    float direct = 0.f, whole = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float x = st[i], y = dp[i];
#pragma unroll
        for (int w = 0; w < 3; ++w) { x += sm.st[w][i / 4][lane][i % 4]; y += sm.dp[w][i / 4][lane][i % 4]; }
        if (8 * (i / 4) + 4 * h + i % 4 <= t + p.Tk - p.Tq) {
            const float w = __builtin_amdgcn_exp2f((x * p.scale - lse) * kLog2e);
            direct += w * y;
            whole += w;
        }
    }
#pragma unroll
    for (int w = 0; w < 3; ++w) all += sm.all[w][lane];
    const float sum = few_or_all(sum_across32(direct), sum_across32(whole), sum_across32(all));
    if (h == 0 && col < count) put_delta(p, row, sum, lse);
}

// `first`, `count`: the queries that the grid's first `heads` blocks take, a block a head.
template <int D>
__global__ __launch_bounds__(256, 4) void attn_delta_kernel(AttnParams p, int first, int count, int heads) {
    constexpr int L = D / 8;
    __shared__ FirstRows sm;
    if (blockIdx.x < (unsigned)heads) return first_rows_delta<D>(p, sm, blockIdx.x / p.Hq, blockIdx.x % p.Hq, first, count);
    const long long row = (long long)(blockIdx.x - heads) * (256 / L) + threadIdx.x / L, all = (long long)p.B * p.Hq * p.Tq;
    if (row >= all) return;
    const int c = threadIdx.x % L;
    const long long bh = row / p.Tq;
    const int t = (int)(row % p.Tq), b = (int)(bh / p.Hq), hq = (int)(bh % p.Hq);
    if ((unsigned)(t - first) < (unsigned)count) return;
    const long long at = b * p.sq.b + hq * p.sq.h + t * p.sq.t + 8 * c;
    const bf8v x = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.o + at));
    const bf8v y = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.dO + at));
    const float lse = p.lse[row];
    int lo = 0;
    // where the row's sequence starts
    if (p.cu_seqlens) lo = max(min(p.cu_seqlens[last_at_most(p.cu_seqlens, p.nseq, t)], t), 0);
    const int end = t + p.Tk - p.Tq + 1;
    if (p.window > 0) lo = max(lo, end - p.window);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (float)x[j] * (float)y[j];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, L);
    if (p.few && end - lo <= kFew) {
        const bf8v q = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.q + at));
        const long long kv = b * p.sk.b + hq / (p.Hq / p.Hkv) * p.sk.h + 8 * c;
        float direct = 0.f, whole = 0.f;
        for (int j0 = lo; j0 < end; j0 += 8) {        // 8 keys' loads at once
            uint4 k[8], v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const long long to = kv + min(j0 + i, end - 1) * p.sk.t;
                k[i] = *reinterpret_cast<const uint4*>((const uint16_t*)p.k + to);
                v[i] = *reinterpret_cast<const uint4*>((const uint16_t*)p.v + to);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bf8v kk = __builtin_bit_cast(bf8v, k[i]), vv = __builtin_bit_cast(bf8v, v[i]);
                float qk = 0.f, gv = 0.f;
#pragma unroll
                for (int c8 = 0; c8 < 8; ++c8) { qk += (float)q[c8] * (float)kk[c8]; gv += (float)y[c8] * (float)vv[c8]; }
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) { qk += __shfl_xor(qk, o, L); gv += __shfl_xor(gv, o, L); }
                if (j0 + i < end) {
                    const float w = __builtin_amdgcn_exp2f((qk * p.scale - lse) * kLog2e);
                    direct += w * gv;
                    whole += w;
                }
            }
        }
        sum = few_or_all(direct, whole, sum);
    }
    if (c == 0) put_delta(p, row, sum, lse);
}

// ---------------------------------------------------------------------------
// query side: dq
// ---------------------------------------------------------------------------

namespace {

constexpr int kQM = 128, kQN = 64, kQWaves = 4;

template <int D>
struct __attribute__((aligned(256))) DqSmem {
    uint16_t k[2][kQN * D];
    uint16_t v[2][kQN * D];
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
__device__ __forceinline__ void query_side(const AttnParams& p, int item, int tiles, char* smem) {
    constexpr int KS = D / 16, DB = D / 32;
    DqSmem<D>& sm = *reinterpret_cast<DqSmem<D>*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;

    int unit, tile;
    work_item(item, p.B * p.Hq, tiles, unit, tile);
    tile = tiles - 1 - tile;
    const int b = unit / p.Hq, hq = unit % p.Hq, hk = hq / (p.Hq / p.Hkv);
    const int r0 = tile * kQM, off = p.Tk - p.Tq;

    SeqRows seq = {p.Tq, 0, 0, 0, false};
    if (p.cu_seqlens) seq = seq_rows<kQM, false>(p.cu_seqlens, p.nseq, p.Tq, r0, r0 + 32 * wave, lane);
    const int used = seq.used;
    if (r0 >= used) return;
    const int row = r0 + 32 * wave + col, at = row + off;
    const bool live = row < used;
    int lo = seq.mine, hi = live ? at + 1 : 0;
    if (p.window > 0 && at - p.window + 1 > lo) lo = at - p.window + 1;
    if (hi <= lo) { lo = 0; hi = 0; }
    const int last_row = min(r0 + kQM, used) - 1, end = last_row + off + 1;
    int begin = seq.first, lo_most = seq.last;
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
    const int last = p.cu_seqlens ? used - 1 : p.Tk - 1;   // of the keys that count
    uint64_t k_rows = loads.rows(kp, j_first), v_rows = loads.rows(vp, j_first);
    const uint64_t tile_bytes = (uint64_t)kQN * 2 * p.sk.t;
    const uint32_t k_lds = lds_address(sm.k[0]), v_lds = lds_address(sm.v[0]);
    if (n > 0) {
        loads.load(k_rows, j_first, last, k_lds, lane);
        loads.load(v_rows, j_first, last, v_lds, lane);
    }
    bf8v qf[KS], gf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.q + qrow + 16 * s + 8 * h));
        gf[s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>((const uint16_t*)p.dO + qrow + 16 * s + 8 * h));
    }
    const float delta = p.delta[stat], lse2 = p.delta[(long long)p.B * p.Hq * p.Tq + stat];

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
            loads.load(k_rows, j0 + kQN, last, k_lds + (BUF ^ 1) * kTile, lane);
            loads.load(v_rows, j0 + kQN, last, v_lds + (BUF ^ 1) * kTile, lane);
        }
        const bool edge = j0 < lo_most || j0 + kQN > hi_least;
        if (edge) {
            // (a masked pair's weight is 0, and its product with dO v - D is, whatever v)
            const bool mine = any_not_finite<D>(sm.k[BUF] + 16 * wave * D, lane);
            if (lane == 0) sm.bad[wave] = mine;
            lds_barrier();
            bad = (sm.bad[0] | sm.bad[1] | sm.bad[2] | sm.bad[3]) != 0;
            if (bad) return false;
        }
        if (!edge || __any(hi > j0 && lo < j0 + kQN)) {
            // Six runs of eight products (d = 128) for the tile's two halves of 32 keys:
            // scores, dO v, scores, dO v, and dq from both; the operands read kAhead
            // products ahead (four 32-cycle products cover a read), the vector work of one
            // run between the products of a later one (see the key-side kernel)
            constexpr int kAhead = 4, kAll = 4 * KS + 4 * DB, PER = 16 / KS;
            auto fixed = [] { __builtin_amdgcn_sched_barrier(0); };
            bf8v f[kAll], ds[4];
            auto read = [&](int u) {
                const int run = u / KS, s = u % KS, t = u - 4 * KS;
                if (run < 4) f[u] = kt.row_frag(32 * (run / 2), s, run % 2 ? kVal : kKey);
                else f[u] = kt.col_frag(16 * (t / DB), t % DB, kKey);
            };
            float16v st[2], dp[2];
            auto weights = [&](int half, int i) { st[half][i] = here(__builtin_amdgcn_exp2f(st[half][i] * to2 - lse2)); };
            auto gradient = [&](int half, int i) {    // a pair at a time, packed
                if (i % 2 == 0) return;
                const float x = weighted(st[half][i - 1], dp[half][i - 1] - delta), y = weighted(st[half][i], dp[half][i] - delta);
                const uint32_t u = here(pack_bf16(x, y));
                const bf2v pair = __builtin_bit_cast(bf2v, u);
                ds[2 * half + i / 8][i % 8 - 1] = pair[0];
                ds[2 * half + i / 8][i % 8] = pair[1];
            };
            auto hide = [&](int half) {
                const int base = j0 + 32 * half + 4 * h - lo;
                const unsigned seen = (unsigned)(hi - lo);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if ((unsigned)(base + 8 * (i / 4) + i % 4) >= seen) st[half][i] = -INFINITY;
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) read(u);
            zero16(st[0]);
            fixed();
#pragma unroll
            for (int u = 0; u < KS; ++u) {
                read(u + kAhead);
                st[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[u], qf[u], st[0], 0, 0, 0);
                fixed();
            }
            if (edge) hide(0);
            zero16(dp[0]);
            fixed();
#pragma unroll
            for (int s = 0; s < KS; ++s) {            // beside dO v, the weights
                read(KS + s + kAhead);
                dp[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[KS + s], gf[s], dp[0], 0, 0, 0);
#pragma unroll
                for (int i = s * PER; i < (s + 1) * PER; ++i) weights(0, i);
                fixed();
            }
            zero16(st[1]);
            fixed();
#pragma unroll
            for (int s = 0; s < KS; ++s) {            // beside the second half's scores, the first's gradients
                read(2 * KS + s + kAhead);
                st[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[2 * KS + s], qf[s], st[1], 0, 0, 0);
#pragma unroll
                for (int i = s * PER; i < (s + 1) * PER; ++i) gradient(0, i);
                fixed();
            }
            if (edge) hide(1);
            zero16(dp[1]);
            fixed();
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                read(3 * KS + s + kAhead);
                dp[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[3 * KS + s], gf[s], dp[1], 0, 0, 0);
#pragma unroll
                for (int i = s * PER; i < (s + 1) * PER; ++i) weights(1, i);
                fixed();
            }
#pragma unroll
            for (int t = 0; t < 4 * DB; ++t) {        // beside dq, the second half's gradients
                if (4 * KS + t + kAhead < kAll) read(4 * KS + t + kAhead);
                dq[t % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[4 * KS + t], ds[t / DB], dq[t % DB], 0, 0, 0);
                if (t < 2 * DB) {
#pragma unroll
                    for (int i = t * PER; i < (t + 1) * PER; ++i) gradient(1, i);
                }
                fixed();
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

constexpr int kKN = 128, kKWaves = 4;                // keys of a workgroup, 32 a wave

// Queries a step.  At d = 128 the sums dk, dv (128 registers) and the keys' operands
// (28 of 32) leave no room for the values' beside the work: those and the last of
// the keys' stay in LDS, and the steps are half as long so that two workgroups
// still fit a compute unit.
template <int D> constexpr int kKM = D == 128 ? 32 : 64;

template <int D>
struct __attribute__((aligned(256))) DkvSmem {
    uint16_t q[2][kKM<D> * D];
    uint16_t g[2][kKM<D> * D];
    uint16_t v[kKN * D];
    uint4 key[kKWaves][64];     // the last operand of each wave's keys
    float delta[2][64];
    float lse2[2][64];
    int4 range[kKN];            // of each key: first query, one past the last, whether alone
    int bad[kKWaves];
};

static_assert(sizeof(DkvSmem<128>) <= 80 * 1024 && sizeof(DkvSmem<64>) <= 80 * 1024, "two workgroups on a compute unit");

// 32 keys from the definition (see dot_row); lane r % 32 holds key r's range of
// queries.
template <int D>
__device__ __forceinline__ void keys_one_by_one(const AttnParams& p, const uint16_t* k, const uint16_t* v, int b, int bh, int hk,
                                                int h0, int split, int first, int used, int i_first, int step, int per, int from,
                                                int to, int lo32, int hi32, int alone32, int lane) {
    const float to2 = p.scale * kLog2e;
    const long long all = (long long)p.B * p.Hq * p.Tq, one = (long long)p.B * p.Hkv * p.Tk * D;
    for (int r = 0; r < 32 && first + r < used; ++r) {
        const int lo = __builtin_amdgcn_readlane(lo32, r), hi = __builtin_amdgcn_readlane(hi32, r);
        const float by = __builtin_amdgcn_readlane(alone32, r) ? 0.f : p.scale;
        const long long j = (long long)(first + r) * p.sk.t;
        float dk[D / 64] = {}, dv[D / 64] = {};
        for (int s = from; s < to; s += per - s % per) {          // the split's steps of one head
            const int hq = h0 + s / per, begin = i_first + s % per * step;
            const int i_lo = max(lo, begin), i_hi = min(hi, begin + min(to - s, per - s % per) * step);
            const long long head = b * p.sq.b + hq * p.sq.h, stat = ((long long)b * p.Hq + hq) * p.Tq;
            const uint16_t* q = (const uint16_t*)p.q + head;
            const uint16_t* g = (const uint16_t*)p.dO + head;
            for (int i0 = i_lo; i0 < i_hi; i0 += 64) {
                float x = 0.f, y = 0.f;
                if (i0 + lane < i_hi) {
                    const long long i = (long long)(i0 + lane) * p.sq.t;
                    x = __builtin_amdgcn_exp2f(dot_row<D>(q + i, k + j) * to2 - p.delta[all + stat + i0 + lane]);
                    y = x * (dot_row<D>(g + i, v + j) - p.delta[stat + i0 + lane]);
                }
                add_rows<D>(dv, x, g + (long long)i0 * p.sq.t, p.sq.t, min(64, i_hi - i0), lane);
                add_rows<D>(dk, y, q + (long long)i0 * p.sq.t, p.sq.t, min(64, i_hi - i0), lane);
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

// Steps of one head's queries that see some key of tile `tile`, without a window.
template <int D> __host__ __device__ inline int key_steps(const AttnParams& p, int tile) {
    const int c0 = tile * kKN, off = p.Tk - p.Tq, begin = c0 > off ? c0 - off : 0;
    return p.Tq > begin ? (p.Tq + kKM<D> - 1) / kKM<D> - begin / kKM<D> : 0;
}
// Workgroups that key tile's queries are dealt to.
template <int D> __host__ __device__ inline int key_splits(const AttnParams& p, int tile) {
    if (p.split_steps == 0) return p.splits;
    const int n = (p.Hq / p.Hkv * key_steps<D>(p, tile) + p.split_steps - 1) / p.split_steps;
    return n < 1 ? 1 : n > p.splits ? p.splits : n;
}

// The key tile of item `split` of all tiles' splits in order; leaves the split's number
// among the tile's and how many it has.  Up to 256 tiles: four a lane and a running sum.
template <int D> __device__ __forceinline__ int tile_of_split(const AttnParams& p, int tiles, int lane, int& split, int& splits) {
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += n[i] = 4 * lane + i < tiles ? key_splits<D>(p, 4 * lane + i) : 0;
    int end = sum;
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(end, o, 64);
        if (lane >= o) end += y;
    }
    const int owner = __builtin_ctzll(__ballot(end > split));
    split -= __builtin_amdgcn_readlane(end - sum, owner);
    int tile = 4 * owner;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        splits = __builtin_amdgcn_readlane(n[i], owner);
        if (split < splits) break;
        split -= splits;
        ++tile;
    }
    return tile;
}

template <int D>
__device__ __forceinline__ void key_side(const AttnParams& p, int item, int tiles, char* smem) {
    constexpr int KS = D / 16, DB = D / 32;
    DkvSmem<D>& sm = *reinterpret_cast<DkvSmem<D>*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;

    int bh, tile, split, splits = p.splits;
    if (p.split_steps == 0) {
        work_item(item, p.B * p.Hkv * splits, tiles, bh, tile);
        split = bh % splits;
        bh /= splits;
    } else {
        bh = item % (p.B * p.Hkv);
        split = item / (p.B * p.Hkv);
        tile = tile_of_split<D>(p, tiles, lane, split, splits);
    }
    const int b = bh / p.Hkv, hk = bh % p.Hkv;
    const int heads = p.Hq / p.Hkv, h0 = hk * heads;
    const int c0 = tile * kKN, off = p.Tk - p.Tq;

    SeqRows seq = {p.Tk, p.Tq, p.Tq, p.Tq, false};
    if (p.cu_seqlens) seq = seq_rows<kKN, true>(p.cu_seqlens, p.nseq, p.Tk, c0, c0 + 32 * wave, lane);
    const int used = seq.used, rows = p.cu_seqlens ? used : p.Tq;
    if (c0 >= used) return;
    const uint16_t* kp = (const uint16_t*)p.k + b * p.sk.b + hk * p.sk.h;
    const uint16_t* vp = (const uint16_t*)p.v + b * p.sk.b + hk * p.sk.h;
    {
        const Stager<D, kKN, kKWaves, false> loads(p.sk.t, wave, lane);
        loads.load(loads.rows(vp, c0), c0, used - 1, lds_address(sm.v), lane);
    }
    bf8v kf[KS - 1];
    {
        const long long kr = (long long)min(c0 + 32 * wave + col, used - 1) * p.sk.t + 8 * h;
#pragma unroll
        for (int s = 0; s < KS - 1; ++s) kf[s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>(kp + kr + 16 * s));
        sm.key[wave][lane] = *reinterpret_cast<const uint4*>(kp + kr + 16 * (KS - 1));
    }
    // the queries that see key j: places j .. j + window - 1, inside its sequence;
    // kept in LDS, for the steps that need them lane by lane
    int see_from, see_to, all_from, all_to;           // queries that see some key of the wave's / every one
    {
        const int in = 32 * wave + col, j = c0 + in;
        int lo = max(j - off, 0), hi = min(seq.mine, rows);
        if (p.window > 0) hi = min(hi, j - off + p.window);
        if (j >= used || hi <= lo) { lo = 0; hi = 0; }
        // seen by one query that sees no other key: the window is one key, or the key is
        // all its sequence has.  The softmax over one key is constant, its gradient 0
        const bool first = j == 0 || seq.starts;
        const bool alone = p.window == 1 || (first && j >= off && hi - lo == 1);
        if (h == 0) sm.range[in] = make_int4(lo, hi, alone, 0);
        see_from = hi > lo ? lo : INT_MAX;
        see_to = hi;
        all_from = hi > lo ? lo : INT_MAX;
        all_to = hi;
    }
    for (int x = 16; x > 0; x >>= 1) {
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
    int end = min(rows, seq.last), hi_least = min(rows, seq.first);
    if (p.window > 0) {
        end = min(end, last_key - off + p.window);
        hi_least = min(hi_least, c0 - off + p.window);
    }
    const int lo_most = c0 + kKN <= used ? max(last_key - off, 0) : rows;   // a tile with dead keys is never whole

    float16v dk[DB], dv[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) { zero16(dk[i]); zero16(dv[i]); }
    const float to2 = p.scale * kLog2e;

    constexpr int KM = kKM<D>, kTile = KM * D * 2;
    constexpr int kG = offsetof(DkvSmem<D>, g) - offsetof(DkvSmem<D>, q);
    const ReadAt<D> at_lane(lane);
    const uint32_t v_lds = lds_address(sm.v) + 32 * wave * D * 2;
    const Stager<D, KM, kKWaves, false> loads(p.sq.t, wave, lane);
    const int i_first = begin / KM * KM;
    // steps of the heads that share the keys, one head after the other; this split's
    const int per = end > begin ? (end - i_first + KM - 1) / KM : 0;
    const int from = (int)((long long)per * heads * split / splits), to = (int)((long long)per * heads * (split + 1) / splits);
    const int n = to - from;
    const long long all = (long long)p.B * p.Hq * p.Tq;
    const uint64_t step_bytes = (uint64_t)KM * 2 * p.sq.t;

    // the step whose loads go out next: queries next_i .. of head next_h; rows behind
    // the last that counts are held at it, so that no step reads what nothing wrote
    const int i_start = n > 0 ? i_first + from % per * KM : 0;
    int next_h = n > 0 ? h0 + from / per : h0, next_i = i_start;
    uint64_t q_rows = 0, g_rows = 0, stats = 0;
    auto fetch = [&](int buf, bool head) {
        if (head || next_i == i_first) {
            q_rows = loads.rows((const uint16_t*)p.q + b * p.sq.b + next_h * p.sq.h, next_i);
            g_rows = loads.rows((const uint16_t*)p.dO + b * p.sq.b + next_h * p.sq.h, next_i);
            stats = (uint64_t)(p.delta + (wave ? all : 0) + ((long long)b * p.Hq + next_h) * p.Tq + next_i);
        }
        loads.load(q_rows, next_i, rows - 1, lds_address(sm.q[0]) + buf * kTile, lane);
        loads.load(g_rows, next_i, rows - 1, lds_address(sm.g[0]) + buf * kTile, lane);
        if (wave < 2)
            direct_load4(4 * min(lane, rows - 1 - next_i), stats, lds_address(wave ? sm.lse2[0] : sm.delta[0]) + buf * 256);
        q_rows += step_bytes;
        g_rows += step_bytes;
        stats += KM * 4;
        next_i += KM;
        if (next_i >= end) { next_i = i_first; ++next_h; }
    };
    if (n > 0) fetch(0, true);
    bool bad = false;
    int i0 = i_start - KM;
    for (int it = 0; it < n; ++it) {
        const int buf = it & 1;
        i0 += KM;
        if (i0 >= end) i0 = i_first;
        wait_loads();
        lds_barrier();
        if (it + 1 < n) fetch(buf ^ 1, false);
        if (i0 < lo_most || i0 + KM > hi_least) {
            constexpr int kMine = KM / kKWaves;
            bool mine = any_not_finite<D, kMine>(sm.q[buf] + kMine * wave * D, lane) ||
                        any_not_finite<D, kMine>(sm.g[buf] + kMine * wave * D, lane);
            // (a masked pair's weight must come out 0; its product with dO v - D then does)
            mine = mine || __any(!(sm.lse2[buf][lane] > -INFINITY));
            if (lane == 0) sm.bad[wave] = mine;
            lds_barrier();
            bad = (sm.bad[0] | sm.bad[1] | sm.bad[2] | sm.bad[3]) != 0;
            if (bad) break;
        }
        const ReadAt<D> at = at_lane.fresh(lds_address(sm.q[0]) + buf * kTile);
        uint32_t v_at = at_lane.row + v_lds;
        asm volatile("" : "+v"(v_at));
#pragma unroll
        for (int ib = 0; ib < KM / 32; ++ib) {
            const int ir = i0 + 32 * ib;
            if (ir >= see_to || ir + 32 <= see_from) continue;
            // Four runs of products, the reads of each issued four products ahead (two in
            // the second, where the registers end), the vector work of one run between
            // the products of the next.  The order is fixed step by step: left alone, the
            // compiler reads right before each product and puts the vector work in one
            // piece, and a wave's 32 products of 32 cycles took about 4,000.
            auto fixed = [] { __builtin_amdgcn_sched_barrier(0); };
            auto v_frag = [&](int s) {
                return __builtin_bit_cast(bf8v, *(const __attribute__((address_space(3))) uint4*)(uintptr_t)(v_at ^ (s << 5)));
            };
            auto g_col = [&](int t) { return at.col_frag(32 * ib + 16 * (t / DB), t % DB, kG); };
            auto q_col = [&](int t) { return at.col_frag(32 * ib + 16 * (t / DB), t % DB); };
            const int half = lane_now() >> 5;
            const float* lse_at = &sm.lse2[buf][32 * ib + 4 * half];
            const float* delta_at = &sm.delta[buf][32 * ib + 4 * half];

            // scores
            float16v st, dp;
            zero16(st);
            bf8v a[KS], g[KS], v[KS], c[2 * DB], e[2 * DB], k_last;
            float4v l4[4], d4[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) a[s] = at.row_frag(32 * ib, s);
            fixed();
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (s + 4 < KS) a[s + 4] = at.row_frag(32 * ib, s + 4);
                if (s + 2 >= KS) { g[s + 2 - KS] = at.row_frag(32 * ib, s + 2 - KS, kG); v[s + 2 - KS] = v_frag(s + 2 - KS); }
                if (s == (KS > 4 ? KS - 5 : 0)) k_last = __builtin_bit_cast(bf8v, sm.key[wave][lane_now()]);
                if (s == KS - 1) l4[0] = *reinterpret_cast<const float4v*>(lse_at);
                st = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[s], s < KS - 1 ? kf[s < KS - 1 ? s : 0] : k_last, st, 0, 0, 0);
                fixed();
            }
            if (ir < all_from || ir + 32 > all_to) {
                const int here = lane_now();
                const int2 see = *reinterpret_cast<const int2*>(&sm.range[32 * wave + (here & 31)]);
                const int from = ir + 4 * (here >> 5) - see.x;
                const unsigned seen = (unsigned)(see.y - see.x);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if ((unsigned)(from + 8 * (i / 4) + i % 4) >= seen) st[i] = -INFINITY;
            }
            // dO v; beside it the weights
            bf8v pf[2], ds[2];
            zero16(dp);
            fixed();
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                constexpr int PER = 16 / KS;          // weights a product
                if (s + 2 < KS) { g[s + 2] = at.row_frag(32 * ib, s + 2, kG); v[s + 2] = v_frag(s + 2); }
                else c[s + 2 - KS] = g_col(s + 2 - KS);
                if ((s + 1) * PER % 4 == 0 && (s + 1) * PER < 16) l4[(s + 1) * PER / 4] = *reinterpret_cast<const float4v*>(lse_at + 2 * (s + 1) * PER);
                if (s == KS - 1) d4[0] = *reinterpret_cast<const float4v*>(delta_at);
                dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(g[s], v[s], dp, 0, 0, 0);
#pragma unroll
                for (int i = s * PER; i < (s + 1) * PER; ++i) {
                    st[i] = __builtin_amdgcn_exp2f(st[i] * to2 - l4[i / 4][i % 4]);
                    pf[i / 8][i % 8] = (__bf16)st[i];
                }
                fixed();
            }
            // dv; beside it the scores' gradients
#pragma unroll
            for (int t = 0; t < 2 * DB; ++t) {
                constexpr int PER = 16 / (2 * DB);
                if (t == 0) {
#pragma unroll
                    for (int x = 2; x < 4 && x < 2 * DB; ++x) c[x] = g_col(x);
                }
                if (t + 4 < 2 * DB) c[t + 4] = g_col(t + 4);
                else e[t + 4 - 2 * DB] = q_col(t + 4 - 2 * DB);
                if ((t + 1) * PER % 4 == 0 && (t + 1) * PER < 16) d4[(t + 1) * PER / 4] = *reinterpret_cast<const float4v*>(delta_at + 2 * (t + 1) * PER);
                dv[t % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c[t], pf[t / DB], dv[t % DB], 0, 0, 0);
#pragma unroll
                for (int i = t * PER; i < (t + 1) * PER; ++i) ds[i / 8][i % 8] = (__bf16)weighted(st[i], dp[i] - d4[i / 4][i % 4]);
                fixed();
            }
            // dk
#pragma unroll
            for (int t = 0; t < 2 * DB; ++t) {
                if (t + 4 < 2 * DB) e[t + 4] = q_col(t + 4);
                dk[t % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e[t], ds[t / DB], dk[t % DB], 0, 0, 0);
                fixed();
            }
        }
    }
    if (bad) {
        wait_loads();                                 // no load into LDS outlives the wave
        const int4 see = sm.range[32 * wave + col];
        keys_one_by_one<D>(p, kp, vp, b, bh, hk, h0, split, c0 + 32 * wave, used, i_first, KM, per, from, to, see.x, see.y, see.z, lane);
        return;
    }
    wait_loads();
    const int key = c0 + 32 * wave + col;
    if (key >= used) return;
    const int4 see = sm.range[32 * wave + col];
    const float by = see.z ? 0.f : p.scale;
    if (see.y <= see.x) {                             // no query sees it: 0, not its 0 * NaN
#pragma unroll
        for (int i = 0; i < DB; ++i) { zero16(dk[i]); zero16(dv[i]); }
    }
    if (p.splits == 1) {
        const long long at = b * p.sk.b + hk * p.sk.h + (long long)key * p.sk.t;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                store4((uint16_t*)p.dk + at + 32 * i + 8 * j + 4 * h, dk[i], j, by);
                store4((uint16_t*)p.dv + at + 32 * i + 8 * j + 4 * h, dv[i], j, 1.f);
            }
    } else {
        const long long one = (long long)p.B * p.Hkv * p.Tk * D;
        float* at = p.part + split * one + ((long long)bh * p.Tk + key) * D;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4v x = {dk[i][4 * j], dk[i][4 * j + 1], dk[i][4 * j + 2], dk[i][4 * j + 3]};
                const float4v y = {dv[i][4 * j], dv[i][4 * j + 1], dv[i][4 * j + 2], dv[i][4 * j + 3]};
                *reinterpret_cast<float4v*>(at + 32 * i + 8 * j + 4 * h) = x * by;
                *reinterpret_cast<float4v*>(at + p.splits * one + 32 * i + 8 * j + 4 * h) = y;
            }
    }
}

static_assert(kQWaves == kKWaves, "one kernel");

template <int D>
__global__ __launch_bounds__(64 * kQWaves, 2) void attn_bwd_kernel(AttnParams p, int key_items, int key_tiles, int query_tiles) {
    extern __shared__ __attribute__((aligned(256))) char smem[];
    // the longest first: on the key side without splits of equal length, else, where every
    // workgroup runs at once, the query side's
    const int item = blockIdx.x, first = p.split_steps > 0 && gridDim.x <= 512 ? gridDim.x - key_items : 0;
    if (item >= first && item - first < key_items) key_side<D>(p, item - first, key_tiles, smem);
    else query_side<D>(p, first ? item : item - key_items, query_tiles, smem);
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
    const int splits = key_splits<D>(p, t / kKN);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const float* src = p.part + side * p.splits * one + at;
        float4v x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < splits; ++s) {
            x += *reinterpret_cast<const float4v*>(src + s * one);
            y += *reinterpret_cast<const float4v*>(src + s * one + 4);
        }
        *reinterpret_cast<uint4*>((uint16_t*)(side ? p.dv : p.dk) + to) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    }
}

constexpr int kSplitQueries = 512;                   // of one head, the least for a split

int attn_bwd_splits(int B, int Hq, int Hkv, int Tq, int Tk) {
    const long long base = (long long)B * Hkv * ((Tk + kKN - 1) / kKN);
    const long long most = (long long)(Hq / Hkv) * (Tq < kSplitQueries ? 1 : Tq / kSplitQueries);
    // one key-side workgroup for every compute unit, beside the query side's, as far as a
    // split has a head or 512 queries of one to walk: each writes its partial sums in fp32
    // (16 heads on 4, T = 2047, as many splits for every tile: 127 us with one, 100 with
    // 256 workgroups, 101 with 512)
    const long long want = base > 0 ? (256 + base - 1) / base : 1;
    return (int)(want < most ? want : most);
}

// the first of K tiles is seen by 2 K / (K + 1) times as many queries as the mean
int attn_bwd_splits_most(int splits, int Tk) {
    const int tiles = (Tk + kKN - 1) / kKN;
    return (int)((2LL * splits * tiles + tiles) / (tiles + 1));
}

long long attn_bwd_workgroups(int B, int Hq, int Hkv, int Tq, int Tk, int d) {
    const long long per = 2048 / d, delta = (long long)B * Hq + ((long long)B * Hq * Tq + per - 1) / per;
    const int splits = attn_bwd_splits(B, Hq, Hkv, Tq, Tk);
    const long long key_items = (long long)B * Hkv * (((long long)Tk + kKN - 1) / kKN) * (splits > 1 ? attn_bwd_splits_most(splits, Tk) : 1);
    const long long items = key_items + (long long)B * Hq * (((long long)Tq + kQM - 1) / kQM);
    return delta > items ? delta : items;
}

template <int D>
static hipError_t launch_bwd_d(AttnParams p, hipStream_t st) {
    static std::atomic<unsigned long long> done{0};
    constexpr size_t kLds = sizeof(DqSmem<D>) > sizeof(DkvSmem<D>) ? sizeof(DqSmem<D>) : sizeof(DkvSmem<D>);
    hipError_t e = ensure_dyn_lds(reinterpret_cast<const void*>(&attn_bwd_kernel<D>), (int)kLds, done);
    if (e != hipSuccess) return e;
    const long long rows = (long long)p.B * p.Hq * p.Tq, per = 2048 / D;
    if (rows > 0) {
        // the queries of each head that see 1 to kFew keys, all of them from the first
        p.few = p.cu_seqlens || (p.window > 0 && p.window <= kFew);
        const int off = p.Tk - p.Tq, first = off < 0 ? -off : 0, behind = p.Tq < kFew - off ? p.Tq : kFew - off;
        const int count = p.few || behind <= first ? 0 : behind - first, heads = count > 0 ? p.B * p.Hq : 0;
        hipLaunchKernelGGL((attn_delta_kernel<D>), dim3((unsigned)(heads + (rows + per - 1) / per)), dim3(256), 0, st, p,
                           first, count, heads);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int query_tiles = (p.Tq + kQM - 1) / kQM, key_tiles = (p.Tk + kKN - 1) / kKN;
    if (p.splits > 1 && !p.cu_seqlens && p.window == 0) {
        // The first keys are seen by most queries: splits of as many steps everywhere
        // (16 heads on 4, T = 2047: 86 us, with as many splits for every tile 100; 16 on 2,
        // T = 4096: 249, 328).  With a window the tiles have about as many as each other
        // (4,096 tokens, window 512: 98, 91), and of packed sequences the host knows none.
        long long steps = 0;
        for (int t = 0; t < key_tiles; ++t) steps += key_steps<D>(p, t);
        const long long all = (long long)key_tiles * p.splits - key_tiles / 2;   // half a split of a tile is lost in rounding
        const long long each = ((long long)(p.Hq / p.Hkv) * steps + all - 1) / all, least = kSplitQueries / kKM<D>;
        p.split_steps = (int)(each > least ? each : least);
        p.splits = attn_bwd_splits_most(p.splits, p.Tk);
    }
    long long key_items = (long long)key_tiles * p.splits;
    if (p.split_steps > 0) {
        key_items = 0;
        for (int t = 0; t < key_tiles; ++t) key_items += key_splits<D>(p, t);
    }
    key_items *= (long long)p.B * p.Hkv;
    const long long items = key_items + (long long)p.B * p.Hq * query_tiles;
    if (items == 0) return hipSuccess;
    hipLaunchKernelGGL((attn_bwd_kernel<D>), dim3((unsigned)items), dim3(64 * kQWaves), kLds, st, p, (int)key_items, key_tiles,
                       query_tiles);
    e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1 || key_tiles == 0) return e;
    const long long sums = (long long)p.B * p.Hkv * p.Tk * D / 8;
    hipLaunchKernelGGL((attn_dkv_sum<D>), dim3((unsigned)((sums + 255) / 256)), dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnParams& p, hipStream_t st) {
    return p.d == 64 ? launch_bwd_d<64>(p, st) : launch_bwd_d<128>(p, st);
}

}  // namespace gdr
