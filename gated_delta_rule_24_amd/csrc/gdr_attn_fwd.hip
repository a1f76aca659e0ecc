// Causal attention, forward, over the whole past or a window, packed sequences
// and shared key heads included:
//   s_ij = scale q_i . k_j   (j <= p_i, j > p_i - window, same sequence; p_i = i + Tk - Tq)
//   o_i = sum_j exp(s_ij - m_i) v_j / l_i,  lse_i = m_i + log l_i
// in one pass over the keys with a running maximum m and sum l (fp32).
//
// A workgroup takes 128 queries of one head, 32 per wave, and walks the keys they
// see in tiles of 64, staged through LDS by direct loads one tile ahead.
//   S^T[key][query] = K Q^T      (32x32x16 MFMA, queries in registers throughout)
//   O^T[channel][query] += V^T P^T
// Both leave a lane with one query (column lane & 31), so the maximum, the sum
// and the rescaling are per lane, and S^T's registers are P^T's operand as they
// stand: an MFMA contracts over any order of the keys that both operands share,
// so the value operand is read with the same order (transposing LDS reads).
//
// The weights are rounded to bf16 for the product with v: the matrix instruction takes
// both operands in one type, and v is bf16 (their sum l is of the fp32 weights).
//
// Bound by matrix cores and vector work taking turns (46% and 44% of the cycles): two workgroups on a
// compute unit, so that one's softmax runs beside the other's products, overlap
// no more of them than that.  On random data the card lowers its clock from 2.4 to about
// 1.9 GHz (all inputs zero: 203 us for 257; a library's product of two 8192 x 8192
// matrices, which has the same clock, 612 for 790: 1,390 TFLOP/s).  Measured, d = 128: 2 x 8,192
// tokens, 16 heads, window 2,048 260 us, 927 TFLOP/s; 16,384 packed tokens as 19
// sequences, 16 heads on 4, 135 us, 628 TFLOP/s (two fifths of the tiles are seen in
// part, and the workgroups' lengths differ); 257 tokens 7.5 us on the GPU, 10 a call.
// Measured and not taken (first case, 254 to 262 beside them): 64 queries a wave and
// one wave a SIMD 296; tiles of 32 keys and three waves a SIMD 273; the scores of a
// tile beside the output of the one before it, in one wave 282.
#include <type_traits>

#include "gdr_attn_tile.h"

namespace gdr {

using namespace attn;

namespace {

constexpr int kBM = 128, kBN = 64, kWaves = 4;

template <int D>
struct __attribute__((aligned(256))) FwdSmem {
    uint16_t k[2][kBN * D];
    uint16_t v[2][kBN * D];
    int bad[kWaves];
};

// The wave's 32 rows from the definition (see dot_row); lane r % 32 holds row r's
// key range.
template <int D>
__device__ __forceinline__ void rows_one_by_one(const AttnParams& p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                                uint16_t* o, float* lse, int first, int used, int lo32, int hi32, int lane) {
    const float to2 = p.scale * kLog2e;
    for (int r = 0; r < 32 && first + r < used; ++r) {
        const int lo = __builtin_amdgcn_readlane(lo32, r), hi = __builtin_amdgcn_readlane(hi32, r);
        const uint16_t* qr = q + (long long)(first + r) * p.sq.t;
        float m = -INFINITY, l = 0.f, acc[D / 64] = {};
        for (int j = lo + lane; j < hi; j += 64) m = fmaxf(m, dot_row<D>(qr, k + (long long)j * p.sk.t) * to2);
        for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
        const float shift = m == -INFINITY ? 0.f : m;
        for (int j0 = lo; j0 < hi; j0 += 64) {
            float w = 0.f;
            if (j0 + lane < hi) w = __builtin_amdgcn_exp2f(dot_row<D>(qr, k + (long long)(j0 + lane) * p.sk.t) * to2 - shift);
            l += w;
            add_rows<D>(acc, w, v + (long long)j0 * p.sk.t, p.sk.t, min(64, hi - j0), lane);
        }
        for (int x = 32; x > 0; x >>= 1) l += __shfl_xor(l, x, 64);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) o[(long long)(first + r) * p.sq.t + lane + 64 * c] = f32_to_bf16(acc[c] * inv);
        if (lse && lane == 0) lse[first + r] = hi <= lo ? -INFINITY : shift / kLog2e + logf(l);
    }
}

}  // namespace

template <int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_fwd_kernel(AttnParams p, int tiles) {
    constexpr int KS = D / 16, DB = D / 32;
    extern __shared__ __attribute__((aligned(256))) char smem[];
    FwdSmem<D>& sm = *reinterpret_cast<FwdSmem<D>*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;

    int unit, tile;
    work_item(blockIdx.x, p.B * p.Hq, tiles, unit, tile);
    tile = tiles - 1 - tile;                          // the rows that see most keys first
    const int b = unit / p.Hq, hq = unit % p.Hq, hk = hq / (p.Hq / p.Hkv);
    const int r0 = tile * kBM;

    const uint16_t* qp = (const uint16_t*)p.q + b * p.sq.b + hq * p.sq.h;
    bf8v qf[KS];
    {
        const uint16_t* qr = qp + (long long)min(r0 + 32 * wave + col, p.Tq - 1) * p.sq.t + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>(qr + 16 * s));
    }
    SeqRows seq = {p.Tq, 0, 0, 0, false};
    if (p.cu_seqlens) seq = seq_rows<kBM, false>(p.cu_seqlens, p.nseq, p.Tq, r0, r0 + 32 * wave, lane);
    const int used = seq.used;
    if (r0 >= used) return;
    const int row = r0 + 32 * wave + col;
    const int at = row + p.Tk - p.Tq;                 // the query's place among the keys
    const bool live = row < used;
    int lo = seq.mine, hi = live ? at + 1 : 0;
    if (p.window > 0 && at - p.window + 1 > lo) lo = at - p.window + 1;
    if (hi <= lo) { lo = 0; hi = 0; }                 // sees nothing
    // the workgroup's keys: rows are in order, so their first and last rows bound them
    const int last_row = min(r0 + kBM, used) - 1;
    const int end = last_row + p.Tk - p.Tq + 1;
    int begin = seq.first;
    if (p.window > 0) begin = max(begin, r0 + p.Tk - p.Tq - p.window + 1);
    begin = max(begin, 0);
    // keys from lo_most on and below hi_least are seen by every row
    int lo_most = seq.last;
    if (p.window > 0) lo_most = max(lo_most, last_row + p.Tk - p.Tq - p.window + 1);
    const int hi_least = r0 + p.Tk - p.Tq + 1;

    const uint16_t* kp = (const uint16_t*)p.k + b * p.sk.b + hk * p.sk.h;
    const uint16_t* vp = (const uint16_t*)p.v + b * p.sk.b + hk * p.sk.h;

    float16v o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float to2 = p.scale * kLog2e;

    // two tiles a turn, so that every LDS address is a fixed register and a constant
    const ReadAt<D> kt = ReadAt<D>(lane).in(lds_address(sm.k[0]));
    const Stager<D, kBN, kWaves, true> loads(p.sk.t, wave, lane);
    const int j_first = begin / kBN * kBN;
    const int n = end > begin ? (end - j_first + kBN - 1) / kBN : 0;
    const int last = p.cu_seqlens ? used - 1 : p.Tk - 1;   // of the keys that count
    uint64_t k_rows = loads.rows(kp, j_first), v_rows = loads.rows(vp, j_first);
    const uint64_t tile_bytes = (uint64_t)kBN * 2 * p.sk.t;
    const uint32_t k_lds = lds_address(sm.k[0]), v_lds = lds_address(sm.v[0]);
    float shift = 0.f;
    bool bad = false;
    int j0 = j_first;
    if (n > 0) {
        loads.load(k_rows, j0, last, k_lds, lane);
        loads.load(v_rows, j0, last, v_lds, lane);
    }
    // one tile, in buffer BUF; false ends the walk
    auto tile_step = [&](auto buffer) {
        constexpr int BUF = decltype(buffer)::value, kTile = kBN * D * 2;
        constexpr int kK = BUF * kTile, kV = (int)(offsetof(FwdSmem<D>, v) - offsetof(FwdSmem<D>, k)) + BUF * kTile;
        wait_loads();
        lds_barrier();
        if (j0 + kBN < end) {
            k_rows += tile_bytes;
            v_rows += tile_bytes;
            loads.load(k_rows, j0 + kBN, last, k_lds + (BUF ^ 1) * kTile, lane);
            loads.load(v_rows, j0 + kBN, last, v_lds + (BUF ^ 1) * kTile, lane);
        }
        // tiles that some row of the workgroup sees in part: infinities and NaN among
        // values that are masked for a row must not reach it through 0 * inf
        const bool edge = j0 < lo_most || j0 + kBN > hi_least;
        if (edge) {
            const bool mine = any_not_finite<D>(sm.v[BUF] + 16 * wave * D, lane);
            if (lane == 0) sm.bad[wave] = mine;
            lds_barrier();
            bad = (sm.bad[0] | sm.bad[1] | sm.bad[2] | sm.bad[3]) != 0;
            if (bad) return false;
        }
        if (!edge || __any(hi > j0 && lo < j0 + kBN)) {
            float16v st[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
                for (int j = 0; j < 16; ++j) st[kb][j] = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    st[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kt.row_frag(32 * kb, s, kK), qf[s], st[kb], 0, 0, 0);
            }
            sched_reads_ahead<4, 2 * KS, 1>();
            if (edge) {
                const int base = j0 + 4 * h - lo;
                const unsigned seen = (unsigned)(hi - lo);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if ((unsigned)(base + 32 * kb + 8 * (i / 4) + i % 4) >= seen) st[kb][i] = -INFINITY;
            }
            float top = st[0][0];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, st[kb][i]);
            top = max_across32(top);
            // m follows the maximum only when that is more than 2^8 ahead: weights up to
            // 2^8 keep their relative precision, and the sums their room, while some row
            // of 32 has a new maximum in most tiles (64 products to rescale o).  Each row
            // goes by its own maximum, the others' factor is 1: the roundings of a row
            // do not depend on keys that only its neighbours see
            const bool ahead = (top - m) * to2 > 8.f;
            if (__any(ahead)) {
                asm volatile("");                         // a branch, not 64 products and selects
                top = ahead ? top : m;
                const float fade = m == top ? 1.f : __builtin_amdgcn_exp2f((m - top) * to2);
                m = top;
                shift = top == -INFINITY ? 0.f : top * to2;
                l *= fade;
#pragma unroll
                for (int i = 0; i < DB; ++i) o[i] *= fade;
            }
            float sum[2] = {0.f, 0.f};
            bf8v pf[4];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = __builtin_amdgcn_exp2f(st[kb][i] * to2 - shift);
                    sum[kb] += x;
                    pf[2 * kb + i / 8][i % 8] = (__bf16)x;
                }
            l += sum[0] + sum[1];
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int i = 0; i < DB; ++i)
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kt.col_frag(16 * s, i, kV), pf[s], o[i], 0, 0, 0);
            sched_reads_ahead<4, 4 * DB, 2>();
        }
        j0 += kBN;
        return j0 < end;
    };
    if (n > 0)
        while (tile_step(std::integral_constant<int, 0>{}) && tile_step(std::integral_constant<int, 1>{})) {
        }
    if (bad) {
        wait_loads();                                 // no load into LDS outlives the wave
        rows_one_by_one<D>(p, qp, kp, vp, (uint16_t*)p.o + b * p.sq.b + hq * p.sq.h,
                           p.lse ? p.lse + ((long long)b * p.Hq + hq) * p.Tq : nullptr, r0 + 32 * wave, used, lo, hi, lane);
        return;
    }

    l = sum_across32(l);
    if (live) {
        // a row that saw nothing has l = 0: its output is 0, its log-sum-exp -inf
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* orow = (uint16_t*)p.o + b * p.sq.b + hq * p.sq.h + (long long)row * p.sq.t;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint2 u = make_uint2(pack_bf16(o[i][4 * j] * inv, o[i][4 * j + 1] * inv),
                                           pack_bf16(o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv));
                *reinterpret_cast<uint2*>(orow + 32 * i + 8 * j + 4 * h) = u;
            }
        if (p.lse && h == 0)
            p.lse[((long long)b * p.Hq + hq) * p.Tq + row] = hi <= lo ? -INFINITY : m * p.scale + logf(l);
    }
}

long long attn_fwd_workgroups(int B, int Hq, int Tq) { return (long long)B * Hq * (((long long)Tq + kBM - 1) / kBM); }

template <int D>
static hipError_t launch_fwd_d(const AttnParams& p, hipStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const void* fn = reinterpret_cast<const void*>(&attn_fwd_kernel<D>);
    const hipError_t e = ensure_dyn_lds(fn, (int)sizeof(FwdSmem<D>), done);
    if (e != hipSuccess) return e;
    const int tiles = (p.Tq + kBM - 1) / kBM;
    if (tiles == 0) return hipSuccess;
    hipLaunchKernelGGL((attn_fwd_kernel<D>), dim3((unsigned)attn_fwd_workgroups(p.B, p.Hq, p.Tq)), dim3(64 * kWaves),
                       sizeof(FwdSmem<D>), st, p, tiles);
    return hipGetLastError();
}

hipError_t launch_attn_fwd(const AttnParams& p, hipStream_t st) {
    return p.d == 64 ? launch_fwd_d<64>(p, st) : launch_fwd_d<128>(p, st);
}

}  // namespace gdr
