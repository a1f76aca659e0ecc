// Tiles of the attention kernels: rows of D bf16 values staged in LDS by direct
// loads, swizzled so that both ways of reading them are free of bank conflicts,
// and the row ranges that packed sequences, the diagonal and the window leave.
//
// One row is CH = D / 8 chunks of 16 bytes; row r keeps chunk c at place
// c ^ swz(r).  The two ways to read:
//   rows     32 rows of one chunk (an operand whose contraction runs along d):
//            the 16 rows of a read phase land on 16 different 16-byte places of
//            the 256-byte bank line;
//   columns  (transposing read: an operand whose contraction runs along the rows)
//            4 rows x 32 bytes per 16 lanes: swz moves neighbouring rows by 64
//            bytes, so 32 lanes cover one bank line exactly.
#pragma once

#include "gdr_attn.h"
#include "gdr_device.h"
#include "gdr_launch.h"

namespace gdr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

template <int D> __device__ __forceinline__ int swz(int r) {
    if constexpr (D == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return ((r & 2) << 1) | ((r >> 2) & 3);
}

// ROWS rows starting at row `first` of a tensor with rows `stride` elements
// apart, into LDS by 16-byte direct loads; row indexes are held inside
// [0, last].  Issued by WAVES waves; complete after the issuing waves' vmcnt
// wait and a barrier.
template <int D, int ROWS, int WAVES>
__device__ __forceinline__ void stage(const uint16_t* src, long long stride, int first, int last, uint16_t* dst,
                                      int wave, int lane) {
    constexpr int CH = D / 8, RPI = 64 / CH;         // rows of one instruction
    constexpr int N = ROWS / RPI / WAVES;
    static_assert(N * RPI * WAVES == ROWS, "rows split over the waves");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r0 = (wave * N + i) * RPI, r = r0 + lane / CH, c = (lane % CH) ^ swz<D>(r);
        int row = first + r;
        row = row < 0 ? 0 : row > last ? last : row;
        const uint16_t* g = src + (long long)row * stride + 8 * c;
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void __attribute__((address_space(1)))*>(
                                             reinterpret_cast<uintptr_t>(g)),
                                         (void __attribute__((address_space(3)))*)(dst + r0 * D), 16, 0, 0);
    }
}

// Operand along d: row `r`, channels 8 c .. 8 c + 7.
template <int D> __device__ __forceinline__ bf8v row_frag(const uint16_t* tile, int r, int c) {
    return __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>(tile + r * D + 8 * (c ^ swz<D>(r))));
}

// Operand along the rows: for the lane's channel 32 db + (lane & 31), rows
// r .. r + 3 and r + 8 .. r + 11 with r = r0 + 4 (lane / 32).
template <int D> __device__ __forceinline__ bf8v col_frag(const uint16_t* tile, int r0, int db, int lane) {
    const int j = (lane & 15) >> 2, h = lane >> 5;
    const int ch = 4 * db + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), in = 4 * (lane & 1);
    bf8v f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * e + 4 * h + j;
        const uint16_t* at = tile + r * D + 8 * (ch ^ swz<D>(r)) + in;
        const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)at);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * e + i] = __builtin_bit_cast(__bf16, (short)x[i]);
    }
    return f;
}

// Whether any of 16 rows of a tile (rows 16 wave ..) holds an infinity or NaN.
template <int D> __device__ __forceinline__ bool any_not_finite(const uint16_t* rows, int lane) {
    typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
    ushort2v top = {0, 0};
#pragma unroll
    for (int i = 0; i < 16 * D / 512; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(rows + 512 * i + 8 * lane);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2v, w[j] & 0x7fff7fffu));
    }
    return __any(top[0] >= 0x7f80 || top[1] >= 0x7f80);
}

// Row by row, for workgroups that met an infinity or NaN in a row that some of
// their other rows do not see (there a matrix product would carry it over as
// 0 * inf): 64 lanes take 64 partners of one row, and each term is formed only
// where the pair is seen.  Slow, and right for every value.
template <int D> __device__ __forceinline__ float dot_row(const uint16_t* x, const uint16_t* y) {
    float sum = 0.f;
#pragma unroll 2
    for (int c = 0; c < D; c += 8) {
        const bf8v a = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>(x + c));
        const bf8v b = __builtin_bit_cast(bf8v, *reinterpret_cast<const uint4*>(y + c));
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += (float)a[j] * (float)b[j];
    }
    return sum;
}
// acc[c] += w of lane t * rows[t][lane + 64 c] for the first n lanes
template <int D>
__device__ __forceinline__ void add_rows(float (&acc)[D / 64], float w, const uint16_t* rows, long long stride, int n, int lane) {
    for (int t = 0; t < n; ++t) {
        const float x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), t));
#pragma unroll
        for (int c = 0; c < D / 64; ++c) acc[c] += x * bf16_to_f32(rows[t * stride + lane + 64 * c]);
    }
}

// Packed sequences: for rows r0 .. r0 + BM - 1 of T, the first row of each one's
// sequence (`from`) or one past its last (`to`).  Values of cu outside [0, T] are
// held inside, so that no content of it leads out of the tensors.  `used` is
// cu[nseq]: rows from there on belong to no sequence.  All threads of the
// workgroup call it; ends with a barrier.
template <int BM, bool TO>
__device__ __forceinline__ void row_bounds(const int* cu, int nseq, int T, int r0, int* bound, int* shared, int tid,
                                           int nthreads, int& used) {
    for (int i = tid; i < BM; i += nthreads) bound[i] = TO ? T : 0;
    if (tid == 0) { shared[0] = TO ? T : 0; shared[1] = 0; }
    __syncthreads();
    int edge = TO ? T : 0;
    for (int s = tid; s <= nseq; s += nthreads) {
        const int raw = cu[s], c = raw < 0 ? 0 : raw > T ? T : raw;
        if (s == nseq) shared[1] = c;
        if constexpr (TO) {                           // the sequence ends at c: rows below c
            if (c >= r0 + BM) edge = c < edge ? c : edge;
            else if (c > r0) bound[c - 1 - r0] = c;
        } else {                                      // a sequence starts at c: rows from c
            if (c <= r0) edge = c > edge ? c : edge;
            else if (c < r0 + BM) bound[c - r0] = c;
        }
    }
    if constexpr (TO) atomicMin(&shared[0], edge);
    else atomicMax(&shared[0], edge);
    __syncthreads();
    // running maximum from the front / minimum from the back, by one wave
    if (tid < 64) {
        constexpr int PER = BM / 64;
        int x[PER];
        int run = shared[0];
        if constexpr (TO) {
            int low = T;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) { const int b = bound[tid * PER + i]; low = b < low ? b : low; x[i] = low; }
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_down(low, o, 64);
                if (tid + o < 64) low = y < low ? y : low;
            }
            int after = __shfl_down(low, 1, 64);
            if (tid == 63) after = T;
            run = after < run ? after : run;
#pragma unroll
            for (int i = 0; i < PER; ++i) bound[tid * PER + i] = x[i] < run ? x[i] : run;
        } else {
            int high = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) { const int b = bound[tid * PER + i]; high = b > high ? b : high; x[i] = high; }
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(high, o, 64);
                if (tid >= o) high = y > high ? y : high;
            }
            int before = __shfl_up(high, 1, 64);
            if (tid == 0) before = 0;
            run = before > run ? before : run;
#pragma unroll
            for (int i = 0; i < PER; ++i) bound[tid * PER + i] = x[i] > run ? x[i] : run;
        }
    }
    __syncthreads();
    used = shared[1];
}

// Work items: unit u of `units` (batch and head), tile t of `tiles`; consecutive
// workgroups go round the 8 XCDs, so each XCD takes a run of units one after the
// other and their keys stay in its L2.
__device__ __forceinline__ void work_item(int bid, int units, int tiles, int& unit, int& tile) {
    if (units % 8 == 0) {
        const int i = bid / 8;
        unit = (bid % 8) * (units / 8) + i / tiles;
        tile = i % tiles;
    } else {
        unit = bid / tiles;
        tile = bid % tiles;
    }
}

}  // namespace attn
}  // namespace gdr
