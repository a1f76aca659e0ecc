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

#include <limits.h>

#include "gdr_attn.h"
#include "gdr_device.h"
#include "gdr_launch.h"

namespace gdr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

// 16 (4) bytes a lane from base + off (unsigned) to LDS at `to` + `more` + 16 (4)
// lane; `base` and `to` uniform.
template <int MORE> __device__ __forceinline__ void direct_load16(int off, uint64_t base, uint32_t to) {
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 ::"v"(off), "s"(base), "s"(to), "i"(MORE) : "memory", "scc");
}
// the same with a 64-bit address per lane
template <int MORE> __device__ __forceinline__ void direct_load16_far(uint64_t at, uint32_t to) {
    asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 ::"v"(at), "s"(to), "i"(MORE) : "memory", "scc");
}
__device__ __forceinline__ void direct_load4(int off, uint64_t base, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(to) : "memory");
}
// every load of this wave has arrived (its own; a barrier makes the others' visible)
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

template <int D> __device__ __forceinline__ int swz(int r) {
    if constexpr (D == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return ((r & 2) << 1) | ((r >> 2) & 3);
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// ROWS rows of a tensor, its rows `stride` elements apart, into LDS by 16-byte
// direct loads of WAVES waves: lane offsets fixed, a scalar address that moves.  Rows
// past the last are held at it.  The loads are issued in assembly, which the
// compiler does not count: with the builtin it makes every later LDS read wait for
// every load in flight (vmcnt(0)), so the next tile's loads could not stay
// in flight across the work on this one.  They have no output registers;
// wait_loads() and a barrier complete them.  What counts beside the bytes is the
// instructions: KEEP holds one offset register per load (three instructions each),
// otherwise one register serves all (six each).
template <int D, int ROWS, int WAVES, bool KEEP>
struct Stager {
    static constexpr int CH = D / 8, RPI = 64 / CH;  // chunks of a row, rows of one instruction
    static constexpr int N = ROWS / RPI / WAVES;
    static_assert(N * RPI * WAVES == ROWS, "rows split over the waves");
    int off[KEEP ? N : 1];
    uint32_t group;                                   // bytes between two instructions' first rows
    int skip;                                         // rows of the waves before this one

    __device__ __forceinline__ Stager(long long stride, int wave, int lane) {
        const int r = lane / CH;
        group = (uint32_t)(2 * RPI * stride);
        skip = wave * N * RPI;
        const int first = (int)(2 * (r * stride + 8 * ((lane % CH) ^ swz<D>(r))));
#pragma unroll
        for (int i = 0; i < (KEEP ? N : 1); ++i)
            off[i] = KEEP ? (first ^ flip(i)) + (int)(i * group) : first;
    }
    // Address of the wave's first row of the tile that starts at row `first`.
    __device__ __forceinline__ uint64_t rows(const uint16_t* src, int first) const {
        return (uint64_t)src + (uint64_t)((long long)(first + skip) * (group / RPI));
    }
    // the tile that starts at row `first`, its rows() given
    __device__ __forceinline__ void load(uint64_t rows, int first, int last, uint32_t to, int lane) const {
        to += 2 * skip * D;
        if (first + ROWS - 1 <= last) {
            load_all<0>(rows, to);
        } else {
            load_held<0>(rows, first + skip, last, to, lane);
        }
    }

private:
    // the swizzle of a row is that of lane / CH xor that of the instruction's first row
    __device__ __forceinline__ int flip(int i) const { return 16 * swz<D>(skip + i * RPI); }
    template <int I> __device__ __forceinline__ void load_all(uint64_t rows, uint32_t to) const {
        if constexpr (KEEP) direct_load16<1024 * I>(off[I], rows, to);
        else direct_load16<1024 * I>(off[0] ^ flip(I), rows + (uint64_t)I * group, to);
        if constexpr (I + 1 < N) load_all<I + 1>(rows, to);
    }
    // the lane offset is unsigned: rows past the last are reached from the last one,
    // not from a base behind it
    template <int I> __device__ __forceinline__ void load_held(uint64_t rows, int first, int last, uint32_t to, int lane) const {
        const int r = lane / CH, row = first + I * RPI + r, held = row < last ? row : last;
        const long long stride = group / RPI;         // bytes
        const int c = (lane % CH) ^ swz<D>(skip + I * RPI + r);
        // this lane's row relative to the tile's: at most ROWS rows before it or behind
        const uint64_t at = rows + (long long)(held - first) * stride + 16 * c;
        direct_load16_far<1024 * I>(at, to);
        if constexpr (I + 1 < N) load_held<I + 1>(rows, first, last, to, lane);
    }
};

// Keeps the computation of x where it stands (the compiler would sink it past the
// next branch, out from between the products).
template <typename T> __device__ __forceinline__ T here(T x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The lane's number, made anew where it is used: two instructions instead of a
// register across the loop.
__device__ __forceinline__ int lane_now() {
    int x;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(x));
    return x;
}

// Order of N products of R LDS reads each: the reads of AHEAD products go first,
// then products and reads in turn.  Left alone, the compiler reads right before
// each product and waits for every read.
template <int AHEAD, int N, int R> __device__ __forceinline__ void sched_reads_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD * R, 0);       // LDS reads
#pragma unroll
    for (int i = 0; i < N - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);           // a product
        __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
}

// A lane's two read addresses inside a tile, from which every other one follows by
// flipping address bits: the swizzle is an exclusive-or of the chunk, and tiles
// start at multiples of 256 bytes.
template <int D> struct ReadAt {
    uint32_t row, col;

    __device__ __forceinline__ explicit ReadAt(int lane) {
        const int r = lane & 31, h = lane >> 5;
        row = 2 * (r * D + 8 * (h ^ swz<D>(r)));
        const int j = 4 * h + ((lane & 15) >> 2), ch = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        col = 2 * (j * D + 8 * (ch ^ swz<D>(j)) + 4 * (lane & 1));
    }
    // inside the tile at LDS address `tile`
    __device__ __forceinline__ ReadAt in(uint32_t tile) const {
        ReadAt x = *this;
        x.row += tile;
        x.col += tile;
        return x;
    }
    // the same, hidden from the compiler, which would keep every address in a register
    // across the loop (16 more than the key-side gradients have)
    __device__ __forceinline__ ReadAt fresh(uint32_t tile) const {
        ReadAt x = in(tile);
        asm volatile("" : "+v"(x.row), "+v"(x.col));
        return x;
    }
    // operand along d: row `r0` + (lane & 31), channels 16 s + 8 (lane / 32) .. + 7
    // (r0 a multiple of 32, `by` bytes further on)
    __device__ __forceinline__ bf8v row_frag(int r0, int s, int by = 0) const {
        return __builtin_bit_cast(bf8v, *(const __attribute__((address_space(3))) uint4*)(uintptr_t)((row ^ (s << 5)) + 2 * r0 * D + by));
    }
    // operand along the rows: channel 32 db + (lane & 31), rows r .. r + 3 and
    // r + 8 .. r + 11 with r = r0 + 4 (lane / 32) (r0 a multiple of 16)
    __device__ __forceinline__ bf8v col_frag(int r0, int db, int by = 0) const {
        bf8v f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t at = (col ^ (db << 6) ^ (e << 5)) + 2 * (r0 + 8 * e) * D + by;
            const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)(uintptr_t)at);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * e + i] = __builtin_bit_cast(__bf16, (short)x[i]);
        }
        return f;
    }
};

// Whether any of ROWS rows of a tile holds an infinity or NaN.
template <int D, int ROWS = 16> __device__ __forceinline__ bool any_not_finite(const uint16_t* rows, int lane) {
    typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
    ushort2v top = {0, 0};
#pragma unroll
    for (int i = 0; i < ROWS * D / 512; ++i) {
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

// Packed sequences.  For the wave's rows w0 .. w0 + 31 (row w0 + lane % 32) of a
// workgroup's r0 .. r0 + BM - 1: where the row's sequence starts (TO: one past its
// end), the same of the workgroup's first and last row, and whether a sequence starts
// at the row.  `used` is cu[nseq]: rows from there on belong to no sequence.  Values of
// cu outside [0, T] are held inside, so that no content of it leads out of the tensors.
//
// Every wave finds them for itself, in registers: 64 entries of cu are one load, what
// lies at or below a row among them one ballot, and more than 64 are first narrowed to
// the 64th part that holds r0.  That is one trip to memory before the first tile
// where passing the bounds through LDS took 5 us of a workgroup's 31.
struct SeqRows {
    int used, mine, first, last;
    bool starts;
};

template <int BM, bool TO>
__device__ __forceinline__ SeqRows seq_rows(const int* cu, int nseq, int T, int r0, int w0, int lane) {
    auto entry = [&](int i, int end) {
        int c = INT_MAX;
        if (i < end) { c = cu[i]; c = c < 0 ? 0 : c > T ? T : c; }
        return c;
    };
    auto last_upto = [&](int c, int x) {              // the last entry <= x, or 0
        const uint64_t m = __ballot(c <= x);
        return m ? __builtin_amdgcn_readlane(c, 63 - __builtin_clzll(m)) : 0;
    };
    auto first_above = [&](int c, int x) {            // the first entry > x, or T
        const uint64_t m = __ballot(c > x);
        return m ? min(__builtin_amdgcn_readlane(c, __builtin_ctzll(m)), T) : T;
    };
    SeqRows z;
    z.used = __builtin_amdgcn_readfirstlane(entry(nseq, nseq + 1));
    int s = 0, n = nseq + 1;                          // the last entry <= r0 is among s .. s + n - 1
    while (n > 64) {
        const int step = (n + 63) / 64;
        const uint64_t m = __ballot(entry(s + lane * step, s + n) <= r0);
        const int k = m ? 63 - __builtin_clzll(m) : 0;
        s += k * step;
        n = min(step, n - k * step);
    }
    const int row = w0 + (lane & 31), last_row = min(r0 + BM, z.used) - 1;
    z.mine = z.first = z.last = TO ? T : 0;
    z.starts = false;
    for (;; s += 64) {
        const int c = entry(s + lane, nseq + 1);
        if constexpr (TO) {
            z.first = min(z.first, first_above(c, r0));
            z.last = min(z.last, first_above(c, last_row));
            z.mine = min(z.mine, first_above(c, w0 + 31));
        } else {
            z.first = max(z.first, last_upto(c, r0));
            z.last = max(z.last, last_upto(c, last_row));
            z.mine = max(z.mine, last_upto(c, w0));
        }
        for (uint64_t m = __ballot(c >= w0 && c <= w0 + 31); m; m &= m - 1) {
            const int v = __builtin_amdgcn_readlane(c, __builtin_ctzll(m));
            if constexpr (TO) {
                if (row < v) z.mine = min(z.mine, v);
                z.starts = z.starts || row == v;
            } else {
                if (row >= v) z.mine = max(z.mine, v);
            }
        }
        if (s + 64 > nseq || __builtin_amdgcn_readlane(c, 63) > r0 + BM) return z;
    }
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
