// The paged 8-bit key/value cache: append of new tokens, and attention of one
// query token per sequence over it.
//
// A page holds 64 tokens of every key head: keys [64][d], values [4][d][16]
// (16 tokens side by side, so that a lane's 16-byte load is one channel of 16
// tokens: the value operand of the matrix instruction, no transposing).  Values
// are e4m3; a (page, head) has one scale for its keys and one for its values,
// a power of two, so that a scale that grows later re-rounds only what falls
// below the type's normal range.
#include "gdr_device.h"
#include "gdr_attn.h"
#include "gdr_kv_tile.h"

namespace gdr {

namespace {

constexpr int kPage = 64;

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Exponent of the smallest power of two s >= 2^-96 with top <= 448 s, from
// top = m 2^x, 1 <= m < 2, and 448 = 1.75 * 2^8 (0 and subnormals give the floor).
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t u = __float_as_uint(top);
    const int x = (int)(u >> 23) - 127;
    const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -96 ? -96 : e;
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// four e4m3 values times a power of two r <= 1, rounded again
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float r) {
    return to_e4m3x4(__builtin_amdgcn_cvt_f32_fp8(w, 0) * r, __builtin_amdgcn_cvt_f32_fp8(w, 1) * r,
                     __builtin_amdgcn_cvt_f32_fp8(w, 2) * r, __builtin_amdgcn_cvt_f32_fp8(w, 3) * r);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

}  // namespace

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
//
// Prompts: one workgroup owns one (touched page, head): it reads the new tokens that
// fall into the page (1 to 64), takes their largest magnitude, raises the scale if
// need be (then it re-rounds the page's older tokens), and writes the new ones.
// Bound by HBM: 2 bytes read, 1 written per value.  The page's other slots are left
// as they were.  One workgroup a page because the page's one scale needs the largest
// of its new values before the first is rounded: they stay in registers between, so
// that each is read once (19 prompts, 16,384 tokens x 8 heads x 128: 25.6 us, 3.9 TB/s).
template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendParams p) {
    constexpr int VPT = D / 8;                        // 16-byte vectors of a token
    constexpr int NV = kPage * VPT / 256;             // vectors a thread may hold
    __shared__ __attribute__((aligned(16))) uint8_t tile[kPage * D];
    __shared__ float s_top[8];
    __shared__ int s_work[4];
    const int tid = threadIdx.x, h = blockIdx.y;

    // which page: sequence, page of it, first new slot, new tokens, their first row
    int seq, page_i, off, n, row;
    {
        // item blockIdx.x of the sequences' touched pages in order: a running
        // sum over 256 sequences at a time
        if (tid == 0) s_work[0] = -1;
        int before = 0;
        bool found = false;
        for (int s0 = 0; s0 < p.nseq && !found; s0 += 256) {
            const int s = s0 + tid;
            int cnt = 0, a = 0, m = 0, len = 0;
            if (s < p.nseq) {
                a = clampi(p.cu_seqlens[s], 0, p.T);
                m = clampi(p.cu_seqlens[s + 1], a, p.T) - a;
                len = max(p.cache_len[s], 0);
                cnt = m > 0 ? (len % kPage + m + kPage - 1) / kPage : 0;
            }
            int run = cnt;
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(run, o, 64);
                if ((tid & 63) >= o) run += y;
            }
            __syncthreads();
            if ((tid & 63) == 63) s_top[tid >> 6] = __int_as_float(run);
            __syncthreads();
            int base = before, total = 0;
            for (int w = 0; w < 4; ++w) {
                const int c = __float_as_int(s_top[w]);
                if (w < (tid >> 6)) base += c;
                total += c;
            }
            const int end = base + run, begin = end - cnt, item = blockIdx.x;
            if (item >= begin && item < end) {
                const int i = item - begin, o = len % kPage;
                const int from = i == 0 ? 0 : i * kPage - o;      // first of the sequence's new tokens here
                s_work[1] = len / kPage + i;
                s_work[2] = i == 0 ? o : 0;
                s_work[3] = a + from;
                s_work[0] = s;
                s_top[4] = __int_as_float(min(m - from, kPage - (i == 0 ? o : 0)));
            }
            __syncthreads();
            found = s_work[0] >= 0;
            before += total;
        }
        if (!found) return;
        seq = s_work[0]; page_i = s_work[1]; off = s_work[2]; row = s_work[3];
        n = __float_as_int(s_top[4]);
        __syncthreads();
    }
    if (page_i >= p.max_pages) return;                // past the table: dropped
    const int page = p.block_table[(size_t)seq * p.max_pages + page_i];
    if ((unsigned)page >= (unsigned)p.n_pages) return;

    const size_t ph = (size_t)page * p.Hkv + h;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint16_t* src = (const uint16_t*)(side ? p.v : p.k) + (long long)row * p.st + (long long)h * p.sh;
        uint8_t* dst = (side ? p.v_cache : p.k_cache) + ph * (kPage * D);
        float* scale_at = (side ? p.v_scale : p.k_scale) + ph;
        const float old = off > 0 ? *scale_at : 0.f;
        uint4 x[NV];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + 256 * i, t = vec / VPT, c = vec % VPT;
            x[i] = make_uint4(0, 0, 0, 0);
            if (t < n) x[i] = *reinterpret_cast<const uint4*>(src + (long long)t * p.st + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {             // infinities and NaN have no part in the scale
                const float a = fabsf(__uint_as_float(w[j] << 16)), b = fabsf(__uint_as_float(w[j] & 0xffff0000u));
                if (a < INFINITY) top = fmaxf(top, a);
                if (b < INFINITY) top = fmaxf(top, b);
            }
        }
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        __syncthreads();
        if ((tid & 63) == 0) s_top[tid >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
        const int e = scale_exponent(top);
        const float s = fmaxf(old, exp2_int(e)), inv = 1.f / s;      // exact: powers of two
        const bool grew = off > 0 && s != old;
        const float r = old * inv;
        if (tid == 0) *scale_at = s;
        // the new tokens' bytes: keys straight to their rows, values through LDS
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vec = tid + 256 * i, t = vec / VPT, c = vec % VPT;
            if (t < n) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = __uint_as_float(w[j] << 16) * inv;
                    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * inv;
                }
                const uint2 y = make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
                if (side == 0) *reinterpret_cast<uint2*>(dst + (size_t)(off + t) * D + 8 * c) = y;
                else *reinterpret_cast<uint2*>(tile + (off + t) * D + 8 * c) = y;
            }
        }
        if (side == 0) {
            if (grew)
                for (int vec = tid; vec < off * (D / 16); vec += 256) {
                    uint4* at = reinterpret_cast<uint4*>(dst + (size_t)vec * 16);
                    const uint4 y = *at;
                    *at = make_uint4(rescale_e4m3x4(y.x, r), rescale_e4m3x4(y.y, r), rescale_e4m3x4(y.z, r),
                                     rescale_e4m3x4(y.w, r));
                }
        } else {
            __syncthreads();
            const int lo = grew ? 0 : off, hi = off + n;
            // 16 slots of one channel: written whole where all are new, else the
            // new bytes one by one, or (scale grown) read, re-rounded and merged
            for (int vec = tid; vec < 4 * D; vec += 256) {
                const int g = vec / D, c = vec % D, first = 16 * g;
                if (first >= hi || first + 16 <= lo) continue;
                uint8_t* at = dst + (size_t)vec * 16;
                if (!grew && (first < off || first + 16 > hi)) {
                    for (int j = max(first, off); j < min(first + 16, hi); ++j) at[j - first] = tile[j * D + c];
                    continue;
                }
                uint32_t w[4] = {0, 0, 0, 0};
                if (first < off || first + 16 > hi) {
                    const uint4 y = *reinterpret_cast<const uint4*>(at);
                    w[0] = y.x; w[1] = y.y; w[2] = y.z; w[3] = y.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t again = rescale_e4m3x4(w[j], r);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int slot = first + 4 * j + b;
                        const uint32_t m = 0xffu << (8 * b);
                        if (slot < off) w[j] = (w[j] & ~m) | (again & m);
                        else if (slot < hi) w[j] = (w[j] & ~m) | ((uint32_t)tile[slot * D + c] << (8 * b));
                    }
                }
                *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// One token of each sequence: 2 L lanes (L = D / 8) own one (sequence, head), L for
// its keys and L for its values, 8 channels a lane, so that the call is one short
// chain of reads (length, page, scale) beside the tokens' own: bound by latency (256
// sequences x 8 heads: 5 us on the GPU at its shortest, 9 in the mean of single calls, and
// 9.9 a call from Python, which the host bounds; with the prompts' kernel the GPU bounded
// it, at 10.9).
template <int D>
__global__ __launch_bounds__(256) void kv_append_one_kernel(KvAppendParams p) {
    constexpr int L = D / 8;
    const long long item = (long long)blockIdx.x * (128 / L) + threadIdx.x / (2 * L);
    const int c = threadIdx.x % L;
    const bool value = (threadIdx.x / L) % 2 != 0;
    if (item >= (long long)p.nseq * p.Hkv) return;
    const int seq = (int)(item / p.Hkv), h = (int)(item % p.Hkv);
    const uint4 x = *reinterpret_cast<const uint4*>((const uint16_t*)(value ? p.v : p.k) + (long long)seq * p.st +
                                                    (long long)h * p.sh + 8 * c);
    const int len = max(p.cache_len[seq], 0), page_i = len / kPage, off = len % kPage;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = fabsf(__uint_as_float(w[j] << 16)), b = fabsf(__uint_as_float(w[j] & 0xffff0000u));
        if (a < INFINITY) top = fmaxf(top, a);
        if (b < INFINITY) top = fmaxf(top, b);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, L));
    if (page_i >= p.max_pages) return;                // past the table: dropped
    const int page = p.block_table[(size_t)seq * p.max_pages + page_i];
    if ((unsigned)page >= (unsigned)p.n_pages) return;
    const size_t ph = (size_t)page * p.Hkv + h;
    uint8_t* dst = (value ? p.v_cache : p.k_cache) + ph * (kPage * D);
    float* scale_at = (value ? p.v_scale : p.k_scale) + ph;
    const float old = off > 0 ? *scale_at : 0.f;
    const float s = fmaxf(old, exp2_int(scale_exponent(top))), inv = 1.f / s;
    if (off > 0 && s != old) {
        // the scale grew: the older tokens again, by this lane group alone, before the
        // new one is written into the same 16 bytes
        const float r = old * inv;
        const int vecs = value ? 4 * D : off * (D / 16);
        for (int vec = c; vec < vecs; vec += L) {
            const int first = 16 * (vec / D);
            if (value && first >= off) break;         // later groups of 16 tokens hold none
            uint4* at = reinterpret_cast<uint4*>(dst + (size_t)vec * 16);
            const uint4 y = *at;
            uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t again = rescale_e4m3x4(u[j], r);
                uint32_t m = 0xffffffffu;
                if (value) {                          // slots from `off` on stay
                    m = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (first + 4 * j + b < off) m |= 0xffu << (8 * b);
                }
                u[j] = (u[j] & ~m) | (again & m);
            }
            *at = make_uint4(u[0], u[1], u[2], u[3]);
        }
        __threadfence();
    }
    if (c == 0) *scale_at = s;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16) * inv;
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * inv;
    }
    const uint2 y = make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
    if (!value) {
        *reinterpret_cast<uint2*>(dst + off * D + 8 * c) = y;
    } else {
        uint8_t* at = dst + ((off / 16) * D + 8 * c) * 16 + off % 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) at[16 * j] = (uint8_t)((j < 4 ? y.x : y.y) >> (8 * (j % 4)));
    }
}

long long kv_append_workgroups(int nseq, int Hkv, int T, int d, bool packed) {
    // a sequence's m new tokens touch at most m / 64 + 2 pages
    if (packed) return (long long)T / kPage + 2LL * nseq;
    const long long pairs = (long long)nseq * Hkv, per = 1024 / d;
    return (pairs + per - 1) / per;
}

hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t st) {
    const unsigned items = (unsigned)kv_append_workgroups(p.nseq, p.Hkv, p.T, p.d, p.cu_seqlens != nullptr);
    if (!p.cu_seqlens) {
        dim3 grid(items), block(256);
        if (p.d == 64) hipLaunchKernelGGL((kv_append_one_kernel<64>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((kv_append_one_kernel<128>), grid, block, 0, st, p);
        return hipGetLastError();
    }
    dim3 grid(items, (unsigned)p.Hkv), block(256);
    if (p.d == 64) hipLaunchKernelGGL((kv_append_kernel<64>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((kv_append_kernel<128>), grid, block, 0, st, p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
//
// o = sum_j p_j v_j / sum_j p_j, p_j = exp2(s_j - m), s_j = scale log2(e) q.k_j,
// over the last `window` of the cached tokens (all: window 0).  Two bytes are
// read per token and channel, and that is the bound: everything else fits beside
// the reads.  A workgroup takes one run of pages of one (sequence, key head); its
// four waves take pages in turn, each with its own running maximum and sum, and
// join at the end.  Up to 16 query heads share the key head's reads as the 16
// columns of one matrix instruction.
//   scores  S^T[key][query] = K Q^T: a lane loads 16 bytes of a key's row (two
//           instructions' worth); the key a tile's row m stands for is
//           16 (m / 4) + 4 tile + m % 4, which leaves lane group g with the
//           scores of keys 16 g .. 16 g + 15: the keys of its value loads.
//   output  O^T[channel][query] += V^T W^T with the weights W = exp2(s + log2 v_scale),
//           relative to their own running maximum and 2^15 times that, as the sum of
//           two f16 values: 22 bits of a weight count, down to 2^-39 of the largest,
//           whatever the pages' scales, so that an fp32 result is one (with two bf16
//           values, 8 bits each, results were 1.3e-6 off).
// e4m3 is exact in bf16 and f16.
// Measured, 32 query heads on 8, d = 128: 256 sequences of up to 8,192 tokens 474 us,
// 5.55 TB/s (a plain sum of as many bytes reads 6.15); one of 50,000 26.8 us: 20 for
// the pages, 4 for the join of the splits, the rest between the two launches (24.1 to 24.6
// where call after call reads the same pages, out of the last cache).
// Two limits.  The splits follow the block table's width, as the host does not know the
// lengths: the sequence of 50,000 tokens takes 28 us behind a table of 782 pages, 35
// behind 2,048 and 190 behind 16,384.  And the cache is read once for each 16 query heads
// of a key head: 32 sequences of up to 8,192 tokens with 16, 32, 64 and 128 heads on one
// take 18, 24, 38 and 65 us.
namespace {

constexpr int kDecWaves = 4;

template <int D>
struct DecodeSmem {
    float o[kDecWaves][16][D + 4];
    float ml[kDecWaves][16][2];
};

__device__ __forceinline__ void store_out(const AttnDecodeParams& p, size_t idx, float x) {
    if (p.flags & GDR_OUT_BF16) reinterpret_cast<uint16_t*>(p.o)[idx] = f32_to_bf16(x);
    else reinterpret_cast<float*>(p.o)[idx] = x;
}

// first and one past the last cached token a query of this sequence sees
__device__ __forceinline__ void decode_range(const AttnDecodeParams& p, int n, int& lo, int& hi) {
    const long long room = (long long)p.max_pages * kPage;
    const int len = p.cache_len[n];
    hi = len < 0 ? 0 : (int)(len > room ? room : len);
    lo = (p.window > 0 && len > p.window) ? min(len - p.window, hi) : 0;
}

}  // namespace

template <int D>
__global__ __launch_bounds__(64 * kDecWaves) void attn_decode_kernel(AttnDecodeParams p, int groups) {
    constexpr int KS = D / 64;                        // 64-channel steps of a key row
    constexpr int VT = D / 16;                        // 16-channel tiles of the output
    __shared__ DecodeSmem<D> sm;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    int w = blockIdx.x;
    const int qg = w % groups; w /= groups;
    const int kh = w % p.Hkv; w /= p.Hkv;
    const int n = w, split = blockIdx.y;
    const int G = p.Hq / p.Hkv, q0 = kh * G + 16 * qg, nq = min(16, G - 16 * qg);

    int lo, hi;
    decode_range(p, n, lo, hi);
    const int pg0 = lo / kPage + split * p.split_pages;
    const int pg1 = min(pg0 + p.split_pages, (hi + kPage - 1) / kPage);
    const bool none = pg0 >= pg1;
    if (none && split > 0) return;                    // the join leaves this split out

    // queries: column col, channels 64 s + 16 g + 8 half ..
    bf8v qf[KS][2];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (col < nq)
                u = *reinterpret_cast<const uint4*>((const uint16_t*)p.q + ((size_t)n * p.Hq + q0 + col) * D + 64 * s +
                                                    16 * g + 8 * hf);
            qf[s][hf] = __builtin_bit_cast(bf8v, u);
        }

    float4v o[VT];
#pragma unroll
    for (int i = 0; i < VT; ++i) o[i] = float4v{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f, wm = -INFINITY;     // maximum and sum of the scores; maximum of the weights
    const float to2 = p.scale * 1.4426950408889634f;
    const int krow = 16 * (col >> 2) + (col & 3);     // key of tile 0's row `col`

    for (int pg = pg0 + wave; pg < pg1; pg += kDecWaves) {
        int page = p.block_table[(size_t)n * p.max_pages + pg];
        const int first = pg * kPage;
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
        for (int i = 0; i < VT; ++i)
            vv[i] = *reinterpret_cast<const uint4*>(vp + (size_t)(g * D + 16 * i + col) * 16);
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
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[t][i] *= ks;
        }
        if (absent || first < lo || first + kPage > hi) {
            // the first and last pages: masked keys count nothing, whatever their bytes
            uint32_t keep[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                keep[t] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = first + 16 * g + 4 * t + i;
                    const bool in = !absent && j >= lo && j < hi;
                    if (!in) sc[t][i] = -INFINITY;
                    else keep[t] |= 0xffu << (8 * i);
                }
            }
#pragma unroll
            for (int i = 0; i < VT; ++i) {
                vv[i].x &= keep[0]; vv[i].y &= keep[1]; vv[i].z &= keep[2]; vv[i].w &= keep[3];
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
        for (int i = 0; i < VT; ++i) o[i] *= fade;
        half8 hi8[2], lo8[2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l += __builtin_amdgcn_exp2f(sc[t][i] - at);
                const float x = __builtin_amdgcn_exp2f(sc[t][i] + up);
                const _Float16 a = (_Float16)x;
                hi8[t >> 1][(t & 1) * 4 + i] = a;
                lo8[t >> 1][(t & 1) * 4 + i] = (_Float16)(x - (float)a);
            }
#pragma unroll
        for (int i = 0; i < VT; ++i) {
            const half8 v0 = e4m3x8_to_f16(vv[i].x, vv[i].y), v1 = e4m3x8_to_f16(vv[i].z, vv[i].w);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, hi8[0], o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, hi8[1], o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, lo8[0], o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, lo8[1], o[i], 0, 0, 0);
        }
    }

    // join the waves: sums over the lane groups, then over the waves
    l += __shfl_xor(l, 16, 64);
    l = sum_across32(l);
    if (g == 0) { sm.ml[wave][col][0] = m; sm.ml[wave][col][1] = l; }
    const float down = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm - m - 15.f);   // to the scores' maximum
#pragma unroll
    for (int i = 0; i < VT; ++i)
        *reinterpret_cast<float4v*>(&sm.o[wave][col][16 * i + 4 * g]) = o[i] * down;
    __syncthreads();
    for (int idx = threadIdx.x; idx < nq * D; idx += 64 * kDecWaves) {
        const int c = idx / D, ch = idx % D;
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < kDecWaves; ++y) top = fmaxf(top, sm.ml[y][c][0]);
        const float at = top == -INFINITY ? 0.f : top;
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int y = 0; y < kDecWaves; ++y) {
            const float f = __builtin_amdgcn_exp2f(sm.ml[y][c][0] - at);
            sum += sm.ml[y][c][1] * f;
            x += sm.o[y][c][ch] * f;
        }
        const size_t head = (size_t)n * p.Hq + q0 + c;
        if (p.splits == 1) {
            store_out(p, head * D + ch, top == -INFINITY && !(x != x) ? 0.f : x / sum);
        } else {
            const size_t at_row = (size_t)split * p.N * p.Hq + head;
            p.part_o[at_row * D + ch] = x;
            if (ch == 0) { p.part_ml[at_row * 2] = top; p.part_ml[at_row * 2 + 1] = sum; }
        }
    }
}

// Joins the splits that have pages: one workgroup per head; its lanes read the
// splits' maxima and sums side by side, then 1024 / D groups of them the outputs.
template <int D>
__global__ __launch_bounds__(256) void attn_decode_join(AttnDecodeParams p) {
    constexpr int GROUPS = 1024 / D;                  // D / 4 lanes each, four channels a lane
    __shared__ float s_x[GROUPS][D], s_ml[8], s_sum;
    const size_t head = blockIdx.x, rows = (size_t)p.N * p.Hq;
    const int tid = threadIdx.x, gi = tid / (D / 4), ch = 4 * (tid % (D / 4));
    int lo, hi;
    decode_range(p, (int)(head / p.Hq), lo, hi);
    const int pages = (hi + kPage - 1) / kPage - lo / kPage;
    const int splits = max(1, (pages + p.split_pages - 1) / p.split_pages);
    float top = -INFINITY, sum = 0.f;
    for (int s = tid; s < splits; s += 256) {
        const float2 ml = *reinterpret_cast<const float2*>(&p.part_ml[(s * rows + head) * 2]);
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
    float4v x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = gi; s < splits; s += GROUPS) {
        const float f = __builtin_amdgcn_exp2f(p.part_ml[(s * rows + head) * 2] - at);
        x += *reinterpret_cast<const float4v*>(&p.part_o[(s * rows + head) * D + ch]) * f;
    }
    *reinterpret_cast<float4v*>(&s_x[gi][ch]) = x;
    __syncthreads();
    if (tid < D) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) y += s_x[i][tid];
        store_out(p, head * D + tid, top == -INFINITY && !(y != y) ? 0.f : y / s_sum);
    }
}

int attn_decode_splits(int N, int Hq, int Hkv, int max_pages, int window, int* split_pages) {
    const int G = Hq / Hkv, groups = (G + 15) / 16;
    const long long base = (long long)N * Hkv * groups;
    int pages = max_pages;
    if (window > 0 && window / kPage + 2 < pages) pages = window / kPage + 2;
    // Few (sequence, head) pairs: at most two workgroups on a compute unit, every
    // one at work at once (one sequence of 50,000 tokens x 8 heads: 24.6 us with 392
    // workgroups, 27.3 with 784, 31.4 with 200; 100,000: 38.5 with 392, 41.8 with 784; on
    // the same pages call after call).
    // Many: splits for balance among ragged lengths, up to about 3,000 workgroups (256
    // sequences of up to 8,192 tokens x 8 heads: 474 us, with up to 2,560 492, 4,096 483;
    // 100 of up to 4,000: 113, 113, 112).  The same pages for each wave, two at least.
    const long long fill = base < 256 ? 512 : 3000;
    long long per = (pages * base + fill - 1) / fill;
    per = (per + kDecWaves - 1) / kDecWaves * kDecWaves;
    if (per < 2 * kDecWaves) per = 2 * kDecWaves;
    *split_pages = (int)per;
    const long long s = (pages + per - 1) / per;
    return s < 1 ? 1 : (int)s;
}

// (the join, a workgroup a head, runs only where these are few: see attn_decode_splits)
long long attn_decode_workgroups(int N, int Hq, int Hkv) { return (long long)N * Hkv * ((Hq / Hkv + 15) / 16); }

hipError_t launch_attn_decode(const AttnDecodeParams& p, hipStream_t st) {
    const int groups = (p.Hq / p.Hkv + 15) / 16;
    dim3 grid((unsigned)attn_decode_workgroups(p.N, p.Hq, p.Hkv), (unsigned)p.splits), block(64 * kDecWaves);
    if (p.d == 64) hipLaunchKernelGGL((attn_decode_kernel<64>), grid, block, 0, st, p, groups);
    else hipLaunchKernelGGL((attn_decode_kernel<128>), grid, block, 0, st, p, groups);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    dim3 jgrid((unsigned)((long long)p.N * p.Hq));
    if (p.d == 64) hipLaunchKernelGGL((attn_decode_join<64>), jgrid, block, 0, st, p);
    else hipLaunchKernelGGL((attn_decode_join<128>), jgrid, block, 0, st, p);
    return hipGetLastError();
}

}  // namespace gdr
