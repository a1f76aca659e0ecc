// Rotary positions of queries and keys (and, inverted, their gradients):
//   y_a = c x_a - s x_b,  y_b = c x_b + s x_a,
//   c = scale cos(pos f_i),  s = scale sin(pos f_i)   (s negated when inverted)
// for the pairs (a, b) = (2i, 2i+1) or (i, i + rot/2), i < rot/2; the channels
// from rot_dim up are copied.
//
// The kernel moves 2 x size bytes per element and computes next to nothing, so
// it is bound by HBM.  The angle is what costs: at position 10^6 a 32-bit
// product is off by up to 0.06 rad, so pos * f is formed in 64 bits, reduced to
// a fraction of a turn there, and only the fraction goes on in 32 bits.  One
// thread owns 2 VE channels (two 16-byte vectors) of one token, computes their VE
// angles once and applies them to `heads` heads of q and k.
// Measured, bf16: 2 x 8,192 tokens of 16 + 16 heads x 128 50 us, 5.4 TB/s read and
// written (a device copy of that size moves 4.8); fp32 gradients, 4,099 tokens of
// 32 + 8 heads x 64 17.5 us, 4.8 TB/s; 64 tokens 4 us on the GPU, 10 a call from Python.
#include "gdr_device.h"
#include "gdr_attn.h"

namespace gdr {

template <bool F32> struct RopeVec;
template <> struct RopeVec<false> {
    static constexpr int VE = 8;
    uint4 u;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct RopeVec<true> {
    static constexpr int VE = 4;
    uint4 u;
    __device__ __forceinline__ void get(float (&f)[4]) const {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    __device__ __forceinline__ void set(const float (&f)[4]) {
        u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// HEADS heads are loaded before the first is stored, so that a thread has
// 2 HEADS loads in flight (in place as well: a thread reads and writes only
// its own channels).
template <bool F32, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeParams p) {
    using V = RopeVec<F32>;
    constexpr int VE = V::VE, ES = F32 ? 4 : 2, HEADS = 4;
    const int units = p.d / (2 * VE);                // threads of one token: a power of two up to 16
    const long long n = (long long)blockIdx.x * (256 / units) + threadIdx.x / units;
    if (n >= p.rows) return;
    const int u = threadIdx.x % units;
    const int turning = p.rot / (2 * VE);            // units that turn; the others copy
    const long long b = n / p.T;
    const int t = (int)(n - b * p.T);

    int e0, e1;                                      // first channels of the two vectors
    if (u >= turning) { e0 = 2 * VE * u; e1 = e0 + VE; }
    else if (INTER) { e0 = 2 * VE * u; e1 = e0 + VE; }
    else { e0 = VE * u; e1 = e0 + p.rot / 2; }

    float c[VE], s[VE];
    if (u < turning) {
        const double pos = p.positions ? (double)p.positions[n] : (double)p.position0 + (double)t;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const double turn = pos * (double)p.inv_freq[VE * u + i] * 0.15915494309189533577;   // 1 / (2 pi)
            const float frac = (float)(turn - rint(turn));
            sincospif(2.f * frac, &s[i], &c[i]);
            c[i] *= p.scale;
            s[i] *= (p.flags & GDR_ROPE_INVERSE) ? -p.scale : p.scale;
        }
    }

    const int h0 = blockIdx.y * p.heads, h1 = min(h0 + p.heads, p.Hq + p.Hk);
    for (int hb = h0; hb < h1; hb += HEADS) {
        V x0[HEADS], x1[HEADS];
        char* out[HEADS];
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
            const int h = hb + j;
            if (h < h1) {
                const bool key = h >= p.Hq;
                const int hh = key ? h - p.Hq : h, H = key ? p.Hk : p.Hq;
                const long long row = (p.flags & GDR_TOKEN_MAJOR) ? (b * p.T + t) * H + hh : (b * H + hh) * (long long)p.T + t;
                const char* in = (const char*)(key ? p.k : p.q) + row * p.d * ES;
                out[j] = (char*)(key ? p.k_out : p.q_out) + row * p.d * ES;
                x0[j].u = *reinterpret_cast<const uint4*>(in + e0 * ES);
                x1[j].u = *reinterpret_cast<const uint4*>(in + e1 * ES);
            }
        }
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
            if (hb + j < h1) {
                if (u < turning) {
                    float f0[VE], f1[VE], g0[VE], g1[VE];
                    x0[j].get(f0);
                    x1[j].get(f1);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        if constexpr (INTER) {       // pairs side by side across the two vectors
                            float& y0 = (2 * i < VE) ? g0[(2 * i) % VE] : g1[(2 * i) % VE];
                            float& y1 = (2 * i < VE) ? g0[(2 * i + 1) % VE] : g1[(2 * i + 1) % VE];
                            const float a = (2 * i < VE) ? f0[(2 * i) % VE] : f1[(2 * i) % VE];
                            const float d = (2 * i < VE) ? f0[(2 * i + 1) % VE] : f1[(2 * i + 1) % VE];
                            y0 = a * c[i] - d * s[i];
                            y1 = d * c[i] + a * s[i];
                        } else {
                            g0[i] = f0[i] * c[i] - f1[i] * s[i];
                            g1[i] = f1[i] * c[i] + f0[i] * s[i];
                        }
                    }
                    x0[j].set(g0);
                    x1[j].set(g1);
                }
                *reinterpret_cast<uint4*>(out[j] + e0 * ES) = x0[j].u;
                *reinterpret_cast<uint4*>(out[j] + e1 * ES) = x1[j].u;
            }
        }
    }
}

long long rope_workgroups(long long rows, int d, uint32_t flags) {
    const int units = d / ((flags & GDR_ACT_F32) ? 8 : 16), per = 256 / units;
    return (rows + per - 1) / per;
}

hipError_t launch_rope(RopeParams p, hipStream_t st) {
    const bool f32 = (p.flags & GDR_ACT_F32) != 0;
    const long long tiles = rope_workgroups(p.rows, p.d, p.flags);
    if (tiles == 0) return hipSuccess;
    const int all = p.Hq + p.Hk;
    // enough workgroups to fill the chip, then as many heads per angle as that leaves
    long long heads = all * tiles / 2048;
    heads = heads < 1 ? 1 : heads > all ? all : heads;
    if (heads < (all + 65534LL) / 65535) heads = (all + 65534LL) / 65535;   // the grid's second axis
    p.heads = (int)heads;
    dim3 grid((unsigned)tiles, (unsigned)((all + heads - 1) / heads)), block(256);
    if (p.flags & GDR_ROPE_INTERLEAVED) {
        if (f32) hipLaunchKernelGGL((rope_kernel<true, true>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((rope_kernel<false, true>), grid, block, 0, st, p);
    } else {
        if (f32) hipLaunchKernelGGL((rope_kernel<true, false>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((rope_kernel<false, false>), grid, block, 0, st, p);
    }
    return hipGetLastError();
}

}  // namespace gdr
