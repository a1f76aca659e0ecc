// Internal interface and device helpers of the attention layer's kernels
// (gdr_rope.hip, gdr_attn_fwd.hip, gdr_attn_bwd.hip, gdr_kv.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr.h"

namespace gdr {

struct RopeParams {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const float* inv_freq;      // [rot / 2]
    const int* positions;       // [rows], or null: position0 + t
    int position0;
    long long rows;             // B * T
    int T, Hq, Hk, d, rot;
    int heads;                  // heads a thread turns with one set of angles
    float scale;
    uint32_t flags;
};
hipError_t launch_rope(RopeParams p, hipStream_t st);
// Workgroups of a call's largest launch, along the grid's first axis (the others' below).
long long rope_workgroups(long long rows, int d, uint32_t flags);

// Element strides of one [.., heads, tokens, d] tensor whose rows of d are
// contiguous; the same for both layouts.
struct AttnStrides {
    long long b, h, t;
};

struct AttnParams {
    const void* q;
    const void* k;
    const void* v;
    void* o;                    // forward: written; backward: read
    float* lse;                 // [B, Hq, Tq]; forward: written, may be null; backward: read
    const void* dO;
    void* dq;
    void* dk;
    void* dv;
    float* delta;               // [B, Hq, Tq]: rowsum(dO o)
    float* part;                // backward: fp32 partial dk, dv of the splits, or null
    const int* cu_seqlens;      // packed sequences, or null
    int nseq;
    int B, Hq, Hkv, Tq, Tk, d;
    int window;                 // 0: none
    int splits;                 // backward: workgroups a key tile's queries (of every head that shares it) are dealt to,
                                // at most
    bool few;                   // backward: any row may be one of few keys (see attn_delta_kernel)
    int split_steps;            // backward: steps of one of them; 0: every tile has `splits`
    float scale;
    AttnStrides sq, sk;         // queries' tensors (q, o, dO, dq); keys' tensors (k, v, dk, dv)
};
hipError_t launch_attn_fwd(const AttnParams& p, hipStream_t st);
hipError_t launch_attn_bwd(const AttnParams& p, hipStream_t st);
long long attn_fwd_workgroups(int B, int Hq, int Tq);
long long attn_bwd_workgroups(int B, int Hq, int Hkv, int Tq, int Tk, int d);
// Splits of the key side's queries, of a tile on average (1: no partials), and the most
// that a tile is given then.
int attn_bwd_splits(int B, int Hq, int Hkv, int Tq, int Tk);
int attn_bwd_splits_most(int splits, int Tk);

struct KvAppendParams {
    const void* k;
    const void* v;
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scale;
    float* v_scale;
    const int* block_table;     // [nseq, max_pages]
    const int* cache_len;       // [nseq]
    const int* cu_seqlens;      // [nseq + 1], or null: one token each
    int nseq, Hkv, T, d, n_pages, max_pages;
    long long st, sh;           // element strides of a token and a head of k and v
};
hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t st);
long long kv_append_workgroups(int nseq, int Hkv, int T, int d, bool packed);

struct AttnDecodeParams {
    const void* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int* block_table;
    const int* cache_len;
    void* o;
    float* part_o;              // [splits, N, Hq, d] unnormalised, or null when splits == 1
    float* part_ml;             // [splits, N, Hq, 2]: running maximum (base 2) and sum
    int N, Hq, Hkv, d, n_pages, max_pages, window;
    int splits, split_pages;    // pages of a split: split s of a sequence is its s-th run of them
    float scale;
    uint32_t flags;
};
// Splits of the pages a call may have to read, and the pages of one split.
int attn_decode_splits(int N, int Hq, int Hkv, int max_pages, int window, int* split_pages);
hipError_t launch_attn_decode(const AttnDecodeParams& p, hipStream_t st);
long long attn_decode_workgroups(int N, int Hq, int Hkv);

// Index of the last of cu[0] .. cu[nseq] that is at most t, or 0.
__host__ __device__ inline int last_at_most(const int* cu, int nseq, int t) {
    int s = 0, z = nseq;
    while (s < z) {
        const int mid = s + (z - s + 1) / 2;       // (s + z may pass 32 bits)
        if (cu[mid] <= t) s = mid;
        else z = mid - 1;
    }
    return s;
}

// ---------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------

#ifdef __HIPCC__
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

// two fp32 values rounded to nearest even, as bf16 bits side by side (one instruction)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bf2v r;
    r[0] = (__bf16)a;
    r[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, r);
}

// The larger / the sum of the two lanes l and l ^ 32, in both: one lane-swap.
__device__ __forceinline__ float max_across32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_across32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
#endif

}  // namespace gdr
