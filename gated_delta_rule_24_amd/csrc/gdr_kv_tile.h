// The cache's values as operands of the matrix instructions: e4m3 is exact in bf16
// and f16.
#pragma once

#include "gdr_attn.h"
#include "gdr_device.h"

namespace gdr {

__device__ __forceinline__ bf8v e4m3x8_to_bf16(uint32_t a, uint32_t b) {
    const bf2v x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf2v x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf2v x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf2v x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    bf8v r;
    r[0] = x0[0]; r[1] = x0[1]; r[2] = x1[0]; r[3] = x1[1];
    r[4] = x2[0]; r[5] = x2[1]; r[6] = x3[0]; r[7] = x3[1];
    return r;
}

__device__ __forceinline__ half8 e4m3x8_to_f16(uint32_t a, uint32_t b) {
    typedef _Float16 half2v __attribute__((ext_vector_type(2)));
    const half2v x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
    const half2v x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
    const half2v x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
    const half2v x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
    return half8{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

}  // namespace gdr
