// NVFP4 values as operands of the FP16 matrix instructions, for gfx950.
//
// An E2M1 code times an E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688], so every NVFP4 value (without its global scale) is exact in
// FP16. Two codes take one conversion (v_cvt_scalef32_pk_f16_fp4) and one
// packed FP16 product with their block's scale. The other operand (BF16 or
// FP32 in memory) is brought into FP16's range by a power of two.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4op {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

// The two codes in byte `byte` (a constant after inlining) of w.
__device__ __forceinline__ half2v fp4x2(uint32_t w, int byte)
{
    switch (byte) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
    }
}

// The two E4M3 values in the low bytes of w.
__device__ __forceinline__ half2v e4m3x2(uint32_t w)
{
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
}

__device__ __forceinline__ half8v join(half2v a, half2v b, half2v c, half2v d)
{
    return half8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight codes of one block times its scale.
__device__ __forceinline__ half8v fp4x8(uint32_t w, _Float16 scale)
{
    const half2v s = {scale, scale};
    return join(fp4x2(w, 0) * s, fp4x2(w, 1) * s, fp4x2(w, 2) * s, fp4x2(w, 3) * s);
}

// The exponent e that puts the largest of some values, given as the bits of its
// magnitude, into [2^14, 2^15) when multiplied by 2^e: values down to 2^-28 of
// it stay normal FP16 numbers, smaller ones are off by at most 2^-39 of it. At
// most 126, so that 2^-e is a normal number; 0 for zero, infinity and NaN,
// which no scaling helps.
__device__ __forceinline__ int fp16_exponent(uint32_t top)
{
    return top == 0 || top >= 0x7f800000u ? 0 : min(14 - ilogbf(__uint_as_float(top)), 126);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

}  // namespace fp4op
