// 4-bit weights on the device: e2m1 codes, two to a byte (the even k in the low
// four bits), and one e8m0 scale 2^(s - 127) for a block of 32 along k.
//
// v_cvt_scalef32_pk_{bf16,f16}_fp4 turns two codes and their scale into two
// values. Code times scale has two significant bits, so in bf16 it is exact for
// every scale (the smallest, 2^-128, is a subnormal that the matrix cores take),
// in fp16 for scales 2^-23 .. 2^13; beyond them it is rounded to fp16's subnormals
// or is infinite, the value that an fp16 weight would have.
#pragma once

#include "device.hpp"

namespace fp8w {

// The scale operand of the conversion for an e8m0 byte (255: NaN).
__device__ __forceinline__ float fp4_scale(uint32_t byte)
{
    return __builtin_bit_cast(float, byte << 23);
}

// Eight codes, the lowest bits first, to eight values of the activation type.
template <typename A>
__device__ __forceinline__ u32x4 decode_fp4(uint32_t w, float scale)
{
    if constexpr (is_bf16<A>::value)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3))};
}

// The first `left` (up to 32) of 32 codes, zeros after them; an odd row's last
// byte holds four bits of no weight.
__device__ __forceinline__ u32x4 first_codes(u32x4 v, int64_t left)
{
    uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = left - 8 * i;
        d[i] = n >= 8 ? d[i] : (n > 0 ? d[i] & ((1u << (4 * n)) - 1) : 0);
    }
    return u32x4{d[0], d[1], d[2], d[3]};
}

}  // namespace fp8w
