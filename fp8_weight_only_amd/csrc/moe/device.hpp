// Device helpers shared by the kernels of libfp8w_moe.so.
#pragma once

#include "../common.hpp"

namespace fp8w {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 16 bytes at any address (the hardware takes unaligned global accesses).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

__device__ __forceinline__ u32x4 load16_any(const void* p)
{
    return *static_cast<const u32x4_any*>(p);
}

__device__ __forceinline__ void store16_any(void* p, u32x4 v)
{
    *static_cast<u32x4_any*>(p) = v;
}

// The first `avail` of 16 bytes at p, zeros after them; reads no byte past them.
__device__ __forceinline__ u32x4 load16_part(const uint8_t* p, int64_t avail)
{
    if (avail >= 16)
        return load16_any(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < avail)
            w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return u32x4{w[0], w[1], w[2], w[3]};
}

template <typename A>
struct is_bf16 {
    static constexpr bool value = false;
};
template <>
struct is_bf16<Bf16> {
    static constexpr bool value = true;
};

template <typename A>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (is_bf16<A>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
}

// Tile (tn, tm) of linear workgroup id L < TN * TM. Workgroups are dealt to the
// 8 XCDs in turn; each XCD is given a contiguous range of tile ids, walked in
// groups of GM row tiles, so the tiles that one XCD holds at a time share
// operand rows in its L2.
template <int GM>
__device__ __forceinline__ void xcd_tile(int64_t L, int64_t TN, int64_t TM, int64_t& tn, int64_t& tm)
{
    const int64_t T = TN * TM;
    const int64_t xcd = L % 8, loc = L / 8, q = T / 8, r = T % 8;
    const int64_t id = xcd * q + (xcd < r ? xcd : r) + loc;
    const int64_t grp = id / (GM * TN), first = grp * GM;
    const int64_t gs = TM - first < GM ? TM - first : GM;
    const int64_t w = id - grp * GM * TN;
    tm = first + w % gs;
    tn = w / gs;
}

// Four consecutive channels of one token: one 8-byte store where it is aligned
// and all four exist.
__device__ __forceinline__ void store4(uint16_t* dst, const uint16_t* o, int64_t left)
{
    if (left >= 4 && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
        u32x2 pk;
        pk.x = (uint32_t)o[0] | ((uint32_t)o[1] << 16);
        pk.y = (uint32_t)o[2] | ((uint32_t)o[3] << 16);
        *reinterpret_cast<u32x2*>(dst) = pk;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < left)
                dst[r] = o[r];
    }
}

}  // namespace fp8w
