// Device helpers shared by the kernels of libfp8w_moe.so.
#pragma once

#include "../common.hpp"

namespace fp8w {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 16 bytes at any address (the hardware takes unaligned global accesses).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ u32x4 load16_any(const void* p)
{
    return *static_cast<const u32x4_any*>(p);
}

// The same for data that is read once.
__device__ __forceinline__ u32x4 load16_once(const void* p)
{
    return __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
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

// The largest v of the wave, in every lane: DPP shifts within rows of 16 lanes,
// row maxima broadcast upwards, lane 63's result read back.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    auto step = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));  // row_shr:1
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));  // row_shr:2
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));  // row_shr:4
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));  // row_shr:8
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast:15
    v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
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

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v)
{
    return __builtin_amdgcn_readfirstlane(v);
}

__device__ __forceinline__ const uint8_t* uniform(const void* p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)v), hi = (uint32_t)uniform((int)(uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
}

// Between one lane's LDS write and another lane's read in the same wave: LDS
// works in order, so only the compiler has to keep it.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Tile (tn, tm) of linear workgroup id L < TN * TM. Workgroups are dealt to the
// 8 XCDs in turn; each XCD is given a contiguous range of tile ids, walked in
// groups of GM row tiles, so the tiles that one XCD holds at a time share
// operand rows in its L2.
template <int GM>
__device__ __forceinline__ void xcd_tile(int L, int TN, int TM, int& tn, int& tm)
{
    const int T = TN * TM;  // fewer than 2^24 (a launch has fewer than 2^32 threads)
    const int xcd = L % 8, loc = L / 8, q = T / 8, r = T % 8;
    const int id = xcd * q + (xcd < r ? xcd : r) + loc;
    const int grp = id / (GM * TN), first = grp * GM;
    const int gs = TM - first < GM ? TM - first : GM;
    const int w = id - grp * GM * TN;
    tm = uniform(first + w % gs);
    tn = uniform(w / gs);
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
