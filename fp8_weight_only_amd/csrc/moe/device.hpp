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
typedef uint32_t u32x4_dword __attribute__((ext_vector_type(4), aligned(4)));  // at any dword
typedef uint32_t u32x2_dword __attribute__((ext_vector_type(2), aligned(4)));

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

// The first `avail` of 16 bytes at p, zeros after them. Reads whole aligned
// dwords, and none that holds no byte of those.
__device__ __forceinline__ u32x4 load16_part(const uint8_t* p, int64_t avail)
{
    if (avail >= 16)
        return load16_any(p);
    u32x4 r{0, 0, 0, 0};
    if (avail > 0) {
        const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u, n = (uint32_t)avail;
        const uint32_t* d = reinterpret_cast<const uint32_t*>(p - shift);
        const uint32_t last = (shift + n - 1) / 4;
        uint32_t v[5], o[4];
#pragma unroll
        for (uint32_t i = 0; i < 5; ++i)
            v[i] = d[i < last ? i : last];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t w = __builtin_amdgcn_alignbyte(v[i + 1], v[i], shift);
            o[i] = n >= 4 * i + 4 ? w : (n > 4 * i ? w & ((1u << (8 * (n - 4 * i))) - 1) : 0);
        }
        r = u32x4{o[0], o[1], o[2], o[3]};
    }
    return r;
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

// A row that is read 16 bytes at a time. SHIFT: it may start at any byte; the
// loads then are of whole aligned dwords, four and the one behind them, shifted
// together. The hardware takes any address, but below dword alignment at 0.4 of
// the rate ([14336, 4100] codes streamed in 26 us, [14336, 4098] in 58). No dword
// is read that holds no byte of the 16.
//
// load() requests them, bytes() puts them together once they are needed.
template <bool SHIFT>
struct Row {
    struct Raw {
        u32x4 v;
        uint32_t e[SHIFT ? 1 : 0];
    };
    const uint8_t* p;
    uint32_t shift, behind;

    Row() = default;
    __device__ __forceinline__ explicit Row(const void* start) : p(static_cast<const uint8_t*>(start))
    {
        if constexpr (SHIFT) {
            shift = (uint32_t)reinterpret_cast<uintptr_t>(start) & 3u;
            p -= shift;
            behind = shift ? 16 : 0;
        }
    }
    // the 16 bytes at off, a multiple of 4
    __device__ __forceinline__ Raw load(int64_t off) const
    {
        Raw r;
        if constexpr (SHIFT) {
            r.v = *reinterpret_cast<const u32x4_dword*>(p + off);
            r.e[0] = *reinterpret_cast<const uint32_t*>(p + off + behind);
        } else {
            r.v = load16_any(p + off);
        }
        return r;
    }
    __device__ __forceinline__ u32x4 bytes(const Raw& r) const
    {
        const u32x4 v = r.v;
        if constexpr (SHIFT)
            return u32x4{__builtin_amdgcn_alignbyte(v.y, v.x, shift), __builtin_amdgcn_alignbyte(v.z, v.y, shift),
                         __builtin_amdgcn_alignbyte(v.w, v.z, shift), __builtin_amdgcn_alignbyte(r.e[0], v.w, shift)};
        return v;
    }
    // the first `avail` of them, zeros after
    __device__ __forceinline__ u32x4 part(int64_t off, int64_t avail) const
    {
        return load16_part(p + (SHIFT ? shift : 0) + off, avail);
    }
    // the same for bytes() to put together: only for rows with a stage of their own
    __device__ __forceinline__ Raw part_raw(int64_t off, int64_t avail) const { return raw(part(off, avail)); }
    // what bytes() makes v of
    __device__ __forceinline__ Raw raw(u32x4 v) const
    {
        Raw r;
        if constexpr (SHIFT) {
            // moved up by the shift that bytes() takes back
            const uint32_t back = 4 - shift;
            r.v = shift ? u32x4{__builtin_amdgcn_alignbyte(v.x, 0, back), __builtin_amdgcn_alignbyte(v.y, v.x, back),
                                __builtin_amdgcn_alignbyte(v.z, v.y, back), __builtin_amdgcn_alignbyte(v.w, v.z, back)}
                        : v;
            r.e[0] = shift ? __builtin_amdgcn_alignbyte(0, v.w, back) : 0;
        } else {
            r.v = v;
        }
        return r;
    }
};

template <typename A>
struct is_bf16 {
    static constexpr bool value = false;
};
template <>
struct is_bf16<Bf16> {
    static constexpr bool value = true;
};

// An fp32 result to the activation type. The empty statement keeps the compiler
// from fusing the last operation with the rounding to fp16 (v_fma_mix rounds
// once where the two instructions round twice): it did so for some elements of
// a kernel and not for others, and a call's bits then depended on the plan.
template <typename A>
__device__ __forceinline__ uint16_t rounded(float v)
{
    asm("" : "+v"(v));
    return A::from_f32(v);
}

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

// A value that is the same in all lanes, in a scalar register. Whatever decides
// whether a matrix instruction runs has to be one: those instructions take no
// notice of masked lanes, and a branch on a per-lane register may be compiled to
// a mask alone.
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

// Four consecutive channels of one token (`left` of them exist): one 8-byte store
// at dword alignment, else a dword between two halves.
__device__ __forceinline__ void store4(uint16_t* dst, const uint16_t* o, int64_t left)
{
    if (left < 4) {
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (r < left)
                dst[r] = o[r];
    } else if ((reinterpret_cast<uintptr_t>(dst) & 3) == 0) {
        u32x2 pk;
        pk.x = (uint32_t)o[0] | ((uint32_t)o[1] << 16);
        pk.y = (uint32_t)o[2] | ((uint32_t)o[3] << 16);
        *reinterpret_cast<u32x2_dword*>(dst) = pk;
    } else {
        dst[0] = o[0];
        *reinterpret_cast<uint32_t*>(dst + 1) = (uint32_t)o[1] | ((uint32_t)o[2] << 16);
        dst[3] = o[3];
    }
}

}  // namespace fp8w
