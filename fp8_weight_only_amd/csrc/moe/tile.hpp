// The main loop of the tiled products: a ring of direct global-to-LDS stage
// loads whose LDS reads run under the matrix instructions.
//
// A stage is 64 k of both operand tiles, consumed in two halves. While the
// products of one half run, the fragments of the next half are read into a
// second register set: half 1 of stage s under half 0's products, half 0 of
// stage s + 1 under half 1's. The barrier stands between the two: behind it all
// waves hold stage s in registers, so its buffer takes stage s + NS, and stage
// s + 1 has landed for everyone. An int8 stage of a 256 x 256 tile takes 0.90 us
// on its own CU, its products 0.52 of that at the clock they run at (1.97 GHz);
// with waits for every read in flight it took 1.02.
//
// The waits are exact as in ../ring.hpp: every stage issues LOADS load
// instructions per wave, the buffers are distinct __shared__ arrays addressed
// through unrolled steps, loads complete in order.
#pragma once

#include "../ring.hpp"
#include "device.hpp"

namespace fp8w {

// Rows at a wave-uniform base, read straight into LDS: 16 bytes per lane, which
// land at dst + 16 * lane. Addressed through a buffer resource: the lane's 32-bit
// offset stays in one register and the stage's in a scalar one, and the compiler
// counts the load in vmcnt alone. The global form also counts as an LDS access
// for it, in no order with the others, and made every wait for a fragment wait
// for all reads in flight.
struct Rows {
    __amdgpu_buffer_rsrc_t rsrc;
    Rows() = default;
    __device__ __forceinline__ explicit Rows(const void* base)
        : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(uniform(base)), 0, -1, 0x00020000))
    {
    }
    __device__ __forceinline__ void load(int lane_off, int off, uint8_t* dst) const
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, FP8W_LDS(dst), 16, lane_off, off, 0, 0);
    }
    // 4 bytes per lane, at dst + 4 * lane
    __device__ __forceinline__ void load4(int lane_off, int off, uint8_t* dst) const
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, FP8W_LDS(dst), 4, lane_off, off, 0, 0);
    }
};

// Workgroup barrier behind which LDS writes before it are seen; loads into
// registers stay in flight over it.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    wait_loads_at_most<63>();
    stage_barrier();
}

// The main loop of the tiles staged through registers, for rows at any byte.
// Stage s + 2 is requested when stage s begins (into the registers that held s),
// stage s + 1 is written to the other LDS buffer when it ends. load(regs, s)
// takes any stage, load_whole one that lies below k; with no branch around them
// the compiler waits for a stage's own loads only (417 tokens, [2368, 3991] int8:
// 35 us, with branches 55). Four stages ahead measured the same or slower.
template <typename Regs, typename Load, typename LoadWhole, typename Put, typename Compute>
__device__ __forceinline__ void run_tile_staged(int S, int whole, const Load& load, const LoadWhole& load_whole,
                                                const Put& put, const Compute& compute)
{
    constexpr int D = 2;
    Regs r[D];
    int s0 = 0;
    if (whole >= 2 * D) {
#pragma unroll
        for (int u = 0; u < D; ++u)
            load_whole(r[u], u);
        put(r[0], 0);
        lds_barrier();
        for (; s0 + 2 * D <= whole; s0 += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                load_whole(r[u], s0 + u + D);
                compute(u & 1);
                put(r[(u + 1) % D], (u + 1) & 1);
                lds_barrier();
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (u < S)
                load(r[u], u);
        put(r[0], 0);
        lds_barrier();
    }
    for (; s0 < S; s0 += D) {
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (s0 + u < S) {
                if (s0 + u + D < S)
                    load(r[u], s0 + u + D);
                compute(u & 1);
                if (s0 + u + 1 < S)
                    put(r[(u + 1) % D], (u + 1) & 1);
                lds_barrier();
            }
    }
}

// Stages 0 .. S - 1 (S >= NS), each multiplied in PARTS (an even number). P: Frags;
// issue(s, buffer), read(buffer, part, frags), mma(frags, acc). buf(integral_constant<int, i>) is stage buffer i.
template <int NS, int LOADS, int PARTS = 2, typename P, typename Buf, typename Acc>
__device__ __forceinline__ void run_tile_ring(const P& p, int S, const Buf& buf, Acc* acc)
{
    static_assert(NS >= 2 && LOADS * (NS - 1) < 64 && PARTS % 2 == 0, "vmcnt range, parts");
    typename P::Frags f0, f1;
    auto at = [&](auto i) { return buf(std::integral_constant<int, decltype(i)::value % NS>{}); };
    // A part's reads are issued before the products of the one before (scheduling barriers); behind
    // those the order is the compiler's, which measured 1 to 2 % faster than holding it too.
    // stage s (step u of a group of NS): `left` later stages may stay in flight
    // at the barrier (-1: this is the last stage), `more` says that stage s + NS exists
    auto step = [&](int s, auto uc, auto left, auto more) {
        constexpr int u = decltype(uc)::value;
        ring_for<1, PARTS>([&](auto h) {
            constexpr int part = decltype(h)::value;
            p.read(at(uc), part, part & 1 ? f1 : f0);
            __builtin_amdgcn_sched_barrier(0);
            p.mma(part & 1 ? f0 : f1, acc);
        });
        if constexpr (decltype(left)::value >= 0) {
            wait_loads_at_most<LOADS * decltype(left)::value>();
            stage_barrier();
            if constexpr (decltype(more)::value)
                p.issue(s + NS, at(uc));
            p.read(at(std::integral_constant<int, u + 1>{}), 0, f0);
            __builtin_amdgcn_sched_barrier(0);
        }
        p.mma(f1, acc);
    };
    ring_for<0, NS>([&](auto i) { p.issue(decltype(i)::value, at(i)); });
    wait_loads_at_most<LOADS*(NS - 1)>();
    stage_barrier();
    p.read(at(std::integral_constant<int, 0>{}), 0, f0);
    int s0 = 0;
    for (; s0 + 2 * NS <= S; s0 += NS)
        ring_for<0, NS>([&](auto u) {
            step(s0 + decltype(u)::value, u, std::integral_constant<int, NS - 2>{}, std::true_type{});
        });
    const int rest = S - s0;  // NS .. 2 NS - 1 stages, the last `rest - NS` of them not yet issued
    ring_for<NS, 2 * NS>([&](auto rc) {
        constexpr int R = decltype(rc)::value;
        if (rest == R)
            ring_for<0, R>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                constexpr int left = R - 2 - u < NS - 2 ? R - 2 - u : NS - 2;
                step(s0 + u, uc, std::integral_constant<int, left>{}, std::integral_constant<bool, (u + NS < R)>{});
            });
    });
}

}  // namespace fp8w
