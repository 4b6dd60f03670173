// A token's choice of experts from its router logits.
//
// G lanes hold a token (64, or 16 where e <= 64 and top <= 16: four
// tokens per wave), J consecutive experts each. A logit becomes an unsigned key
// of the same order (NaN above everything, both zeros equal, -inf key 0 = not to
// be taken). A round is an integer maximum over registers and lanes (DPP
// rotations within rows of 16 lanes, row swaps across them), the first lane and
// register that hold it (the lowest index, since a lane's experts are
// consecutive), and that key cleared.
#pragma once

#include <math.h>

#include "device.hpp"
#include "moe.hpp"

namespace fp8w {

__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 becomes 0
    uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    key = f == -INFINITY ? 0 : key;
    return f != f ? 0xffffffffu : key;
}

// the logit of a key (a NaN for a NaN's key, -inf for key 0)
__device__ __forceinline__ float logit_of(uint32_t key)
{
    if (key == 0)
        return -INFINITY;
    return __builtin_bit_cast(float, (key >> 31) ? key ^ 0x80000000u : ~key);
}

template <int CTRL>
__device__ __forceinline__ uint32_t rotated(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

// OP over the G lanes of a group, in all of them.
template <int G, typename OP>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, OP op)
{
    static_assert(G == 16 || G == 64, "a row of lanes or the wave");
    v = op(v, rotated<0x128>(v));  // row_ror:8
    v = op(v, rotated<0x124>(v));
    v = op(v, rotated<0x122>(v));
    v = op(v, rotated<0x121>(v));
    if constexpr (G == 64) {
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // even rows' and odd rows' values
        v = op(a[0], a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(b[0], b[1]);
    }
    return v;
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (G == 64)
        return wave_max_u32(v);  // in a scalar register
    else
        return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    return __builtin_bit_cast(float, group_reduce<G>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
                                  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) +
                                                                          __builtin_bit_cast(float, b));
                              }));
}

// A lane's J logits of a row, -inf past its end.
template <int J>
__device__ __forceinline__ void load_logits(const void* logits, Act type, int64_t row, int e, int first, float* l)
{
    if (type == Act::FP32) {
        const float* p = static_cast<const float*>(logits) + row * e + first;
        if (J == 4 && first + 4 <= e) {
            const u32x4 v = load16_any(p);
            const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < J; ++j)
                l[j] = __builtin_bit_cast(float, d[j & 3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            l[j] = first + j < e ? p[j] : -INFINITY;
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(logits) + row * e + first;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint16_t b = first + j < e ? p[j] : (uint16_t)0;
        const float f = type == Act::BF16 ? Bf16::to_f32(b) : F16::to_f32(b);
        l[j] = first + j < e ? f : -INFINITY;
    }
}

// A group's next choice: the largest key left among its lanes' (0: none left),
// taken out, and its expert. A lane's keys are sorted where they are few (a
// choice is then its first key, and taking it a shift), else searched each time.
template <int G, int J>
struct Keys {
    static constexpr bool kSorted = J <= 4;
    uint32_t key[J];
    uint32_t order;  // sorted: the registers' original numbers, a byte each, first key's lowest

    __device__ __forceinline__ void set(const float (&l)[J])
    {
#pragma unroll
        for (int j = 0; j < J; ++j)
            key[j] = key_of(l[j]);
        if constexpr (kSorted) {
            uint32_t id[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                id[j] = j;
            // neighbours exchanged only where the later is larger: equal keys stay in order
#pragma unroll
            for (int n = J - 1; n >= 1; --n)
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const bool swap = key[j + 1] > key[j];
                    const uint32_t hi = swap ? key[j + 1] : key[j], lo = swap ? key[j] : key[j + 1];
                    const uint32_t a = swap ? id[j + 1] : id[j], b = swap ? id[j] : id[j + 1];
                    key[j] = hi;
                    key[j + 1] = lo;
                    id[j] = a;
                    id[j + 1] = b;
                }
            order = 0;
#pragma unroll
            for (int j = 0; j < J; ++j)
                order |= id[j] << (8 * j);
        }
    }

    __device__ __forceinline__ uint32_t take(int& expert)
    {
        const int lane = threadIdx.x & 63, in = lane % G;
        uint32_t head = key[0];
        int at = 0;
        if constexpr (kSorted) {
            at = (int)(order & 255u);
        } else {
#pragma unroll
            for (int j = 1; j < J; ++j)
                head = head > key[j] ? head : key[j];
#pragma unroll
            for (int j = J - 1; j >= 1; --j)
                at = key[j] == head ? j : at;
            at = key[0] == head ? 0 : at;
        }
        const uint32_t best = group_max<G>(head);
        bool mine;
        if constexpr (G == 64) {
            const int win = (int)__builtin_ctzll(__ballot(head == best));  // never empty
            expert = __builtin_amdgcn_readlane(at, win) + win * J;
            mine = lane == win;
        } else {
            expert = (int)group_reduce<G>(head == best ? (uint32_t)(in * J + at) : 0xffffffffu,
                                          [](uint32_t a, uint32_t b) { return a < b ? a : b; });
            mine = expert / J == in;
        }
        if constexpr (kSorted) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[j] = mine ? (j + 1 < J ? key[j + 1 < J ? j + 1 : j] : 0) : key[j];
            order = mine ? order >> 8 : order;
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[j] = mine && j == at ? 0 : key[j];
        }
        return best;
    }
};

// U tokens per group at a time (two: their chains of dependent steps overlap), from
// l[u][j], the token's logit of expert in * J + j. Lane r of a group gets its
// tokens' r-th choice in id[u] (-1: none) and its weight.
template <int G, int J, int U>
__device__ __forceinline__ void choose(const float (&l)[U][J], int top, bool renorm, float (&weight)[U], int (&id)[U])
{
    const int in = (threadIdx.x & 63) % G;
    uint32_t mine[U], peak[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        mine[u] = peak[u] = 0;
        id[u] = -1;
    }
    Keys<G, J> keys[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        keys[u].set(l[u]);
    for (int r = 0; r < top; ++r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int first;
            const uint32_t best = keys[u].take(first);
            if (r == 0)
                peak[u] = best;
            const bool take = in == r && best != 0;
            mine[u] = take ? best : mine[u];
            id[u] = take ? first : id[u];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float top_logit = logit_of(peak[u]);
        const float num = mine[u] ? expf(logit_of(mine[u]) - top_logit) : 0.0f;
        float part = num;
        if (!renorm) {
            part = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
                part += l[u][j] == -INFINITY ? 0.0f : expf(l[u][j] - top_logit);
        }
        const float total = group_sum<G>(part);
        weight[u] = id[u] >= 0 ? num / total : 0.0f;
    }
}

// Chooses for tokens [t0, t1), the workgroup's WAVES waves in turn, and calls
// done(token, choice number, expert, weight) from the lanes that hold them.
template <int G, int J, int WAVES, typename F>
__device__ __forceinline__ void choose_chunk(const void* logits, Act type, int64_t t0, int64_t t1, int e, int top,
                                             bool renorm, F&& done)
{
    constexpr int U = 2, T = U * kWave / G;  // tokens per wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, in = lane % G;
    auto load = [&](int64_t t, float (&l)[U][J]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = t + u * (kWave / G) + lane / G;
            load_logits<J>(logits, type, row < t1 ? row : t1 - 1, e, in * J, l[u]);
        }
    };
    int64_t t = t0 + (int64_t)wave * T;
    float next[U][J];
    if (t < t1)
        load(t, next);
    for (; t < t1; t += WAVES * T) {
        float l[U][J];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < J; ++j)
                l[u][j] = next[u][j];
        if (t + WAVES * T < t1)
            load(t + WAVES * T, next);
        float weight[U];
        int id[U];
        choose<G, J, U>(l, top, renorm, weight, id);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = t + u * (kWave / G) + lane / G;
            if (in < top && row < t1)
                done(row, in, id[u], weight[u]);
        }
    }
}

// Lanes per token.
__host__ __device__ inline int choice_lanes(int64_t e, int64_t top)
{
    return e <= 64 && top <= 16 ? 16 : 64;
}

}  // namespace fp8w
