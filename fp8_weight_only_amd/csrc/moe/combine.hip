// The weighted sum of a token's expert outputs:
//   out[t, c] = sum_j weights[t, j] * y[t * top + j, c],
// fp32 products and sums in the order of j, one rounding to the activation type.
//
// A stream of top + 1 rows per token, bound by memory. Each thread owns eight
// channels (16 bytes) of one token. Where top is 1, 2, 4, 6 or 8 (known when
// compiled) it loads them from every row before the first product needs them,
// past the caches, since nothing is read twice: 8192 tokens, 8 rows of 4096 in
// 96 us, 6.3 TB/s (a loop over the rows with cached loads: 113; a large copy: 5.2
// TB/s); rows below dword alignment by whole dwords shifted (8 rows of 4095: 116
// us). Any other top takes the loop: 8192 tokens, 3 rows of 4096 in 47 us, 5.7 TB/s,
// and 3 rows of 4095 in 55, where 2 rows of 4096 by the loads ahead take 32, 6.4.
#include "device.hpp"
#include "moe.hpp"

namespace fp8w {
namespace {

constexpr int kThreads = 256;

// TOP > 0: top, known when compiled; 0: any (a loop, rows at any byte).
template <typename A, int TOP, bool SHIFT>
__global__ __launch_bounds__(kThreads) void combine_kernel(const uint16_t* __restrict__ y,
                                                           const float* __restrict__ weights,
                                                           uint16_t* __restrict__ out, int64_t items, int top,
                                                           int64_t n, int64_t chunks)
{
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= items)
        return;
    const int64_t t = item / chunks, c = (item - t * chunks) * 8;
    const uint16_t* src = y + t * top * n + c;
    const float* w = weights + t * top;
    const int64_t left = 2 * (n - c);  // bytes
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        acc[i] = 0.0f;
    auto add = [&](u32x4 v, float wj) {
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] = __builtin_fmaf(wj, A::lo_f32(d[i]), acc[2 * i]);
            acc[2 * i + 1] = __builtin_fmaf(wj, A::hi_f32(d[i]), acc[2 * i + 1]);
        }
    };
    if constexpr (TOP > 0) {
        u32x4 v[TOP];
        if (left >= 16) {
            if constexpr (SHIFT) {
                typename Row<true>::Raw raw[TOP];
#pragma unroll
                for (int j = 0; j < TOP; ++j)
                    raw[j] = Row<true>(src + j * n).load(0);
#pragma unroll
                for (int j = 0; j < TOP; ++j)
                    v[j] = Row<true>(src + j * n).bytes(raw[j]);
            } else {
#pragma unroll
                for (int j = 0; j < TOP; ++j)
                    v[j] = load16_once(src + j * n);
            }
        } else {
#pragma unroll
            for (int j = 0; j < TOP; ++j)
                v[j] = load16_part(reinterpret_cast<const uint8_t*>(src + j * n), left);
        }
#pragma unroll
        for (int j = 0; j < TOP; ++j)
            add(v[j], w[j]);
    } else {
        for (int j = 0; j < top; ++j)
            add(load16_part(reinterpret_cast<const uint8_t*>(src + j * n), left), w[j]);
    }
    uint16_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = rounded<A>(acc[i]);
    uint16_t* dst = out + t * n + c;
    if (left >= 16) {
        u32x4 pk;
        pk.x = (uint32_t)o[0] | ((uint32_t)o[1] << 16);
        pk.y = (uint32_t)o[2] | ((uint32_t)o[3] << 16);
        pk.z = (uint32_t)o[4] | ((uint32_t)o[5] << 16);
        pk.w = (uint32_t)o[6] | ((uint32_t)o[7] << 16);
        store16_any(dst, pk);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i < left)
                dst[i] = o[i];
    }
}

}  // namespace

hipError_t launch_combine(const void* y, Act act, const float* weights, int64_t t, int64_t top, int64_t n, void* out,
                          hipStream_t stream)
{
    const int64_t chunks = (n + 7) / 8, items = t * chunks, groups = (items + kThreads - 1) / kThreads;
    if (!grid_fits(groups, kThreads))
        return hipErrorInvalidValue;
    const uint16_t* src = static_cast<const uint16_t*>(y);
    uint16_t* dst = static_cast<uint16_t*>(out);
    const bool shift = ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(2 * n)) & 3) != 0;
    const dim3 grid((unsigned)groups), block(kThreads);
#define FP8W_COMBINE(A, TOP)                                                                                           \
    return launch(shift && TOP ? combine_kernel<A, TOP, (TOP > 0)> : combine_kernel<A, TOP, false>, grid, block,       \
                  stream, src, weights, dst, items, top, n, chunks)
#define FP8W_COMBINE_TOP(A)                                                                                            \
    switch (top) {                                                                                                     \
    case 1: FP8W_COMBINE(A, 1);                                                                                        \
    case 2: FP8W_COMBINE(A, 2);                                                                                        \
    case 4: FP8W_COMBINE(A, 4);                                                                                        \
    case 6: FP8W_COMBINE(A, 6);                                                                                        \
    case 8: FP8W_COMBINE(A, 8);                                                                                        \
    default: FP8W_COMBINE(A, 0);                                                                                       \
    }
    if (act == Act::BF16) {
        FP8W_COMBINE_TOP(Bf16)
    } else {
        FP8W_COMBINE_TOP(F16)
    }
#undef FP8W_COMBINE_TOP
#undef FP8W_COMBINE
}

}  // namespace fp8w
