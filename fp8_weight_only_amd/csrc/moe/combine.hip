// The weighted sum of a token's expert outputs:
//   out[t, c] = sum_j weights[t, j] * y[t * top + j, c],
// fp32 products and sums in the order of j, one rounding to the activation type.
//
// A stream of top + 1 rows per token. Each thread owns eight channels (16 bytes)
// of one token and loads them from every row before the first product needs
// them; loads and stores take any alignment, so odd widths run the same code.
#include "device.hpp"
#include "moe.hpp"

namespace fp8w {
namespace {

constexpr int kThreads = 256;

template <typename A>
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
    for (int j = 0; j < top; ++j) {
        const u32x4 v = load16_part(reinterpret_cast<const uint8_t*>(src + j * n), left);
        const float wj = w[j];
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] = __builtin_fmaf(wj, A::lo_f32(d[i]), acc[2 * i]);
            acc[2 * i + 1] = __builtin_fmaf(wj, A::hi_f32(d[i]), acc[2 * i + 1]);
        }
    }
    uint16_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = A::from_f32(acc[i]);
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
    const dim3 grid((unsigned)groups), block(kThreads);
    if (act == Act::BF16)
        hipLaunchKernelGGL(combine_kernel<Bf16>, grid, block, 0, stream, static_cast<const uint16_t*>(y), weights,
                           static_cast<uint16_t*>(out), items, (int)top, n, chunks);
    else
        hipLaunchKernelGGL(combine_kernel<F16>, grid, block, 0, stream, static_cast<const uint16_t*>(y), weights,
                           static_cast<uint16_t*>(out), items, (int)top, n, chunks);
    return hipGetLastError();
}

}  // namespace fp8w
