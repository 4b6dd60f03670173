// The linear layer on 8-bit integers, a scale for each token and each output
// channel:
//   sx[t] = max_k |x[t, k]| / 127,  qx[t, k] = round(127 x[t, k] / max_k |x[t, k]|)
//   y[t, c] = (sum_k qx[t, k] * q[c, k]) * sx[t] * sw[c] + bias[c]
// The sum is exact in 32-bit integers (k <= 131072); the scales and the bias are
// applied in fp32 and the result is rounded once.
//
// Codes of 16-bit activations are the exact quotient's nearest integers, ties to
// even: 127 x has at most 18 significant bits, so it is exact in fp32; the fp32
// quotient by the maximum is off by at most 2^-24 of its value, and a quotient
// that is no half lies at least 1 / (254 * 2^11), above 2^-19, of its value away
// from one (x and the maximum have at most 11 significant bits), so rounding the rounded quotient gives what
// rounding the exact one would.
#include <math.h>
#include <stdio.h>

#include "device.hpp"
#include "moe.hpp"

namespace fp8w {
namespace {

__device__ __forceinline__ float value_at(const void* p, Act type, int64_t i)
{
    if (type == Act::FP32)
        return static_cast<const float*>(p)[i];
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return type == Act::BF16 ? Bf16::to_f32(b) : F16::to_f32(b);
}

// Rows with very large values are divided by 2^64 first (exactly; what that
// rounds away is far below half a code), so that 127 x stays finite.
__device__ __forceinline__ float prescale(float amax)
{
    return amax > 0x1p100f ? 0x1p-64f : 1.0f;
}

__device__ __forceinline__ int code_of(float x, float amax, float pre)
{
    return (int)rintf(__fdiv_rn(127.0f * (x * pre), amax * pre));
}

// One workgroup per row: the maximum, then the codes from a second read.
__global__ __launch_bounds__(256) void quantize_int8_kernel(const void* __restrict__ x, Act type, int64_t k,
                                                            int8_t* __restrict__ q, int64_t kx,
                                                            float* __restrict__ scale)
{
    __shared__ float part[4];
    __shared__ int bad[4];
    const int64_t row = blockIdx.x, base = row * k;
    float amax = 0.0f;
    int nf = 0;
    for (int64_t j = threadIdx.x; j < k; j += 256) {
        const float a = fabsf(value_at(x, type, base + j));
        nf |= !(a <= 3.402823466e38f);
        amax = fmaxf(amax, a);
    }
    amax = wave_max(amax);
    nf = __any(nf);
    if ((threadIdx.x & 63) == 0) {
        part[threadIdx.x >> 6] = amax;
        bad[threadIdx.x >> 6] = nf;
    }
    __syncthreads();
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    nf = bad[0] | bad[1] | bad[2] | bad[3];
    if (threadIdx.x == 0)
        scale[row] = nf ? __builtin_nanf("") : amax / 127.0f;
    const float pre = prescale(amax);
    for (int64_t j = threadIdx.x; j < kx; j += 256)
        q[row * kx + j] =
            j < k && amax > 0.0f && !nf ? (int8_t)code_of(value_at(x, type, base + j), amax, pre) : (int8_t)0;
}

template <typename A>
__device__ __forceinline__ uint16_t finish(int acc, float sx, float sw, float bias)
{
    return A::from_f32(__builtin_fmaf((float)acc * sx, sw, bias));
}

// Any k, any alignment: 64 channels x 64 tokens, four waves of 32 x 32, stages
// of 64 k through registers into LDS.
template <typename A>
__global__ __launch_bounds__(256) void int8_any_kernel(const int8_t* __restrict__ qx, int64_t kx,
                                                       const float* __restrict__ sx, const int8_t* __restrict__ qw,
                                                       const float* __restrict__ sw,
                                                       const uint16_t* __restrict__ bias, uint16_t* __restrict__ y,
                                                       int64_t m, int64_t n, int64_t k, int64_t TN, int64_t TM)
{
    constexpr int LD = 80;  // row pitch in bytes
    __shared__ __attribute__((aligned(16))) uint8_t lw[2][64 * LD];
    __shared__ __attribute__((aligned(16))) uint8_t lx[2][64 * LD];
    int64_t tn, tm;
    xcd_tile<4>(blockIdx.x, TN, TM, tn, tm);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int i = lane & 31, h = lane >> 5, wn = wave & 1, wm = wave >> 1;
    const int r = tid >> 2, ch = 16 * (tid & 3);
    const int64_t wrow = tn * 64 + r, xrow = tm * 64 + r;
    const uint8_t* wp = reinterpret_cast<const uint8_t*>(qw) + (wrow < n ? wrow : 0) * k + ch;
    const uint8_t* xp = reinterpret_cast<const uint8_t*>(qx) + (xrow < m ? xrow : 0) * kx + ch;
    u32x4 wv, xv;
    auto load = [&](int64_t kb) {
        wv = load16_part(wp + kb, wrow < n ? k - kb - ch : 0);
        xv = load16_part(xp + kb, xrow < m ? k - kb - ch : 0);
    };
    auto put = [&](int b) {
        *reinterpret_cast<u32x4*>(&lw[b][r * LD + ch]) = wv;
        *reinterpret_cast<u32x4*>(&lx[b][r * LD + ch]) = xv;
    };
    i32x16 acc = i32x16{0};
    int b = 0;
    if (k > 0) {
        load(0);
        put(0);
    }
    __syncthreads();
    for (int64_t kb = 0; kb < k; kb += 64, b ^= 1) {
        const bool more = kb + 64 < k;
        if (more)
            load(kb + 64);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const i32x4 a = *reinterpret_cast<const i32x4*>(&lw[b][(32 * wn + i) * LD + 32 * j + 16 * h]);
            const i32x4 c = *reinterpret_cast<const i32x4*>(&lx[b][(32 * wm + i) * LD + 32 * j + 16 * h]);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, c, acc, 0, 0, 0);
        }
        if (more)
            put(b ^ 1);
        __syncthreads();
    }
    const int64_t t = tm * 64 + 32 * wm + i;
    if (t >= m)
        return;
    const float st = sx[t];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t c0 = tn * 64 + 32 * wn + 8 * j + 4 * h;
        uint16_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t cc = c0 + e < n ? c0 + e : n - 1;
            o[e] = finish<A>(acc[4 * j + e], st, sw[cc], A::to_f32(bias_bits(bias, cc)));
        }
        if (c0 < n)
            store4(y + t * n + c0, o, n - c0);
    }
}

int64_t padded_k(int64_t k)
{
    return (k + 63) / 64 * 64;
}

}  // namespace

hipError_t launch_quantize_int8(const void* x, Act type, int64_t rows, int64_t k, int8_t* q, int64_t kx, float* scale,
                                hipStream_t stream)
{
    if (rows == 0)
        return hipSuccess;
    if (!grid_fits(rows, 256))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(quantize_int8_kernel, dim3((unsigned)rows), dim3(256), 0, stream, x, type, k, q, kx, scale);
    return hipGetLastError();
}

hipError_t launch_gemm_int8(const int8_t* qx, int64_t kx, const float* sx, int64_t m, int64_t k, const int8_t* qw,
                            const float* sw, const void* bias, int64_t n, void* y, Act out, hipStream_t stream)
{
    if (m == 0 || n == 0)
        return hipSuccess;
    const int64_t TN = (n + 63) / 64, TM = (m + 63) / 64;
    if (!grid_fits(TN * TM, 256))
        return hipErrorInvalidValue;
    if (out == Act::BF16)
        hipLaunchKernelGGL(int8_any_kernel<Bf16>, dim3((unsigned)(TN * TM)), dim3(256), 0, stream, qx, kx, sx, qw, sw,
                           static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), m, n, k, TN, TM);
    else
        hipLaunchKernelGGL(int8_any_kernel<F16>, dim3((unsigned)(TN * TM)), dim3(256), 0, stream, qx, kx, sx, qw, sw,
                           static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), m, n, k, TN, TM);
    return hipGetLastError();
}

// codes [m, k rounded up to 64], then scales [m]
size_t linear_int8_workspace_bytes(int64_t m, int64_t, int64_t k, const void*, const int8_t*)
{
    return (size_t)m * (size_t)padded_k(k) + (size_t)m * 4;
}

hipError_t launch_linear_int8(const void* x, Act act, int64_t m, int64_t k, const int8_t* qw, const float* sw,
                              const void* bias, int64_t n, void* y, void* ws, hipStream_t stream)
{
    if (m == 0 || n == 0)
        return hipSuccess;
    const int64_t kx = padded_k(k);
    int8_t* qx = static_cast<int8_t*>(ws);
    float* sx = reinterpret_cast<float*>(qx + m * kx);
    const hipError_t e = launch_quantize_int8(x, act, m, k, qx, kx, sx, stream);
    return e != hipSuccess ? e : launch_gemm_int8(qx, kx, sx, m, k, qw, sw, bias, n, y, act, stream);
}

const char* linear_int8_kernel_name(int64_t, int64_t, int64_t, const void*, const int8_t*)
{
    return "quantize_int8_kernel+int8_any_kernel";
}

}  // namespace fp8w
