// C ABI of libfp8w_moe.so: argument validation and dispatch. Declarations and
// the contract of each call are in include/fp8w_moe.h.
#include <math.h>
#include <stdint.h>

#include <new>
#include <vector>

#include "../../../include/fp8w_moe.h"
#include "moe.hpp"

namespace {

thread_local int g_last_hip_error = 0;

constexpr int64_t kMaxDim = (int64_t)0x7fffffff;
constexpr int64_t kMaxElems = (int64_t)1 << 62;

fp8w_status_t hip_status(hipError_t e)
{
    if (e == hipSuccess)
        return FP8W_SUCCESS;
    g_last_hip_error = (int)e;
    return FP8W_ERR_HIP;
}

bool aligned(const void* p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool valid_dtype(fp8w_dtype_t t)
{
    return t == FP8W_BF16 || t == FP8W_FP16 || t == FP8W_FP32;
}

bool valid_act(fp8w_dtype_t t)
{
    return t == FP8W_BF16 || t == FP8W_FP16;
}

size_t elem_bytes(fp8w_dtype_t t)
{
    return t == FP8W_FP32 ? 4 : 2;
}

fp8w::Act act_of(fp8w_dtype_t t)
{
    return t == FP8W_BF16 ? fp8w::Act::BF16 : (t == FP8W_FP16 ? fp8w::Act::FP16 : fp8w::Act::FP32);
}

bool dim_ok(int64_t v)
{
    return v >= 0 && v <= kMaxDim;
}

// a * b * c elements stay far from overflowing a byte count
bool product_ok(int64_t a, int64_t b, int64_t c = 1)
{
    if (a == 0 || b == 0 || c == 0)
        return true;
    return a <= kMaxElems / b && a * b <= kMaxElems / c;
}

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(Span a, Span b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0)
        return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return pa < pb + b.bytes && pb < pa + a.bytes;
}

template <size_t N>
bool overlaps_any(Span a, const Span (&list)[N])
{
    for (const Span& s : list)
        if (overlap(a, s))
            return true;
    return false;
}

bool route_sizes_ok(int64_t t, int64_t e, int64_t top)
{
    return t >= 0 && e >= 1 && e <= fp8w::kMaxExperts && top >= 1 && top <= e && top <= fp8w::kMaxTop &&
           t <= kMaxDim / top;
}

bool int8_sizes_ok(int64_t m, int64_t n, int64_t k)
{
    return dim_ok(m) && dim_ok(n) && k >= 0 && k <= fp8w::kMaxInt8K && product_ok(m, n) && product_ok(m, k + 64) &&
           product_ok(n, k) && fp8w::tiles_fit((m + 63) / 64, n);
}

bool expert_sizes_ok(int64_t m, int64_t e, int64_t n, int64_t k)
{
    return dim_ok(m) && e >= 1 && e <= fp8w::kMaxExperts && dim_ok(n) && dim_ok(k) && product_ok(e, n, k) &&
           product_ok(m, n) && fp8w::tiles_fit(fp8w::max_row_tiles(m, e, 64), n);
}

}  // namespace

extern "C" {

size_t fp8w_route_workspace_bytes(int64_t t, int64_t e, int64_t top_k)
{
    return route_sizes_ok(t, e, top_k) ? fp8w::route_workspace_bytes(t, e, top_k) : 0;
}

fp8w_status_t fp8w_route(const void* logits, fp8w_dtype_t dtype, int64_t t, int64_t e, int64_t top_k, int renormalize,
                         float* weights, int32_t* experts, int32_t* offsets, int32_t* slots, int32_t* tokens,
                         void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!valid_dtype(dtype) || !route_sizes_ok(t, e, top_k) || !offsets)
        return FP8W_ERR_INVALID_VALUE;
    if (t > 0 && (!logits || !weights || !experts || !slots || !tokens))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(logits, elem_bytes(dtype)) || !aligned(weights, 4) || !aligned(experts, 4) || !aligned(offsets, 4) ||
        !aligned(slots, 4) || !aligned(tokens, 4))
        return FP8W_ERR_MISALIGNED;
    size_t need = fp8w::route_workspace_bytes(t, e, top_k);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return FP8W_ERR_WORKSPACE;
    if (!aligned(workspace, 4))
        return FP8W_ERR_MISALIGNED;
    if (need == 0 && workspace_bytes > 0)
        need = 1;  // one that is passed without need is not an output's place either
    const size_t lists = t > 0 ? (size_t)t * (size_t)top_k * 4 : 0;
    const Span all[] = {{logits, (size_t)t * (size_t)e * elem_bytes(dtype)}, {weights, lists}, {experts, lists},
                        {offsets, ((size_t)e + 1) * 4}, {slots, lists}, {tokens, lists}, {workspace, need}};
    for (size_t a = 1; a < sizeof all / sizeof all[0]; ++a)
        for (size_t b = 0; b < a; ++b)
            if (overlap(all[a], all[b]))
                return FP8W_ERR_INVALID_VALUE;
    return hip_status(fp8w::launch_route(logits, act_of(dtype), t, e, top_k, renormalize != 0, weights, experts,
                                         offsets, slots, tokens, workspace, stream));
}

fp8w_status_t fp8w_combine(const void* y, fp8w_dtype_t act_dtype, const float* weights, int64_t t, int64_t top_k,
                           int64_t n, void* out, hipStream_t stream)
{
    if (!valid_act(act_dtype) || !dim_ok(t) || !dim_ok(n) || top_k < 0 || top_k > fp8w::kMaxTop ||
        !product_ok(t, n, top_k + 1) || t * ((n + 7) / 8) > ((int64_t)1 << 32) - 512)
        return FP8W_ERR_INVALID_VALUE;
    if (t == 0 || n == 0)
        return FP8W_SUCCESS;
    if (!out || (top_k > 0 && (!y || !weights)))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(y, 2) || !aligned(out, 2) || !aligned(weights, 4))
        return FP8W_ERR_MISALIGNED;
    const Span in[] = {{y, (size_t)t * (size_t)top_k * (size_t)n * 2}, {weights, (size_t)t * (size_t)top_k * 4}};
    if (overlaps_any({out, (size_t)t * (size_t)n * 2}, in))
        return FP8W_ERR_INVALID_VALUE;
    return hip_status(fp8w::launch_combine(y, act_of(act_dtype), weights, t, top_k, n, out, stream));
}

size_t fp8w_linear_experts_workspace_bytes(int64_t, int64_t, int64_t, int64_t, const void*, const uint8_t*)
{
    return 0;  // k is split over the waves of a workgroup, or not at all
}

const char* fp8w_linear_experts_kernel(int64_t m, int64_t e, int64_t n, int64_t k, const void* x, const uint8_t* q)
{
    if (!expert_sizes_ok(m, e, n, k) || m == 0 || n == 0)
        return nullptr;
    return fp8w::experts_kernel_name(m, e, n, k, x, q);
}

fp8w_status_t fp8w_linear_experts(const void* x, fp8w_dtype_t act_dtype, int64_t x_count, int64_t k, const uint8_t* q,
                                  const float* scale, const void* bias, int64_t e, int64_t n, const int32_t* offsets,
                                  int64_t m, const int32_t* x_rows, const int32_t* y_rows, void* y, void*, size_t,
                                  hipStream_t stream)
{
    if (!valid_act(act_dtype) || !dim_ok(x_count) || !expert_sizes_ok(m, e, n, k) || !product_ok(x_count, k))
        return FP8W_ERR_INVALID_VALUE;
    if (!x_rows && x_count != m)
        return FP8W_ERR_INVALID_VALUE;
    if (m == 0 || n == 0)
        return FP8W_SUCCESS;
    if (!offsets || !scale || !y || (k > 0 && (!q || (x_count > 0 && !x))))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(x, 2) || !aligned(y, 2) || !aligned(bias, 2) || !aligned(scale, 4) || !aligned(offsets, 4) ||
        !aligned(x_rows, 4) || !aligned(y_rows, 4))
        return FP8W_ERR_MISALIGNED;
    const Span in[] = {{x, (size_t)x_count * (size_t)k * 2},
                       {q, (size_t)e * (size_t)n * (size_t)k},
                       {scale, (size_t)e * (size_t)n * 4},
                       {bias, (size_t)e * (size_t)n * 2},
                       {offsets, ((size_t)e + 1) * 4},
                       {x_rows, (size_t)m * 4},
                       {y_rows, (size_t)m * 4}};
    const Span out{y, (size_t)m * (size_t)n * 2};
    if (overlaps_any(out, in))
        return FP8W_ERR_INVALID_VALUE;
    const fp8w::ExpertCall c{x, x_count, k, q, scale, bias, e, n, offsets, m, x_rows, y_rows, y};
    return hip_status(fp8w::launch_experts(c, act_of(act_dtype), stream));
}

fp8w_status_t fp8w_quantize_int8(const void* w, fp8w_dtype_t w_dtype, int64_t n, int64_t k, int8_t* q, float* scale,
                                 hipStream_t stream)
{
    if (!valid_dtype(w_dtype) || !int8_sizes_ok(0, n, k))
        return FP8W_ERR_INVALID_VALUE;
    if (n == 0)
        return FP8W_SUCCESS;
    if (!scale || (k > 0 && (!w || !q)))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(w, elem_bytes(w_dtype)) || !aligned(scale, 4))
        return FP8W_ERR_MISALIGNED;
    const Span sw{w, (size_t)n * (size_t)k * elem_bytes(w_dtype)}, sq{q, (size_t)n * (size_t)k},
        ss{scale, (size_t)n * 4};
    if (overlap(sw, sq) || overlap(sw, ss) || overlap(sq, ss))
        return FP8W_ERR_INVALID_VALUE;
    std::vector<float> host;
    try {
        host.resize((size_t)n);
    } catch (const std::bad_alloc&) {
        return hip_status(hipErrorOutOfMemory);
    }
    fp8w_status_t st = hip_status(fp8w::launch_quantize_int8(w, act_of(w_dtype), n, k, q, k, scale, stream));
    if (st != FP8W_SUCCESS)
        return st;
    st = hip_status(
        fp8w::own_status(hipMemcpyAsync(host.data(), scale, (size_t)n * 4, hipMemcpyDeviceToHost, stream)));
    if (st != FP8W_SUCCESS)
        return st;
    st = hip_status(fp8w::own_status(hipStreamSynchronize(stream)));
    if (st != FP8W_SUCCESS)
        return st;
    for (float s : host)
        if (!isfinite(s))
            return FP8W_ERR_NONFINITE;
    return FP8W_SUCCESS;
}

fp8w_status_t fp8w_quantize_activations_int8(const void* x, fp8w_dtype_t act_dtype, int64_t m, int64_t k, int8_t* qx,
                                             float* sx, hipStream_t stream)
{
    if (!valid_act(act_dtype) || !int8_sizes_ok(m, 0, k))
        return FP8W_ERR_INVALID_VALUE;
    if (m == 0)
        return FP8W_SUCCESS;
    if (!sx || (k > 0 && (!x || !qx)))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(x, 2) || !aligned(sx, 4))
        return FP8W_ERR_MISALIGNED;
    const Span s0{x, (size_t)m * (size_t)k * 2}, s1{qx, (size_t)m * (size_t)k}, s2{sx, (size_t)m * 4};
    if (overlap(s0, s1) || overlap(s0, s2) || overlap(s1, s2))
        return FP8W_ERR_INVALID_VALUE;
    return hip_status(fp8w::launch_quantize_int8(x, act_of(act_dtype), m, k, qx, k, sx, stream));
}

fp8w_status_t fp8w_gemm_int8(const int8_t* qx, const float* sx, int64_t m, int64_t k, const int8_t* q,
                             const float* scale, const void* bias, int64_t n, void* y, fp8w_dtype_t out_dtype,
                             hipStream_t stream)
{
    if (!valid_act(out_dtype) || !int8_sizes_ok(m, n, k))
        return FP8W_ERR_INVALID_VALUE;
    if (m == 0 || n == 0)
        return FP8W_SUCCESS;
    if (!sx || !scale || !y || (k > 0 && (!qx || !q)))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(sx, 4) || !aligned(scale, 4) || !aligned(bias, 2) || !aligned(y, 2))
        return FP8W_ERR_MISALIGNED;
    const Span in[] = {{qx, (size_t)m * (size_t)k}, {sx, (size_t)m * 4}, {q, (size_t)n * (size_t)k},
                       {scale, (size_t)n * 4}, {bias, (size_t)n * 2}};
    if (overlaps_any({y, (size_t)m * (size_t)n * 2}, in))
        return FP8W_ERR_INVALID_VALUE;
    return hip_status(
        fp8w::launch_gemm_int8(qx, sx, m, k, q, scale, bias, n, y, act_of(out_dtype), stream));
}

size_t fp8w_linear_int8_workspace_bytes(int64_t m, int64_t n, int64_t k, const void* x, const int8_t* q)
{
    if (!int8_sizes_ok(m, n, k) || m == 0 || n == 0)
        return 0;
    return fp8w::linear_int8_workspace_bytes(m, n, k, x, q);
}

const char* fp8w_linear_int8_kernel(int64_t m, int64_t n, int64_t k, const void* x, const int8_t* q)
{
    if (!int8_sizes_ok(m, n, k) || m == 0 || n == 0)
        return nullptr;
    return fp8w::linear_int8_kernel_name(m, n, k, x, q);
}

fp8w_status_t fp8w_linear_int8(const void* x, fp8w_dtype_t act_dtype, int64_t m, int64_t k, const int8_t* q,
                               const float* scale, const void* bias, int64_t n, void* y, void* workspace,
                               size_t workspace_bytes, hipStream_t stream)
{
    if (!valid_act(act_dtype) || !int8_sizes_ok(m, n, k))
        return FP8W_ERR_INVALID_VALUE;
    if (m == 0 || n == 0)
        return FP8W_SUCCESS;
    if (!scale || !y || (k > 0 && (!x || !q)))
        return FP8W_ERR_INVALID_VALUE;
    if (!aligned(x, 2) || !aligned(scale, 4) || !aligned(bias, 2) || !aligned(y, 2))
        return FP8W_ERR_MISALIGNED;
    const Span in[] = {{x, (size_t)m * (size_t)k * 2}, {q, (size_t)n * (size_t)k}, {scale, (size_t)n * 4},
                       {bias, (size_t)n * 2}};
    const Span out{y, (size_t)m * (size_t)n * 2};
    if (overlaps_any(out, in))
        return FP8W_ERR_INVALID_VALUE;
    const size_t need = fp8w::linear_int8_workspace_bytes(m, n, k, x, q);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return FP8W_ERR_WORKSPACE;
        if (!aligned(workspace, 16))
            return FP8W_ERR_MISALIGNED;
        if (overlaps_any({workspace, need}, in) || overlap({workspace, need}, out))
            return FP8W_ERR_INVALID_VALUE;
    }
    return hip_status(
        fp8w::launch_linear_int8(x, act_of(act_dtype), m, k, q, scale, bias, n, y, workspace, stream));
}

int fp8w_moe_last_hip_error(void)
{
    return g_last_hip_error;
}

}  // extern "C"
