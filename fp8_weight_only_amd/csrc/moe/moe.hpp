// Host-side launchers of libfp8w_moe.so (routing, products grouped by expert,
// their weighted sum, the int8 linear layer). Internal: the public interface is
// the C ABI in include/fp8w_moe.h. Every launcher enqueues on the given stream,
// returns the launch status, and assumes that the C-ABI layer has validated
// sizes, pointers and alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <tuple>

namespace fp8w {

enum class Act { BF16 = 0, FP16 = 1, FP32 = 2 };

constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 64;
constexpr int64_t kMaxInt8K = 131072;  // 128 * 128 * k is at most 2^31

// A HIP call's status. What a failed one leaves for hipGetLastError() is taken
// back, for the status goes to the caller by itself.
inline hipError_t own_status(hipError_t e)
{
    if (e != hipSuccess)
        (void)hipGetLastError();
    return e;
}

// Launches a kernel and returns the launch's own status. hipGetLastError() behind
// it would return, and clear, an error that an earlier call of the thread left for
// its own caller.
template <typename... P, typename... Q>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t stream, Q... args)
{
    std::tuple<P...> values{static_cast<P>(args)...};
    return std::apply(
        [&](P&... v) {
            void* pointers[] = {const_cast<void*>(static_cast<const void*>(&v))...};
            return own_status(
                hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, pointers, 0, stream));
        },
        values);
}

// A grid of this many workgroups of `threads` stays under the 2^32 threads a
// launch can have.
inline bool grid_fits(int64_t groups, int64_t threads)
{
    return groups <= ((int64_t)1 << 32) / threads - 1;
}

// The kernels that take every shape run 256-thread workgroups on 64 x 64 tiles.
inline bool tiles_fit(int64_t row_tiles, int64_t n)
{
    const int64_t tn = (n + 63) / 64;
    return row_tiles == 0 || tn == 0 || tn <= (((int64_t)1 << 32) / 256 - 1) / row_tiles;
}

// Most row tiles of `bm` rows that m rows in e ragged groups (and one group of
// rows without an expert) can make: every non-empty group may end inside a tile.
inline int64_t max_row_tiles(int64_t m, int64_t e, int64_t bm)
{
    const int64_t g = m < e + 1 ? m : e + 1;
    return g + (m - g) / bm;
}

size_t route_workspace_bytes(int64_t t, int64_t e, int64_t top);
hipError_t launch_route(const void* logits, Act type, int64_t t, int64_t e, int64_t top, bool renorm, float* weights,
                        int32_t* experts, int32_t* offsets, int32_t* slots, int32_t* tokens, void* ws,
                        hipStream_t stream);

hipError_t launch_combine(const void* y, Act act, const float* weights, int64_t t, int64_t top, int64_t n, void* out,
                          hipStream_t stream);

struct ExpertCall {
    const void* x;
    int64_t xr, k;  // x is [xr, k]
    const uint8_t* q;
    const float* scale;
    const void* bias;
    int64_t e, n;
    const int32_t* offsets;
    int64_t m;
    const int32_t *x_rows, *y_rows;
    void* y;
};
hipError_t launch_experts(const ExpertCall& c, Act act, hipStream_t stream);
const char* experts_kernel_name(int64_t m, int64_t e, int64_t n, int64_t k, const void* x, const uint8_t* q);

// The same on 4-bit weights: q rows of row_bytes = (k + 1) / 2 bytes, row_scales =
// (k + 31) / 32 e8m0 scales of a row, no scale of a channel. Without offsets e == 1
// and all rows are that expert's.
struct Fp4Call : ExpertCall {
    const uint8_t* block_scale;
    int64_t row_bytes, row_scales;
    float* parts;  // the linear layer's workspace, where its plan needs one
};
struct Fp4Shape {
    int64_t m, e, n, k, xr;
    bool grouped;
    int64_t row_tiles(int64_t bm) const { return grouped ? max_row_tiles(m, e, bm) : (m + bm - 1) / bm; }
};
hipError_t launch_fp4(const Fp4Call& c, Act act, hipStream_t stream);
size_t linear_fp4_workspace_bytes(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale);
const char* fp4_kernel_name(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale);
hipError_t launch_quantize_fp4(const void* w, Act type, int64_t n, int64_t k, uint8_t* q, uint8_t* scale,
                               hipStream_t stream);
hipError_t launch_dequantize_fp4(const uint8_t* q, const uint8_t* scale, int64_t n, int64_t k, void* out, Act type,
                                 hipStream_t stream);

constexpr int kMaxLayerTokens = 64;
constexpr int64_t kMaxLayerWidth = (int64_t)1 << 22;  // units of k times experts fit an int
constexpr int64_t kMaxLayerValues = (int64_t)1 << 27;  // silu(gate) * up of all places, four rows for one: bytes fit an int

struct LayerWeights {
    const uint8_t* q;
    const void* scale;  // [e, n] fp32 of e4m3 codes, [e, n, (k + 31) / 32] bytes of 4-bit ones
    const void* bias;   // [e, n] or null
};
struct LayerCall {
    const void* x;  // [t, hidden]
    const void* logits;
    Act logits_type;
    int top, renorm;
    int64_t t, e, hidden, inner;
    LayerWeights up, down;  // [e, 2 inner, hidden], [e, hidden, inner]
    void* out;
    // the workspace's parts, set by launch_layer
    uint16_t* h;
    int64_t pitch;
    int32_t* plan;
    uint32_t* arrived;  // per 16 output channels, null where one workgroup has them
    float* parts;
};
size_t layer_workspace_bytes(int64_t t, int64_t e, int64_t top, int64_t hidden, int64_t inner);
hipError_t launch_layer(LayerCall c, bool fp4, Act act, void* ws, hipStream_t stream);

// qx rows are kx >= k bytes apart (kx > k: bytes k .. kx - 1 of every row are
// written as zeros).
hipError_t launch_quantize_int8(const void* x, Act type, int64_t rows, int64_t k, int8_t* q, int64_t kx, float* scale,
                                hipStream_t stream);
// qx [m, k] dense.
hipError_t launch_gemm_int8(const int8_t* qx, const float* sx, int64_t m, int64_t k, const int8_t* qw,
                            const float* sw, const void* bias, int64_t n, void* y, Act out, hipStream_t stream);
size_t linear_int8_workspace_bytes(int64_t m, int64_t n, int64_t k, const void* x, const int8_t* q);
hipError_t launch_linear_int8(const void* x, Act act, int64_t m, int64_t k, const int8_t* qw, const float* sw,
                              const void* bias, int64_t n, void* y, void* ws, hipStream_t stream);
const char* linear_int8_kernel_name(int64_t m, int64_t n, int64_t k, const void* x, const int8_t* q);

}  // namespace fp8w
