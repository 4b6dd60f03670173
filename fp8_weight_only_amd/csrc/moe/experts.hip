// Matrix products grouped by expert, ragged sizes:
//   y[dst(p), c] = scale[i, c] * sum_k x[src(p), k] * value(q[i, c, k]) + bias[i, c]
// for the positions p of expert i, offsets[i] <= p < offsets[i + 1]; e4m3 codes
// with one fp32 scale per expert and output channel, bf16 / fp16 activations,
// fp32 accumulation, one rounding. src and dst are the optional row lists
// (gather from tokens, scatter to slots). Positions from offsets[e] on belong to
// no expert: their rows are zeros. A position whose source row does not exist
// gives NaN; one whose destination does not exist is not written.
//
// The offsets stay on the GPU: the grid holds the most tiles that m rows in e
// ragged groups can make, and a workgroup finds its tile from the offsets
// (groups.hpp); those past the last tile end at once.
#include <stdio.h>

#include "device.hpp"
#include "groups.hpp"
#include "moe.hpp"

namespace fp8w {
namespace {

template <typename A>
__device__ __forceinline__ void store_tile_row(const ExpertCall& c, int64_t pos, int expert, int64_t c0, int count,
                                               const float* acc)
{
    int64_t dst = pos;
    if (c.y_rows) {
        dst = c.y_rows[pos];
        if (dst < 0 || dst >= c.m)
            return;
    }
    bool ok = true;
    if (c.x_rows && expert < (int)c.e) {
        const int64_t src = c.x_rows[pos];
        ok = src >= 0 && src < c.xr;
    }
    uint16_t o[4];
    uint16_t* out = static_cast<uint16_t*>(c.y) + dst * c.n + c0;
    const uint16_t* bias = static_cast<const uint16_t*>(c.bias);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (r >= count || expert >= (int)c.e) {
            o[r] = 0;
            continue;
        }
        const int64_t ch = (int64_t)expert * c.n + c0 + r;
        o[r] = epilogue<A>(ok ? acc[r] : __builtin_nanf(""), c.scale[ch], bias, ch);
    }
    store4(out, o, count);
}

// Any k, any alignment: 64 channels x 64 rows, four waves of 32 x 32. Stages of
// 64 k pass through registers (the next stage's loads are in flight during this
// one's products) into LDS, the codes decoded on the way.
template <typename A>
__global__ __launch_bounds__(256) void experts_any_kernel(ExpertCall c, int64_t TN)
{
    constexpr int BN = 64, BM = 64, LD = 72;  // LD: row pitch in elements; 16-byte reads of 16 rows spread over banks
    __shared__ __attribute__((aligned(16))) uint16_t sw[2][BN * LD];
    __shared__ __attribute__((aligned(16))) uint16_t sx[2][BM * LD];
    int64_t tn = 0;
    const int64_t L = blockIdx.x;
    const RowTile tile = find_row_tile<BM>(c.offsets, (int)c.e, c.m, [&](int64_t total) -> int64_t {
        if (L >= TN * total)
            return -1;
        int64_t tm;
        xcd_tile<4>(L, TN, total, tn, tm);
        return tm;
    });
    if (tile.expert < 0)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int i = lane & 31, h = lane >> 5, wn = wave & 1, wm = wave >> 1;
    const int64_t n0 = tn * BN;
    f32x16 acc = f32x16{0.0f};
    if (tile.expert < (int)c.e) {
        // this thread's 16 codes of one weight row and 8 values of two rows of x in each stage
        const int64_t wrow = n0 + (tid >> 2);
        const uint8_t* wp = c.q + ((int64_t)tile.expert * c.n + (wrow < c.n ? wrow : 0)) * c.k + 16 * (tid & 3);
        const bool won = wrow < c.n;
        const uint8_t* xp[2];
        bool xon[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (tid >> 3) + 32 * u;
            int64_t src = tile.row + r;
            xon[u] = r < tile.rows;
            if (xon[u] && c.x_rows)
                src = c.x_rows[src];
            xon[u] = xon[u] && src >= 0 && src < c.xr;
            xp[u] = static_cast<const uint8_t*>(c.x) + 2 * ((xon[u] ? src : 0) * c.k + 8 * (tid & 7));
        }
        u32x4 wv, xv[2];
        auto load = [&](int64_t kb) {
            wv = load16_part(wp + kb, won ? c.k - kb - 16 * (tid & 3) : 0);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                xv[u] = load16_part(xp[u] + 2 * kb, xon[u] ? 2 * (c.k - kb - 8 * (tid & 7)) : 0);
        };
        auto put = [&](int b) {
            const uint32_t w4[4] = {wv.x, wv.y, wv.z, wv.w};
            uint16_t* d = &sw[b][(tid >> 2) * LD + 16 * (tid & 3)];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const u32x2 p0 = A::decode4(w4[2 * v]), p1 = A::decode4(w4[2 * v + 1]);
                *reinterpret_cast<u32x4*>(d + 8 * v) = u32x4{p0.x, p0.y, p1.x, p1.y};
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                *reinterpret_cast<u32x4*>(&sx[b][((tid >> 3) + 32 * u) * LD + 8 * (tid & 7)]) = xv[u];
        };
        int b = 0;
        if (c.k > 0) {
            load(0);
            put(0);
        }
        __syncthreads();
        for (int64_t kb = 0; kb < c.k; kb += 64, b ^= 1) {
            const bool more = kb + 64 < c.k;
            if (more)
                load(kb + 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(&sw[b][(32 * wn + i) * LD + 16 * j + 8 * h]);
                const u32x4 bb = *reinterpret_cast<const u32x4*>(&sx[b][(32 * wm + i) * LD + 16 * j + 8 * h]);
                acc = mfma32<A>(a, bb, acc);
            }
            if (more)
                put(b ^ 1);
            __syncthreads();
        }
    }
    // lane (i, h) holds channels 8 j + 4 h + r of row i in accumulators 4 j + r
    const int rl = 32 * wm + i;
    if (rl >= tile.rows)
        return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t c0 = n0 + 32 * wn + 8 * j + 4 * h;
        const int64_t left = c.n - c0;
        const float v[4] = {acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]};
        if (left > 0)
            store_tile_row<A>(c, tile.row + rl, tile.expert, c0, left < 4 ? (int)left : 4, v);
    }
}

}  // namespace

size_t experts_workspace_bytes(int64_t, int64_t, int64_t, int64_t, const void*, const uint8_t*)
{
    return 0;
}

hipError_t launch_experts(const ExpertCall& c, Act act, void*, size_t, hipStream_t stream)
{
    const int64_t TN = (c.n + 63) / 64, groups = TN * max_row_tiles(c.m, c.e, 64);
    if (!grid_fits(groups, 256))
        return hipErrorInvalidValue;
    if (act == Act::BF16)
        hipLaunchKernelGGL(experts_any_kernel<Bf16>, dim3((unsigned)groups), dim3(256), 0, stream, c, TN);
    else
        hipLaunchKernelGGL(experts_any_kernel<F16>, dim3((unsigned)groups), dim3(256), 0, stream, c, TN);
    return hipGetLastError();
}

const char* experts_kernel_name(int64_t, int64_t, int64_t, int64_t, const void*, const uint8_t*)
{
    return "experts_any_kernel";
}

}  // namespace fp8w
