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

// Few rows per expert (decode): the weights stream once, straight into the
// matrix cores' operand registers.
//
// A workgroup owns 16 CT channels of up to 16 rows of one expert. Its W waves
// split k in blocks of 128: a lane holds 16 codes of channel lane % 16 at k =
// 16 (lane / 16) of either half of a block (one 16-byte load each; 16 rows of
// 64 consecutive bytes per instruction), decodes them in registers, and feeds
// eight to each of two v_mfma_f32_16x16x32, the row's values at the same k on
// the other side. Which k meet in one instruction does not matter as long as
// both operands agree. The next block's loads are in flight during a block's
// products. The waves' sums meet in LDS and are added in wave order.
//
// Any k and any alignment: whole blocks take unaligned 16-byte loads, the last
// k % 128 a masked step.
template <typename A, int CT, int W>
__global__ __launch_bounds__(W* kWave) void experts_stream_kernel(ExpertCall c, int TN)
{
    __shared__ __attribute__((aligned(16))) f32x4 part[W][CT][kWave];
    TileFinder<16> finder(c.offsets, (int)c.e, (int)c.m);
    const int tn = blockIdx.x % TN;
    const RowTile tile = finder.find(blockIdx.x / TN);
    if (tile.expert < 0)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)tn * (16 * CT);
    f32x4 acc[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
        acc[t] = f32x4{0.0f};
    if (tile.expert < (int)c.e && c.xr > 0) {
        const uint8_t* wp[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int64_t ch = n0 + 16 * t + r < c.n ? n0 + 16 * t + r : c.n - 1;
            wp[t] = c.q + ((int64_t)tile.expert * c.n + ch) * c.k + 16 * g;
        }
        int64_t src = tile.row + (r < tile.rows ? r : 0);  // rows past the tile's: any row, not stored
        if (c.x_rows)
            src = c.x_rows[src];
        if (src < 0 || src >= c.xr)
            src = 0;  // stored as NaN
        const uint8_t* xp = static_cast<const uint8_t*>(c.x) + 2 * (src * c.k + 16 * g);
        struct Block {
            u32x4 w[CT][2], x[2][2];
        };
        auto load = [&](Block& b, int64_t kb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    b.w[t][h] = load16_any(wp[t] + kb + 64 * h);
                b.x[h][0] = load16_any(xp + 2 * kb + 128 * h);
                b.x[h][1] = load16_any(xp + 2 * kb + 128 * h + 16);
            }
        };
        auto compute = [&](const Block& b) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const u32x4 v = b.w[t][h];
                    const u32x2 d0 = A::decode4(v.x), d1 = A::decode4(v.y), d2 = A::decode4(v.z), d3 = A::decode4(v.w);
                    acc[t] = A::mfma(u32x4{d0.x, d0.y, d1.x, d1.y}, b.x[h][0], acc[t]);
                    acc[t] = A::mfma(u32x4{d2.x, d2.y, d3.x, d3.y}, b.x[h][1], acc[t]);
                }
        };
        const int64_t whole = c.k / 128;
        int64_t b = wave;
        if (b < whole) {
            Block cur;
            load(cur, 128 * b);
            for (b += W; b < whole; b += W) {
                Block next;
                load(next, 128 * b);
                compute(cur);
                cur = next;
            }
            compute(cur);
        }
        const int64_t kb = 128 * whole;
        if (kb < c.k && wave == (int)(whole % W)) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int64_t left = c.k - kb - 64 * h - 16 * g;
                const u32x4 x0 = load16_part(xp + 2 * kb + 128 * h, 2 * left);
                const u32x4 x1 = load16_part(xp + 2 * kb + 128 * h + 16, 2 * left - 16);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const u32x4 v = load16_part(wp[t] + kb + 64 * h, left);
                    const u32x2 d0 = A::decode4(v.x), d1 = A::decode4(v.y), d2 = A::decode4(v.z), d3 = A::decode4(v.w);
                    acc[t] = A::mfma(u32x4{d0.x, d0.y, d1.x, d1.y}, x0, acc[t]);
                    acc[t] = A::mfma(u32x4{d2.x, d2.y, d3.x, d3.y}, x1, acc[t]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < CT; ++t)
        part[wave][t][lane] = acc[t];
    __syncthreads();
    // lane (r, g) holds channels 4 g .. 4 g + 3 of row r
    for (int t = wave; t < CT; t += W) {
        f32x4 sum = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += part[w][t][lane];
        const int64_t c0 = n0 + 16 * t + 4 * g, left = c.n - c0;
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
        if (r < tile.rows && left > 0)
            store_tile_row<A>(c, tile.row + r, tile.expert, c0, left < 4 ? (int)left : 4, v);
    }
}

// Any k, any alignment: 64 channels x 64 rows, four waves of 32 x 32. Stages of
// 64 k pass through registers (the next stage's loads are in flight during this
// one's products) into LDS, the codes decoded on the way.
template <typename A>
__global__ __launch_bounds__(256) void experts_any_kernel(ExpertCall c, int TN)
{
    constexpr int BN = 64, BM = 64, LD = 72;  // LD: row pitch in elements; 16-byte reads of 16 rows spread over banks
    __shared__ __attribute__((aligned(16))) uint16_t sw[2][BN * LD];
    __shared__ __attribute__((aligned(16))) uint16_t sx[2][BM * LD];
    const int L = blockIdx.x;
    TileFinder<BM> finder(c.offsets, (int)c.e, (int)c.m);
    const int total = finder.total();
    if (L >= TN * total)
        return;
    int tn, tm;
    xcd_tile<4>(L, TN, total, tn, tm);
    const RowTile tile = finder.find(tm);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int i = lane & 31, h = lane >> 5, wn = wave & 1, wm = wave >> 1;
    const int64_t n0 = (int64_t)tn * BN;
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

template <typename A, int CT, int W>
hipError_t launch_stream(const ExpertCall& c, hipStream_t stream)
{
    const int64_t TN = (c.n + 16 * CT - 1) / (16 * CT), groups = TN * max_row_tiles(c.m, c.e, 16);
    hipLaunchKernelGGL((experts_stream_kernel<A, CT, W>), dim3((unsigned)groups), dim3(W * kWave), 0, stream, c,
                       (int)TN);
    return hipGetLastError();
}

struct ExpertPlan {
    bool stream;
    int ct, w;
};

ExpertPlan experts_plan(int64_t m, int64_t e, int64_t n, int64_t k)
{
    const int64_t active = m < e ? m : e;  // at most so many experts have rows
    ExpertPlan p{m <= 16 * active, 4, 8};
    const int64_t tiles = max_row_tiles(m, e, 16);
    auto groups = [&](int ct) { return (n + 16 * ct - 1) / (16 * ct) * active; };
    while (p.ct > 1 && groups(p.ct) < 256)
        p.ct /= 2;
    p.w = k >= 2048 ? 8 : 4;
    if (!grid_fits((n + 16 * p.ct - 1) / (16 * p.ct) * tiles, p.w * kWave))
        p.stream = false;
    return p;
}

template <typename A>
hipError_t launch_typed(const ExpertCall& c, hipStream_t stream)
{
    const ExpertPlan p = experts_plan(c.m, c.e, c.n, c.k);
    if (p.stream) {
        if (p.w == 8)
            return p.ct == 4   ? launch_stream<A, 4, 8>(c, stream)
                   : p.ct == 2 ? launch_stream<A, 2, 8>(c, stream)
                               : launch_stream<A, 1, 8>(c, stream);
        return p.ct == 4   ? launch_stream<A, 4, 4>(c, stream)
               : p.ct == 2 ? launch_stream<A, 2, 4>(c, stream)
                           : launch_stream<A, 1, 4>(c, stream);
    }
    const int64_t TN = (c.n + 63) / 64, groups = TN * max_row_tiles(c.m, c.e, 64);
    hipLaunchKernelGGL(experts_any_kernel<A>, dim3((unsigned)groups), dim3(256), 0, stream, c, (int)TN);
    return hipGetLastError();
}

}  // namespace

size_t experts_workspace_bytes(int64_t, int64_t, int64_t, int64_t, const void*, const uint8_t*)
{
    return 0;
}

hipError_t launch_experts(const ExpertCall& c, Act act, void*, size_t, hipStream_t stream)
{
    return act == Act::BF16 ? launch_typed<Bf16>(c, stream) : launch_typed<F16>(c, stream);
}

const char* experts_kernel_name(int64_t m, int64_t e, int64_t n, int64_t k, const void*, const uint8_t*)
{
    thread_local char name[96];
    const ExpertPlan p = experts_plan(m, e, n, k);
    if (!p.stream)
        return "experts_any_kernel";
    snprintf(name, sizeof name, "experts_stream_kernel<CT=%d,W=%d>", p.ct, p.w);
    return name;
}

}  // namespace fp8w
