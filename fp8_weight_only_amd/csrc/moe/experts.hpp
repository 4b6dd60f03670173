// What the kernels of products grouped by expert share, whatever the weights'
// format: which rows a tile has, and how its results are stored.
//
// SCALED: each output channel has an fp32 scale that enters here (e4m3 codes);
// without it the products are of whole weights already (4-bit codes, whose block
// scales enter when they are decoded).
#pragma once

#include "groups.hpp"
#include "moe.hpp"

namespace fp8w {

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
        o[r] = rounded<A>(
            __builtin_fmaf(c.scale[ch], ok ? acc[r] : __builtin_nanf(""), A::to_f32(bias_bits(bias, ch))));
    }
    store4(out, o, count);
}

// What a tile's epilogue needs: the channels' scales and biases, and where each
// row goes (-1: nowhere) and whether its source exists.
template <int BN, int BM>
struct ExpertEpilogue {
    float scale[BN];
    uint16_t bias[BN];
    int dst[BM];
    bool bad[BM];
};

// The source row of a tile's row; rows past the tile's and rows that do not
// exist read some row of x, and are not stored or stored as NaN.
__device__ __forceinline__ int64_t source_row(const ExpertCall& c, const RowTile& tile, int r)
{
    int64_t src = tile.row + (r < tile.rows ? r : 0);
    if (c.x_rows)
        src = c.x_rows[src];
    return src < 0 || src >= c.xr ? 0 : src;
}

// Fills the epilogue's operands (any thread its share); the caller's barrier
// stands before their use.
template <int BN, int BM, int NT, bool SCALED = true>
__device__ __forceinline__ void fill_epilogue(const ExpertCall& c, const RowTile& tile, int64_t n0,
                                              ExpertEpilogue<BN, BM>& e)
{
    for (int j = threadIdx.x; j < BN; j += NT) {
        const int64_t ch = n0 + j < c.n ? n0 + j : c.n - 1, at = (int64_t)tile.expert * c.n + ch;
        const bool on = tile.expert < (int)c.e;
        e.scale[j] = SCALED ? (on ? c.scale[at] : 0.0f) : 1.0f;
        e.bias[j] = on ? bias_bits(static_cast<const uint16_t*>(c.bias), at) : (uint16_t)0;
    }
    for (int j = threadIdx.x; j < BM; j += NT) {
        int dst = -1;
        bool bad = false;
        if (j < tile.rows) {
            const int pos = tile.row + j;
            dst = c.y_rows ? c.y_rows[pos] : pos;
            if (dst >= (int)c.m)
                dst = -1;
            if (c.x_rows && tile.expert < (int)c.e) {
                const int src = c.x_rows[pos];
                bad = src < 0 || src >= c.xr;
            }
        }
        e.dst[j] = dst;
        e.bad[j] = bad;
    }
}

// Lane (i, h) holds channels 8 j + 4 h + r of row i in accumulators 4 j + r of
// each fragment.
template <typename A, int BN, int BM, int WN, int WM, typename P>
__device__ __forceinline__ void store_tile(const ExpertCall& c, const P& p, int64_t n0,
                                           const ExpertEpilogue<BN, BM>& e, const f32x16* acc)
{
    const int i = p.lane & 31, h = p.lane >> 5;
#pragma unroll
    for (int fm = 0; fm < P::FM; ++fm) {
        const int rl = p.wm * (BM / WM) + 32 * fm + i, dst = e.dst[rl];
        if (dst < 0)
            continue;
        const bool bad = e.bad[rl];
        uint16_t* out = static_cast<uint16_t*>(c.y) + (int64_t)dst * c.n;
#pragma unroll
        for (int fn = 0; fn < P::FN; ++fn)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int cl = p.wn * (BN / WN) + 32 * fn + 8 * j + 4 * h;
                const int64_t c0 = n0 + cl;
                const f32x4 s4 = *reinterpret_cast<const f32x4*>(&e.scale[cl]);
                const u32x2 b4 = *reinterpret_cast<const u32x2*>(&e.bias[cl]);
                const float bf[4] = {A::lo_f32(b4.x), A::hi_f32(b4.x), A::lo_f32(b4.y), A::hi_f32(b4.y)};
                uint16_t o[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[r] = rounded<A>(bad ? __builtin_nanf("")
                                           : __builtin_fmaf(s4[r], acc[fn * P::FM + fm][4 * j + r], bf[r]));
                if (c0 < c.n)
                    store4(out + c0, o, c.n - c0);
            }
    }
}

// Which tile this workgroup is (false: none).
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertCall& c, int TN, int& tn, RowTile& tile)
{
    TileFinder<BM> finder(c.offsets, (int)c.e, (int)c.m);
    const int total = uniform(finder.total());
    if ((int)blockIdx.x >= TN * total)
        return false;
    int tm;
    xcd_tile<4>(blockIdx.x, TN, total, tn, tm);
    tile = finder.find(tm);
    tile.expert = uniform(tile.expert);
    tile.row = uniform(tile.row);
    tile.rows = uniform(tile.rows);
    return true;
}

}  // namespace fp8w
