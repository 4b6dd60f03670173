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

#include "experts.hpp"
#include "tile.hpp"

namespace fp8w {
namespace {

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
// Any k and any alignment: whole blocks take 16-byte loads from any dword (below
// that, Row), the last k % 128 a masked step.
//
// Bound by the weight stream: one token, two of eight [14336, 4096] experts read
// 117 MB in 27.6 us on 448 workgroups of eight waves, 4.3 TB/s, when calls go
// through all eight experts in turn (470 MB; a large copy: 4.9 to 5.2 TB/s). With
// two pairs of experts in turn the memory-side cache (256 MB) holds part of them:
// 22 us. Measured against those 22: four waves the same; 32 or 16 channels per
// workgroup 23 to 25 us (more waves load the same activations); four blocks per
// wave in flight 26, for fewer waves per CU; loads that bypass the caches 27 to
// 30 (two lanes' 64-byte halves of a line come by separate instructions).
template <typename A, int CT, int W, bool SHIFT>
__global__ __launch_bounds__(W* kWave) void experts_stream_kernel(ExpertCall c, int TN)
{
    __shared__ __attribute__((aligned(16))) f32x4 part[W][CT][kWave];
    TileFinder<16> finder(c.offsets, (int)c.e, (int)c.m);
    const int tn = blockIdx.x % TN;
    const RowTile tile = finder.find(blockIdx.x / TN);
    if (tile.expert < 0)
        return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)tn * (16 * CT);
    f32x4 acc[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
        acc[t] = f32x4{0.0f};
    if (tile.expert < (int)c.e && c.xr > 0) {
        Row<SHIFT> wp[CT], xp;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int64_t ch = n0 + 16 * t + r < c.n ? n0 + 16 * t + r : c.n - 1;
            wp[t] = Row<SHIFT>(c.q + ((int64_t)tile.expert * c.n + ch) * c.k + 16 * g);
        }
        int64_t src = tile.row + (r < tile.rows ? r : 0);  // rows past the tile's: any row, not stored
        if (c.x_rows)
            src = c.x_rows[src];
        if (src < 0 || src >= c.xr)
            src = 0;  // stored as NaN
        xp = Row<SHIFT>(static_cast<const uint8_t*>(c.x) + 2 * (src * c.k + 16 * g));
        struct Block {
            typename Row<SHIFT>::Raw w[CT][2], x[2][2];
        };
        auto load = [&](Block& b, int64_t kb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    b.w[t][h] = wp[t].load(kb + 64 * h);
                b.x[h][0] = xp.load(2 * kb + 128 * h);
                b.x[h][1] = xp.load(2 * kb + 128 * h + 16);
            }
        };
        auto compute = [&](const Block& b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 x0 = xp.bytes(b.x[h][0]), x1 = xp.bytes(b.x[h][1]);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const u32x4 v = wp[t].bytes(b.w[t][h]);
                    const u32x2 d0 = A::decode4(v.x), d1 = A::decode4(v.y), d2 = A::decode4(v.z), d3 = A::decode4(v.w);
                    acc[t] = A::mfma(u32x4{d0.x, d0.y, d1.x, d1.y}, x0, acc[t]);
                    acc[t] = A::mfma(u32x4{d2.x, d2.y, d3.x, d3.y}, x1, acc[t]);
                }
            }
        };
        // this wave's blocks: wave, wave + W, .. below k / 128
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
                const u32x4 x0 = xp.part(2 * kb + 128 * h, 2 * left);
                const u32x4 x1 = xp.part(2 * kb + 128 * h + 16, 2 * left - 16);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const u32x4 v = wp[t].part(kb + 64 * h, left);
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

// ------------------------------------------------------------------ tiles
// More rows per expert: BN channels x BM rows of one expert, WN x WM waves of
// 32 x 32 fragments, stages of 64 k. In LDS a stage holds BN rows of 64 codes,
// their four 16-byte chunks rotated by row / 4, and BM rows of 64 activations,
// their eight chunks rotated by row / 2, so the 16 lanes of a read's phase (16
// rows, same chunk) hit distinct banks. The codes are decoded on their way from
// LDS to the matrix cores: every e4m3 value is a bf16 and an fp16 value.
//
// Two waves per SIMD and 256 x 256 tiles (128 x 64 per wave) where the rows fill
// them: 4096 tokens, two of eight [14336, 4096] experts take 838 to 871 us from
// card to card, 1.1 PFLOP/s with the matrix cores busy 66 % of the time at a clock
// of 1.7 to 1.9 GHz and no bank conflicts; a large bf16 product of the vendor's
// library runs at 1.2 to 1.3 PFLOP/s there. Raised wave priority around the products, another grouping of tiles per
// XCD (2, 8) and no stagger of k measured the same within 2 %.
//
// A half of a stage is 32 k: lane (i, h) takes the 16 codes and the 16 values at
// k = 16 h of its rows, eight for each of two v_mfma_f32_32x32x16. Which k meet
// in one instruction does not matter as long as both operands agree.
template <typename A, int BN, int BM, int WN, int WM>
struct ExpertTile {
    static constexpr int W = WN * WM, NT = W * kWave, FN = BN / WN / 32, FM = BM / WM / 32;
    static constexpr int ABYTES = BN * 64, STAGE = ABYTES + BM * 128;
    static_assert(BN == FN * WN * 32 && BM == FM * WM * 32, "tile and wave layout");
    struct Frags {
        u32x4 a[FN], x[FM][2];
    };
    int lane, wave, wn, wm;

    __device__ __forceinline__ void read(const uint8_t* buf, int j, Frags& f) const
    {
        const int i = lane & 31, h = lane >> 5;
        // one addition to the buffer's address per read: through longer chains the compiler
        // loses which buffer is read, and waits for every load in flight
        const int oa = 64 * (wn * (BN / WN) + i) + 16 * ((2 * j + h + (i >> 2)) & 3);
        const int ox = ABYTES + 128 * (wm * (BM / WM) + i);
        const int o0 = ox + 16 * ((4 * j + 2 * h + (i >> 1)) & 7), o1 = ox + 16 * ((4 * j + 2 * h + 1 + (i >> 1)) & 7);
#pragma unroll
        for (int q = 0; q < FN; ++q)
            f.a[q] = *reinterpret_cast<const u32x4*>(buf + (oa + 2048 * q));
#pragma unroll
        for (int q = 0; q < FM; ++q)
            f.x[q][0] = *reinterpret_cast<const u32x4*>(buf + (o0 + 4096 * q));
#pragma unroll
        for (int q = 0; q < FM; ++q)
            f.x[q][1] = *reinterpret_cast<const u32x4*>(buf + (o1 + 4096 * q));
    }

    __device__ __forceinline__ void mma(const Frags& f, f32x16* acc) const
    {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            u32x4 a[FN];
#pragma unroll
            for (int q = 0; q < FN; ++q) {
                const u32x4 v = f.a[q];
                const u32x2 d0 = A::decode4(t ? v.z : v.x), d1 = A::decode4(t ? v.w : v.y);
                a[q] = u32x4{d0.x, d0.y, d1.x, d1.y};
            }
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int fm = 0; fm < FM; ++fm)
                    acc[fn * FM + fm] = mfma32<A>(a[fn], f.x[fm][t], acc[fn * FM + fm]);
        }
    }
};

// Any k, any alignment, any number of rows in x: a stage passes through
// registers into LDS (run_tile_staged).
template <typename A, int BN, int BM, int WN, int WM, bool SHIFT>
__global__ __launch_bounds__(WN* WM* kWave) void experts_tile_kernel(ExpertCall c, int TN)
{
    using P = ExpertTile<A, BN, BM, WN, WM>;
    constexpr int LW = BN * 4 / P::NT, LX = BM * 8 / P::NT;
    static_assert(BN * 4 == LW * P::NT && BM * 8 == LX * P::NT, "chunks split evenly");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][P::STAGE];
    __shared__ __attribute__((aligned(16))) ExpertEpilogue<BN, BM> epi;
    int tn;
    RowTile tile;
    if (!find_tile<BM>(c, TN, tn, tile))
        return;
    const int64_t n0 = (int64_t)tn * BN;
    const int tid = threadIdx.x;
    P p;
    p.lane = tid & 63;
    p.wave = uniform(tid >> 6);
    p.wn = p.wave % WN;
    p.wm = p.wave / WN;
    fill_epilogue<BN, BM, P::NT>(c, tile, n0, epi);
    f32x16 acc[P::FN * P::FM];
#pragma unroll
    for (int f = 0; f < P::FN * P::FM; ++f)
        acc[f] = f32x16{0.0f};
    const int64_t S = tile.expert < (int)c.e && c.xr > 0 ? (c.k + 63) / 64 : 0;
    if (S > 0) {
        Row<SHIFT> wp[LW], xp[LX];
        int wo[LW], xo[LX];
        const int wc = tid & 3, xc = tid & 7;
#pragma unroll
        for (int u = 0; u < LW; ++u) {
            const int r = (tid >> 2) + P::NT / 4 * u;
            wp[u] = Row<SHIFT>(c.q + ((int64_t)tile.expert * c.n + (n0 + r < c.n ? n0 + r : c.n - 1)) * c.k + 16 * wc);
            wo[u] = 64 * r + 16 * ((wc + (r >> 2)) & 3);
        }
#pragma unroll
        for (int u = 0; u < LX; ++u) {
            const int r = (tid >> 3) + P::NT / 8 * u;
            xp[u] = Row<SHIFT>(static_cast<const uint8_t*>(c.x) + 2 * (source_row(c, tile, r) * c.k + 8 * xc));
            xo[u] = P::ABYTES + 128 * r + 16 * ((xc + (r >> 1)) & 7);
        }
        struct Regs {
            typename Row<SHIFT>::Raw w[LW], x[LX];
        };
        auto load_whole = [&](Regs& g, int s) {
            const int64_t kb = 64 * (int64_t)s;
#pragma unroll
            for (int u = 0; u < LW; ++u)
                g.w[u] = wp[u].load(kb);
#pragma unroll
            for (int u = 0; u < LX; ++u)
                g.x[u] = xp[u].load(2 * kb);
        };
        auto load = [&](Regs& g, int s) {
            const int64_t kb = 64 * (int64_t)s;
            if (kb + 64 <= c.k) {
                load_whole(g, s);
            } else {
#pragma unroll
                for (int u = 0; u < LW; ++u)
                    g.w[u] = wp[u].part_raw(kb, c.k - kb - 16 * wc);
#pragma unroll
                for (int u = 0; u < LX; ++u)
                    g.x[u] = xp[u].part_raw(2 * kb, 2 * (c.k - kb - 8 * xc));
            }
        };
        auto put = [&](const Regs& g, int b) {
#pragma unroll
            for (int u = 0; u < LW; ++u)
                *reinterpret_cast<u32x4*>(&lds[b][wo[u]]) = wp[u].bytes(g.w[u]);
#pragma unroll
            for (int u = 0; u < LX; ++u)
                *reinterpret_cast<u32x4*>(&lds[b][xo[u]]) = xp[u].bytes(g.x[u]);
        };
        auto compute = [&](int b) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                typename P::Frags f;
                p.read(lds[b], j, f);
                p.mma(f, acc);
            }
        };
        run_tile_staged<Regs>((int)S, (int)(c.k / 64), load, load_whole, put, compute);
    } else {
        __syncthreads();
    }
    store_tile<A, BN, BM, WN, WM>(c, p, n0, epi, acc);
}

// Rows at 16-byte boundaries, k a multiple of 64, x below 2 GiB: the same tiles
// fed by a ring of NS direct-to-LDS stages (tile.hpp).
template <typename A, int BN, int BM, int WN, int WM>
struct ExpertRing : ExpertTile<A, BN, BM, WN, WM> {
    using T = ExpertTile<A, BN, BM, WN, WM>;
    static constexpr int LW = BN / 16 / T::W, LX = BM / 8 / T::W, LOADS = LW + LX;  // 1 KB loads per wave and stage
    static_assert(BN == LW * 16 * T::W && BM == LX * 8 * T::W, "loads split evenly");
    Rows w, x;
    int off[LOADS];  // this lane's 16 bytes of each load at k = 0
    int S, rot;

    __device__ __forceinline__ void issue(int s, uint8_t* buf) const
    {
        const int kb = 64 * (s + rot < S ? s + rot : s + rot - S);
#pragma unroll
        for (int u = 0; u < LW; ++u)
            w.load(off[u], kb, buf + 1024 * (u * T::W + this->wave));
#pragma unroll
        for (int u = 0; u < LX; ++u)
            x.load(off[LW + u], 2 * kb, buf + T::ABYTES + 1024 * (u * T::W + this->wave));
    }
};

// A wave whose rows all lie past the tile's: it loads its share and keeps the
// barriers, and leaves the matrix cores to the others.
template <typename A, int BN, int BM, int WN, int WM>
struct ExpertRingIdle : ExpertRing<A, BN, BM, WN, WM> {
    struct Frags {};
    __device__ __forceinline__ void read(const uint8_t*, int, Frags&) const {}
    __device__ __forceinline__ void mma(const Frags&, f32x16*) const {}
};

template <typename A, int BN, int BM, int WN, int WM, int NS>
__global__ __launch_bounds__(WN* WM* kWave) void experts_ring_kernel(ExpertCall c, int TN)
{
    using P = ExpertRing<A, BN, BM, WN, WM>;
    using T = ExpertTile<A, BN, BM, WN, WM>;
    static_assert(NS >= 3 && NS <= 8, "stages");
    __shared__ __attribute__((aligned(1024))) uint8_t b0[T::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[T::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[T::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[NS > 3 ? T::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b4[NS > 4 ? T::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b5[NS > 5 ? T::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b6[NS > 6 ? T::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b7[NS > 7 ? T::STAGE : 16];
    __shared__ __attribute__((aligned(16))) ExpertEpilogue<BN, BM> epi;
    auto buf = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < 4)
            return ring_buf<i>(b0, b1, b2, b3);
        else
            return ring_buf<i - 4>(b4, b5, b6, b7);
    };
    int tn;
    RowTile tile;
    if (!find_tile<BM>(c, TN, tn, tile))
        return;
    const int64_t n0 = (int64_t)tn * BN;
    const int tid = threadIdx.x;
    P p;
    p.lane = tid & 63;
    p.wave = uniform(tid >> 6);
    p.wn = p.wave % WN;
    p.wm = p.wave / WN;
    f32x16 acc[T::FN * T::FM];
#pragma unroll
    for (int f = 0; f < T::FN * T::FM; ++f)
        acc[f] = f32x16{0.0f};
    fill_epilogue<BN, BM, T::NT>(c, tile, n0, epi);
    if (tile.expert < (int)c.e && c.xr > 0) {
        p.S = (int)(c.k / 64);
        p.rot = (int)(blockIdx.x % 8) * (p.S / 8);
        p.w = Rows(c.q + ((int64_t)tile.expert * c.n + n0) * c.k);
        p.x = Rows(c.x);
#pragma unroll
        for (int u = 0; u < P::LW; ++u) {
            const int r = 16 * (u * T::W + p.wave) + (p.lane >> 2);
            p.off[u] = (int)((n0 + r < c.n ? r : c.n - 1 - n0) * c.k) + 16 * (((p.lane & 3) - (r >> 2)) & 3);
        }
#pragma unroll
        for (int u = 0; u < P::LX; ++u) {
            const int r = 8 * (u * T::W + p.wave) + (p.lane >> 3);
            p.off[P::LW + u] = (int)(2 * source_row(c, tile, r) * c.k) + 16 * (((p.lane & 7) - (r >> 1)) & 7);
        }
        if (p.wm * (BM / WM) < tile.rows) {
            run_tile_ring<NS, P::LOADS>(p, p.S, buf, acc);
        } else {
            ExpertRingIdle<A, BN, BM, WN, WM> idle;
            static_cast<P&>(idle) = p;
            run_tile_ring<NS, P::LOADS>(idle, p.S, buf, acc);
        }
    }
    __syncthreads();
    store_tile<A, BN, BM, WN, WM>(c, p, n0, epi, acc);
}

// ------------------------------------------------------------------ plans
enum class ExpertKind { STREAM, TILE, RING };

struct ExpertPlan {
    ExpertKind kind;
    int a, b, w;  // stream: CT, rows of a tile, W; tile, ring: BN, BM, waves
    int64_t groups(int64_t m, int64_t e, int64_t n) const
    {
        const int64_t bn = kind == ExpertKind::STREAM ? 16 * a : a;
        return (n + bn - 1) / bn * max_row_tiles(m, e, b);
    }
    bool fits(int64_t m, int64_t e, int64_t n) const { return grid_fits(groups(m, e, n), w * kWave); }
};

constexpr ExpertPlan kRings[] = {{ExpertKind::RING, 256, 256, 8}, {ExpertKind::RING, 256, 128, 8},
                                 {ExpertKind::RING, 128, 128, 8}, {ExpertKind::RING, 256, 64, 8},
                                 {ExpertKind::RING, 128, 64, 4},  {ExpertKind::RING, 64, 64, 4},
                                 {ExpertKind::RING, 256, 32, 4},  {ExpertKind::RING, 128, 32, 4},
                                 {ExpertKind::RING, 64, 32, 2}};
constexpr ExpertPlan kTiles[] = {{ExpertKind::TILE, 256, 128, 8}, {ExpertKind::TILE, 128, 64, 4},
                                 {ExpertKind::TILE, 64, 64, 4}, {ExpertKind::TILE, 128, 32, 4}};

// Stages of a ring's tile: what LDS holds.
constexpr int ring_depth(int bn, int bm)
{
    return bn == 256 && bm == 256 ? 3 : 4;
}

ExpertPlan stream_plan(int64_t active, int64_t n, int64_t k)
{
    ExpertPlan p{ExpertKind::STREAM, 4, 16, k >= 2048 ? 8 : 4};
    while (p.a > 1 && (n + 16 * p.a - 1) / (16 * p.a) * active < 256)
        p.a /= 2;
    return p;
}

// The plan goes by the rows per expert, were they spread evenly over as many
// experts as can have any (how they are spread only the GPU knows). Measured, us,
// rows of random tokens, weights of over 800 MB in turn:
//                       [14336, 4096] x 8                     [4096, 1024] x 128
//   rows per expert     4    16    32    64   128  256  1024     5    32   128
//   stream             93   120   208   352   -    -    -       89    -     -
//   256 x 32           88    89   118   180  268  503  1873    105   174   443
//   128 x 32           90    94   132   202  260  472  1724     84   162   367
//   128 x 64           93    98   104   151  218  334  1236     98   149   298
//   256 x 64           92    95   101   138  217  334  1208    105   154   309
//   128 x 128         109   113   121   139  216  325  1086    134   203   342
//   256 x 128          95    99   106   126  181  305   964    110   164   279
//   256 x 256         106   111   118   138  178  309   920    129   181   336
// A tile's channels are halved while it leaves CUs idle; 128 x 32 where k is
// short (several workgroups per CU then overlap their starts: 84 against 105 us
// at k = 1024, 5 rows), 256 x 32 where it is long (89 against 94 at k = 4096, 16
// rows). 128 x 128 is ahead of 128 x 64 at k = 4096 and behind it at 1024.
// Layers too small for their tiles to fill the CUs: the stream kernel, whose
// waves split k ([256, 14080] x 5, five rows each: 17 us against 35).
// Rows that the ring cannot load, and k below 320 (its starts and ends are most
// of it then): the register-staged tiles, 128 x 32 up to 16 rows ([4096, 1023] x
// 128, four rows: 127 us; 128 x 64 169, the stream 171; but 23 rows, unevenly
// spread, [1030, 1001] x 60: 33 against 27), 128 x 64 up to 96 ([11904, 256] x 40,
// 83 rows: 110 us; 256 x 128 123), 256 x 128 above.
ExpertPlan experts_plan(int64_t m, int64_t e, int64_t n, int64_t k, int64_t xr, const void* x, const uint8_t* q)
{
    const int64_t active = m < e ? m : e, rows = (m + active - 1) / active;
    const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    const bool ring = aligned && k % 64 == 0 && k >= 320 && k <= (1 << 22) && xr <= ((int64_t)1 << 30) / k;
    const ExpertPlan st = stream_plan(active, n, k);
    const bool streams = st.fits(m, e, n);
    if (rows <= 2 && streams)
        return st;
    auto fills = [&](const ExpertPlan& p, int64_t least) {
        return (n + p.a - 1) / p.a * active * ((rows + p.b - 1) / p.b) >= least && p.fits(m, e, n);
    };
    if (ring) {
        const int bm = rows <= 16 ? 32 : (rows <= 48 ? 64 : (rows <= 192 ? 128 : 256));
        for (const ExpertPlan& p : kRings) {
            if (p.b > bm || (p.a == 256 && p.b == 32 && k < 2048))
                continue;
            if (fills(p, p.b == 256 ? 128 : 224))
                return p;
        }
    } else {
        const int bm = rows <= 16 ? 32 : (rows <= 96 ? 64 : 128);
        for (const ExpertPlan& p : kTiles)
            if (p.b <= bm && fills(p, 224))
                return p;
    }
    if (rows <= 64 && streams)
        return st;
    for (const ExpertPlan& p : kRings)
        if (ring && p.a == 64 && p.b == 64 && p.fits(m, e, n))
            return p;
    return {ExpertKind::TILE, 64, 64, 4};
}

// Whether some row starts below dword alignment.
bool shifted(const ExpertCall& c)
{
    return ((reinterpret_cast<uintptr_t>(c.x) | reinterpret_cast<uintptr_t>(c.q) | (uintptr_t)c.k) & 3) != 0;
}

template <typename A, int CT, int W>
hipError_t run_stream(const ExpertCall& c, hipStream_t stream)
{
    const int64_t TN = (c.n + 16 * CT - 1) / (16 * CT), groups = TN * max_row_tiles(c.m, c.e, 16);
    return launch(shifted(c) ? experts_stream_kernel<A, CT, W, true> : experts_stream_kernel<A, CT, W, false>,
                  dim3((unsigned)groups), dim3(W * kWave), stream, c, TN);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_tile(const ExpertCall& c, hipStream_t stream)
{
    const int64_t TN = (c.n + BN - 1) / BN, groups = TN * max_row_tiles(c.m, c.e, BM);
    return launch(shifted(c) ? experts_tile_kernel<A, BN, BM, WN, WM, true>
                             : experts_tile_kernel<A, BN, BM, WN, WM, false>,
                  dim3((unsigned)groups), dim3(WN * WM * kWave), stream, c, TN);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_ring(const ExpertCall& c, hipStream_t stream)
{
    const int64_t TN = (c.n + BN - 1) / BN, groups = TN * max_row_tiles(c.m, c.e, BM);
    return launch(experts_ring_kernel<A, BN, BM, WN, WM, ring_depth(BN, BM)>, dim3((unsigned)groups),
                  dim3(WN * WM * kWave), stream, c, TN);
}

template <typename A>
hipError_t launch_typed(const ExpertCall& c, hipStream_t stream)
{
    const ExpertPlan p = experts_plan(c.m, c.e, c.n, c.k, c.xr, c.x, c.q);
    if (p.kind == ExpertKind::STREAM) {
        if (p.w == 8)
            return p.a == 4   ? run_stream<A, 4, 8>(c, stream)
                   : p.a == 2 ? run_stream<A, 2, 8>(c, stream)
                              : run_stream<A, 1, 8>(c, stream);
        return p.a == 4   ? run_stream<A, 4, 4>(c, stream)
               : p.a == 2 ? run_stream<A, 2, 4>(c, stream)
                          : run_stream<A, 1, 4>(c, stream);
    }
    if (p.kind == ExpertKind::TILE)
        return p.a == 256   ? run_tile<A, 256, 128, 2, 4>(c, stream)
               : p.b == 32  ? run_tile<A, 128, 32, 4, 1>(c, stream)
               : p.a == 128 ? run_tile<A, 128, 64, 2, 2>(c, stream)
                            : run_tile<A, 64, 64, 2, 2>(c, stream);
    if (p.b == 256)
        return run_ring<A, 256, 256, 2, 4>(c, stream);
    if (p.b == 128)
        return p.a == 256 ? run_ring<A, 256, 128, 4, 2>(c, stream) : run_ring<A, 128, 128, 4, 2>(c, stream);
    if (p.b == 64)
        return p.a == 256   ? run_ring<A, 256, 64, 4, 2>(c, stream)
               : p.a == 128 ? run_ring<A, 128, 64, 2, 2>(c, stream)
                            : run_ring<A, 64, 64, 2, 2>(c, stream);
    return p.a == 256   ? run_ring<A, 256, 32, 4, 1>(c, stream)
           : p.a == 128 ? run_ring<A, 128, 32, 4, 1>(c, stream)
                        : run_ring<A, 64, 32, 2, 1>(c, stream);
}

}  // namespace

hipError_t launch_experts(const ExpertCall& c, Act act, hipStream_t stream)
{
    return act == Act::BF16 ? launch_typed<Bf16>(c, stream) : launch_typed<F16>(c, stream);
}

const char* experts_kernel_name(int64_t m, int64_t e, int64_t n, int64_t k, const void* x, const uint8_t* q)
{
    thread_local char name[96];
    const ExpertPlan p = experts_plan(m, e, n, k, m, x, q);
    if (p.kind == ExpertKind::STREAM)
        snprintf(name, sizeof name, "experts_stream_kernel<CT=%d,W=%d>", p.a, p.w);
    else
        snprintf(name, sizeof name, "experts_%s_kernel<BN=%d,BM=%d,W=%d>",
                 p.kind == ExpertKind::TILE ? "tile" : "ring", p.a, p.b, p.w);
    return name;
}

}  // namespace fp8w
