// The linear layer and the products grouped by expert on 4-bit weights (fp4.hpp):
//   y[dst(p), c] = sum_k x[src(p), k] * value(q[i, c, k]) 2^(s[i, c, k / 32] - 127) + bias[i, c]
// bf16 / fp16 activations, fp32 accumulation, one rounding. The linear layer is
// one expert that has every row (no offsets); else groups, row lists and rows that
// do not exist are those of experts.hip.
//
// The block scales enter when the codes are decoded, so the matrix cores see
// whole weights and nothing is rescaled between their sums.
#include <math.h>
#include <stdio.h>

#include "experts.hpp"
#include "fp4.hpp"
#include "tile.hpp"

namespace fp8w {
namespace {

// A workgroup's tile of one expert's rows, or of all rows without offsets.
template <int BM>
__device__ __forceinline__ RowTile row_tile(const Fp4Call& c, int want)
{
    RowTile tile;
    if (c.offsets) {
        TileFinder<BM> finder(c.offsets, (int)c.e, (int)c.m);
        tile = finder.find(want);
    } else {
        const int row = want * BM, left = (int)c.m - row;
        tile = RowTile{left > 0 ? 0 : -1, row, left < BM ? left : BM};
    }
    return tile;
}

// Few rows (decode): the weights stream once, straight into the matrix cores'
// operand registers.
//
// A workgroup owns 16 CT channels of up to 16 RT rows of one expert. Its W waves
// split k in blocks of 256: a lane holds 32 codes, one scale's block, of channel
// lane % 16 at k = 32 (lane / 16) of either half (one 16-byte load each), decodes
// them, and feeds eight to each of four v_mfma_f32_16x16x32, the row's values at
// the same k on the other side. A block's eight scales of a channel come in one
// load. The next block's loads are in flight during a block's products. The waves'
// sums meet in LDS and are added in wave order.
//
// Any k and any alignment: whole blocks take 16-byte loads from any dword (below
// that, Row), the last k % 256 a masked step.
template <typename A, int CT, int RT, int W, bool SHIFT>
__global__ __launch_bounds__(W* kWave) void fp4_stream_kernel(Fp4Call c, int TN)
{
    __shared__ __attribute__((aligned(16))) f32x4 part[W][CT * RT][kWave];
    const int tn = blockIdx.x % TN;
    const RowTile tile = row_tile<16 * RT>(c, blockIdx.x / TN);
    if (tile.expert < 0)
        return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)tn * (16 * CT);
    f32x4 acc[CT][RT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int u = 0; u < RT; ++u)
            acc[t][u] = f32x4{0.0f};
    if (tile.expert < (int)c.e && c.xr > 0) {
        Row<SHIFT> wp[CT], xp[RT];
        const uint8_t* sp[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int64_t ch = n0 + 16 * t + r < c.n ? n0 + 16 * t + r : c.n - 1, row = (int64_t)tile.expert * c.n + ch;
            wp[t] = Row<SHIFT>(c.q + row * c.row_bytes + 16 * g);
            sp[t] = c.block_scale + row * c.row_scales;
        }
#pragma unroll
        for (int u = 0; u < RT; ++u)
            xp[u] = Row<SHIFT>(static_cast<const uint8_t*>(c.x) + 2 * (source_row(c, tile, 16 * u + r) * c.k + 32 * g));
        struct Block {
            typename Row<SHIFT>::Raw w[CT][2], x[RT][2][4];
            u32x2 s[CT];
        };
        auto load = [&](Block& b, int64_t kb) {
#pragma unroll
            for (int t = 0; t < CT; ++t)
                b.s[t] = *reinterpret_cast<const u32x2_any*>(sp[t] + kb / 32);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    b.w[t][h] = wp[t].load(kb / 2 + 64 * h);
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        b.x[u][h][j] = xp[u].load(2 * kb + 256 * h + 16 * j);
            }
        };
        auto products = [&](const u32x4 (&w)[CT], const float (&s)[CT], const u32x4 (&x)[RT][4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const u32x4 v = w[t];
                    const u32x4 a = decode_fp4<A>(j == 0 ? v.x : (j == 1 ? v.y : (j == 2 ? v.z : v.w)), s[t]);
#pragma unroll
                    for (int u = 0; u < RT; ++u)
                        acc[t][u] = A::mfma(a, x[u][j], acc[t][u]);
                }
        };
        auto compute = [&](const Block& b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 w[CT], x[RT][4];
                float s[CT];
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    w[t] = wp[t].bytes(b.w[t][h]);
                    const u32x2 s8 = b.s[t];
                    s[t] = fp4_scale(((h ? s8.y : s8.x) >> (8 * g)) & 255u);
                }
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[u][j] = xp[u].bytes(b.x[u][h][j]);
                products(w, s, x);
            }
        };
        // this wave's blocks: wave, wave + W, .. below k / 256
        const int64_t whole = c.k / 256;
        int64_t b = wave;
        if (b < whole) {
            Block cur;
            load(cur, 256 * b);
            for (b += W; b < whole; b += W) {
                Block next;
                load(next, 256 * b);
                compute(cur);
                cur = next;
            }
            compute(cur);
        }
        const int64_t kb = 256 * whole;
        if (kb < c.k && wave == (int)(whole % W)) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int64_t left = c.k - kb - 128 * h - 32 * g;  // weights from this lane's first on
                u32x4 w[CT], x[RT][4];
                float s[CT];
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    w[t] = first_codes(wp[t].part(kb / 2 + 64 * h, (left + 1) / 2), left);
                    s[t] = fp4_scale(left > 0 ? sp[t][kb / 32 + 4 * h + g] : 127);
                }
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[u][j] = xp[u].part(2 * kb + 256 * h + 16 * j, 2 * left - 16 * j);
                products(w, s, x);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int u = 0; u < RT; ++u)
            part[wave][t * RT + u][lane] = acc[t][u];
    __syncthreads();
    // lane (r, g) holds channels 4 g .. 4 g + 3 of row r
    for (int t = wave; t < CT * RT; t += W) {
        f32x4 sum = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += part[w][t][lane];
        const int64_t c0 = n0 + 16 * (t / RT) + 4 * g, left = c.n - c0;
        const int row = 16 * (t % RT) + r;
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
        if (row < tile.rows && left > 0)
            store_tile_row<A, false>(c, tile.row + row, tile.expert, c0, left < 4 ? (int)left : 4, v);
    }
}

// ------------------------------------------------------------------ tiles
// More rows: the tiles of experts.hip (BN channels x BM rows, WN x WM waves of
// 32 x 32 fragments, stages of 64 k), a weight row of 32 bytes in a stage. Its
// two 16-byte chunks change places every eight rows: a fragment's read of eight
// bytes per row then meets each bank twice, without it four times. Eight bytes are
// 16 codes, for two v_mfma_f32_32x32x16 of eight k each; both lie in one scale's
// block (a half of a stage is 32 k).
template <typename A, int BN, int BM, int WN, int WM>
struct Fp4Tile {
    static constexpr int W = WN * WM, NT = W * kWave, FN = BN / WN / 32, FM = BM / WM / 32;
    static constexpr int ABYTES = BN * 32, STAGE = ABYTES + BM * 128;
    static_assert(BN == FN * WN * 32 && BM == FM * WM * 32, "tile and wave layout");
    struct Frags {
        u32x2 a[FN];
        float s[FN];
        u32x4 x[FM][2];
    };
    int lane, wave, wn, wm;

    // everything but the scales
    __device__ __forceinline__ void read_operands(const uint8_t* buf, int j, Frags& f) const
    {
        const int i = lane & 31, h = lane >> 5;
        const int oa = 32 * (wn * (BN / WN) + i) + 16 * ((j + (i >> 3)) & 1) + 8 * h;
        const int ox = ABYTES + 128 * (wm * (BM / WM) + i);
        const int o0 = ox + 16 * ((4 * j + 2 * h + (i >> 1)) & 7), o1 = ox + 16 * ((4 * j + 2 * h + 1 + (i >> 1)) & 7);
#pragma unroll
        for (int q = 0; q < FN; ++q)
            f.a[q] = *reinterpret_cast<const u32x2*>(buf + (oa + 1024 * q));
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
                const u32x2 v = f.a[q];
                a[q] = decode_fp4<A>(t ? v.y : v.x, f.s[q]);
            }
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int fm = 0; fm < FM; ++fm)
                    acc[fn * FM + fm] = mfma32<A>(a[fn], f.x[fm][t], acc[fn * FM + fm]);
        }
    }
};

// Which tile this workgroup is (false: none).
template <int BM>
__device__ __forceinline__ bool find_fp4_tile(const Fp4Call& c, int TN, int& tn, RowTile& tile)
{
    if (c.offsets)
        return find_tile<BM>(c, TN, tn, tile);
    int tm;
    const int TM = (int)((c.m + BM - 1) / BM);
    xcd_tile<4>(blockIdx.x, TN, TM, tn, tm);
    const int left = (int)c.m - tm * BM;
    tile = RowTile{0, tm * BM, left < BM ? left : BM};
    return true;
}

// Any k, any alignment, any number of rows in x: a stage passes through
// registers into LDS (run_tile_staged), a chunk's scale beside it.
template <typename A, int BN, int BM, int WN, int WM, bool SHIFT>
__global__ __launch_bounds__(WN* WM* kWave) void fp4_tile_kernel(Fp4Call c, int TN)
{
    using P = Fp4Tile<A, BN, BM, WN, WM>;
    constexpr int LW = BN * 2 > P::NT ? BN * 2 / P::NT : 1, LX = BM * 8 / P::NT;
    static_assert((BN * 2) % P::NT == 0 || P::NT % (BN * 2) == 0, "weight chunks split evenly, or threads share one");
    static_assert(BM * 8 == LX * P::NT, "activation chunks split evenly");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][P::STAGE];
    __shared__ uint8_t scales[2][BN * 2];
    __shared__ __attribute__((aligned(16))) ExpertEpilogue<BN, BM> epi;
    int tn;
    RowTile tile;
    if (!find_fp4_tile<BM>(c, TN, tn, tile))
        return;
    const int64_t n0 = (int64_t)tn * BN;
    const int tid = threadIdx.x;
    P p;
    p.lane = tid & 63;
    p.wave = uniform(tid >> 6);
    p.wn = p.wave % WN;
    p.wm = p.wave / WN;
    fill_epilogue<BN, BM, P::NT, false>(c, tile, n0, epi);
    f32x16 acc[P::FN * P::FM];
#pragma unroll
    for (int f = 0; f < P::FN * P::FM; ++f)
        acc[f] = f32x16{0.0f};
    const int64_t S = tile.expert < (int)c.e && c.xr > 0 ? (c.k + 63) / 64 : 0;
    if (S > 0) {
        Row<SHIFT> wp[LW], xp[LX];
        const uint8_t* sp[LW];
        int wo[LW], so[LW], xo[LX];
        const int wc = tid & 1, xc = tid & 7;
#pragma unroll
        for (int u = 0; u < LW; ++u) {
            const int r = ((tid >> 1) + P::NT / 2 * u) % BN;
            const int64_t row = (int64_t)tile.expert * c.n + (n0 + r < c.n ? n0 + r : c.n - 1);
            wp[u] = Row<SHIFT>(c.q + row * c.row_bytes + 16 * wc);
            sp[u] = c.block_scale + row * c.row_scales + wc;
            wo[u] = 32 * r + 16 * ((wc + (r >> 3)) & 1);
            so[u] = 2 * r + wc;
        }
#pragma unroll
        for (int u = 0; u < LX; ++u) {
            const int r = (tid >> 3) + P::NT / 8 * u;
            xp[u] = Row<SHIFT>(static_cast<const uint8_t*>(c.x) + 2 * (source_row(c, tile, r) * c.k + 8 * xc));
            xo[u] = P::ABYTES + 128 * r + 16 * ((xc + (r >> 1)) & 7);
        }
        struct Regs {
            typename Row<SHIFT>::Raw w[LW], x[LX];
            uint8_t s[LW];
        };
        auto load_whole = [&](Regs& g, int s) {
            const int64_t kb = 64 * (int64_t)s;
#pragma unroll
            for (int u = 0; u < LW; ++u) {
                g.w[u] = wp[u].load(kb / 2);
                g.s[u] = sp[u][2 * (int64_t)s];
            }
#pragma unroll
            for (int u = 0; u < LX; ++u)
                g.x[u] = xp[u].load(2 * kb);
        };
        auto load = [&](Regs& g, int s) {
            const int64_t kb = 64 * (int64_t)s;
            if (kb + 64 <= c.k) {
                load_whole(g, s);
            } else {
                const int64_t left = c.k - kb - 32 * wc;
#pragma unroll
                for (int u = 0; u < LW; ++u) {
                    g.w[u] = wp[u].raw(first_codes(wp[u].part(kb / 2, (left + 1) / 2), left));
                    g.s[u] = left > 0 ? sp[u][2 * (int64_t)s] : (uint8_t)127;
                }
#pragma unroll
                for (int u = 0; u < LX; ++u)
                    g.x[u] = xp[u].part_raw(2 * kb, 2 * (c.k - kb - 8 * xc));
            }
        };
        auto put = [&](const Regs& g, int b) {
#pragma unroll
            for (int u = 0; u < LW; ++u) {
                *reinterpret_cast<u32x4*>(&lds[b][wo[u]]) = wp[u].bytes(g.w[u]);
                scales[b][so[u]] = g.s[u];
            }
#pragma unroll
            for (int u = 0; u < LX; ++u)
                *reinterpret_cast<u32x4*>(&lds[b][xo[u]]) = xp[u].bytes(g.x[u]);
        };
        auto compute = [&](int b) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                typename P::Frags f;
                p.read_operands(lds[b], j, f);
#pragma unroll
                for (int q = 0; q < P::FN; ++q)
                    f.s[q] = fp4_scale(scales[b][2 * (p.wn * (BN / WN) + 32 * q + (p.lane & 31)) + j]);
                p.mma(f, acc);
            }
        };
        run_tile_staged<Regs>((int)S, (int)(c.k / 64), load, load_whole, put, compute);
    } else {
        __syncthreads();
    }
    store_tile<A, BN, BM, WN, WM>(c, p, n0, epi, acc);
}

// Rows at 16-byte boundaries, k a multiple of 128, scales at dword boundaries, x
// below 2 GiB: the same tiles fed by a ring of NS direct-to-LDS stages (tile.hpp).
// A stage brings each channel's four scales of 128 k, of which it uses two: the
// lower pair in an even stage, the upper in an odd one.
template <int I>
struct RingSlot {
    static constexpr int index = I;
    uint8_t* p;
};

template <typename A, int BN, int BM, int WN, int WM, int NS>
struct Fp4Ring : Fp4Tile<A, BN, BM, WN, WM> {
    using T = Fp4Tile<A, BN, BM, WN, WM>;
    using Frags = typename T::Frags;
    static constexpr int STAGE = T::STAGE + BN * 4;
    // 1 KB pieces of a stage's codes, 256-byte pieces of its scales; where there are fewer than waves, some load the same
    static constexpr int KW = BN / 32, KS = BN / 64;
    static constexpr int LW = KW > T::W ? KW / T::W : 1, LX = BM / 8 / T::W, LOADS = LW + LX + 1;
    static_assert(KW % T::W == 0 || T::W % KW == 0, "code pieces split evenly, or waves load the same");
    static_assert(BM == LX * 8 * T::W && KS >= 1 && KS <= T::W, "loads split evenly");
    Rows w, x, sc;
    int off[LOADS];  // this lane's part of each load at k = 0
    int S, rot;
    mutable int upper[NS];  // the bit in its dword where a stage's pair of scales starts

    template <int I>
    __device__ __forceinline__ void issue(int s, RingSlot<I> slot) const
    {
        const int st = s + rot < S ? s + rot : s + rot - S, kb = 64 * st;
        upper[I] = 16 * (st & 1);
#pragma unroll
        for (int u = 0; u < LW; ++u)
            w.load(off[u], kb / 2, slot.p + 1024 * ((u * T::W + this->wave) % KW));
#pragma unroll
        for (int u = 0; u < LX; ++u)
            x.load(off[LW + u], 2 * kb, slot.p + T::ABYTES + 1024 * (u * T::W + this->wave));
        sc.load4(off[LW + LX], 4 * (st / 2), slot.p + T::STAGE + 256 * (this->wave % KS));
    }

    template <int I>
    __device__ __forceinline__ void read(RingSlot<I> slot, int j, Frags& f) const
    {
        this->read_operands(slot.p, j, f);
        const int os = T::STAGE + 4 * (this->wn * (BN / WN) + (this->lane & 31));
#pragma unroll
        for (int q = 0; q < T::FN; ++q)
            f.s[q] = fp4_scale((*reinterpret_cast<const uint32_t*>(slot.p + (os + 128 * q)) >> (upper[I] + 8 * j)) & 255u);
    }
};

// A wave whose rows all lie past the tile's: it loads its share and keeps the
// barriers, and leaves the matrix cores to the others.
template <typename A, int BN, int BM, int WN, int WM, int NS>
struct Fp4RingIdle : Fp4Ring<A, BN, BM, WN, WM, NS> {
    struct Frags {};
    template <int I>
    __device__ __forceinline__ void read(RingSlot<I>, int, Frags&) const
    {
    }
    __device__ __forceinline__ void mma(const Frags&, f32x16*) const {}
};

template <typename A, int BN, int BM, int WN, int WM, int NS>
__global__ __launch_bounds__(WN* WM* kWave) void fp4_ring_kernel(Fp4Call c, int TN)
{
    using P = Fp4Ring<A, BN, BM, WN, WM, NS>;
    using T = Fp4Tile<A, BN, BM, WN, WM>;
    static_assert(NS >= 3 && NS <= 4, "stages");
    __shared__ __attribute__((aligned(1024))) uint8_t b0[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[NS > 3 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(16))) ExpertEpilogue<BN, BM> epi;
    auto buf = [&](auto ic) {
        constexpr int i = decltype(ic)::value;
        return RingSlot<i>{ring_buf<i>(b0, b1, b2, b3)};
    };
    int tn;
    RowTile tile;
    if (!find_fp4_tile<BM>(c, TN, tn, tile))
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
    fill_epilogue<BN, BM, T::NT, false>(c, tile, n0, epi);
    if (tile.expert < (int)c.e && c.xr > 0) {
        p.S = (int)(c.k / 64);
        p.rot = (int)(blockIdx.x % 8) * (p.S / 8);
        const int64_t first = (int64_t)tile.expert * c.n + n0;
        p.w = Rows(c.q + first * c.row_bytes);
        p.sc = Rows(c.block_scale + first * c.row_scales);
        p.x = Rows(c.x);
        auto row = [&](int r) { return (int)(n0 + r < c.n ? r : c.n - 1 - n0); };
#pragma unroll
        for (int u = 0; u < P::LW; ++u) {
            const int r = 32 * ((u * T::W + p.wave) % P::KW) + (p.lane >> 1);
            p.off[u] = row(r) * (int)c.row_bytes + 16 * (((p.lane & 1) - (r >> 3)) & 1);
        }
#pragma unroll
        for (int u = 0; u < P::LX; ++u) {
            const int r = 8 * (u * T::W + p.wave) + (p.lane >> 3);
            p.off[P::LW + u] = (int)(2 * source_row(c, tile, r) * c.k) + 16 * (((p.lane & 7) - (r >> 1)) & 7);
        }
        p.off[P::LW + P::LX] = row(64 * (p.wave % P::KS) + p.lane) * (int)c.row_scales;
        if (p.wm * (BM / WM) < tile.rows) {
            run_tile_ring<NS, P::LOADS>(p, p.S, buf, acc);
        } else {
            Fp4RingIdle<A, BN, BM, WN, WM, NS> idle;
            static_cast<P&>(idle) = p;
            run_tile_ring<NS, P::LOADS>(idle, p.S, buf, acc);
        }
    }
    __syncthreads();
    store_tile<A, BN, BM, WN, WM>(c, p, n0, epi, acc);
}

// ------------------------------------------------------------------ quantizer
// Blocks of 32 weights, eight lanes a block, four weights a lane. The scale is
// the power of two with amax / scale in [4, 8): 2^(floor(log2 amax) - 2), codes the
// nearest e2m1 values, ties to the even code, beyond 6 the code of 6 (the OCP
// formats' own conversion). Build time: not tuned.
constexpr int kQuantThreads = 256;

template <typename T>
__device__ __forceinline__ float weight_at(const T* p, int64_t i);
template <>
__device__ __forceinline__ float weight_at<float>(const float* p, int64_t i)
{
    return p[i];
}
template <>
__device__ __forceinline__ float weight_at<Bf16>(const Bf16* p, int64_t i)
{
    return Bf16::to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <>
__device__ __forceinline__ float weight_at<F16>(const F16* p, int64_t i)
{
    return F16::to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

// The nearest e2m1 code, ties to the even one.
__device__ __forceinline__ uint32_t e2m1_code(float v)
{
    const float m = fabsf(v);
    const uint32_t mag = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) + (m >= 3.5f) + (m > 5.0f);
    return mag | ((__builtin_bit_cast(uint32_t, v) >> 31) << 3);
}

template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_fp4_kernel(const T* __restrict__ w, int64_t n, int64_t k,
                                                                     uint8_t* __restrict__ q,
                                                                     uint8_t* __restrict__ scale)
{
    const int64_t scales = (k + 31) / 32, bytes = (k + 1) / 2, blocks = n * scales;
    const int in = threadIdx.x & 7;
    for (int64_t b = ((int64_t)blockIdx.x * kQuantThreads + threadIdx.x) >> 3; b < blocks;
         b += (int64_t)gridDim.x * (kQuantThreads / 8)) {
        const int64_t row = b / scales, k0 = 32 * (b - row * scales) + 4 * in;
        float v[4];
        uint32_t top = 0;  // the largest magnitude's bits: ordered as the values, NaN above infinity
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = k0 + j < k ? weight_at<T>(w, row * k + k0 + j) : 0.0f;
            const uint32_t mag = __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu;
            top = mag > top ? mag : top;
        }
#pragma unroll
        for (int off = 1; off < 8; off *= 2) {
            const uint32_t other = (uint32_t)__shfl_xor((int)top, off, kWave);
            top = other > top ? other : top;
        }
        // amax below 2^-125 (subnormals among them) has the smallest scale, 2^-127
        const int field = (int)(top >> 23);
        const bool finite = field < 255;
        const int s = finite ? (field > 2 ? field - 2 : 0) : 255;
        uint32_t code = 0;
        if (finite) {
            const float by = __builtin_bit_cast(float, (uint32_t)(254 - s) << 23);  // 1 / scale, s <= 252
#pragma unroll
            for (int j = 0; j < 4; ++j)
                code |= e2m1_code(v[j] * by) << (4 * j);
        }
        const int64_t at = row * bytes + k0 / 2;
        if (k0 < k)
            q[at] = (uint8_t)code;
        if (k0 + 2 < k)
            q[at + 1] = (uint8_t)(code >> 8);
        if (in == 0)
            scale[row * scales + k0 / 32] = (uint8_t)s;
    }
}

// Eight weights a thread.
__global__ __launch_bounds__(kQuantThreads) void dequantize_fp4_kernel(const uint8_t* __restrict__ q,
                                                                       const uint8_t* __restrict__ scale, int64_t n,
                                                                       int64_t k, void* __restrict__ out, Act type)
{
    const int64_t scales = (k + 31) / 32, bytes = (k + 1) / 2, per = (k + 7) / 8, all = n * per;
    for (int64_t b = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; b < all;
         b += (int64_t)gridDim.x * kQuantThreads) {
        const int64_t row = b / per, k0 = 8 * (b - row * per);
        const float s = fp4_scale(scale[row * scales + k0 / 32]);
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w |= k0 + 2 * j < k ? (uint32_t)q[row * bytes + k0 / 2 + j] << (8 * j) : 0;
        const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3)};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f32x2 two = p[j / 2];
            const float v = j % 2 ? two.y : two.x;
            const int64_t at = row * k + k0 + j;
            if (k0 + j >= k)
                continue;
            if (type == Act::FP32)
                static_cast<float*>(out)[at] = v;
            else
                static_cast<uint16_t*>(out)[at] = type == Act::BF16 ? Bf16::from_f32(v) : F16::from_f32(v);
        }
    }
}

unsigned capped_grid(int64_t threads)
{
    const int64_t groups = (threads + kQuantThreads - 1) / kQuantThreads;
    return (unsigned)(groups < 65536 ? groups : 65536);
}

// ------------------------------------------------------------------ plans
enum class Fp4Kind { STREAM, TILE, RING };

struct Fp4Plan {
    Fp4Kind kind;
    int a, b, w;  // stream: CT, RT, W; tile, ring: BN, BM, waves
    int64_t channels() const { return kind == Fp4Kind::STREAM ? 16 * a : a; }
    int64_t rows() const { return kind == Fp4Kind::STREAM ? 16 * b : b; }
    bool fits(const Fp4Shape& s) const { return grid_fits(groups(s), w * kWave); }
    int64_t groups(const Fp4Shape& s) const { return (s.n + channels() - 1) / channels() * s.row_tiles(rows()); }
};

constexpr Fp4Plan kRings[] = {{Fp4Kind::RING, 256, 256, 8}, {Fp4Kind::RING, 256, 128, 8}, {Fp4Kind::RING, 128, 128, 8},
                              {Fp4Kind::RING, 256, 64, 8},  {Fp4Kind::RING, 128, 64, 4},  {Fp4Kind::RING, 64, 64, 4},
                              {Fp4Kind::RING, 256, 32, 4},  {Fp4Kind::RING, 128, 32, 4},  {Fp4Kind::RING, 64, 32, 2}};
constexpr Fp4Plan kTiles[] = {{Fp4Kind::TILE, 256, 128, 8},
                              {Fp4Kind::TILE, 128, 64, 4},
                              {Fp4Kind::TILE, 64, 64, 4},
                              {Fp4Kind::TILE, 128, 32, 4}};

constexpr int ring_depth(int bn, int bm)
{
    return bn == 256 && bm == 256 ? 3 : 4;
}

Fp4Plan stream_plan(const Fp4Shape& s, int64_t active, int64_t rows)
{
    const int rt = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
    Fp4Plan p{Fp4Kind::STREAM, rt == 1 ? 4 : (rt == 2 ? 2 : 1), rt, s.k >= 2048 ? 8 : 4};
    while (p.a > 1 && (s.n + 16 * p.a - 1) / (16 * p.a) * active < 256)
        p.a /= 2;
    return p;
}

Fp4Plan fp4_plan(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale)
{
    const int64_t active = !s.grouped ? 1 : (s.m < s.e ? s.m : s.e), rows = (s.m + active - 1) / active;
    const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) & 15) == 0 &&
                         (reinterpret_cast<uintptr_t>(scale) & 3) == 0;
    const bool ring =
        aligned && s.k % 128 == 0 && s.k >= 320 && s.k <= (1 << 22) && s.xr <= ((int64_t)1 << 30) / s.k;
    const Fp4Plan st = stream_plan(s, active, rows);
    const bool streams = st.fits(s);
    if (rows <= 16 && streams)
        return st;
    auto fills = [&](const Fp4Plan& p, int64_t least) {
        return (s.n + p.a - 1) / p.a * active * ((rows + p.b - 1) / p.b) >= least && p.fits(s);
    };
    if (ring) {
        const int bm = rows <= 16 ? 32 : (rows <= 48 ? 64 : (rows <= 192 ? 128 : 256));
        for (const Fp4Plan& p : kRings) {
            if (p.b > bm || (p.a == 256 && p.b == 32 && s.k < 2048))
                continue;
            if (fills(p, p.b == 256 ? 128 : 224))
                return p;
        }
    } else {
        const int bm = rows <= 16 ? 32 : (rows <= 96 ? 64 : 128);
        for (const Fp4Plan& p : kTiles)
            if (p.b <= bm && fills(p, 224))
                return p;
    }
    if (rows <= 64 && streams)
        return st;
    for (const Fp4Plan& p : kRings)
        if (ring && p.a == 64 && p.b == 64 && p.fits(s))
            return p;
    return {Fp4Kind::TILE, 64, 64, 4};
}

Fp4Shape shape_of(const Fp4Call& c)
{
    return {c.m, c.e, c.n, c.k, c.xr, c.offsets != nullptr};
}

// Whether some row starts below dword alignment.
bool shifted(const Fp4Call& c)
{
    return ((reinterpret_cast<uintptr_t>(c.x) | reinterpret_cast<uintptr_t>(c.q) | (uintptr_t)(2 * c.k) |
             (uintptr_t)c.row_bytes) &
            3) != 0;
}

template <typename A, int CT, int RT, int W>
hipError_t run_stream(const Fp4Call& c, hipStream_t stream)
{
    const int64_t TN = (c.n + 16 * CT - 1) / (16 * CT), groups = TN * shape_of(c).row_tiles(16 * RT);
    return launch(shifted(c) ? fp4_stream_kernel<A, CT, RT, W, true> : fp4_stream_kernel<A, CT, RT, W, false>,
                  dim3((unsigned)groups), dim3(W * kWave), stream, c, TN);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_tile(const Fp4Call& c, hipStream_t stream)
{
    const int64_t TN = (c.n + BN - 1) / BN, groups = TN * shape_of(c).row_tiles(BM);
    return launch(shifted(c) ? fp4_tile_kernel<A, BN, BM, WN, WM, true> : fp4_tile_kernel<A, BN, BM, WN, WM, false>,
                  dim3((unsigned)groups), dim3(WN * WM * kWave), stream, c, TN);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_ring(const Fp4Call& c, hipStream_t stream)
{
    const int64_t TN = (c.n + BN - 1) / BN, groups = TN * shape_of(c).row_tiles(BM);
    return launch(fp4_ring_kernel<A, BN, BM, WN, WM, ring_depth(BN, BM)>, dim3((unsigned)groups),
                  dim3(WN * WM * kWave), stream, c, TN);
}

template <typename A, int W>
hipError_t run_streams(const Fp4Call& c, const Fp4Plan& p, hipStream_t stream)
{
    if (p.b == 1)
        return p.a == 4   ? run_stream<A, 4, 1, W>(c, stream)
               : p.a == 2 ? run_stream<A, 2, 1, W>(c, stream)
                          : run_stream<A, 1, 1, W>(c, stream);
    if (p.b == 2)
        return p.a == 2 ? run_stream<A, 2, 2, W>(c, stream) : run_stream<A, 1, 2, W>(c, stream);
    return run_stream<A, 1, 4, W>(c, stream);
}

template <typename A>
hipError_t launch_typed(const Fp4Call& c, hipStream_t stream)
{
    const Fp4Plan p = fp4_plan(shape_of(c), c.x, c.q, c.block_scale);
    if (p.kind == Fp4Kind::STREAM)
        return p.w == 8 ? run_streams<A, 8>(c, p, stream) : run_streams<A, 4>(c, p, stream);
    if (p.kind == Fp4Kind::TILE)
        return p.a == 256   ? run_tile<A, 256, 128, 2, 4>(c, stream)
               : p.b == 32  ? run_tile<A, 128, 32, 4, 1>(c, stream)
               : p.a == 128 ? run_tile<A, 128, 64, 2, 2>(c, stream)
                            : run_tile<A, 64, 64, 2, 2>(c, stream);
    if (p.b == 256)
        return run_ring<A, 256, 256, 4, 2>(c, stream);
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

hipError_t launch_fp4(const Fp4Call& c, Act act, hipStream_t stream)
{
    return act == Act::BF16 ? launch_typed<Bf16>(c, stream) : launch_typed<F16>(c, stream);
}

size_t linear_fp4_workspace_bytes(const Fp4Shape&, const void*, const uint8_t*, const uint8_t*)
{
    return 0;
}

const char* fp4_kernel_name(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale)
{
    thread_local char name[96];
    const Fp4Plan p = fp4_plan(s, x, q, scale);
    if (p.kind == Fp4Kind::STREAM)
        snprintf(name, sizeof name, "fp4_stream_kernel<CT=%d,RT=%d,W=%d>", p.a, p.b, p.w);
    else
        snprintf(name, sizeof name, "fp4_%s_kernel<BN=%d,BM=%d,W=%d>", p.kind == Fp4Kind::TILE ? "tile" : "ring", p.a,
                 p.b, p.w);
    return name;
}

hipError_t launch_quantize_fp4(const void* w, Act type, int64_t n, int64_t k, uint8_t* q, uint8_t* scale,
                               hipStream_t stream)
{
    const dim3 grid(capped_grid(8 * n * ((k + 31) / 32))), block(kQuantThreads);
    if (type == Act::FP32)
        return launch(quantize_fp4_kernel<float>, grid, block, stream, static_cast<const float*>(w), n, k, q, scale);
    if (type == Act::BF16)
        return launch(quantize_fp4_kernel<Bf16>, grid, block, stream, static_cast<const Bf16*>(w), n, k, q, scale);
    return launch(quantize_fp4_kernel<F16>, grid, block, stream, static_cast<const F16*>(w), n, k, q, scale);
}

hipError_t launch_dequantize_fp4(const uint8_t* q, const uint8_t* scale, int64_t n, int64_t k, void* out, Act type,
                                 hipStream_t stream)
{
    return launch(dequantize_fp4_kernel, dim3(capped_grid(n * ((k + 7) / 8))), dim3(kQuantThreads), stream, q, scale, n,
                  k, out, type);
}

}  // namespace fp8w
