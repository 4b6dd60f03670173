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
#include "stream.hpp"
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
// operand registers (stream.hpp).
//
// A workgroup has up to 16 rows of one expert and every cols-th tile of 16 CT WC
// channels. Its waves are WC times WK: each owns 16 CT of a tile's channels and takes
// every WK-th step of k; the sums of WK waves meet in LDS and are added in wave order.
// A wave's loads run a step ahead, into the next tile's weights.
//
// One row, [14336, 4096] from memory: 10.7 us, 2.9 TB/s, on 224 workgroups with one of a wave's eight
// steps in flight (9.3 where the weights are in the memory-side cache); [28672, 8192]: 31 us, 4.0 TB/s.
// 512 rows over 128 experts [4096, 1024]: 62 us, 3.7 TB/s, the address unit busy 67 %.
template <typename A, int CT, int WK, int WC, Way WAY>
__global__ __launch_bounds__(WK* WC* kWave) void fp4_stream_kernel(Fp4Call c, int TN, int cols)
{
    using S = Stream<Fp4, A, CT, 1, 1, WAY, false>;
    constexpr int W = WK * WC;
    __shared__ __attribute__((aligned(16))) uint8_t ring[W][S::LDS];
    __shared__ __attribute__((aligned(16))) f32x4 part[WK > 1 ? W : 1][CT][kWave];
    const RowTile tile = row_tile<16>(c, blockIdx.x / cols);
    if (tile.expert < 0)
        return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int wk = wave % WK, wc = wave / WK, rows = uniform(tile.rows), expert = uniform(tile.expert);
    const bool on = expert < (int)c.e;
    // where this lane's row goes (-1: nowhere), and whether what it comes from exists
    const int at = r < rows ? tile.row + r : tile.row;
    int dst = c.y_rows ? c.y_rows[at] : at;
    if (r >= rows || dst >= (int)c.m)
        dst = -1;
    const int64_t from = c.x_rows && on ? c.x_rows[at] : 0;
    const bool ok = from >= 0 && (!c.x_rows || !on || from < c.xr);
    // without a row list the rows are the tile's, from its first on
    const int64_t first = c.x_rows ? 0 : uniform(tile.row);
    S st(c.k, static_cast<const uint16_t*>(c.x) + first * c.k, on ? 2 * (c.xr - first) * c.k : 0, ring[wave]);
    typename S::Source src;
    st.rows(src, rows, [&](int i) { return (source_row(c, tile, i) - first) * c.k; });
    auto enter = [&](int tn) {
        const int64_t n0 = ((int64_t)tn * WC + wc) * (16 * CT);
        st.weights(src, 0, c.q, c.block_scale, expert * c.n + n0, on ? c.e * c.n : 0);
    };
    const int NU = on ? (st.steps + WK - 1) / WK : 0;
    int tn = blockIdx.x % cols;
    enter(tn);
    st.load(src, wk, wk < st.steps);
#pragma unroll 1
    for (; tn < TN; tn += cols) {
        const int64_t n0 = ((int64_t)tn * WC + wc) * (16 * CT);
        uint16_t bias[CT][4];
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ch = n0 + 16 * t + 4 * g + i;
                bias[t][i] = bias_bits(static_cast<const uint16_t*>(c.bias), on && ch < c.n ? expert * c.n + ch : 0);
            }
        f32x4 acc[CT][1];
#pragma unroll
        for (int t = 0; t < CT; ++t)
            acc[t][0] = f32x4{0.0f};
#pragma unroll 1
        for (int v = 0; v < NU; ++v) {
            int ahead = v + 1;
            bool more = true;
            if (ahead == NU) {
                ahead = 0;
                more = tn + cols < TN;
                if (more)
                    enter(tn + cols);
            }
            ahead = wk + WK * ahead;
            st.consume(wk + WK * v, src, ahead, more && ahead < st.steps, acc);
        }
        // lane (r, g) holds channels 4 g .. 4 g + 3 of row r
        auto store = [&](int t, f32x4 sum) {
            const int64_t c0 = n0 + 16 * t + 4 * g;
            const float v[4] = {sum.x, sum.y, sum.z, sum.w};
            uint16_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = on ? rounded<A>((ok ? v[i] : __builtin_nanf("")) + A::to_f32(bias[t][i])) : (uint16_t)0;
            if (dst >= 0 && c0 < c.n)
                store4(static_cast<uint16_t*>(c.y) + (int64_t)dst * c.n + c0, o, c.n - c0);
        };
        if constexpr (WK == 1) {
#pragma unroll
            for (int t = 0; t < CT; ++t)
                store(t, acc[t][0]);
        } else {
#pragma unroll
            for (int t = 0; t < CT; ++t)
                part[wave][t][lane] = acc[t][0];
            lds_barrier();
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (t % WK == wk) {
                    f32x4 sum = part[wc * WK][t][lane];
#pragma unroll
                    for (int w = 1; w < WK; ++w)
                        sum += part[wc * WK + w][t][lane];
                    store(t, sum);
                }
            if (tn + cols < TN)
                lds_barrier();
        }
    }
}

// ------------------------------------------------------------------ tiles
// More rows: the tiles of experts.hip (BN channels x BM rows, WN x WM waves of
// 32 x 32 fragments, stages of 64 k), a weight row of 32 bytes in a stage. Its
// two 16-byte chunks change places every eight rows: a fragment's read of eight
// bytes per row then meets each bank twice, without it four times. Eight bytes are
// 16 codes, for two v_mfma_f32_32x32x16 of eight k each; both lie in one scale's
// block (a part of a stage is 32 k). Unaligned rows bind by latency, not by a unit: 333 tokens, 4 of
// 60 experts [1030, 1001], 24 us with the address unit busy 29 %, the matrix cores 17 %; stages of 128
// and 256 k, with fewer workgroups on a CU, took 25 to 38.
template <typename A, int BN, int BM, int WN, int WM, int Q = 1>
struct Fp4Tile {
    static constexpr int W = WN * WM, NT = W * kWave, FN = BN / WN / 32, FM = BM / WM / 32;
    static constexpr int ABYTES = BN * 32 * Q, XBYTES = BM * 128, STAGE = ABYTES + XBYTES * Q;
    static_assert(BN == FN * WN * 32 && BM == FM * WM * 32, "tile and wave layout");
    struct Frags {
        u32x2 a[FN];
        float s[FN];
        u32x4 x[FM][2];
    };
    int lane, wave, wn, wm;

    // where a row's 16-byte chunk of codes lies in its 2 Q: 256 bytes of chunks of one number hold 16 rows'
    __device__ __forceinline__ static int place(int r, int chunk) { return (chunk ^ (r / (8 / Q))) & (2 * Q - 1); }

    // everything but the scales, of 32 k: part j of the stage's 2 Q
    __device__ __forceinline__ void read_operands(const uint8_t* buf, int j, Frags& f) const
    {
        const int i = lane & 31, h = lane >> 5, t = 4 * (j & 1) + 2 * h + (i >> 1);
        const int oa = 32 * Q * (wn * (BN / WN) + i) + 16 * place(i, j) + 8 * h;
        const int ox = ABYTES + XBYTES * (j / 2) + 128 * (wm * (BM / WM) + i);
        const int o0 = ox + 16 * (t & 7), o1 = ox + 16 * ((t + 1) & 7);
#pragma unroll
        for (int q = 0; q < FN; ++q)
            f.a[q] = *reinterpret_cast<const u32x2*>(buf + (oa + 1024 * Q * q));
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
__device__ __forceinline__ bool find_fp4_tile(const Fp4Call& c, int TN, int block, int& tn, RowTile& tile)
{
    if (c.offsets)
        return find_tile<BM>(c, TN, tn, tile);
    int tm;
    const int TM = (int)((c.m + BM - 1) / BM);
    xcd_tile<4>(block, TN, TM, tn, tm);
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
    if (!find_fp4_tile<BM>(c, TN, blockIdx.x, tn, tile))
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

// Rows at 16-byte boundaries, k a multiple of 64 Q (and of 128), scales at dword
// boundaries, experts' x below 2 GiB: the same tiles fed by a ring of NS direct-to-LDS stages
// (tile.hpp) of 64 Q k. Scales come as dwords of 128 k: a stage of 64 k uses half of
// it, the lower pair in an even stage, the upper in an odd one.
template <int I>
struct RingSlot {
    static constexpr int index = I;
    uint8_t* p;
};

template <typename A, int BN, int BM, int WN, int WM, int NS, int Q>
struct Fp4Ring : Fp4Tile<A, BN, BM, WN, WM, Q> {
    using T = Fp4Tile<A, BN, BM, WN, WM, Q>;
    using Frags = typename T::Frags;
    static constexpr int SD = Q > 1 ? Q / 2 : 1;  // dwords of a channel's scales
    static constexpr int STAGE = T::STAGE + BN * 4 * SD;
    // 1 KB pieces of a stage's codes, 256-byte pieces of its scales; where there are fewer than waves, some load the same
    static constexpr int KW = BN * Q / 32, KS = BN * SD / 64;
    static constexpr int LW = KW > T::W ? KW / T::W : 1, LX = BM * Q / 8 / T::W, LS = KS > T::W ? KS / T::W : 1;
    static constexpr int LOADS = LW + LX + LS;
    static_assert(KW % T::W == 0 || T::W % KW == 0, "code pieces split evenly, or waves load the same");
    static_assert(KS % T::W == 0 || T::W % KS == 0, "scale pieces split evenly, or waves load the same");
    static_assert(BM * Q == LX * 8 * T::W && KS >= 1, "loads split evenly");
    Rows w, x, sc;
    int off[LOADS];  // this lane's part of each load at k = 0
    int S, rot, s0;  // stages, the one to begin with, the slice's first
    mutable int upper[NS];  // the bit in its dword where a stage's pair of scales starts

    template <int I>
    __device__ __forceinline__ void issue(int s, RingSlot<I> slot) const
    {
        const int st = s0 + (s + rot < S ? s + rot : s + rot - S), kb = 64 * Q * st;
        upper[I] = Q == 1 ? 16 * (st & 1) : 0;
#pragma unroll
        for (int u = 0; u < LW; ++u)
            w.load(off[u], kb / 2, slot.p + 1024 * ((u * T::W + this->wave) % KW));
#pragma unroll
        for (int u = 0; u < LX; ++u)
            x.load(off[LW + u], 2 * kb, slot.p + T::ABYTES + 1024 * (u * T::W + this->wave));
#pragma unroll
        for (int u = 0; u < LS; ++u)
            sc.load4(off[LW + LX + u], kb / 128 * 4, slot.p + T::STAGE + 256 * ((u * T::W + this->wave) % KS));
    }

    template <int I>
    __device__ __forceinline__ void read(RingSlot<I> slot, int j, Frags& f) const
    {
        this->read_operands(slot.p, j, f);
        const int os = T::STAGE + 4 * SD * (this->wn * (BN / WN) + (this->lane & 31));
#pragma unroll
        for (int q = 0; q < T::FN; ++q) {
            const uint8_t* at = slot.p + (os + 128 * SD * q);
            if constexpr (Q == 1)
                f.s[q] = fp4_scale((*reinterpret_cast<const uint32_t*>(at) >> (upper[I] + 8 * j)) & 255u);
            else
                f.s[q] = fp4_scale(at[j]);
        }
    }
};

// A wave whose rows all lie past the tile's: it loads its share and keeps the
// barriers, and leaves the matrix cores to the others.
template <typename A, int BN, int BM, int WN, int WM, int NS, int Q>
struct Fp4RingIdle : Fp4Ring<A, BN, BM, WN, WM, NS, Q> {
    struct Frags {};
    template <int I>
    __device__ __forceinline__ void read(RingSlot<I>, int, Frags&) const
    {
    }
    __device__ __forceinline__ void mma(const Frags&, f32x16*) const {}
};

// A k split's sums: parts[slice, row, channel], rows of whole fours.
constexpr int kJoinThreads = 256;
__host__ __device__ constexpr int64_t parts_row(int64_t n) { return (n + 3) / 4 * 4; }

template <int BN, int BM, int WN, int WM, typename P>
__device__ __forceinline__ void store_sums(const Fp4Call& c, const P& p, float* part, const RowTile& tile, int64_t n0,
                                           const f32x16* acc)
{
    const int i = p.lane & 31, h = p.lane >> 5;
#pragma unroll
    for (int fm = 0; fm < P::FM; ++fm) {
        const int row = p.wm * (BM / WM) + 32 * fm + i;
        if (row >= tile.rows)
            continue;
#pragma unroll
        for (int fn = 0; fn < P::FN; ++fn)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c0 = n0 + p.wn * (BN / WN) + 32 * fn + 8 * j + 4 * h;
                const f32x16& a = acc[fn * P::FM + fm];
                if (c0 < c.n)
                    *reinterpret_cast<f32x4*>(part + (tile.row + row) * parts_row(c.n) + c0) =
                        f32x4{a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]};
            }
    }
}

// Adds the slices of a k split in their order: four channels of a row a thread.
template <typename A>
__global__ __launch_bounds__(kJoinThreads) void fp4_join_kernel(Fp4Call c, int slices)
{
    const int64_t row4 = parts_row(c.n), item = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
    const int64_t row = 4 * item / row4, c0 = 4 * item - row * row4;
    if (row >= c.m)
        return;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int z = 0; z < slices; ++z)
        sum += *reinterpret_cast<const f32x4*>(c.parts + (z * c.m + row) * row4 + c0);
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = rounded<A>(sum[e] + A::to_f32(bias_bits(static_cast<const uint16_t*>(c.bias), c0 + e < c.n ? c0 + e : 0)));
    store4(static_cast<uint16_t*>(c.y) + row * c.n + c0, o, c.n - c0);
}

template <typename A, int BN, int BM, int WN, int WM, int NS, int Q>
__global__ __launch_bounds__(WN* WM* kWave) void fp4_ring_kernel(Fp4Call c, int TN, int tiles, int slices)
{
    using P = Fp4Ring<A, BN, BM, WN, WM, NS, Q>;
    using T = Fp4Tile<A, BN, BM, WN, WM, Q>;
    static_assert(NS >= 2 && NS <= 4, "stages");
    __shared__ __attribute__((aligned(1024))) uint8_t b0[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[NS > 2 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[NS > 3 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(16))) ExpertEpilogue<BN, BM> epi;
    auto buf = [&](auto ic) {
        constexpr int i = decltype(ic)::value;
        return RingSlot<i>{ring_buf<i>(b0, b1, b2, b3)};
    };
    int tn;
    RowTile tile;
    const int slice = slices > 1 ? (int)blockIdx.x / tiles : 0;
    if (!find_fp4_tile<BM>(c, TN, (int)blockIdx.x - slice * tiles, tn, tile))
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
        const int S = (int)(c.k / (64 * Q));
        p.s0 = slice * S / slices;
        p.S = (slice + 1) * S / slices - p.s0;
        p.rot = (int)(blockIdx.x % 8) * (p.S / 8);
        const int64_t first = (int64_t)tile.expert * c.n + n0;
        p.w = Rows(c.q + first * c.row_bytes);
        p.sc = Rows(c.block_scale + first * c.row_scales);
        // the linear layer's rows are offset from the tile's first, so that x may be of any size (past 2 GiB
        // only the stream was left: 74899 tokens [4096, 14336] 36.9 ms, 74898 and now both 7.8)
        const int64_t from = c.offsets ? 0 : tile.row * c.k;
        p.x = Rows(static_cast<const uint16_t*>(c.x) + from);
        auto row = [&](int r) { return (int)(n0 + r < c.n ? r : c.n - 1 - n0); };
#pragma unroll
        for (int u = 0; u < P::LW; ++u) {
            const int r = 32 / Q * ((u * T::W + p.wave) % P::KW) + p.lane / (2 * Q);
            p.off[u] = row(r) * (int)c.row_bytes + 16 * T::place(r, p.lane % (2 * Q));
        }
#pragma unroll
        for (int u = 0; u < P::LX; ++u) {
            const int piece = u * T::W + p.wave, r = 8 * (piece % (BM / 8)) + (p.lane >> 3);
            p.off[P::LW + u] = (int)(2 * (source_row(c, tile, r) * c.k - from)) + 128 * (piece / (BM / 8)) +
                               16 * (((p.lane & 7) - (r >> 1)) & 7);
        }
#pragma unroll
        for (int u = 0; u < P::LS; ++u) {
            const int at = 64 * ((u * T::W + p.wave) % P::KS) + p.lane;
            p.off[P::LW + P::LX + u] = row(at / P::SD) * (int)c.row_scales + 4 * (at % P::SD);
        }
        if (p.wm * (BM / WM) < tile.rows) {
            run_tile_ring<NS, P::LOADS, 2 * Q>(p, p.S, buf, acc);
        } else {
            Fp4RingIdle<A, BN, BM, WN, WM, NS, Q> idle;
            static_cast<P&>(idle) = p;
            run_tile_ring<NS, P::LOADS, 2 * Q>(idle, p.S, buf, acc);
        }
    }
    __syncthreads();
    if (slices > 1) {
        store_sums<BN, BM, WN, WM>(c, p, c.parts + slice * c.m * parts_row(c.n), tile, n0, acc);
        return;
    }
    store_tile<A, BN, BM, WN, WM>(c, p, n0, epi, acc);
}

// ------------------------------------------------------------------ quantizer
// Blocks of 32 weights, eight lanes a block, four weights a lane. The scale is
// the power of two with amax / scale in [4, 8): 2^(floor(log2 amax) - 2), codes the
// nearest e2m1 values, ties to the even code, beyond 6 the code of 6 (the OCP
// formats' own conversion). Build time, not tuned: [14336, 4096] of fp32 76 us, of bf16 91 (its bytes 52 and
// 29); a call takes 250 with the scales' copy to the host.
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

// Eight weights a thread; [14336, 4096] to fp32 139 us, its bytes 52: not tuned either.
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

// A kernel's tile, and what its calls take: start us, and for every 64 k of a
// workgroup's k, wait and for every workgroup on its CU each + rows_part (of 16 rows in use;
// less of fewer) us. Fitted to sweeps over layers of [1024, 1024] to [28672, 8192] with 1 to
// 4096 rows, weights from memory (a stream's own three: one row, [28672, 8192], {2, 1, 4} 30.2, {2, 2, 2}
// 30.5, {1, 4, 1} 37.0; [14336, 4096]: 15.0, 10.8, 13.4; [4096, 4096]: 13.9, 9.0, 5.9). The plan with the lowest
// modelled time was the fastest measured or within 5 % of it in 42 of 44 calls, 21 % off at worst.
struct Fp4Plan {
    Fp4Kind kind;
    int a, b, w;  // stream: CT, 16, WK; tile, ring: BN, BM, waves
    int c;        // stream: WC
    double start, wait, each, rows_part;
    int slices = 1;  // ring: parts of k
    int64_t channels() const { return kind == Fp4Kind::STREAM ? 16 * a * c : a; }
    int64_t groups(const Fp4Shape& s) const { return (s.n + channels() - 1) / channels() * s.row_tiles(b) * slices; }
    bool fits(const Fp4Shape& s) const { return grid_fits(groups(s), w * c * kWave); }
    // active experts of rows rows each
    double us(const Fp4Shape& s, int64_t active, int64_t rows) const
    {
        const int64_t tiles = (s.n + channels() - 1) / channels() * active * ((rows + b - 1) / b);
        const double share = (double)(rows < 16 ? rows : 16) / 16.0;
        double t = start + (double)s.k / (64.0 * slices) *
                               (wait + (double)((tiles * slices + 255) / 256) * (each + rows_part * share));
        if (slices > 1)  // the join's launch, the sums it reads
            t += 3.0 + 2.9e-6 * (double)slices * (double)s.m * (double)s.n;
        return t;
    }
};

constexpr Fp4Plan kStreams[] = {{Fp4Kind::STREAM, 1, 16, 4, 1, 3.0, 0.0, 0.035, 0.035},
                                {Fp4Kind::STREAM, 2, 16, 2, 2, 3.0, 0.0, 0.086, 0.058},
                                {Fp4Kind::STREAM, 2, 16, 1, 4, 3.0, 0.0, 0.17, 0.11}};
constexpr Fp4Plan kRings[] = {
    {Fp4Kind::RING, 64, 32, 2, 1, 3.8, 0.05, 0.099, 0.0},  {Fp4Kind::RING, 128, 32, 4, 1, 3.8, 0.0, 0.191, 0.0},
    {Fp4Kind::RING, 64, 64, 4, 1, 3.8, 0.0, 0.198, 0.0},   {Fp4Kind::RING, 128, 64, 4, 1, 3.8, 0.0, 0.36, 0.0},
    {Fp4Kind::RING, 128, 128, 8, 1, 3.8, 0.0, 0.70, 0.0},  {Fp4Kind::RING, 256, 128, 8, 1, 3.8, 0.0, 1.13, 0.0},
    {Fp4Kind::RING, 256, 256, 8, 1, 3.8, 0.0, 1.78, 0.0}};
constexpr Fp4Plan kTiles[] = {{Fp4Kind::TILE, 256, 128, 8, 1, 0.0, 0.0, 0.0, 0.0},
                              {Fp4Kind::TILE, 128, 64, 4, 1, 0.0, 0.0, 0.0, 0.0},
                              {Fp4Kind::TILE, 64, 64, 4, 1, 0.0, 0.0, 0.0, 0.0},
                              {Fp4Kind::TILE, 128, 32, 4, 1, 0.0, 0.0, 0.0, 0.0}};

// Where LDS has room, a stage is 256 k: whole 128-byte lines of codes. With stages of 64 k
// each line is fetched four times, and [4096, 14336] with 22 rows takes 20.0 us instead of 15.1,
// [14336, 4096] with 64 rows 24.4 instead of 17.8.
constexpr int ring_units(int bm)
{
    return bm <= 64 ? 4 : 1;
}

constexpr int ring_depth(int bn, int bm)
{
    return bm <= 64 || bn * bm == 65536 ? 3 : 4;
}

// Workgroups on a row tile's channels: all of the channel tiles while there are few, else
// each goes on to the next tile with loads in flight (512 rows above: 70 us a workgroup
// a tile, 65 with 1024 workgroups, 62 with 2048).
int64_t stream_columns(int64_t tiles, int64_t TN)
{
    const int64_t most = (2048 + tiles - 1) / tiles;
    return TN < most ? TN : most;
}

// Offsets of an int.
bool stream_fits(const Fp4Shape& s, const Fp4Plan& p)
{
    const int64_t rows = s.grouped ? s.xr : 16;
    return p.fits(s) && s.k <= (1 << 22) && rows * s.k < (1 << 29);
}

// Whether some row starts below dword alignment.
bool rows_shifted(const void* x, const uint8_t* q, int64_t k)
{
    return ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q) | (uintptr_t)(2 * k) |
             (uintptr_t)Fp4::row_bytes(k)) &
            3) != 0;
}

// aligned: rows and scales as the ring and the stream's LDS way take them.
Fp4Plan fp4_plan(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale)
{
    const int64_t most = s.m < s.e ? s.m : s.e, active = s.grouped && most > 0 ? most : 1, rows = (s.m + active - 1) / active;
    const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) & 15) == 0 &&
                         (reinterpret_cast<uintptr_t>(scale) & 3) == 0 && s.k % 128 == 0;
    Fp4Plan found{};
    double low = 0.0;
    bool any = false;
    auto offer = [&](const Fp4Plan& p) {
        const double us = p.us(s, active, rows);
        if (!any || us < low) {
            found = p;
            any = true;
            low = us;
        }
    };
    for (const Fp4Plan& p : kStreams)
        if ((rows <= 16 || aligned) && stream_fits(s, p))
            offer(p);
    // Few rows to an expert: rings of 32 rows load and multiply mostly nothing, and are modelled too fast (128
    // experts [4096, 1024], 4 and 16 rows each: 113 and 117 us, streams 75 and 104; 32 experts [1024, 2048], 4
    // rows: 12.8, 11.8). Only at 16 rows of few experts is a ring faster (8 experts [4096, 4096]: 20, 25).
    const bool few = s.grouped && rows <= 16 && any;
    if (aligned && !few && s.k > 0 && s.k <= (1 << 22) && (!s.grouped || s.xr <= ((int64_t)1 << 30) / s.k)) {
        for (const Fp4Plan& p : kRings)
            for (int z = 1; z <= (s.grouped ? 1 : 16); z *= 2) {
                Fp4Plan v = p;
                v.slices = z;
                const int64_t stage = 64 * ring_units(p.b);
                if (s.k % stage == 0 && s.k / stage / z >= ring_depth(p.a, p.b) && v.fits(s))
                    offer(v);
            }
    }
    if (any)
        return found;
    const int bm = rows <= 16 ? 32 : (rows <= 96 ? 64 : 128);
    for (const Fp4Plan& p : kTiles)
        if (p.b <= bm && (s.n + p.a - 1) / p.a * active * ((rows + p.b - 1) / p.b) >= 224 && p.fits(s))
            return p;
    // Few tiles, which walk a long k on a part of the CUs: a stream that is modelled a quarter faster (of rows at
    // any byte it takes up to 1.3 times its model) than the one round of 64 x 64 tiles takes. Measured, us:
    // [4096, 14330] with 17, 64, 128 tokens 33, 48, 88, tiles 110, 139, 131; [1024, 8128] with 17, 200 tokens
    // 11.8, 23, tiles 37, 37; two experts [4096, 14330], 20 rows each, 45, tiles 113; eight [512, 4090], 64 rows
    // each, 17, tiles 34. From 224 tiles on they are even or slower: [4096, 14330] with 200 tokens 158, tiles 108.
    const double tile_us = 3.0 + (double)s.k / 64.0 * (rows_shifted(x, q, s.k) ? 0.47 : 0.34);
    for (const Fp4Plan& p : kStreams)
        if (stream_fits(s, p))
            offer(p);
    return any && low < 0.75 * tile_us ? found : kTiles[2];
}

Fp4Shape shape_of(const Fp4Call& c)
{
    return {c.m, c.e, c.n, c.k, c.xr, c.offsets != nullptr};
}

bool shifted(const Fp4Call& c)
{
    return rows_shifted(c.x, c.q, c.k);
}

// LDS takes rows at 16-byte boundaries, and scales at dwords, in steps of four units: where
// those are fewer than the waves they are for, the shorter steps keep more of them busy
// (one row, [1024, 1024]: 3.6 us against 5.0; of [1024, 2048] it is 4.3 against 3.9).
Way stream_way(const Fp4Call& c, int wk)
{
    if (shifted(c))
        return Way::SHIFTED;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(c.x) | reinterpret_cast<uintptr_t>(c.q) | (uintptr_t)(2 * c.k) |
                           (uintptr_t)c.row_bytes;
    const uintptr_t scales = reinterpret_cast<uintptr_t>(c.block_scale) | (uintptr_t)c.row_scales;
    return (rows & 15) == 0 && (scales & 3) == 0 && c.k > 4 * Fp4::kUnit * (wk - 1) ? Way::LDS : Way::ROWS;
}

template <typename A, int CT, int WK, int WC>
hipError_t run_stream(const Fp4Call& c, hipStream_t stream)
{
    const int64_t TN = (c.n + 16 * CT * WC - 1) / (16 * CT * WC), tiles = shape_of(c).row_tiles(16);
    const int64_t cols = stream_columns(tiles, TN);
    const Way way = stream_way(c, WK);
    return launch(way == Way::LDS    ? fp4_stream_kernel<A, CT, WK, WC, Way::LDS>
                  : way == Way::ROWS ? fp4_stream_kernel<A, CT, WK, WC, Way::ROWS>
                                     : fp4_stream_kernel<A, CT, WK, WC, Way::SHIFTED>,
                  dim3((unsigned)(tiles * cols)), dim3(WK * WC * kWave), stream, c, TN, cols);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_tile(const Fp4Call& c, hipStream_t stream)
{
    const int64_t TN = (c.n + BN - 1) / BN, groups = TN * shape_of(c).row_tiles(BM);
    return launch(shifted(c) ? fp4_tile_kernel<A, BN, BM, WN, WM, true> : fp4_tile_kernel<A, BN, BM, WN, WM, false>,
                  dim3((unsigned)groups), dim3(WN * WM * kWave), stream, c, TN);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_ring(const Fp4Call& c, int slices, hipStream_t stream)
{
    const int64_t TN = (c.n + BN - 1) / BN, tiles = TN * shape_of(c).row_tiles(BM);
    const hipError_t status = launch(fp4_ring_kernel<A, BN, BM, WN, WM, ring_depth(BN, BM), ring_units(BM)>, dim3((unsigned)(tiles * slices)),
                                     dim3(WN * WM * kWave), stream, c, TN, tiles, slices);
    if (status != hipSuccess || slices == 1)
        return status;
    const int64_t items = c.m * (parts_row(c.n) / 4);
    return launch(fp4_join_kernel<A>, dim3((unsigned)((items + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), stream,
                  c, slices);
}

template <typename A>
hipError_t run_streams(const Fp4Call& c, const Fp4Plan& p, hipStream_t stream)
{
    return p.c == 4 ? run_stream<A, 2, 1, 4>(c, stream)
           : p.c == 2 ? run_stream<A, 2, 2, 2>(c, stream)
                      : run_stream<A, 1, 4, 1>(c, stream);
}

template <typename A>
hipError_t launch_typed(const Fp4Call& c, hipStream_t stream)
{
    const Fp4Plan p = fp4_plan(shape_of(c), c.x, c.q, c.block_scale);
    if (p.kind == Fp4Kind::STREAM)
        return run_streams<A>(c, p, stream);
    if (p.kind == Fp4Kind::TILE)
        return p.a == 256   ? run_tile<A, 256, 128, 2, 4>(c, stream)
               : p.b == 32  ? run_tile<A, 128, 32, 4, 1>(c, stream)
               : p.a == 128 ? run_tile<A, 128, 64, 2, 2>(c, stream)
                            : run_tile<A, 64, 64, 2, 2>(c, stream);
    if (p.b == 256)
        return run_ring<A, 256, 256, 4, 2>(c, p.slices, stream);
    if (p.b == 128)
        return p.a == 256 ? run_ring<A, 256, 128, 4, 2>(c, p.slices, stream)
                          : run_ring<A, 128, 128, 4, 2>(c, p.slices, stream);
    if (p.b == 64)
        return p.a == 128 ? run_ring<A, 128, 64, 2, 2>(c, p.slices, stream) : run_ring<A, 64, 64, 2, 2>(c, p.slices, stream);
    return p.a == 128 ? run_ring<A, 128, 32, 4, 1>(c, p.slices, stream) : run_ring<A, 64, 32, 2, 1>(c, p.slices, stream);
}

}  // namespace

hipError_t launch_fp4(const Fp4Call& c, Act act, hipStream_t stream)
{
    return act == Act::BF16 ? launch_typed<Bf16>(c, stream) : launch_typed<F16>(c, stream);
}

size_t linear_fp4_workspace_bytes(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale)
{
    const Fp4Plan p = fp4_plan(s, x, q, scale);
    return p.slices > 1 ? (size_t)(p.slices * s.m * parts_row(s.n)) * sizeof(float) : 0;
}

const char* fp4_kernel_name(const Fp4Shape& s, const void* x, const uint8_t* q, const uint8_t* scale)
{
    thread_local char name[96];
    const Fp4Plan p = fp4_plan(s, x, q, scale);
    char join[32] = "";
    if (p.slices > 1)
        snprintf(join, sizeof join, "*%d+fp4_join_kernel", p.slices);
    if (p.kind == Fp4Kind::STREAM)
        snprintf(name, sizeof name, "fp4_stream_kernel<CT=%d,WK=%d,WC=%d>", p.a, p.w, p.c);
    else
        snprintf(name, sizeof name, "fp4_%s_kernel<BN=%d,BM=%d,W=%d>%s", p.kind == Fp4Kind::TILE ? "tile" : "ring", p.a,
                 p.b, p.w, join);
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
