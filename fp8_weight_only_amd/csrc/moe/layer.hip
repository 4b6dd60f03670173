// A whole mixture-of-experts layer for a few tokens (t <= 64), two launches:
//   h[s, i]  = silu(g) * u of slot s = token * top + j, g and u the gate and up
//              products of token s / top with its j-th expert's rows i and inner + i
//   out[t, c] = sum_j weights[t, j] * (sum_i h[s, i] * down[expert, c, i] + bias)
// The choice and the weights are the router's (choose.hpp). Weights are e4m3 codes
// with a scale per output channel, or 4-bit codes with block scales (fp4.hpp).
//
// First launch: every workgroup chooses for all tokens (a few microseconds at most,
// under the other workgroups' loads) rather than wait for a launch that does, and
// makes the lists of the active experts and their slots in LDS. Its items are
// 16 CT channels of one active expert, gate and up rows together, with all the
// expert's rows (up to 64), so every weight is read once. The first workgroup
// leaves choices and weights for the second launch.
//
// Second launch: a workgroup owns 16 CT output channels of every token. The active
// experts' blocks of k, in one line, are split evenly over its waves; a wave adds
// weights[t, j] times its part of an expert's sums to its own fp32 accumulators in
// LDS, and the waves' accumulators are added in wave order. No slot's result goes
// through memory, and no sum depends on the order of anything.
//
// Sums, scales, biases, the activation and the weighted sum are fp32; h is rounded
// once to the activation type, as the matrix cores take it (half a step of it per
// value), and out once.
#include <stdio.h>

#include "choose.hpp"
#include "fp4.hpp"
#include "groups.hpp"

namespace fp8w {
namespace {

constexpr int kMaxSlots = kMaxLayerTokens * kMaxTop;

struct E4m3 {
    static constexpr bool kBlockScales = false;
    static constexpr int kUnit = 64;   // k of a 16-byte load by the four lane groups
    static constexpr int kParts = 2;   // matrix instructions of a unit
    __device__ static int64_t row_bytes(int64_t k) { return k; }
    template <typename A>
    __device__ __forceinline__ static u32x4 values(u32x4 v, int part, float)
    {
        const u32x2 a = A::decode4(part ? v.z : v.x), b = A::decode4(part ? v.w : v.y);
        return u32x4{a.x, a.y, b.x, b.y};
    }
};

struct Fp4 {
    static constexpr bool kBlockScales = true;
    static constexpr int kUnit = 128;
    static constexpr int kParts = 4;
    __device__ static int64_t row_bytes(int64_t k) { return (k + 1) / 2; }
    template <typename A>
    __device__ __forceinline__ static u32x4 values(u32x4 v, int part, float scale)
    {
        return decode_fp4<A>(part == 0 ? v.x : (part == 1 ? v.y : (part == 2 ? v.z : v.w)), scale);
    }
};

typedef uint32_t u32_any __attribute__((aligned(1)));

// NT tiles of 16 weight rows times RC tiles of 16 activation rows, straight from
// memory into operand registers; the next block's loads run under a block's
// products. A block is two units of k (one where the rows' registers would not
// leave room for two).
template <typename F, typename A, int NT, int RC, bool SHIFT, bool XSHIFT>
struct Product {
    static constexpr int U = RC == 1 ? 2 : 1, BK = U * F::kUnit, LANE = F::kUnit / 4;
    Row<SHIFT> w[NT];
    Row<XSHIFT> x[RC];
    const uint8_t* s[NT];
    int64_t k;
    int g;
    struct Block {
        typename Row<SHIFT>::Raw w[NT][U];
        typename Row<XSHIFT>::Raw x[RC][U][F::kParts];
        uint32_t s[F::kBlockScales ? NT : 1][U];
    };

    __device__ __forceinline__ void weight_row(int t, const uint8_t* q, const void* scale, int64_t row)
    {
        w[t] = Row<SHIFT>(q + row * F::row_bytes(k) + 16 * g);
        if constexpr (F::kBlockScales)
            s[t] = static_cast<const uint8_t*>(scale) + row * ((k + 31) / 32);
    }
    __device__ __forceinline__ void x_row(int u, const void* p, int64_t first)
    {
        x[u] = Row<XSHIFT>(static_cast<const uint8_t*>(p) + 2 * (first + LANE * g));
    }
    __device__ __forceinline__ void load(Block& b, int64_t kb) const
    {
        if constexpr (F::kBlockScales)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < U; ++h)
                    b.s[t][h] = *reinterpret_cast<const u32_any*>(s[t] + kb / 32 + 4 * h);
#pragma unroll
        for (int h = 0; h < U; ++h) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                b.w[t][h] = w[t].load(F::row_bytes(kb) + 64 * h);
#pragma unroll
            for (int u = 0; u < RC; ++u)
#pragma unroll
                for (int p = 0; p < F::kParts; ++p)
                    b.x[u][h][p] = x[u].load(2 * (kb + F::kUnit * h) + 16 * p);
        }
    }
    __device__ __forceinline__ void products(const u32x4 (&v)[NT], const float (&scale)[NT],
                                             const u32x4 (&xs)[RC][F::kParts], f32x4 (&acc)[NT][RC]) const
    {
#pragma unroll
        for (int p = 0; p < F::kParts; ++p)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const u32x4 a = F::template values<A>(v[t], p, scale[t]);
#pragma unroll
                for (int u = 0; u < RC; ++u)
                    acc[t][u] = A::mfma(a, xs[u][p], acc[t][u]);
            }
    }
    __device__ __forceinline__ void compute(const Block& b, f32x4 (&acc)[NT][RC]) const
    {
#pragma unroll
        for (int h = 0; h < U; ++h) {
            u32x4 v[NT], xs[RC][F::kParts];
            float scale[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                v[t] = w[t].bytes(b.w[t][h]);
                scale[t] = F::kBlockScales ? fp4_scale((b.s[F::kBlockScales ? t : 0][h] >> (8 * g)) & 255u) : 1.0f;
            }
#pragma unroll
            for (int u = 0; u < RC; ++u)
#pragma unroll
                for (int p = 0; p < F::kParts; ++p)
                    xs[u][p] = x[u].bytes(b.x[u][h][p]);
            products(v, scale, xs, acc);
        }
    }
    // what is left of k behind the whole blocks
    __device__ __forceinline__ void tail(int64_t kb, f32x4 (&acc)[NT][RC]) const
    {
#pragma unroll 1
        for (int h = 0; h < U; ++h) {
            const int64_t left = k - kb - F::kUnit * h - LANE * g;
            u32x4 v[NT], xs[RC][F::kParts];
            float scale[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (F::kBlockScales) {
                    v[t] = first_codes(w[t].part(F::row_bytes(kb) + 64 * h, (left + 1) / 2), left);
                    scale[t] = fp4_scale(left > 0 ? s[t][kb / 32 + 4 * h + g] : 127);
                } else {
                    v[t] = w[t].part(kb + 64 * h, left);
                    scale[t] = 1.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < RC; ++u)
#pragma unroll
                for (int p = 0; p < F::kParts; ++p)
                    xs[u][p] = x[u].part(2 * (kb + F::kUnit * h) + 16 * p, 2 * left - 16 * p);
            products(v, scale, xs, acc);
        }
    }
    // blocks b, b + step, .. below end (all of them the same in every lane)
    __device__ __forceinline__ void run(int64_t b, int64_t end, int step, f32x4 (&acc)[NT][RC]) const
    {
        const int64_t whole = k / BK, last = end < whole ? end : whole;
        int64_t i = b;
        if (i < last) {
            Block cur;
            load(cur, BK * i);
            for (i += step; i < last; i += step) {
                Block next;
                load(next, BK * i);
                compute(cur, acc);
                cur = next;
            }
            compute(cur, acc);
        }
        if (i == whole && whole < end && BK * whole < k)
            tail(BK * whole, acc);
    }
};

// The active experts in order, each one's slots, in LDS.
struct Lists {
    int cursor[kMaxExperts];
    int16_t id[kMaxSlots];
    uint16_t row[kMaxSlots];
    uint16_t active[kMaxExperts], start[kMaxExperts + 1];
    int count;

    template <int NT>
    __device__ __forceinline__ void clear(int e)
    {
        for (int i = threadIdx.x; i < e; i += NT)
            cursor[i] = 0;
    }
    // From id[] and the experts' counts in cursor[], both written before a barrier. An
    // expert's slots stand in any order: a slot's sums do not depend on its place.
    template <int NT>
    __device__ __forceinline__ void build(int slots, int e)
    {
        if (threadIdx.x < kWave) {
            const int lane = threadIdx.x;
            int experts = 0, rows = 0;
            for (int i0 = 0; i0 < e; i0 += kWave) {
                const int i = i0 + lane, n = i < e ? cursor[i] : 0, incl = wave_prefix(n);
                const uint64_t on = __ballot(n > 0);
                if (n > 0) {
                    const int at = experts + __popcll(on & (((uint64_t)1 << lane) - 1));
                    active[at] = (uint16_t)i;
                    start[at] = (uint16_t)(rows + incl - n);
                    cursor[i] = rows + incl - n;
                }
                experts += __popcll(on);
                rows += __builtin_amdgcn_readlane(incl, 63);
            }
            if (lane == 0) {
                start[experts] = (uint16_t)rows;
                count = experts;
            }
        }
        __syncthreads();
        for (int s = threadIdx.x; s < slots; s += NT)
            if (id[s] >= 0)
                row[atomicAdd(&cursor[id[s]], 1)] = (uint16_t)s;
        __syncthreads();
    }
};

// f(integral_constant<int, RC>) for the row tiles that `rows` rows need.
template <int RCMAX, typename Fn>
__device__ __forceinline__ void with_row_tiles(int rows, Fn&& f)
{
    if constexpr (RCMAX > 1) {
        if (rows > 32)
            return f(std::integral_constant<int, 4>{});
        if (rows > 16)
            return f(std::integral_constant<int, 2>{});
    }
    f(std::integral_constant<int, 1>{});
}

__device__ __forceinline__ float channel_scale(const void* scale, int64_t at)
{
    return static_cast<const float*>(scale)[at];
}

template <int WAVES, typename Fn>
__device__ __forceinline__ void choose_all(const LayerCall& c, Fn&& done)
{
#define FP8W_CHOOSE(G, J) \
    return choose_chunk<G, J, WAVES>(c.logits, c.logits_type, 0, c.t, (int)c.e, c.top, c.renorm != 0, done)
    if (choice_lanes(c.e, c.top) == 16) {
        if (c.e <= 16)
            FP8W_CHOOSE(16, 1);
        FP8W_CHOOSE(16, 4);
    }
    if (c.e <= 64)
        FP8W_CHOOSE(64, 1);
    if (c.e <= 128)
        FP8W_CHOOSE(64, 2);
    if (c.e <= 256)
        FP8W_CHOOSE(64, 4);
    FP8W_CHOOSE(64, 16);
#undef FP8W_CHOOSE
}

template <typename F, typename A, int CT, int RCMAX, int W, bool SHIFT>
__global__ __launch_bounds__(W* kWave) void layer_up_kernel(LayerCall c, int TN)
{
    constexpr int NT = W * kWave;
    __shared__ Lists lists;
    __shared__ __attribute__((aligned(16))) f32x4 part[W][2 * CT][kWave];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int slots = (int)c.t * c.top;
    lists.clear<NT>((int)c.e);
    __syncthreads();
    choose_all<W>(c, [&](int64_t tok, int j, int id, float weight) {
        const int s = (int)tok * c.top + j;
        lists.id[s] = (int16_t)id;
        if (id >= 0)
            atomicAdd(&lists.cursor[id], 1);
        if (blockIdx.x == 0) {
            c.ids[s] = id;
            c.weights[s] = weight;
        }
    });
    __syncthreads();
    lists.build<NT>(slots, (int)c.e);
    const int items = TN * uniform(lists.count);
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int a = uniform(it / TN), expert = uniform(lists.active[a]), first = uniform(lists.start[a]);
        const int rows = uniform(lists.start[a + 1]) - first;
        const int64_t n0 = (int64_t)(it - a * TN) * (16 * CT), up = (int64_t)expert * 2 * c.inner;
        with_row_tiles<RCMAX>(rows, [&](auto rc) {
            constexpr int RC = decltype(rc)::value;
            Product<F, A, 2 * CT, RC, SHIFT, SHIFT> p;
            p.k = c.hidden;
            p.g = g;
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const int64_t ch = n0 + 16 * t + r < c.inner ? n0 + 16 * t + r : c.inner - 1;
                p.weight_row(t, c.up.q, c.up.scale, up + ch);
                p.weight_row(CT + t, c.up.q, c.up.scale, up + c.inner + ch);
            }
#pragma unroll
            for (int u = 0; u < RC; ++u) {
                const int i = 16 * u + r < rows ? 16 * u + r : 0;  // rows past the expert's: any row, not stored
                p.x_row(u, c.x, (int64_t)((uint32_t)lists.row[first + i] / (uint32_t)c.top) * c.hidden);
            }
            f32x4 acc[2 * CT][RC];
#pragma unroll
            for (int t = 0; t < 2 * CT; ++t)
#pragma unroll
                for (int u = 0; u < RC; ++u)
                    acc[t][u] = f32x4{0.0f};
            p.run(wave, (c.hidden + p.BK - 1) / p.BK, W, acc);
#pragma unroll
            for (int u = 0; u < RC; ++u) {
#pragma unroll
                for (int t = 0; t < 2 * CT; ++t)
                    part[wave][t][lane] = acc[t][u];
                __syncthreads();
                // lane (r, g): channels 4 g .. 4 g + 3 of row r
                for (int t = wave; t < CT; t += W) {
                    f32x4 gs = part[0][t][lane], us = part[0][CT + t][lane];
#pragma unroll
                    for (int v = 1; v < W; ++v) {
                        gs += part[v][t][lane];
                        us += part[v][CT + t][lane];
                    }
                    const int64_t c0 = n0 + 16 * t + 4 * g;
                    if (16 * u + r < rows && c0 < c.inner) {
                        const float gv[4] = {gs.x, gs.y, gs.z, gs.w}, uv[4] = {us.x, us.y, us.z, us.w};
                        const uint16_t* bias = static_cast<const uint16_t*>(c.up.bias);
                        uint16_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int64_t gc = up + (c0 + i < c.inner ? c0 + i : c.inner - 1), uc = gc + c.inner;
                            const float sg = F::kBlockScales ? 1.0f : channel_scale(c.up.scale, gc);
                            const float su = F::kBlockScales ? 1.0f : channel_scale(c.up.scale, uc);
                            const float gate = __builtin_fmaf(sg, gv[i], A::to_f32(bias_bits(bias, gc)));
                            const float lift = __builtin_fmaf(su, uv[i], A::to_f32(bias_bits(bias, uc)));
                            o[i] = rounded<A>(gate / (1.0f + expf(-gate)) * lift);
                        }
                        const u32x2 pk{(uint32_t)o[0] | ((uint32_t)o[1] << 16), (uint32_t)o[2] | ((uint32_t)o[3] << 16)};
                        *reinterpret_cast<u32x2*>(c.h + lists.row[first + 16 * u + r] * c.pitch + c0) = pk;
                    }
                }
                __syncthreads();
            }
        });
    }
}

template <typename F, typename A, int CT, int RCMAX, int W, bool SHIFT>
__global__ __launch_bounds__(W* kWave) void layer_down_kernel(LayerCall c)
{
    constexpr int NT = W * kWave, TOKENS = 16 * RCMAX;
    __shared__ Lists lists;
    __shared__ float weight[RCMAX == 1 ? 16 * kMaxTop : kMaxSlots];
    __shared__ __attribute__((aligned(16))) f32x4 sum[W][TOKENS][4 * CT];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int slots = (int)c.t * c.top;
    lists.clear<NT>((int)c.e);
    for (int i = threadIdx.x; i < W * TOKENS * 4 * CT; i += NT)
        (&sum[0][0][0])[i] = f32x4{0.0f};
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += NT) {
        const int id = c.ids[s];
        lists.id[s] = (int16_t)id;
        weight[s] = c.weights[s];
        if (id >= 0)
            atomicAdd(&lists.cursor[id], 1);
    }
    __syncthreads();
    lists.build<NT>(slots, (int)c.e);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * CT);
    // this wave's blocks of two units among all experts'
    const int per = (int)((c.inner + 2 * F::kUnit - 1) / (2 * F::kUnit)), all = per * uniform(lists.count);
    const int hi = uniform(all * (wave + 1) / W);
    for (int at = uniform(all * wave / W); at < hi;) {
        const int a = uniform(at / per), b0 = at - a * per, b1 = b0 + hi - at < per ? b0 + hi - at : per;
        at += b1 - b0;
        const int expert = uniform(lists.active[a]), first = uniform(lists.start[a]);
        const int rows = uniform(lists.start[a + 1]) - first;
        with_row_tiles<RCMAX>(rows, [&](auto rc) {
            constexpr int RC = decltype(rc)::value;
            Product<F, A, CT, RC, SHIFT, false> p;
            p.k = c.inner;
            p.g = g;
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const int64_t ch = n0 + 16 * t + r < c.hidden ? n0 + 16 * t + r : c.hidden - 1;
                p.weight_row(t, c.down.q, c.down.scale, (int64_t)expert * c.hidden + ch);
            }
#pragma unroll
            for (int u = 0; u < RC; ++u) {
                const int i = 16 * u + r < rows ? 16 * u + r : 0;
                p.x_row(u, c.h, lists.row[first + i] * c.pitch);
            }
            f32x4 acc[CT][RC];
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int u = 0; u < RC; ++u)
                    acc[t][u] = f32x4{0.0f};
            p.run(b0 * (2 / p.U), b1 * (2 / p.U), 1, acc);
            // lane (r, g): channels 4 g .. 4 g + 3 of row r; an expert has a token once
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const int64_t c0 = n0 + 16 * t + 4 * g;
                float scale[4], bias[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t ch = (int64_t)expert * c.hidden + (c0 + i < c.hidden ? c0 + i : c.hidden - 1);
                    scale[i] = F::kBlockScales ? 1.0f : channel_scale(c.down.scale, ch);
                    bias[i] = b0 == 0 ? A::to_f32(bias_bits(static_cast<const uint16_t*>(c.down.bias), ch)) : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < RC; ++u) {
                    if (16 * u + r < rows) {
                        const int s = lists.row[first + 16 * u + r];
                        const float wt = weight[s];
                        f32x4& to = sum[wave][(uint32_t)s / (uint32_t)c.top][4 * t + g];
                        const f32x4 v = acc[t][u];
                        f32x4 z = to;
                        z.x = __builtin_fmaf(wt, __builtin_fmaf(scale[0], v.x, bias[0]), z.x);
                        z.y = __builtin_fmaf(wt, __builtin_fmaf(scale[1], v.y, bias[1]), z.y);
                        z.z = __builtin_fmaf(wt, __builtin_fmaf(scale[2], v.z, bias[2]), z.z);
                        z.w = __builtin_fmaf(wt, __builtin_fmaf(scale[3], v.w, bias[3]), z.w);
                        to = z;
                    }
                }
            }
            wave_sync();
        });
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (int)c.t * 4 * CT; i += NT) {
        const int tok = i / (4 * CT), q = i % (4 * CT);
        f32x4 z = sum[0][tok][q];
#pragma unroll
        for (int v = 1; v < W; ++v)
            z += sum[v][tok][q];
        const int64_t c0 = n0 + 4 * q;
        const uint16_t o[4] = {rounded<A>(z.x), rounded<A>(z.y), rounded<A>(z.z), rounded<A>(z.w)};
        if (c0 < c.hidden)
            store4(static_cast<uint16_t*>(c.out) + tok * c.hidden + c0, o, c.hidden - c0);
    }
}

// ------------------------------------------------------------------ plans
constexpr int kUpGroups = 1024;

bool rows_shifted(const void* a, const void* b, int64_t bytes)
{
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | (uintptr_t)bytes) & 3) != 0;
}

template <typename F, typename A, int CT, int RCMAX, bool SHIFT>
hipError_t run_up(const LayerCall& c, hipStream_t stream)
{
    const int64_t TN = (c.inner + 16 * CT - 1) / (16 * CT), most = c.t * c.top < c.e ? c.t * c.top : c.e;
    const int64_t items = TN * most;
    return launch(layer_up_kernel<F, A, CT, RCMAX, 8, SHIFT>, dim3((unsigned)(items < kUpGroups ? items : kUpGroups)),
                  dim3(8 * kWave), stream, c, TN);
}

template <typename F, typename A, int CT, int RCMAX, bool SHIFT>
hipError_t run_down(const LayerCall& c, hipStream_t stream)
{
    return launch(layer_down_kernel<F, A, CT, RCMAX, 8, SHIFT>, dim3((unsigned)((c.hidden + 16 * CT - 1) / (16 * CT))),
                  dim3(8 * kWave), stream, c);
}

template <typename F, typename A>
hipError_t launch_typed(const LayerCall& c, int64_t up_bytes, int64_t down_bytes, hipStream_t stream)
{
    const bool us = rows_shifted(c.up.q, c.x, up_bytes | (2 * c.hidden)), ds = rows_shifted(c.down.q, nullptr, down_bytes);
    hipError_t st;
    if (c.t <= 16)
        st = us ? run_up<F, A, 2, 1, true>(c, stream) : run_up<F, A, 2, 1, false>(c, stream);
    else
        st = us ? run_up<F, A, 1, 4, true>(c, stream) : run_up<F, A, 1, 4, false>(c, stream);
    if (st != hipSuccess)
        return st;
    if (c.t <= 16)
        return ds ? run_down<F, A, 1, 1, true>(c, stream) : run_down<F, A, 1, 1, false>(c, stream);
    return ds ? run_down<F, A, 1, 4, true>(c, stream) : run_down<F, A, 1, 4, false>(c, stream);
}

int64_t h_pitch(int64_t inner)
{
    return (inner + 63) / 64 * 64;
}

}  // namespace

size_t layer_workspace_bytes(int64_t t, int64_t top, int64_t inner)
{
    const size_t slots = (size_t)t * (size_t)top;
    return (slots * 8 + 15) / 16 * 16 + slots * (size_t)h_pitch(inner) * 2;
}

hipError_t launch_layer(LayerCall c, bool fp4, Act act, void* ws, hipStream_t stream)
{
    const size_t slots = (size_t)c.t * (size_t)c.top;
    c.ids = static_cast<int32_t*>(ws);
    c.weights = reinterpret_cast<float*>(c.ids + slots);
    c.h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + (slots * 8 + 15) / 16 * 16);
    c.pitch = h_pitch(c.inner);
    if (fp4)
        return act == Act::BF16 ? launch_typed<Fp4, Bf16>(c, (c.hidden + 1) / 2, (c.inner + 1) / 2, stream)
                                : launch_typed<Fp4, F16>(c, (c.hidden + 1) / 2, (c.inner + 1) / 2, stream);
    return act == Act::BF16 ? launch_typed<E4m3, Bf16>(c, c.hidden, c.inner, stream)
                            : launch_typed<E4m3, F16>(c, c.hidden, c.inner, stream);
}

}  // namespace fp8w
