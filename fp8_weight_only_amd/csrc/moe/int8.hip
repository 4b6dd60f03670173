// The linear layer on 8-bit integers, a scale for each token and each output
// channel:
//   sx[t] = max_k |x[t, k]| / 127,  qx[t, k] = round(127 x[t, k] / max_k |x[t, k]|)
//   y[t, c] = (sum_k qx[t, k] * q[c, k]) * sx[t] * sw[c] + bias[c]
// The sum is exact in 32-bit integers (k <= 131072), in whatever order (its one
// value of 2^31: see sum_f32); the scales and the bias are applied in fp32 and
// the result is rounded once.
//
// Codes of 16-bit activations are the exact quotient's nearest integers, ties to
// even. 127 x has at most 18 significant bits, so it is exact in fp32, and x and
// the maximum a have at most 11 significant bits, so a quotient that is no half
// lies at least 1 / (254 * 2^11), above 2^-19, of its value away from one. The
// rounded quotient (fp32 weights: an IEEE division) is off by 2^-24. For 16-bit
// rows the division is a product with the row's fl(1 / a), off by 2^-23, and one
// correction q + (127 x - q a) fl(1 / a): a tie h is then hit exactly, since the
// residual (h - q) a is exact and what the correction rounds away is far below
// half a step of h.
#include <math.h>
#include <stdio.h>

#include "device.hpp"
#include "moe.hpp"
#include "tile.hpp"

namespace fp8w {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float value_at(const void* p, Act type, int64_t i)
{
    if (type == Act::FP32)
        return static_cast<const float*>(p)[i];
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return type == Act::BF16 ? Bf16::to_f32(b) : F16::to_f32(b);
}

// ------------------------------------------------------------------ quantizers
// Any type and length, one workgroup per row: the maximum, then the codes from
// a second read. Rows with very large values are divided by 2^64 first (exactly;
// what that rounds away is far below half a code), so that 127 x stays finite.
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
    const float pre = amax > 0x1p100f ? 0x1p-64f : 1.0f;
    for (int64_t j = threadIdx.x; j < kx; j += 256)
        q[row * kx + j] = j < k && amax > 0.0f && !nf
                              ? (int8_t)(int)rintf(__fdiv_rn(127.0f * (value_at(x, type, base + j) * pre), amax * pre))
                              : (int8_t)0;
}

// The quantization of one 16-bit row, from its largest magnitude's bits.
template <typename A>
struct RowCodes {
    float a, inv, pre, scale;
    bool zero;  // codes are all zero: a zero row, or one with a NaN or an infinity

    __device__ __forceinline__ explicit RowCodes(uint32_t bits)
    {
        constexpr uint32_t kInf = is_bf16<A>::value ? 0x7f80 : 0x7c00;
        const float amax = A::to_f32((uint16_t)bits);
        scale = bits >= kInf ? __builtin_nanf("") : amax / 127.0f;
        zero = bits >= kInf || bits == 0;
        // very large and very small rows are moved by 2^64 (exactly, but for what is far
        // below half a code), so that 127 x and 1 / a stay finite and residuals normal
        pre = amax > 0x1p100f ? 0x1p-64f : (amax < 0x1p-60f ? 0x1p64f : 1.0f);
        a = zero ? 1.0f : amax * pre;
        inv = 1.0f / a;
    }

    __device__ __forceinline__ uint32_t code(float x) const
    {
        const float n = 127.0f * (x * pre);
        const float q = n * inv;
        const float r = __builtin_fmaf(__builtin_fmaf(-q, a, n), inv, q);
        return (uint32_t)(int)rintf(r) & 255u;
    }

    // codes of eight values
    __device__ __forceinline__ u32x2 code8(u32x4 v) const
    {
        if (zero)
            return u32x2{0, 0};
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            o[i] = code(A::lo_f32(d[2 * i])) | (code(A::hi_f32(d[2 * i])) << 8) |
                   (code(A::lo_f32(d[2 * i + 1])) << 16) | (code(A::hi_f32(d[2 * i + 1])) << 24);
        return u32x2{o[0], o[1]};
    }
};

// Largest magnitude's bits in v, as two 16-bit halves.
__device__ __forceinline__ uint32_t max_bits(u32x4 v, uint32_t so_far)
{
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = d[i] & 0x7fff7fffu;
        so_far = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, w),
                                                                        __builtin_bit_cast(u16x2, so_far)));
    }
    return so_far;
}

// Eight codes at q + off of a row of kx.
__device__ __forceinline__ void put_codes(int8_t* q, int64_t off, int64_t kx, u32x2 c)
{
    if (off + 8 <= kx) {
        *reinterpret_cast<u32x2_any*>(q + off) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (off + i < kx)
                q[off + i] = (int8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

// 16-bit rows of up to 8 NT CH values, one workgroup of NT threads per row, read
// once: each thread keeps CH runs of eight values.
template <typename A, int NT, int CH, bool SHIFT>
__global__ __launch_bounds__(NT) void quantize_row_kernel(const uint16_t* __restrict__ x, int64_t k,
                                                          int8_t* __restrict__ q, int64_t kx,
                                                          float* __restrict__ scale)
{
    __shared__ uint32_t part[NT / kWave];
    const int64_t row = blockIdx.x;
    const Row<SHIFT> src(x + row * k);
    typename Row<SHIFT>::Raw raw[CH];
    u32x4 v[CH];
    uint32_t big = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int64_t off = 8 * ((int64_t)threadIdx.x + NT * c);
        raw[c] = off + 8 <= k ? src.load(2 * off) : src.part_raw(2 * off, 2 * (k - off));
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        v[c] = src.bytes(raw[c]);
        big = max_bits(v[c], big);
    }
    big = (big >> 16) > (big & 0xffffu) ? big >> 16 : big & 0xffffu;
    big = wave_max_u32(big);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w)
        big = big > part[w] ? big : part[w];
    const RowCodes<A> codes(big);
    if (threadIdx.x == 0)
        scale[row] = codes.scale;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int64_t off = 8 * ((int64_t)threadIdx.x + NT * c);
        if (off < kx)
            put_codes(q + row * kx, off, kx, codes.code8(v[c]));
    }
}

// ------------------------------------------------------------------ products
// A sum in fp32. -128 * -128 taken 131072 times is 2^31, which wraps to -2^31;
// no other sum is there, the lowest being -128 * 127 * 131072.
__device__ __forceinline__ float sum_f32(int acc)
{
    return acc == INT32_MIN ? 0x1p31f : (float)acc;
}

template <typename A>
__device__ __forceinline__ uint16_t finish(int acc, float sx, float sw, float bias)
{
    return rounded<A>(__builtin_fmaf(sum_f32(acc) * sx, sw, bias));
}

struct Int8Call {
    const uint16_t* x;  // the layer's 16-bit activations (one token: quantized in the product's kernel)
    const int8_t* qx;
    int64_t kx;
    const float* sx;
    const int8_t* qw;
    const float* sw;
    const uint16_t* bias;
    uint16_t* y;
    int64_t m, n, k;
};

constexpr int kFusedK = 16384;

// Few tokens (decode): the weights stream once, straight into the matrix cores'
// operand registers.
//
// A workgroup owns 16 CT channels of up to 16 RT tokens. Its W waves split k in
// blocks of 128: a lane holds 16 codes of channel lane % 16 at k = 16 (lane / 16)
// of either half of a block (16 rows of 64 consecutive bytes per load), and the
// tokens' codes at the same k on the other side of v_mfma_i32_16x16x64. U blocks
// per wave are in flight. The waves' sums meet in LDS; integers, so in any order.
//
// FUSED (one token): the row is quantized by every workgroup for itself, into
// LDS, behind the first weight loads: 14.0 us (then) against 14.4 and a launch of
// 2.3 for the quantizer on [14336, 4096].
//
// Any k and any alignment: whole blocks take 16-byte loads from any dword (below
// that, Row), the last k % 128 a masked step.
//
// Bound by the weight stream: one token on [14336, 4096] (59 MB) takes 13.5 us, 4.4
// TB/s, when 600 MB of weights are taken in turn, 12.0 when the memory-side cache
// holds them. Before the first loads lost the branches between them it took 14.0
// there; against that, two column tiles per workgroup 14.8, four waves 15.3, two
// blocks in flight 14.9. From five tokens on the ring below is faster where it can run: every wave here loads the tokens' codes
// for itself (16 tokens, [14336, 4096]: 16.6 us against 13.7).
template <typename A, int RT, int CT, int W, int U, bool FUSED, bool SHIFT>
__global__ __launch_bounds__(W* kWave) void int8_stream_kernel(Int8Call c, int TN, int TM)
{
    static_assert(!FUSED || RT == 1, "one token");
    __shared__ __attribute__((aligned(16))) i32x4 part[W][RT * CT][kWave];
    __shared__ __attribute__((aligned(16))) int8_t row[FUSED ? kFusedK : 16];
    __shared__ uint32_t row_max[W];
    int tn, tm;
    xcd_tile<8>(blockIdx.x, TN, TM, tn, tm);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)tn * (16 * CT), m0 = (int64_t)tm * (16 * RT);
    Row<SHIFT> wp[CT], xp[RT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const int64_t ch = n0 + 16 * t + r < c.n ? n0 + 16 * t + r : c.n - 1;
        wp[t] = Row<SHIFT>(c.qw + ch * c.k + 16 * g);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int64_t tok = m0 + 16 * t + r < c.m ? m0 + 16 * t + r : c.m - 1;
        if constexpr (!FUSED)
            xp[t] = Row<SHIFT>(c.qx + tok * c.kx + 16 * g);
    }
    struct Block {
        typename Row<SHIFT>::Raw w[CT][2], x[FUSED ? 1 : RT][2];
    };
    auto load = [&](Block& b, int64_t i) {
        const int64_t kb = 128 * i;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int t = 0; t < CT; ++t)
                b.w[t][h] = wp[t].load(kb + 64 * h);
            if constexpr (!FUSED) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    b.x[t][h] = xp[t].load(kb + 64 * h);
            }
        }
    };
    i32x4 acc[RT * CT];
#pragma unroll
    for (int t = 0; t < RT * CT; ++t)
        acc[t] = i32x4{0};
    auto compute = [&](const Block& b, int64_t i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 w[CT];
#pragma unroll
            for (int u = 0; u < CT; ++u)
                w[u] = wp[u].bytes(b.w[u][h]);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                u32x4 xv;
                if constexpr (FUSED)
                    xv = *reinterpret_cast<const u32x4*>(row + 16 * g + 128 * i + 64 * h);
                else
                    xv = xp[t].bytes(b.x[t][h]);
#pragma unroll
                for (int u = 0; u < CT; ++u)
                    acc[t * CT + u] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[u]),
                                                              __builtin_bit_cast(i32x4, xv), acc[t * CT + u], 0, 0, 0);
            }
        }
    };
    // this wave's blocks: wave, wave + W, .. below k / 128
    const int whole = (int)(c.k / 128), mine = whole > wave ? (whole - wave + W - 1) / W : 0;
    Block buf[U];
    if (mine >= U) {  // no branch between the first loads
#pragma unroll
        for (int u = 0; u < U; ++u)
            load(buf[u], wave + u * W);
    } else {
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (u < mine)
                load(buf[u], wave + u * W);
    }
    float token_scale = 0.0f;
    if constexpr (FUSED) {
        constexpr int NT = W * kWave, CH = kFusedK / 8 / NT;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(c.x);
        u32x4 v[CH];
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int64_t off = 8 * ((int64_t)threadIdx.x + NT * j);
            if (off < c.k) {
                v[j] = load16_part(src + 2 * off, 2 * (c.k - off));
                big = max_bits(v[j], big);
            }
        }
        big = (big >> 16) > (big & 0xffffu) ? big >> 16 : big & 0xffffu;
        big = wave_max_u32(big);
        if (lane == 0)
            row_max[wave] = big;
        __syncthreads();
        for (int w = 0; w < W; ++w)
            big = big > row_max[w] ? big : row_max[w];
        const RowCodes<A> codes(big);
        token_scale = codes.scale;
        const int64_t kp = (c.k + 127) / 128 * 128;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int64_t off = 8 * ((int64_t)threadIdx.x + NT * j);
            if (off < kp)
                *reinterpret_cast<u32x2*>(row + off) = off < c.k ? codes.code8(v[j]) : u32x2{0, 0};
        }
        __syncthreads();
    }
    if (mine >= U) {
        int done = 0;
        for (; done + 2 * U <= mine; done += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                compute(buf[u], wave + (done + u) * W);
                load(buf[u], wave + (done + u + U) * W);
            }
        }
        const int rest = mine - done - U;  // fewer than U
#pragma unroll
        for (int u = 0; u < U; ++u) {
            compute(buf[u], wave + (done + u) * W);
            if (u < rest)
                load(buf[u], wave + (done + u + U) * W);
        }
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (u < rest)
                compute(buf[u], wave + (done + u + U) * W);
    } else {
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (u < mine)
                compute(buf[u], wave + u * W);
    }
    const int64_t kb = 128 * (int64_t)whole;
    if (kb < c.k && wave == whole % W) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const int64_t left = c.k - kb - 64 * h - 16 * g;
            u32x4 w[CT];
#pragma unroll
            for (int u = 0; u < CT; ++u)
                w[u] = wp[u].part(kb + 64 * h, left);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                u32x4 xv;
                if constexpr (FUSED)
                    xv = *reinterpret_cast<const u32x4*>(row + 16 * g + kb + 64 * h);  // zeros from k on
                else
                    xv = xp[t].part(kb + 64 * h, left);
#pragma unroll
                for (int u = 0; u < CT; ++u)
                    acc[t * CT + u] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[u]),
                                                              __builtin_bit_cast(i32x4, xv), acc[t * CT + u], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT * CT; ++t)
        part[wave][t][lane] = acc[t];
    __syncthreads();
    // lane (r, g) holds channels 4 g .. 4 g + 3 of token r
    for (int t = wave; t < RT * CT; t += W) {
        u32x4 sum = __builtin_bit_cast(u32x4, part[0][t][lane]);  // unsigned: 2^31 may wrap
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += __builtin_bit_cast(u32x4, part[w][t][lane]);
        const int64_t tok = m0 + 16 * (t / CT) + r, c0 = n0 + 16 * (t % CT) + 4 * g;
        if (tok < c.m && c0 < c.n) {
            const float st = FUSED ? token_scale : c.sx[tok];
            const int v[4] = {(int)sum.x, (int)sum.y, (int)sum.z, (int)sum.w};
            uint16_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t cc = c0 + e < c.n ? c0 + e : c.n - 1;
                o[e] = finish<A>(v[e], st, c.sw[cc], A::to_f32(bias_bits(c.bias, cc)));
            }
            store4(c.y + tok * c.n + c0, o, c.n - c0);
        }
    }
}

// The tiles' epilogue: lane (i, h) holds channels 8 j + 4 h + e of token i in
// accumulators 4 j + e of each 32 x 32 fragment.
template <typename A, int BN, int BM, int WN, int WM>
__device__ __forceinline__ void store_tile(const Int8Call& c, int64_t n0, int64_t m0, int wn, int wm, int lane,
                                           const float* e_sw, const uint16_t* e_bias, const float* e_sx,
                                           const i32x16* acc)
{
    constexpr int FN = BN / WN / 32, FM = BM / WM / 32;
    const int i = lane & 31, h = lane >> 5;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int tl = wm * (BM / WM) + 32 * fm + i;
        const int64_t t = m0 + tl;
        if (t >= c.m)
            continue;
        const float st = e_sx[tl];
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int cl = wn * (BN / WN) + 32 * fn + 8 * j + 4 * h;
                const int64_t c0 = n0 + cl;
                const f32x4 s4 = *reinterpret_cast<const f32x4*>(&e_sw[cl]);
                const u32x2 b4 = *reinterpret_cast<const u32x2*>(&e_bias[cl]);
                const float bf[4] = {A::lo_f32(b4.x), A::hi_f32(b4.x), A::lo_f32(b4.y), A::hi_f32(b4.y)};
                uint16_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = finish<A>(acc[fn * FM + fm][4 * j + e], st, s4[e], bf[e]);
                if (c0 < c.n)
                    store4(c.y + t * c.n + c0, o, c.n - c0);
            }
    }
}

// A k slice's sums.
template <int BN, int BM, int WN, int WM>
__device__ __forceinline__ void store_sums(const Int8Call& c, int* part, int64_t n0, int64_t m0, int wn, int wm,
                                           int lane, const i32x16* acc)
{
    constexpr int FN = BN / WN / 32, FM = BM / WM / 32;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int64_t t = m0 + wm * (BM / WM) + 32 * fm + (lane & 31);
        if (t >= c.m)
            continue;
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c0 = n0 + wn * (BN / WN) + 32 * fn + 8 * j + 4 * (lane >> 5);
                int* dst = part + t * c.n + c0;
                if (c0 + 4 <= c.n) {
                    *reinterpret_cast<u32x4_any*>(dst) =
                        u32x4{(uint32_t)acc[fn * FM + fm][4 * j], (uint32_t)acc[fn * FM + fm][4 * j + 1],
                              (uint32_t)acc[fn * FM + fm][4 * j + 2], (uint32_t)acc[fn * FM + fm][4 * j + 3]};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c0 + e < c.n)
                            dst[e] = acc[fn * FM + fm][4 * j + e];
                }
            }
    }
}

// Adds the slices' sums and applies the epilogue, four channels per thread.
template <typename A>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Call c, const int* __restrict__ part, int slices)
{
    const int64_t quads = (c.n + 3) / 4, item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = item / quads, c0 = (item - t * quads) * 4;
    if (t >= c.m)
        return;
    int v[4] = {0, 0, 0, 0};
    const int* src = part + t * c.n + c0;
    if (c0 + 4 <= c.n) {
#pragma unroll 4
        for (int s = 0; s < slices; ++s) {
            const u32x4 d = *reinterpret_cast<const u32x4_any*>(src + (int64_t)s * c.m * c.n);
            v[0] += (int)d.x;
            v[1] += (int)d.y;
            v[2] += (int)d.z;
            v[3] += (int)d.w;
        }
    } else {
        for (int s = 0; s < slices; ++s)
            for (int e = 0; e < 4; ++e)
                v[e] += c0 + e < c.n ? src[(int64_t)s * c.m * c.n + e] : 0;
    }
    const float st = c.sx[t];
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t cc = c0 + e < c.n ? c0 + e : c.n - 1;
        o[e] = finish<A>(v[e], st, c.sw[cc], A::to_f32(bias_bits(c.bias, cc)));
    }
    store4(c.y + t * c.n + c0, o, c.n - c0);
}

// Many tokens (prefill): BN channels x BM tokens, WN x WM waves of 32 x 32
// fragments, stages of 64 k. A stage passes through registers into LDS, so any
// k and any alignment take the same code (run_tile_staged). In LDS every 64-byte
// row keeps its four 16-byte chunks rotated by row / 4, so the 16 lanes of a
// read's phase (16 rows, same chunk) hit distinct banks. part: k is split into
// slices of `stages` stages, as for the ring below.
template <typename A, int BN, int BM, int WN, int WM, bool SHIFT>
__global__ __launch_bounds__(WN* WM* kWave) void int8_tile_kernel(Int8Call c, int TN, int TM, int stages, int* part)
{
    constexpr int NT = WN * WM * kWave, FN = BN / WN / 32, FM = BM / WM / 32;
    constexpr int LW = BN * 4 / NT, LX = BM * 4 / NT;  // 16-byte chunks per thread and stage
    static_assert(LW >= 1 && LX >= 1 && BN * 4 == LW * NT && BM * 4 == LX * NT, "chunks split evenly");
    static_assert(BN <= NT && BM <= NT, "one epilogue operand per thread");
    __shared__ __attribute__((aligned(16))) uint8_t lw[2][BN * 64];
    __shared__ __attribute__((aligned(16))) uint8_t lx[2][BM * 64];
    __shared__ __attribute__((aligned(16))) float e_sw[BN];
    __shared__ __attribute__((aligned(16))) uint16_t e_bias[BN];
    __shared__ __attribute__((aligned(16))) float e_sx[BM];
    int tn, tm;
    const int slice = blockIdx.x / (TN * TM);
    xcd_tile<4>(blockIdx.x - slice * (TN * TM), TN, TM, tn, tm);
    // this workgroup's part of k
    const int64_t k0 = (int64_t)slice * stages * 64, kl = c.k - k0 < (int64_t)stages * 64 ? c.k - k0 : (int64_t)stages * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int i = lane & 31, h = lane >> 5, wn = wave % WN, wm = wave / WN;
    const int64_t n0 = (int64_t)tn * BN, m0 = (int64_t)tm * BM;
    if (tid < BN) {
        const int64_t ch = n0 + tid < c.n ? n0 + tid : c.n - 1;
        e_sw[tid] = c.sw[ch];
        e_bias[tid] = bias_bits(c.bias, ch);
    }
    if (tid < BM)
        e_sx[tid] = c.sx[m0 + tid < c.m ? m0 + tid : c.m - 1];
    Row<SHIFT> wp[LW], xp[LX];
    int wo[LW], xo[LX];
    const int ch = tid & 3;
#pragma unroll
    for (int u = 0; u < LW; ++u) {
        const int r = (tid >> 2) + NT / 4 * u;
        wp[u] = Row<SHIFT>(c.qw + (n0 + r < c.n ? n0 + r : c.n - 1) * c.k + k0 + 16 * ch);
        wo[u] = 64 * r + 16 * ((ch + (r >> 2)) & 3);
    }
#pragma unroll
    for (int u = 0; u < LX; ++u) {
        const int r = (tid >> 2) + NT / 4 * u;
        xp[u] = Row<SHIFT>(c.qx + (m0 + r < c.m ? m0 + r : c.m - 1) * c.kx + k0 + 16 * ch);
        xo[u] = 64 * r + 16 * ((ch + (r >> 2)) & 3);
    }
    const int S = (int)((kl + 63) / 64);
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
            g.x[u] = xp[u].load(kb);
    };
    auto load = [&](Regs& g, int s) {
        const int64_t kb = 64 * (int64_t)s, left = kl - kb - 16 * ch;
        if (kb + 64 <= kl) {
            load_whole(g, s);
        } else {
#pragma unroll
            for (int u = 0; u < LW; ++u)
                g.w[u] = wp[u].part_raw(kb, left);
#pragma unroll
            for (int u = 0; u < LX; ++u)
                g.x[u] = xp[u].part_raw(kb, left);
        }
    };
    auto put = [&](const Regs& g, int b) {
#pragma unroll
        for (int u = 0; u < LW; ++u)
            *reinterpret_cast<u32x4*>(&lw[b][wo[u]]) = wp[u].bytes(g.w[u]);
#pragma unroll
        for (int u = 0; u < LX; ++u)
            *reinterpret_cast<u32x4*>(&lx[b][xo[u]]) = xp[u].bytes(g.x[u]);
    };
    i32x16 acc[FN * FM];
#pragma unroll
    for (int f = 0; f < FN * FM; ++f)
        acc[f] = i32x16{0};
    auto compute = [&](int b) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            i32x4 a[FN], x[FM];
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const int r = wn * (BN / WN) + 32 * f + i;
                a[f] = *reinterpret_cast<const i32x4*>(&lw[b][64 * r + 16 * ((2 * j + h + (r >> 2)) & 3)]);
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const int r = wm * (BM / WM) + 32 * f + i;
                x[f] = *reinterpret_cast<const i32x4*>(&lx[b][64 * r + 16 * ((2 * j + h + (r >> 2)) & 3)]);
            }
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int fm = 0; fm < FM; ++fm)
                    acc[fn * FM + fm] =
                        __builtin_amdgcn_mfma_i32_32x32x32_i8(a[fn], x[fm], acc[fn * FM + fm], 0, 0, 0);
        }
    };
    if (S > 0) {
        run_tile_staged<Regs>(S, (int)(kl / 64), load, load_whole, put, compute);
    } else {
        __syncthreads();
    }
    if (part)
        store_sums<BN, BM, WN, WM>(c, part + (int64_t)slice * c.m * c.n, n0, m0, wn, wm, lane, acc);
    else
        store_tile<A, BN, BM, WN, WM>(c, n0, m0, wn, wm, lane, e_sw, e_bias, e_sx, acc);
}

// More tokens, weight rows at 16-byte boundaries, k a multiple of 64: the same
// tiles fed by a ring of NS direct-to-LDS stages (tile.hpp).
//
// 4096 tokens on [14336, 4096]: 246 us, 2.0 POP/s (256 x 256 tiles, two waves per
// SIMD; matrix cores busy 59 % of the time at 1.9 GHz, no bank conflicts), where
// the register-staged tiles take 301 and the vendor's library 234. 22 tokens on
// [4096, 14336]: 128 x 64 tiles are 32 workgroups; k in eight slices takes 12 us
// and the join 4, where the call without a split (fp8w_gemm_int8) takes 32.5.
template <int BN, int BM, int WN, int WM>
struct Int8Ring {
    static constexpr int W = WN * WM, FN = BN / WN / 32, FM = BM / WM / 32;
    static constexpr int LOADS = (BN + BM) / 16 / W;  // 1 KB load instructions per wave and stage
    static constexpr int STAGE = (BN + BM) * 64;
    static_assert(BN % (16 * W) == 0 && BM % (16 * W) == 0, "loads split evenly");
    struct Frags {
        i32x4 a[FN], x[FM];
    };
    Rows w, x;       // the tile's rows of weight and activation codes
    int off[LOADS];  // this lane's 16 bytes of each load at k = 0
    int S, rot;
    int lane, wave, wn, wm;

    __device__ __forceinline__ void issue(int s, uint8_t* buf) const
    {
        const int kb = 64 * (s + rot < S ? s + rot : s + rot - S);
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
            (u < BN / 16 / W ? w : x).load(off[u], kb, buf + 1024 * (u * W + wave));
    }
    __device__ __forceinline__ void read(const uint8_t* buf, int j, Frags& f) const
    {
        // fragment q's row is 32 q further: the same rotation. One addition to the buffer's
        // address per read: through longer chains the compiler loses which buffer is read,
        // and waits for every load in flight
        const int i = lane & 31, c = 16 * ((2 * j + (lane >> 5) + (i >> 2)) & 3);
        const int oa = 64 * (wn * (BN / WN) + i) + c, ox = 64 * (BN + wm * (BM / WM) + i) + c;
#pragma unroll
        for (int q = 0; q < FN; ++q)
            f.a[q] = *reinterpret_cast<const i32x4*>(buf + (oa + 2048 * q));
#pragma unroll
        for (int q = 0; q < FM; ++q)
            f.x[q] = *reinterpret_cast<const i32x4*>(buf + (ox + 2048 * q));
    }
    __device__ __forceinline__ void mma(const Frags& f, i32x16* acc) const
    {
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
                acc[fn * FM + fm] =
                    __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[fn], f.x[fm], acc[fn * FM + fm], 0, 0, 0);
    }
};

// part: k is split over gridDim.x / (TN TM) slices of whole stages, whose sums
// go to part[slice, token, channel] for int8_join_kernel.
template <typename A, int BN, int BM, int WN, int WM, int NS>
__global__ __launch_bounds__(WN* WM* kWave) void int8_ring_kernel(Int8Call c, int TN, int TM, int S, int* part)
{
    using P = Int8Ring<BN, BM, WN, WM>;
    static_assert(NS == 4 || NS == 8, "stages");
    static_assert(BN <= WN * WM * kWave && BM <= WN * WM * kWave, "one epilogue operand per thread");
    __shared__ __attribute__((aligned(1024))) uint8_t b0[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[P::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b4[NS > 4 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b5[NS > 4 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b6[NS > 4 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b7[NS > 4 ? P::STAGE : 16];
    __shared__ __attribute__((aligned(16))) float e_sw[BN];
    __shared__ __attribute__((aligned(16))) uint16_t e_bias[BN];
    __shared__ __attribute__((aligned(16))) float e_sx[BM];
    auto buf = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < 4)
            return ring_buf<i>(b0, b1, b2, b3);
        else
            return ring_buf<i - 4>(b4, b5, b6, b7);
    };
    int tn, tm;
    const int slice = blockIdx.x / (TN * TM);
    xcd_tile<4>(blockIdx.x - slice * (TN * TM), TN, TM, tn, tm);
    const int tid = threadIdx.x;
    const int64_t n0 = (int64_t)tn * BN, m0 = (int64_t)tm * BM, k0 = (int64_t)slice * S * 64;
    P p;
    p.lane = tid & 63;
    p.wave = uniform(tid >> 6);
    p.wn = p.wave % WN;
    p.wm = p.wave / WN;
    p.S = S;
    p.rot = (int)(blockIdx.x % 8) * (S / 8);
    p.w = Rows(c.qw + n0 * c.k + k0);
    p.x = Rows(c.qx + m0 * c.kx + k0);
#pragma unroll
    for (int u = 0; u < P::LOADS; ++u) {
        // row of the stage's combined tile; its chunks are rotated by row / 4
        const int r = 16 * (u * P::W + p.wave) + (p.lane >> 2), chunk = ((p.lane & 3) - (r >> 2)) & 3;
        const int64_t row = r < BN ? (n0 + r < c.n ? r : c.n - 1 - n0) : (m0 + r - BN < c.m ? r - BN : c.m - 1 - m0);
        p.off[u] = (int)(row * (r < BN ? c.k : c.kx)) + 16 * chunk;
    }
    float r_sw = 0.0f, r_sx = 0.0f;
    uint16_t r_bias = 0;
    if (tid < BN) {
        const int64_t ch = n0 + tid < c.n ? n0 + tid : c.n - 1;
        r_sw = c.sw[ch];
        r_bias = bias_bits(c.bias, ch);
    }
    if (tid < BM)
        r_sx = c.sx[m0 + tid < c.m ? m0 + tid : c.m - 1];
    i32x16 acc[P::FN * P::FM];
#pragma unroll
    for (int f = 0; f < P::FN * P::FM; ++f)
        acc[f] = i32x16{0};
    run_tile_ring<NS, P::LOADS>(p, S, buf, acc);
    if (part) {
        store_sums<BN, BM, WN, WM>(c, part + (int64_t)slice * c.m * c.n, n0, m0, p.wn, p.wm, p.lane, acc);
        return;
    }
    if (tid < BN) {
        e_sw[tid] = r_sw;
        e_bias[tid] = r_bias;
    }
    if (tid < BM)
        e_sx[tid] = r_sx;
    __syncthreads();
    store_tile<A, BN, BM, WN, WM>(c, n0, m0, p.wn, p.wm, p.lane, e_sw, e_bias, e_sx, acc);
}

// ------------------------------------------------------------------ plans
enum class Int8Kind { STREAM, TILE, RING };

struct Int8Plan {
    Int8Kind kind;
    int a, b, w;  // stream: RT, CT, W; tile, ring: BN, BM, waves
    int64_t TN, TM;
    int slices;  // ring: of k
    bool fits() const { return grid_fits(TN * TM * slices, w * kWave); }
};

Int8Plan stream_plan(int64_t m, int64_t n, int rt, int ct, int w)
{
    return {Int8Kind::STREAM, rt, ct, w, (n + 16 * ct - 1) / (16 * ct), (m + 16 * rt - 1) / (16 * rt), 1};
}

Int8Plan tile_plan(Int8Kind kind, int64_t m, int64_t n, int bn, int bm, int slices)
{
    return {kind, bn, bm, bm == 64 ? 4 : 8, (n + bn - 1) / bn, (m + bm - 1) / bm, slices};
}

// Stages of the ring: 8 on the 64-wide tile, whose stages are short, else 4.
int ring_depth(int bn)
{
    return bn == 64 ? 8 : 4;
}

// The ring's tile and k split with the lowest modelled time: rounds of 256
// workgroups, each taking the measured time of a stage of its tile (one
// workgroup per CU), plus what writing and joining a split's sums costs. On
// [14336, 4096], [4096, 14336] and [4096, 4096] layers with 64 to 4096 tokens it
// takes the fastest unsplit tile of a sweep or one within 5 %.
bool ring_plan(int64_t m, int64_t n, int64_t k, bool split, Int8Plan& best)
{
    const struct {
        int bn, bm;
        double us;
    } shapes[] = {{256, 256, 0.92}, {256, 128, 0.63}, {128, 128, 0.40}, {128, 64, 0.33}, {64, 64, 0.19}};
    double low = 0.0;
    bool found = false;
    for (const auto& s : shapes)
        for (int z = 1; z <= (split ? 16 : 1); z *= 2) {
            const int64_t stages = k / 64;
            if (stages % z != 0 || stages / z < ring_depth(s.bn))
                continue;
            const Int8Plan p = tile_plan(Int8Kind::RING, m, n, s.bn, s.bm, z);
            const int64_t rounds = (p.TN * p.TM * z + 255) / 256;
            const double us = (double)rounds * (1.0 + s.us * (double)(stages / z)) +
                              (z > 1 ? 3.0 + 8e-6 * (double)z * (double)m * (double)n / 3.0 : 0.0);
            if (p.fits() && (!found || us < low)) {
                low = us;
                best = p;
                found = true;
            }
        }
    return found;
}

// Few tokens, or weight rows that the ring cannot load: the stream kernel up to
// 64 tokens, register-staged tiles above. split: the caller has a workspace for
// the sums of a k split.
Int8Plan int8_plan(int64_t m, int64_t n, int64_t k, int64_t kx, const int8_t* qw, const int8_t* qx, bool split)
{
    const bool ring = k % 64 == 0 && kx % 16 == 0 &&
                      ((reinterpret_cast<uintptr_t>(qw) | reinterpret_cast<uintptr_t>(qx)) & 15) == 0;
    Int8Plan p{};
    if (ring && m > 4 && ring_plan(m, n, k, split, p))
        return p;
    if (m <= 64) {
        const int rt = m <= 16 ? 1 : (m <= 32 ? 2 : 4), w = k >= 2048 ? 8 : 4;
        // two column tiles where that leaves two workgroups per CU
        const int ct = m > 1 && (n + 31) / 32 >= 448 ? 2 : 1;
        p = stream_plan(m, n, rt, ct, w);
        if (p.fits())
            return p;
    }
    const int shapes[3][2] = {{256, 256}, {256, 128}, {128, 128}};
    for (const auto& s : shapes) {
        p = tile_plan(Int8Kind::TILE, m, n, s[0], s[1], 1);
        if (p.TN * p.TM >= 224)
            return p;
    }
    p = tile_plan(Int8Kind::TILE, m, n, 64, 64, 1);
    // few tiles and a long k: slices of eight stages or more (428 tokens, [256, 12149], 28 tiles: 71 us in one piece)
    while (split && p.slices < 8 && p.TN * p.TM * p.slices < 128 && (k + 63) / 64 >= 16 * p.slices)
        p.slices *= 2;
    return p;
}

// Whether some row of codes starts below dword alignment.
bool shifted(const Int8Call& c)
{
    return ((reinterpret_cast<uintptr_t>(c.qw) | reinterpret_cast<uintptr_t>(c.qx) | (uintptr_t)c.k |
             (uintptr_t)c.kx) & 3) != 0;
}

template <typename A, int RT, int CT, int W, int U, bool FUSED>
hipError_t run_stream(const Int8Call& c, const Int8Plan& p, hipStream_t stream)
{
    const dim3 grid((unsigned)(p.TN * p.TM)), block(W * kWave);
    return launch(shifted(c) ? int8_stream_kernel<A, RT, CT, W, U, FUSED, true>
                             : int8_stream_kernel<A, RT, CT, W, U, FUSED, false>,
                  grid, block, stream, c, p.TN, p.TM);
}

// Joins the slices of a k split, behind a products' launch of this status.
template <typename A>
hipError_t join(hipError_t products, const Int8Call& c, const Int8Plan& p, int* part, hipStream_t stream)
{
    if (products != hipSuccess || p.slices == 1)
        return products;
    const int64_t items = c.m * ((c.n + 3) / 4);
    return launch(int8_join_kernel<A>, dim3((unsigned)((items + 255) / 256)), dim3(256), stream, c, part, p.slices);
}

template <typename A, int BN, int BM, int WN, int WM>
hipError_t run_tile(const Int8Call& c, const Int8Plan& p, int* part, hipStream_t stream)
{
    const dim3 grid((unsigned)(p.TN * p.TM * p.slices)), block(WN * WM * kWave);
    const int stages = (int)(((c.k + 63) / 64 + p.slices - 1) / p.slices);
    int* sums = p.slices > 1 ? part : nullptr;
    const hipError_t st = launch(shifted(c) ? int8_tile_kernel<A, BN, BM, WN, WM, true>
                                            : int8_tile_kernel<A, BN, BM, WN, WM, false>,
                                 grid, block, stream, c, p.TN, p.TM, stages, sums);
    return join<A>(st, c, p, part, stream);
}

template <typename A, int BN, int BM, int WN, int WM, int NS>
hipError_t run_ring(const Int8Call& c, const Int8Plan& p, int* part, hipStream_t stream)
{
    const hipError_t st =
        launch(int8_ring_kernel<A, BN, BM, WN, WM, NS>, dim3((unsigned)(p.TN * p.TM * p.slices)),
               dim3(WN * WM * kWave), stream, c, p.TN, p.TM, c.k / 64 / p.slices, p.slices > 1 ? part : nullptr);
    return join<A>(st, c, p, part, stream);
}

template <typename A>
hipError_t run_plan(const Int8Call& c, const Int8Plan& p, bool fuse, int* part, hipStream_t stream)
{
    if (p.kind == Int8Kind::RING) {
        if (p.a == 256)
            return p.b == 256 ? run_ring<A, 256, 256, 2, 4, 4>(c, p, part, stream)
                              : run_ring<A, 256, 128, 2, 4, 4>(c, p, part, stream);
        if (p.a == 128)
            return p.b == 128 ? run_ring<A, 128, 128, 2, 4, 4>(c, p, part, stream)
                              : run_ring<A, 128, 64, 2, 2, 4>(c, p, part, stream);
        return run_ring<A, 64, 64, 2, 2, 8>(c, p, part, stream);
    }
    if (p.kind == Int8Kind::TILE) {
        if (p.a == 256)
            return p.b == 256 ? run_tile<A, 256, 256, 2, 4>(c, p, part, stream) : run_tile<A, 256, 128, 2, 4>(c, p, part, stream);
        return p.a == 128 ? run_tile<A, 128, 128, 2, 4>(c, p, part, stream) : run_tile<A, 64, 64, 2, 2>(c, p, part, stream);
    }
    if (fuse)
        return p.w == 8 ? run_stream<A, 1, 1, 8, 4, true>(c, p, stream)
                        : run_stream<A, 1, 1, 4, 4, true>(c, p, stream);
#define FP8W_STREAM(RT, CT, U)                                                                                         \
    if (p.a == RT && p.b == CT)                                                                                        \
        return p.w == 8 ? run_stream<A, RT, CT, 8, U, false>(c, p, stream)                                             \
                        : run_stream<A, RT, CT, 4, U, false>(c, p, stream);
    FP8W_STREAM(1, 1, 2)
    FP8W_STREAM(1, 2, 2)
    FP8W_STREAM(2, 1, 4)
    FP8W_STREAM(2, 2, 2)
    FP8W_STREAM(4, 1, 1)
    FP8W_STREAM(4, 2, 1)
#undef FP8W_STREAM
    return hipErrorInvalidValue;
}

// One token: quantized in the product's own kernel.
bool fused(int64_t m, int64_t n, int64_t k)
{
    return m == 1 && k <= kFusedK && stream_plan(m, n, 1, 1, 8).fits();
}

// whole cache lines of codes
int64_t padded_k(int64_t k)
{
    return (k + 127) / 128 * 128;
}

// The layer's plan: codes in its workspace, 16-byte aligned.
Int8Plan layer_plan(int64_t m, int64_t n, int64_t k, const int8_t* qw)
{
    return int8_plan(m, n, k, padded_k(k), qw, nullptr, true);
}

// Rows of many values: 256 threads where there are rows enough to fill the CUs
// several times (fewer waves to join), 1024 below (22 rows of 14336: 4.3 us with
// 256 threads).
template <typename A>
hipError_t run_quantize(const void* x, int64_t rows, int64_t k, int8_t* q, int64_t kx, float* scale, hipStream_t stream)
{
    const uint16_t* src = static_cast<const uint16_t*>(x);
    const bool shift = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(2 * k)) & 3) != 0;
    const bool few = rows < 1024;
#define FP8W_ROW(NT, CH)                                                                                               \
    return launch(shift ? quantize_row_kernel<A, NT, CH, true> : quantize_row_kernel<A, NT, CH, false>,                \
                  dim3((unsigned)rows), dim3(NT), stream, src, k, q, kx, scale)
    if (kx <= 2048)
        FP8W_ROW(256, 1);
    if (few && kx <= 8192)
        FP8W_ROW(1024, 1);
    if (few)
        FP8W_ROW(1024, 2);
    if (kx <= 4096)
        FP8W_ROW(256, 2);
    if (kx <= 8192)
        FP8W_ROW(256, 4);
    FP8W_ROW(256, 8);
#undef FP8W_ROW
}

}  // namespace

hipError_t launch_quantize_int8(const void* x, Act type, int64_t rows, int64_t k, int8_t* q, int64_t kx, float* scale,
                                hipStream_t stream)
{
    // a workgroup per row: 2^23 rows of 256 threads are half of what a launch can have
    constexpr int64_t kRows = (int64_t)1 << 23;
    const uint8_t* src = static_cast<const uint8_t*>(x);
    for (int64_t r = 0; r < rows; r += kRows) {
        const int64_t part = rows - r < kRows ? rows - r : kRows;
        const void* from = src + r * k * (type == Act::FP32 ? 4 : 2);
        int8_t* codes = q + r * kx;
        hipError_t st;
        if (type == Act::FP32 || kx > 16384)
            st = launch(quantize_int8_kernel, dim3((unsigned)part), dim3(256), stream, from, type, k, codes, kx,
                        scale + r);
        else
            st = type == Act::BF16 ? run_quantize<Bf16>(from, part, k, codes, kx, scale + r, stream)
                                   : run_quantize<F16>(from, part, k, codes, kx, scale + r, stream);
        if (st != hipSuccess)
            return st;
    }
    return hipSuccess;
}

hipError_t launch_gemm_int8(const int8_t* qx, const float* sx, int64_t m, int64_t k, const int8_t* qw,
                            const float* sw, const void* bias, int64_t n, void* y, Act out, hipStream_t stream)
{
    if (m == 0 || n == 0)
        return hipSuccess;
    const Int8Plan p = int8_plan(m, n, k, k, qw, qx, false);
    if (!p.fits())
        return hipErrorInvalidValue;
    const Int8Call c{nullptr, qx, k, sx, qw, sw, static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y),
                     m, n, k};
    return out == Act::BF16 ? run_plan<Bf16>(c, p, false, nullptr, stream)
                            : run_plan<F16>(c, p, false, nullptr, stream);
}

// The layer's workspace: codes [m, padded k], scales [m], and a k split's sums.
size_t linear_int8_workspace_bytes(int64_t m, int64_t n, int64_t k, const void*, const int8_t* q)
{
    if (fused(m, n, k))
        return 0;
    const Int8Plan p = layer_plan(m, n, k, q);
    const size_t codes = (size_t)m * (size_t)padded_k(k) + (size_t)((m * 4 + 15) & ~(int64_t)15);
    return codes + (p.slices > 1 ? (size_t)p.slices * (size_t)m * (size_t)n * 4 : 0);
}

hipError_t launch_linear_int8(const void* x, Act act, int64_t m, int64_t k, const int8_t* qw, const float* sw,
                              const void* bias, int64_t n, void* y, void* ws, hipStream_t stream)
{
    if (m == 0 || n == 0)
        return hipSuccess;
    Int8Call c{static_cast<const uint16_t*>(x), nullptr, 0, nullptr, qw, sw, static_cast<const uint16_t*>(bias),
               static_cast<uint16_t*>(y), m, n, k};
    if (fused(m, n, k)) {
        const Int8Plan p = stream_plan(m, n, 1, 1, k >= 2048 ? 8 : 4);
        return act == Act::BF16 ? run_plan<Bf16>(c, p, true, nullptr, stream)
                                : run_plan<F16>(c, p, true, nullptr, stream);
    }
    const Int8Plan p = layer_plan(m, n, k, qw);
    if (!p.fits())
        return hipErrorInvalidValue;
    int8_t* qx = static_cast<int8_t*>(ws);
    float* sx = reinterpret_cast<float*>(qx + m * padded_k(k));
    int* part = reinterpret_cast<int*>(sx + ((m + 3) & ~(int64_t)3));
    c.qx = qx;
    c.kx = padded_k(k);
    c.sx = sx;
    const hipError_t e = launch_quantize_int8(x, act, m, k, qx, c.kx, sx, stream);
    if (e != hipSuccess)
        return e;
    return act == Act::BF16 ? run_plan<Bf16>(c, p, false, part, stream) : run_plan<F16>(c, p, false, part, stream);
}

const char* linear_int8_kernel_name(int64_t m, int64_t n, int64_t k, const void*, const int8_t* q)
{
    thread_local char name[160];
    if (fused(m, n, k)) {
        snprintf(name, sizeof name, "int8_stream_kernel<RT=1,CT=1,W=%d,FUSED>", k >= 2048 ? 8 : 4);
        return name;
    }
    const Int8Plan p = layer_plan(m, n, k, q);
    const char* first = padded_k(k) > 16384 ? "quantize_int8_kernel" : "quantize_row_kernel";
    if (p.kind == Int8Kind::STREAM)
        snprintf(name, sizeof name, "%s+int8_stream_kernel<RT=%d,CT=%d,W=%d>", first, p.a, p.b, p.w);
    else {
        char slices[32] = "";
        if (p.slices > 1)
            snprintf(slices, sizeof slices, "*%d+int8_join_kernel", p.slices);
        if (p.kind == Int8Kind::TILE)
            snprintf(name, sizeof name, "%s+int8_tile_kernel<BN=%d,BM=%d,W=%d>%s", first, p.a, p.b, p.w, slices);
        else
            snprintf(name, sizeof name, "%s+int8_ring_kernel<BN=%d,BM=%d,W=%d,NS=%d>%s", first, p.a, p.b, p.w,
                     ring_depth(p.a), slices);
    }
    return name;
}

}  // namespace fp8w
