// The router of a mixture of experts, from logits to the row lists that the
// products grouped by expert take.
//
//   experts[t, j]  the j-th largest logit's expert, equal logits by the lower
//                  index; an expert with logit -inf is never taken: its place
//                  holds -1 and weight 0
//   weights[t, j]  exp(l_j - l_0) / sum, the sum over the chosen experts
//                  (renormalized) or over all of the token's (softmax)
//   slots          the slots t * top + j ordered by expert, in slot order
//                  within an expert; slots without an expert last
//   offsets[i]     the first position in slots of expert i; offsets[e] the
//                  number of slots with an expert
//   tokens         slots / top
//
// Choice: one wave per token, expert 64 j + lane in register j of a lane. A
// logit becomes an unsigned key of the same order (NaN above everything, both
// zeros equal, -inf key 0 = not to be taken), so a round is an integer maximum
// over registers and lanes, a comparison of each register with it (the first
// register and lane that hold it are the lowest index), and a key cleared.
//
// Order: a counting sort without atomics on global memory, so the lists do not
// depend on timing. Tokens are cut into at most 256 chunks; the first kernel
// writes each chunk's count of every expert, the second adds the counts of the
// experts before (for the offsets) and of the chunks before, and places its
// slots: every wave owns a run of the chunk's slots and ranks 64 at a time by
// the lanes that hold the same expert.
#include <math.h>

#include "device.hpp"
#include "moe.hpp"

namespace fp8w {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kChunks = 256;

__device__ __forceinline__ float logit_at(const void* p, Act type, int64_t i)
{
    if (type == Act::FP32)
        return static_cast<const float*>(p)[i];
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return type == Act::BF16 ? Bf16::to_f32(b) : F16::to_f32(b);
}

__device__ __forceinline__ uint32_t key_of(float f)
{
    if (f != f)
        return 0xffffffffu;
    if (f == -INFINITY)
        return 0;
    const uint32_t u = __builtin_bit_cast(uint32_t, f == 0.0f ? 0.0f : f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// the logit of a key (a NaN for a NaN's key, -inf for key 0)
__device__ __forceinline__ float logit_of(uint32_t key)
{
    if (key == 0)
        return -INFINITY;
    return __builtin_bit_cast(float, (key >> 31) ? key ^ 0x80000000u : ~key);
}

// J registers of logits per lane: e <= 64 J.
template <int J>
__device__ __forceinline__ void choose(const void* logits, Act type, int64_t t, int e, int top, bool renorm,
                                       float* weights, int32_t* experts, int lane)
{
    uint32_t key[J];
    float l[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int i = 64 * j + lane;
        l[j] = i < e ? logit_at(logits, type, t * e + i) : -INFINITY;
        key[j] = key_of(l[j]);
    }
    uint32_t my_key = 0;
    int my_id = -1;
    for (int r = 0; r < top; ++r) {
        uint32_t best = key[0];
#pragma unroll
        for (int j = 1; j < J; ++j)
            best = best > key[j] ? best : key[j];
        best = wave_max_u32(best);
        if (best == 0)
            break;  // nothing left to take
        int id = -1;
#pragma unroll
        for (int j = J - 1; j >= 0; --j) {
            const uint64_t hit = __ballot(key[j] == best);
            if (hit)
                id = 64 * j + (int)__builtin_ctzll(hit);
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            key[j] = 64 * j + lane == id ? 0 : key[j];
        if (lane == r) {
            my_key = best;
            my_id = id;
        }
    }
    const float mine = logit_of(my_key);
    const float peak = __shfl(mine, 0, kWave);
    const float num = my_key ? expf(mine - peak) : 0.0f;
    float part = num;
    if (!renorm) {
        part = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j)
            part += l[j] == -INFINITY ? 0.0f : expf(l[j] - peak);
    }
    const float total = wave_sum(part);
    if (lane < top) {
        weights[t * top + lane] = my_id >= 0 ? num / total : 0.0f;
        experts[t * top + lane] = my_id;
    }
}

// Chunk c holds tokens [c * per, min(t, (c + 1) * per)); counts[c][i] (i <= e;
// i == e: slots without an expert). gridDim.x chunks.
template <int J>
__global__ __launch_bounds__(kThreads) void route_choose_kernel(const void* __restrict__ logits, Act type, int64_t t,
                                                                int e, int top, int renorm, int64_t per,
                                                                float* __restrict__ weights,
                                                                int32_t* __restrict__ experts,
                                                                int32_t* __restrict__ counts)
{
    __shared__ int hist[kMaxExperts + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i <= e; i += kThreads)
        hist[i] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * per, t1 = t0 + per < t ? t0 + per : t;
    for (int64_t tt = t0 + wave; tt < t1; tt += kWaves) {
        choose<J>(logits, type, tt, e, top, renorm != 0, weights, experts, lane);
        if (lane < top) {
            const int id = experts[tt * top + lane];
            atomicAdd(&hist[id < 0 ? e : id], 1);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= e; i += kThreads)
        counts[(int64_t)blockIdx.x * (e + 1) + i] = hist[i];
}

__global__ __launch_bounds__(kThreads) void route_place_kernel(const int32_t* __restrict__ experts,
                                                               const int32_t* __restrict__ counts, int64_t t, int e,
                                                               int top, int64_t per, int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ slots,
                                                               int32_t* __restrict__ tokens)
{
    __shared__ int next[kMaxExperts + 1];               // this chunk's first position of every expert
    __shared__ int scan[kThreads];
    __shared__ int mine[kWaves][kMaxExperts + 1];       // each wave's count, then its first position
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int chunks = gridDim.x, chunk = blockIdx.x;
    // every expert's total and the part of the chunks before this one
    int before = 0, total = 0;
    const int i = threadIdx.x;
    if (i <= e) {
        for (int c = 0; c < chunks; ++c) {
            const int v = counts[(int64_t)c * (e + 1) + i];
            total += v;
            before += c < chunk ? v : 0;
        }
    }
    // group e (no expert) only needs a start: with 1024 experts it is thread 0's extra
    scan[i] = i < e ? total : 0;
    for (int w = 0; w < kWaves; ++w)
        for (int j = threadIdx.x; j <= e; j += kThreads)
            mine[w][j] = 0;
    __syncthreads();
    for (int off = 1; off < kThreads; off <<= 1) {
        const int v = i >= off ? scan[i - off] : 0;
        __syncthreads();
        scan[i] += v;
        __syncthreads();
    }
    if (i < e) {
        next[i] = scan[i] - total + before;
        if (chunk == 0)
            offsets[i] = scan[i] - total;
    }
    if (i == 0) {
        int b = 0;  // slots without an expert in the chunks before
        for (int c = 0; c < chunk; ++c)
            b += counts[(int64_t)c * (e + 1) + e];
        next[e] = scan[kThreads - 1] + b;
        if (chunk == 0)
            offsets[e] = scan[kThreads - 1];
    }
    const int64_t s0 = (int64_t)chunk * per * top;
    const int64_t s1 = ((int64_t)chunk + 1) * per < t ? ((int64_t)chunk + 1) * per * top : t * top;
    const int64_t run = (s1 - s0 + kWaves - 1) / kWaves;
    const int64_t w0 = s0 + wave * run < s1 ? s0 + wave * run : s1;
    const int64_t w1 = w0 + run < s1 ? w0 + run : s1;
    for (int64_t s = w0 + lane; s < w1; s += 64) {
        const int id = experts[s];
        atomicAdd(&mine[wave][id < 0 ? e : id], 1);
    }
    __syncthreads();
    for (int j = threadIdx.x; j <= e; j += kThreads) {
        int at = next[j];
        for (int w = 0; w < kWaves; ++w) {
            const int c = mine[w][j];
            mine[w][j] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t s = w0; s < w1; s += 64) {
        const bool on = s + lane < w1;
        int id = on ? experts[s + lane] : e;
        id = id < 0 ? e : id;
        uint64_t same = __ballot(on);
        for (int b = 1; b <= e; b <<= 1) {  // lanes whose expert agrees in every bit
            const uint64_t set = __ballot(id & b);
            same &= (id & b) ? set : ~set;
        }
        const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        const int at = mine[wave][id] + rank;
        __builtin_amdgcn_wave_barrier();
        if (on) {
            slots[at] = (int32_t)(s + lane);
            tokens[at] = (int32_t)((s + lane) / top);
            if (rank == 0)
                mine[wave][id] = at + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

int64_t tokens_per_chunk(int64_t t)
{
    const int64_t per = (t + kChunks - 1) / kChunks;
    return per < kWaves ? kWaves : per;
}

int64_t chunk_count(int64_t t)
{
    const int64_t per = tokens_per_chunk(t);
    return (t + per - 1) / per;
}

}  // namespace

size_t route_workspace_bytes(int64_t t, int64_t e, int64_t top)
{
    return t > 0 ? (size_t)chunk_count(t) * (size_t)(e + 1) * 4 : (size_t)(e + 1) * 4;
}

hipError_t launch_route(const void* logits, Act type, int64_t t, int64_t e, int64_t top, bool renorm, float* weights,
                        int32_t* experts, int32_t* offsets, int32_t* slots, int32_t* tokens, void* ws,
                        hipStream_t stream)
{
    const int64_t per = tokens_per_chunk(t), chunks = t > 0 ? chunk_count(t) : 1;
    int32_t* counts = static_cast<int32_t*>(ws);
    const dim3 grid((unsigned)chunks), block(kThreads);
#define FP8W_CHOOSE(J)                                                                                                 \
    hipLaunchKernelGGL(route_choose_kernel<J>, grid, block, 0, stream, logits, type, t, (int)e, (int)top, (int)renorm, \
                       per, weights, experts, counts)
    if (e <= 64)
        FP8W_CHOOSE(1);
    else if (e <= 128)
        FP8W_CHOOSE(2);
    else if (e <= 256)
        FP8W_CHOOSE(4);
    else
        FP8W_CHOOSE(16);
#undef FP8W_CHOOSE
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess)
        return st;
    hipLaunchKernelGGL(route_place_kernel, grid, block, 0, stream, experts, counts, t, (int)e, (int)top, per, offsets,
                       slots, tokens);
    return hipGetLastError();
}

}  // namespace fp8w
