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
// Choice: G lanes hold a token (64, or 16 where e <= 64 and top <= 16: four
// tokens per wave), J consecutive experts each. A logit becomes an unsigned key
// of the same order (NaN above everything, both zeros equal, -inf key 0 = not to
// be taken). A round is an integer maximum over registers and lanes (DPP
// rotations within rows of 16 lanes, row swaps across them), the first lane and
// register that hold it (the lowest index, since a lane's experts are
// consecutive), and that key cleared.
//
// Order: a counting sort without atomics on global memory, so the lists do not
// depend on timing. Tokens are cut into at most 256 chunks; the first kernel
// writes each chunk's count of every expert, the second adds the counts of the
// experts before (for the offsets) and of the chunks before, and places its
// slots: every wave owns a run of the chunk's slots and ranks 64 at a time by
// the lanes that hold the same expert. Few tokens are one chunk: one workgroup
// does all of it in a single launch.
//
// 32768 tokens, 8 of 256 experts, fp32: 24 us for the choice and 10 for the
// order, where the logits alone take 7 at the rate of a large copy. The choice is
// bound by vector instructions (one more choice of 32768 costs 1.9 us; with one,
// 11), the order by its chain of short steps (8 us for 4096 tokens). One token, 8
// of 128: 5.1 us in its launch, where a launch with little to do takes 2.
#include <math.h>

#include "device.hpp"
#include "moe.hpp"

namespace fp8w {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kChunks = 256;

__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 becomes 0
    uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    key = f == -INFINITY ? 0 : key;
    return f != f ? 0xffffffffu : key;
}

// the logit of a key (a NaN for a NaN's key, -inf for key 0)
__device__ __forceinline__ float logit_of(uint32_t key)
{
    if (key == 0)
        return -INFINITY;
    return __builtin_bit_cast(float, (key >> 31) ? key ^ 0x80000000u : ~key);
}

template <int CTRL>
__device__ __forceinline__ uint32_t rotated(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

// OP over the G lanes of a group, in all of them.
template <int G, typename OP>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, OP op)
{
    static_assert(G == 16 || G == 64, "a row of lanes or the wave");
    v = op(v, rotated<0x128>(v));  // row_ror:8
    v = op(v, rotated<0x124>(v));
    v = op(v, rotated<0x122>(v));
    v = op(v, rotated<0x121>(v));
    if constexpr (G == 64) {
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // even rows' and odd rows' values
        v = op(a[0], a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(b[0], b[1]);
    }
    return v;
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (G == 64)
        return wave_max_u32(v);  // in a scalar register
    else
        return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    return __builtin_bit_cast(float, group_reduce<G>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
                                  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) +
                                                                          __builtin_bit_cast(float, b));
                              }));
}

// A lane's J logits of a row, -inf past its end.
template <int J>
__device__ __forceinline__ void load_logits(const void* logits, Act type, int64_t row, int e, int first, float* l)
{
    if (type == Act::FP32) {
        const float* p = static_cast<const float*>(logits) + row * e + first;
        if (J == 4 && first + 4 <= e) {
            const u32x4 v = load16_any(p);
            const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < J; ++j)
                l[j] = __builtin_bit_cast(float, d[j & 3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            l[j] = first + j < e ? p[j] : -INFINITY;
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(logits) + row * e + first;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint16_t b = first + j < e ? p[j] : (uint16_t)0;
        const float f = type == Act::BF16 ? Bf16::to_f32(b) : F16::to_f32(b);
        l[j] = first + j < e ? f : -INFINITY;
    }
}

// A group's next choice: the largest key left among its lanes' (0: none left),
// taken out, and its expert. A lane's keys are sorted where they are few (a
// choice is then its first key, and taking it a shift), else searched each time.
template <int G, int J>
struct Keys {
    static constexpr bool kSorted = J <= 4;
    uint32_t key[J];
    uint32_t order;  // sorted: the registers' original numbers, a byte each, first key's lowest

    __device__ __forceinline__ explicit Keys(const float (&l)[J])
    {
#pragma unroll
        for (int j = 0; j < J; ++j)
            key[j] = key_of(l[j]);
        if constexpr (kSorted) {
            uint32_t id[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                id[j] = j;
            // neighbours exchanged only where the later is larger: equal keys stay in order
#pragma unroll
            for (int n = J - 1; n >= 1; --n)
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const bool swap = key[j + 1] > key[j];
                    const uint32_t hi = swap ? key[j + 1] : key[j], lo = swap ? key[j] : key[j + 1];
                    const uint32_t a = swap ? id[j + 1] : id[j], b = swap ? id[j] : id[j + 1];
                    key[j] = hi;
                    key[j + 1] = lo;
                    id[j] = a;
                    id[j + 1] = b;
                }
            order = 0;
#pragma unroll
            for (int j = 0; j < J; ++j)
                order |= id[j] << (8 * j);
        }
    }

    __device__ __forceinline__ uint32_t take(int& expert)
    {
        const int lane = threadIdx.x & 63, in = lane % G;
        uint32_t head = key[0];
        int at = 0;
        if constexpr (kSorted) {
            at = (int)(order & 255u);
        } else {
#pragma unroll
            for (int j = 1; j < J; ++j)
                head = head > key[j] ? head : key[j];
#pragma unroll
            for (int j = J - 1; j >= 1; --j)
                at = key[j] == head ? j : at;
            at = key[0] == head ? 0 : at;
        }
        const uint32_t best = group_max<G>(head);
        bool mine;
        if constexpr (G == 64) {
            const int win = (int)__builtin_ctzll(__ballot(head == best));  // never empty
            expert = __builtin_amdgcn_readlane(at, win) + win * J;
            mine = lane == win;
        } else {
            expert = (int)group_reduce<G>(head == best ? (uint32_t)(in * J + at) : 0xffffffffu,
                                          [](uint32_t a, uint32_t b) { return a < b ? a : b; });
            mine = expert / J == in;
        }
        if constexpr (kSorted) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[j] = mine ? (j + 1 < J ? key[j + 1 < J ? j + 1 : j] : 0) : key[j];
            order = mine ? order >> 8 : order;
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[j] = mine && j == at ? 0 : key[j];
        }
        return best;
    }
};

// Two tokens per group at a time (their chains of dependent steps overlap), from
// l[u][j], the token's logit of expert in * J + j. Lane r of a group gets its
// tokens' r-th choice in id[u] (-1: none) and its weight.
template <int G, int J, int U>
__device__ __forceinline__ void choose(const float (&l)[U][J], int top, bool renorm, float (&weight)[U], int (&id)[U])
{
    static_assert(U == 2, "two tokens");
    const int in = (threadIdx.x & 63) % G;
    uint32_t mine[U], peak[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        mine[u] = peak[u] = 0;
        id[u] = -1;
    }
    Keys<G, J> keys[U] = {Keys<G, J>(l[0]), Keys<G, J>(l[U - 1])};
    for (int r = 0; r < top; ++r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int first;
            const uint32_t best = keys[u].take(first);
            if (r == 0)
                peak[u] = best;
            const bool take = in == r && best != 0;
            mine[u] = take ? best : mine[u];
            id[u] = take ? first : id[u];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float top_logit = logit_of(peak[u]);
        const float num = mine[u] ? expf(logit_of(mine[u]) - top_logit) : 0.0f;
        float part = num;
        if (!renorm) {
            part = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
                part += l[u][j] == -INFINITY ? 0.0f : expf(l[u][j] - top_logit);
        }
        const float total = group_sum<G>(part);
        weight[u] = id[u] >= 0 ? num / total : 0.0f;
    }
}

// Chooses for tokens [t0, t1), the workgroup's waves in turn, and calls
// done(token, choice number, expert) from the lanes that hold them.
template <int G, int J, typename F>
__device__ __forceinline__ void choose_chunk(const void* logits, Act type, int64_t t0, int64_t t1, int e, int top,
                                             bool renorm, float* weights, int32_t* experts, F&& done)
{
    constexpr int U = 2, T = U * kWave / G;  // tokens per wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, in = lane % G;
    auto load = [&](int64_t t, float (&l)[U][J]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = t + u * (kWave / G) + lane / G;
            load_logits<J>(logits, type, row < t1 ? row : t1 - 1, e, in * J, l[u]);
        }
    };
    int64_t t = t0 + (int64_t)wave * T;
    float next[U][J];
    if (t < t1)
        load(t, next);
    for (; t < t1; t += kWaves * T) {
        float l[U][J];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < J; ++j)
                l[u][j] = next[u][j];
        if (t + kWaves * T < t1)
            load(t + kWaves * T, next);
        float weight[U];
        int id[U];
        choose<G, J, U>(l, top, renorm, weight, id);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = t + u * (kWave / G) + lane / G;
            if (in < top && row < t1) {
                weights[row * top + in] = weight[u];
                experts[row * top + in] = id[u];
                done(row, in, id[u]);
            }
        }
    }
}

// counts[c][i]: chunk c's slots of expert i, rows of `pitch`.
template <int G, int J>
__global__ __launch_bounds__(kThreads) void route_choose_kernel(const void* __restrict__ logits, Act type, int64_t t,
                                                                int e, int top, int renorm, int64_t per,
                                                                float* __restrict__ weights,
                                                                int32_t* __restrict__ experts,
                                                                int32_t* __restrict__ counts, int pitch)
{
    __shared__ int hist[kMaxExperts];
    for (int i = threadIdx.x; i < e; i += kThreads)
        hist[i] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * per, t1 = t0 + per < t ? t0 + per : t;
    choose_chunk<G, J>(logits, type, t0, t1, e, top, renorm != 0, weights, experts, [&](int64_t, int, int id) {
                           if (id >= 0)
                               atomicAdd(&hist[id], 1);
                       });
    __syncthreads();
    for (int i = threadIdx.x; i < pitch; i += kThreads)
        counts[(int64_t)blockIdx.x * pitch + i] = i < e ? hist[i] : 0;
}

// LDS of a workgroup that places a chunk's slots.
struct Place {
    int next[kMaxExperts + 1];          // the chunk's first position of every expert (e: none)
    int mine[kWaves][kMaxExperts + 1];  // each wave's count, then its first position
    int waves[kWaves];
};

// The sum of v over this thread and those below it (one barrier before the
// result is used by others is the caller's).
__device__ __forceinline__ int block_prefix(int v, int* waves)
{
    const int wave = threadIdx.x >> 6;
    v += rotated<0x111>((uint32_t)v);
    v += rotated<0x112>((uint32_t)v);
    v += rotated<0x114>((uint32_t)v);
    v += rotated<0x118>((uint32_t)v);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    if ((threadIdx.x & 63) == 63)
        waves[wave] = v;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        before += w < wave ? waves[w] : 0;
    return v + before;
}

__device__ __forceinline__ void clear_counts(Place& p, int e)
{
    for (int w = 0; w < kWaves; ++w)
        for (int j = threadIdx.x; j <= e; j += kThreads)
            p.mine[w][j] = 0;
}

// A wave's run [w0, w1) of a chunk's slots.
struct Run {
    int64_t w0, w1;
    __device__ __forceinline__ Run(int64_t s0, int64_t s1)
    {
        const int64_t run = (s1 - s0 + kWaves - 1) / kWaves, wave = threadIdx.x >> 6;
        w0 = s0 + wave * run < s1 ? s0 + wave * run : s1;
        w1 = w0 + run < s1 ? w0 + run : s1;
    }
};

// Places a chunk's slots, whose experts expert(s) returns (-1: none), from
// p.next on. first: this lane's expert in the run's first 64. p.mine is clear;
// the caller's barrier stands before.
template <typename F>
__device__ __forceinline__ void place_chunk(Place& p, Run run, int first, int e, int top, int32_t* slots,
                                            int32_t* tokens, F&& expert)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t w0 = run.w0, w1 = run.w1;
    for (int64_t s = w0 + lane; s < w1; s += 64) {
        const int id = s < w0 + 64 ? first : expert(s);
        atomicAdd(&p.mine[wave][id < 0 ? e : id], 1);
    }
    __syncthreads();
    for (int j = threadIdx.x; j <= e; j += kThreads) {
        int at = p.next[j];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = p.mine[w][j];
            p.mine[w][j] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t s = w0; s < w1; s += 64) {
        const bool on = s + lane < w1;
        int id = !on ? e : (s == w0 ? first : expert(s + lane));
        id = id < 0 ? e : id;
        uint64_t same = __ballot(on);
        for (int b = 1; b <= e; b <<= 1) {  // lanes whose expert agrees in every bit
            const uint64_t set = __ballot(id & b);
            same &= (id & b) ? set : ~set;
        }
        const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        const int at = p.mine[wave][id] + rank;
        wave_sync();
        if (on) {
            slots[at] = (int32_t)(s + lane);
            tokens[at] = (int32_t)((uint32_t)(s + lane) / (uint32_t)top);
            if (rank == 0)
                p.mine[wave][id] = at + __popcll(same);
        }
        wave_sync();
    }
}

__global__ __launch_bounds__(kThreads) void route_place_kernel(const int32_t* __restrict__ experts,
                                                               const int32_t* __restrict__ counts, int pitch,
                                                               int64_t t, int e, int top, int64_t per,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ slots,
                                                               int32_t* __restrict__ tokens)
{
    __shared__ Place p;
    __shared__ int total[kMaxExperts], before[kMaxExperts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = threadIdx.x;
    const int chunks = gridDim.x, chunk = blockIdx.x;
    const int64_t s0 = (int64_t)chunk * per * top;
    const int64_t s1 = ((int64_t)chunk + 1) * per < t ? ((int64_t)chunk + 1) * per * top : t * top;
    const Run run(s0, s1);
    const int first = run.w0 + lane < run.w1 ? experts[run.w0 + lane] : -1;
    total[i] = 0;
    before[i] = 0;
    clear_counts(p, e);
    __syncthreads();
    // every expert's total and the part of the chunks before this one: a wave adds every
    // 16th chunk, four experts per lane, eight chunks in flight
    for (int b = 0; b < pitch; b += 4 * kWave) {
        const int at = b + 4 * lane;
        if (at < pitch) {
            int sum[4] = {0, 0, 0, 0}, low[4] = {0, 0, 0, 0};
            for (int c0 = wave; c0 < chunks; c0 += 8 * kWaves) {
                u32x4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int c = c0 + u * kWaves;
                    v[u] = load16_any(counts + (int64_t)(c < chunks ? c : c0) * pitch + at);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int c = c0 + u * kWaves;
                    const int d[4] = {(int)v[u].x, (int)v[u].y, (int)v[u].z, (int)v[u].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        sum[q] += c < chunks ? d[q] : 0;
                        low[q] += c < chunk ? d[q] : 0;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (at + q < e) {
                    atomicAdd(&total[at + q], sum[q]);
                    atomicAdd(&before[at + q], low[q]);
                }
        }
    }
    __syncthreads();
    const int mine = i < e ? total[i] : 0, low = i < e ? before[i] : 0;
    const int incl = block_prefix(mine, p.waves);
    __syncthreads();
    const int incl_low = block_prefix(low, p.waves);
    if (i < e) {
        p.next[i] = incl - mine + low;
        if (chunk == 0)
            offsets[i] = incl - mine;
    }
    if (i == e - 1) {
        p.next[e] = incl + (int)(s0 - incl_low);  // behind all of them: the slots before that have no expert
        if (chunk == 0)
            offsets[e] = incl;
    }
    __syncthreads();
    place_chunk(p, run, first, e, top, slots, tokens, [&](int64_t s) { return experts[s]; });
}

constexpr int kSmallSlots = 4096;

template <int G, int J>
__global__ __launch_bounds__(kThreads) void route_small_kernel(const void* __restrict__ logits, Act type, int64_t t,
                                                               int e, int top, int renorm,
                                                               float* __restrict__ weights,
                                                               int32_t* __restrict__ experts,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ slots,
                                                               int32_t* __restrict__ tokens)
{
    __shared__ Place p;
    __shared__ int total[kMaxExperts];
    __shared__ int16_t chosen[kSmallSlots];
    const int i = threadIdx.x;
    total[i] = 0;
    clear_counts(p, e);
    __syncthreads();
    choose_chunk<G, J>(logits, type, 0, t, e, top, renorm != 0, weights, experts, [&](int64_t tok, int r, int id) {
                           chosen[tok * top + r] = (int16_t)id;
                           if (id >= 0)
                               atomicAdd(&total[id], 1);
                       });
    __syncthreads();
    const int mine = i < e ? total[i] : 0;
    const int incl = block_prefix(mine, p.waves);
    if (i < e)
        p.next[i] = offsets[i] = incl - mine;
    if (i == e - 1)
        p.next[e] = offsets[e] = incl;
    __syncthreads();
    const Run run(0, t * top);
    const int64_t mine_first = run.w0 + (threadIdx.x & 63);
    place_chunk(p, run, mine_first < run.w1 ? chosen[mine_first] : -1, e, top, slots, tokens,
                [&](int64_t s) { return (int)chosen[s]; });
}

// Tokens of a chunk: a round of every wave at least.
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

int count_pitch(int64_t e)
{
    return (int)((e + 3) / 4 * 4);
}

// Lanes per token.
int lanes(int64_t e, int64_t top)
{
    return e <= 64 && top <= 16 ? 16 : 64;
}

// One workgroup, one launch: one round of its waves, or few choices. The two
// launches take 9 to 11 us however few the tokens; a round of one workgroup adds
// about 0.35 us per choice (235 tokens, 6 of 44, in two rounds: 14.8 us against
// 11.0; 250 tokens, 2 of 8: 7.4 against 9.3).
bool small(int64_t t, int64_t e, int64_t top)
{
    const int64_t rounds = (t * lanes(e, top) + 2 * kThreads - 1) / (2 * kThreads);
    return t * top <= kSmallSlots && (rounds <= 1 || rounds * (top + 2) <= 8);
}

template <int G, int J>
hipError_t run(const void* logits, Act type, int64_t t, int e, int top, bool renorm, float* weights, int32_t* experts,
               int32_t* offsets, int32_t* slots, int32_t* tokens, void* ws, hipStream_t stream)
{
    if (small(t, e, top))
        return launch(route_small_kernel<G, J>, dim3(1), dim3(kThreads), stream, logits, type, t, e, top, renorm,
                      weights, experts, offsets, slots, tokens);
    const int64_t per = tokens_per_chunk(t);
    const int pitch = count_pitch(e);
    int32_t* counts = static_cast<int32_t*>(ws);
    const dim3 grid((unsigned)chunk_count(t)), block(kThreads);
    const hipError_t st = launch(route_choose_kernel<G, J>, grid, block, stream, logits, type, t, e, top, renorm, per,
                                 weights, experts, counts, pitch);
    if (st != hipSuccess)
        return st;
    return launch(route_place_kernel, grid, block, stream, experts, counts, pitch, t, e, top, per, offsets, slots,
                  tokens);
}

}  // namespace

size_t route_workspace_bytes(int64_t t, int64_t e, int64_t top)
{
    return small(t, e, top) ? 0 : (size_t)chunk_count(t) * (size_t)count_pitch(e) * 4;
}

hipError_t launch_route(const void* logits, Act type, int64_t t, int64_t e, int64_t top, bool renorm, float* weights,
                        int32_t* experts, int32_t* offsets, int32_t* slots, int32_t* tokens, void* ws,
                        hipStream_t stream)
{
#define FP8W_ROUTE(G, J)                                                                                               \
    return run<G, J>(logits, type, t, (int)e, (int)top, renorm, weights, experts, offsets, slots, tokens, ws, stream)
    if (lanes(e, top) == 16) {
        if (e <= 16)
            FP8W_ROUTE(16, 1);
        if (e <= 32)
            FP8W_ROUTE(16, 2);
        FP8W_ROUTE(16, 4);
    }
    if (e <= 64)
        FP8W_ROUTE(64, 1);
    if (e <= 128)
        FP8W_ROUTE(64, 2);
    if (e <= 256)
        FP8W_ROUTE(64, 4);
    if (e <= 512)
        FP8W_ROUTE(64, 8);
    FP8W_ROUTE(64, 16);
#undef FP8W_ROUTE
}

}  // namespace fp8w
