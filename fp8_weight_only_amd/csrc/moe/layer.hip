// A whole mixture-of-experts layer for a few tokens (t <= 64), two launches:
//   h[s, i]  = silu(g) * u, for each place s of a token with an expert: g and u the
//              products of the token with the expert's rows i and inner + i
//   out[t, c] = sum over t's places of weight * (sum_i h[s, i] * down[expert, c, i] + bias)
// The choice and the weights are the router's. Weights are e4m3 codes
// with a scale per output channel, or 4-bit codes with block scales (fp4.hpp).
//
// First launch: every workgroup chooses for all tokens rather than wait for a launch
// that does. Its items are 16 channels of one active expert, gate and up rows
// together, with up to 32 of its rows: an expert with more is read twice. The
// first workgroup leaves the plan for the second launch.
//
// Second launch: a workgroup has 16 output channels of every token, or where there
// are few channels a part of their steps. The active experts' blocks of k, in one
// line, are split evenly over its waves (over all waves of the workgroups that share
// the channels); a wave adds weights[t, j] times its part of an expert's sums to its
// own fp32 accumulators in LDS, and the waves' accumulators are added in wave order.
// Workgroups that share channels leave those fp32 sums in the workspace and the last
// one adds them in their order. What goes through memory besides is h: no slot's down
// product does, and no sum depends on the order of anything.
//
// Sums, scales, biases, the activation and the weighted sum are fp32; h is rounded
// once to the activation type, as the matrix cores take it (half a step of it per
// value), and out once. With both roundings the error to the 64-bit result is 1.4
// times that of rounding out alone (bf16 2.4e-3 against 1.7e-3 of the norm, fp16 3.0e-4
// against 2.1e-4), without a second pass of the matrix cores over h's lower bits. In
// fp16 an h above 65504 is infinite, as a tensor of that type between separate calls
// would be; it stays in its token.
#include <algorithm>

#include <stdio.h>

#include "choose.hpp"
#include "groups.hpp"
#include "stream.hpp"
#include "tile.hpp"

namespace fp8w {
namespace {

// A wave's choices for U tokens, lane r the r-th of each (-1: none) and its weight,
// as route's: a lane holds the keys of experts lane, lane + 64, ..; a choice is the
// largest key, of equal ones the lowest expert's. Short code rather than few
// instructions: it runs once, on a cold instruction cache.
template <int J, int U>
__device__ __forceinline__ void choose_keys(const LayerCall& c, int token, float (&weight)[U], int (&id)[U])
{
    const int lane = threadIdx.x & 63, e = (int)c.e;
    float l[U][J];
    uint32_t key[U][J], mine[U], peak[U];
    auto load = [&](auto&& get) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = (int64_t)(token + u < (int)c.t ? token + u : (int)c.t - 1) * e;
#pragma unroll
            for (int j = 0; j < J; ++j)
                l[u][j] = get(row + (lane + 64 * j < e ? lane + 64 * j : e - 1));
        }
    };
    if (c.logits_type == Act::FP32)
        load([&](int64_t at) { return static_cast<const float*>(c.logits)[at]; });
    else if (c.logits_type == Act::BF16)
        load([&](int64_t at) { return Bf16::to_f32(static_cast<const uint16_t*>(c.logits)[at]); });
    else
        load([&](int64_t at) { return F16::to_f32(static_cast<const uint16_t*>(c.logits)[at]); });
#pragma unroll
    for (int u = 0; u < U; ++u) {
        mine[u] = peak[u] = 0;
        id[u] = -1;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            l[u][j] = lane + 64 * j < e ? l[u][j] : -INFINITY;
            key[u][j] = key_of(l[u][j]);
        }
    }
#pragma unroll 1
    for (int r = 0; r < c.top; ++r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t head = key[u][0];
#pragma unroll
            for (int j = 1; j < J; ++j)
                head = head > key[u][j] ? head : key[u][j];
            const uint32_t best = wave_max_u32(head);
            int expert = 0;
#pragma unroll
            for (int j = J - 1; j >= 0; --j) {
                const uint64_t has = __ballot(key[u][j] == best);
                expert = has ? 64 * j + (int)__builtin_ctzll(has) : expert;
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[u][j] = lane + 64 * j == expert ? 0 : key[u][j];
            peak[u] = r == 0 ? best : peak[u];
            const bool take = lane == r && best != 0;
            mine[u] = take ? best : mine[u];
            id[u] = take ? expert : id[u];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float top_logit = logit_of(peak[u]);
        float num = mine[u] ? expf(logit_of(mine[u]) - top_logit) : 0.0f, part = num;
        if (!c.renorm) {
            part = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
                part += l[u][j] == -INFINITY ? 0.0f : expf(l[u][j] - top_logit);
        }
        const float total = group_sum<kWave>(part);
        weight[u] = id[u] >= 0 ? num / total : 0.0f;
    }
}

template <int U>
__device__ __forceinline__ void choose_by_wave(const LayerCall& c, int token, float (&weight)[U], int (&id)[U])
{
    if (c.e <= 64)
        choose_keys<1, U>(c, token, weight, id);
    else if (c.e <= 128)
        choose_keys<2, U>(c, token, weight, id);
    else if (c.e <= 256)
        choose_keys<4, U>(c, token, weight, id);
    else
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            float w[1];
            int i[1];
            choose_keys<16, 1>(c, token + u, w, i);
#pragma unroll
            for (int q = 0; q < U; ++q) {
                weight[q] = u == q ? w[0] : weight[q];
                id[q] = u == q ? i[0] : id[q];
            }
        }
}

// What the first launch leaves for the second: the active experts in order, their first
// rows and each row's token and weight, and the choices by token, for the biases. A row
// is a token's place with one expert; an expert's rows stand by rising token.
//
// h keeps an expert's rows in groups of four, eight values of each in turn: group G has
// value i of its row b at (G * pitch + i / 8 * 8) * 4 + 8 b + i % 8 (stream.hpp).
struct Plan {
    int32_t *count, *active, *start, *group, *token, *choice;
    float *weight, *share;
};

// Rows that are multiplied together: an expert with more (t > 32 only) stands in the
// plan again for the next ones, and its weights are read again.
constexpr int kRows = 32;
constexpr int kMaxEntries = kMaxExperts + kMaxLayerTokens * kMaxTop / kRows;

__device__ __host__ inline int64_t most_entries(int64_t t, int64_t e, int64_t top)
{
    const int64_t slots = t * top;
    return (slots < e ? slots : e) + (t > kRows ? slots / kRows : 0);
}

// Rows of h: every entry's last group may have up to three of no token.
__device__ __host__ inline int64_t h_rows(int64_t t, int64_t e, int64_t top)
{
    return t * top + 3 * most_entries(t, e, top);
}

__device__ __host__ inline Plan plan_of(const LayerCall& c)
{
    const int64_t slots = c.t * c.top, most = most_entries(c.t, c.e, c.top);
    Plan p;
    p.count = c.plan;
    p.active = p.count + 1;
    p.start = p.active + most;
    p.group = p.start + most + 1;
    p.token = p.group + most;
    p.choice = p.token + slots;
    p.weight = reinterpret_cast<float*>(p.choice + slots);
    p.share = p.weight + slots;
    return p;
}

__device__ __host__ inline int64_t output_tiles(int64_t hidden)
{
    return (hidden + 15) / 16;
}

constexpr int kPlanNumbers = 4;  // per slot, besides 2 and 3 per expert

// LDS of the first launch: the tokens of every expert as bits (t <= 64), the active
// experts and their first rows. The first workgroup's choices, for the plan, stand where
// the stream begins afterwards.
struct Lists {
    uint64_t tokens[kMaxExperts];
    uint16_t active[kMaxEntries], start[kMaxEntries + 1], group[kMaxEntries], of[kMaxExperts];
    int count;
};
template <int SLOTS>
struct Choices {
    float weight[SLOTS];
    int16_t id[SLOTS];
};

// The token of row `lane` of an expert whose tokens are these bits.
__device__ __forceinline__ int token_of_row(uint64_t tokens)
{
    const int lane = threadIdx.x & 63;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    const int to = (tokens >> lane) & 1 ? __popcll(tokens & below) : __popcll(tokens) + __popcll(~tokens & below);
    return __builtin_amdgcn_ds_permute(4 * to, lane);  // a permutation: every lane is written once
}

// An item is 16 channels of gate and of up of one active expert; a workgroup has
// every gridDim.x-th. Its W waves take the steps of k in turn. A wave's loads run a step
// ahead, into the next item while this one's sums meet in LDS, so the stream of weights
// does not stop between items.
//
// RC: tiles of 16 rows (0: one token, whose choices every wave makes for itself, with
// no barrier before the first loads).
//
// One token, two of eight e4m3 experts [28672, 4096]: 47 us, 5.0 TB/s. 64 tokens over all eight: 234 us,
// the address unit busy 80 % (two tiles of channels, half the activations' loads: 233). 16 tokens over 128 4-bit experts [2048, 4096]: 88.
template <typename F, typename A, int RC, int W, Way WAY>
__global__ __launch_bounds__(W* kWave, 2) void layer_up_kernel(LayerCall c, int TN)
{
    constexpr int NT = W * kWave, CH = 16, RT = RC == 0 ? 1 : RC;  // a thread's values are of one channel
    constexpr bool ONE = RC == 0;
    constexpr int SLOTS = (RC <= 1 ? 16 : kMaxLayerTokens) * kMaxTop;
    using S = Stream<F, A, 2, 2, RT, WAY, false>;  // gate, up
    using C = Choices<SLOTS>;
    constexpr size_t kRing = (size_t)W * S::LDS, kChoices = ONE ? 16 : sizeof(C);
    __shared__ std::conditional_t<ONE, char, Lists> lists;
    __shared__ __attribute__((aligned(16))) uint8_t ring[kRing > kChoices ? kRing : kChoices];
    __shared__ __attribute__((aligned(16))) float part[W][2][4 * kWave];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const Plan plan = plan_of(c);
    if (blockIdx.x == 0 && c.arrived)
        for (int i = tid; i < (int)output_tiles(c.hidden); i += NT)
            c.arrived[i] = 0;
    int count, one_id = -1;
    if constexpr (ONE) {
        float weight[1];
        int id[1];
        choose_by_wave<1>(c, 0, weight, id);
        one_id = id[0];
        count = __popcll(__ballot(one_id >= 0));
        if (blockIdx.x == 0 && wave == 0) {
            if (lane == 0) {
                *plan.count = count;
                plan.start[0] = 0;
            }
            if (lane < count) {
                plan.active[lane] = one_id;
                plan.start[lane + 1] = lane + 1;
                plan.group[lane] = lane;
                plan.token[lane] = 0;
                plan.weight[lane] = weight[0];
            }
            if (lane < c.top) {
                plan.choice[lane] = one_id;
                plan.share[lane] = weight[0];
            }
        }
    } else {
        const int e = (int)c.e, slots = (int)c.t * c.top;
        C& mine = *reinterpret_cast<C*>(ring);
        for (int i = tid; i < e; i += NT)
            lists.tokens[i] = 0;
        __syncthreads();
#pragma unroll 1
        for (int t = 2 * wave; t < (int)c.t; t += 2 * W) {
            float weight[2];
            int id[2];
            choose_by_wave<2>(c, t, weight, id);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (t + u < (int)c.t && lane < c.top) {
                    if (id[u] >= 0)
                        atomicOr(reinterpret_cast<uint32_t*>(&lists.tokens[id[u]]) + ((t + u) >> 5), 1u << ((t + u) & 31));
                    if (blockIdx.x == 0) {
                        const int s = (t + u) * c.top + lane;
                        mine.id[s] = (int16_t)id[u];
                        mine.weight[s] = weight[u];
                        plan.choice[s] = id[u];
                        plan.share[s] = weight[u];
                    }
                }
        }
        __syncthreads();
        if (wave == 0) {
            int experts = 0, rows = 0, groups = 0;
#pragma unroll 1
            for (int i0 = 0; i0 < e; i0 += kWave) {
                const int i = i0 + lane, n = i < e ? __popcll(lists.tokens[i]) : 0, incl = wave_prefix(n);
                const int entries = (n + 16 * RT - 1) / (16 * RT), upto = wave_prefix(entries);
                const int fours = wave_prefix((n + 3) / 4);
                if (n > 0) {
                    const int at = experts + upto - entries, row = rows + incl - n;
                    lists.of[i] = (uint16_t)row;
                    for (int q = 0; q < entries; ++q) {
                        lists.active[at + q] = (uint16_t)i;
                        lists.start[at + q] = (uint16_t)(row + 16 * RT * q);
                        lists.group[at + q] = (uint16_t)(groups + fours - (n + 3) / 4 + 4 * RT * q);
                    }
                }
                experts += __builtin_amdgcn_readlane(upto, 63);
                rows += __builtin_amdgcn_readlane(incl, 63);
                groups += __builtin_amdgcn_readlane(fours, 63);
            }
            if (lane == 0) {
                lists.start[experts] = (uint16_t)rows;
                lists.count = experts;
            }
        }
        __syncthreads();
        count = uniform(lists.count);
        if (blockIdx.x == 0) {
            if (tid == 0)
                *plan.count = count;
            for (int i = tid; i <= count; i += NT) {
                plan.start[i] = lists.start[i];
                if (i < count) {
                    plan.active[i] = lists.active[i];
                    plan.group[i] = lists.group[i];
                }
            }
            for (int s = tid; s < slots; s += NT) {
                const int id = mine.id[s], tok = s / c.top;
                if (id >= 0) {
                    const int at = lists.of[id] + __popcll(lists.tokens[id] & (((uint64_t)1 << tok) - 1));
                    plan.token[at] = tok;
                    plan.weight[at] = mine.weight[s];
                }
            }
            __syncthreads();
        }
    }

    S st(c.hidden, c.x, 2 * c.t * c.hidden, ring + wave * S::LDS);
    struct Item {
        int group, rows;
        int64_t n0, up;  // first channel; the expert's first gate row
    };
    const int items = TN * count, NU = (st.steps + W - 1) / W;  // steps of a wave in an item
    auto enter = [&](int it, Item& item, typename S::Source& src) {
        const int a = uniform(it / TN);
        int expert, tok = 0, before = 0;  // the expert's rows before the item's
        item.group = a;
        item.rows = 1;
        if constexpr (ONE) {
            expert = __builtin_amdgcn_readlane(one_id, a);
        } else {
            expert = uniform(lists.active[a]);
            const int first = uniform(lists.start[a]);
            item.group = uniform(lists.group[a]);
            item.rows = uniform(lists.start[a + 1]) - first;
            before = first - uniform(lists.of[expert]);
            tok = token_of_row(lists.tokens[expert]);
        }
        item.n0 = (int64_t)(it - a * TN) * CH;
        item.up = (int64_t)expert * 2 * c.inner;
        st.weights(src, 0, c.up.q, c.up.scale, item.up + item.n0, 2 * c.e * c.inner);
        st.weights(src, 1, c.up.q, c.up.scale, item.up + c.inner + item.n0, 2 * c.e * c.inner);
        // rows past the item's: any row, not stored
        st.rows(src, item.rows, [&](int i) {
            return ONE ? 0 : (int64_t)__shfl(tok, before + (i < item.rows ? i : 0), kWave) * c.hidden;
        });
    };
    int it = blockIdx.x;
    if (it >= items)
        return;
    Item item, next;
    typename S::Source src;
    enter(it, item, src);
    st.load(src, wave, wave < st.steps);
#pragma unroll 1
    for (; it < items; it += gridDim.x, item = next) {
        // the scales and biases of this thread's channel
        const int ch = tid % CH, channels = (int)(c.inner - item.n0 < CH ? c.inner - item.n0 : CH);
        const int64_t gc = item.up + item.n0 + (ch < channels ? ch : 0), uc = gc + c.inner;
        const uint16_t* bias = static_cast<const uint16_t*>(c.up.bias);
        const float* scale = static_cast<const float*>(c.up.scale);
        const float gs = F::kBlockScales ? 1.0f : scale[gc], us = F::kBlockScales ? 1.0f : scale[uc];
        const uint16_t gb = bias_bits(bias, gc), ub = bias_bits(bias, uc);
        f32x4 acc[2][RT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < RT; ++u)
                acc[t][u] = f32x4{0.0f};
#pragma unroll 1
        for (int v = 0; v < NU; ++v) {
            int ahead = v + 1;
            bool more = true;
            if (ahead == NU) {
                ahead = 0;
                more = it + (int)gridDim.x < items;
                if (more)
                    enter(it + gridDim.x, next, src);
            }
            ahead = wave + W * ahead;
            st.consume(wave + W * v, src, ahead, more && ahead < st.steps, acc);
        }
#pragma unroll 1
        for (int u = 0; u < RT; ++u) {
            if (16 * u >= item.rows)
                break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 sums = acc[t][0];
#pragma unroll
                for (int q = 1; q < RT; ++q)
                    sums = u == q ? acc[t][q] : sums;
                *reinterpret_cast<f32x4*>(&part[wave][t][4 * lane]) = sums;
            }
            lds_barrier();
            // lane (r, g) of a tile has its channels 4 g .. 4 g + 3 of row r
            const int here = item.rows - 16 * u < 16 ? item.rows - 16 * u : 16;
#pragma unroll 1
            for (int row = tid / CH; row < here; row += NT / CH) {
                const int at = 4 * (row + 16 * (ch >> 2)) + (ch & 3);
                float gate = 0.0f, lift = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    gate += part[w][0][at];
                    lift += part[w][1][at];
                }
                gate = __builtin_fmaf(gs, gate, A::to_f32(gb));
                lift = __builtin_fmaf(us, lift, A::to_f32(ub));
                const int64_t i = item.n0 + ch;
                if (ch < channels)
                    c.h[((item.group + 4 * u + row / 4) * c.pitch + i / 8 * 8) * 4 + 8 * (row & 3) + i % 8] =
                        rounded<A>(gate / (1.0f + expf(-gate)) * lift);
            }
            lds_barrier();
        }
    }
}

// A workgroup has 16 output channels of every token. A wave's steps run over the active
// experts; at an expert's end (or the wave's own) its sums go to the wave's accumulators
// of the tokens. One token, two of eight e4m3 experts [4096, 14336]: 25.5 us, 4.6 TB/s; 64 tokens
// over all eight: 122.
//
// Where there are few channels the steps are shared by `slices` workgroups: each leaves its
// sums in the workspace and counts itself in (the first launch cleared the counts), and the last
// to come adds all of them, in the slices' order whichever came last. Sums pass by stores and loads
// of device scope, past the L2 that each XCD has for itself, one release and one acquire to a
// workgroup around the count. 13 tokens over 60 e4m3 experts of [1030, 513]: 19.8 us in four slices, 25.8
// in one on a quarter of the CUs (and 77 with a fence in every wave: it empties an L2).
template <typename F, typename A, int RC, int W, Way WAY>
__global__ __launch_bounds__(W* kWave) void layer_down_kernel(LayerCall c, int slices)
{
    constexpr int NT = W * kWave, RT = RC == 0 ? 1 : RC;
    constexpr int TOKENS = RC == 0 ? 1 : (RC == 1 ? 16 : kMaxLayerTokens);
    __shared__ __attribute__((aligned(16))) f32x4 sum[W][TOKENS][4];
    __shared__ uint16_t active[kMaxEntries], start[kMaxEntries + 1], group[kMaxEntries];
    __shared__ uint8_t token[TOKENS * kMaxTop];
    __shared__ float weight[TOKENS * kMaxTop];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 15, g = lane >> 4;
    const int slots = (int)c.t * c.top, most = (int)most_entries(c.t, c.e, c.top);
    __shared__ bool last;
    const int tile = (int)blockIdx.x / slices, slice = (int)blockIdx.x % slices;
    const int64_t n0 = (int64_t)tile * 16;
    const Plan plan = plan_of(c);
    const int count = uniform(*plan.count);
    // what lies behind the lists' ends is of no use, and not used
    for (int i = tid; i <= most; i += NT) {
        start[i] = (uint16_t)plan.start[i];
        if (i < most) {
            active[i] = (uint16_t)plan.active[i];
            group[i] = (uint16_t)plan.group[i];
        }
    }
    for (int i = tid; i < slots; i += NT) {
        token[i] = (uint8_t)plan.token[i];
        weight[i] = plan.weight[i];
    }
    for (int i = tid; i < W * TOKENS * 4; i += NT)
        (&sum[0][0][0])[i] = f32x4{0.0f};
    __syncthreads();
    if (c.down.bias && slice == 0) {
#pragma unroll 1
        for (int i = tid; i < (int)c.t * 16; i += NT) {
            float z = 0.0f;
#pragma unroll 1
            for (int j = 0; j < c.top && n0 + i % 16 < c.hidden; ++j) {
                const int s = i / 16 * c.top + j, id = plan.choice[s];
                if (id >= 0)
                    z = __builtin_fmaf(plan.share[s], A::to_f32(static_cast<const uint16_t*>(
                                                          c.down.bias)[id * c.hidden + n0 + i % 16]), z);
            }
            reinterpret_cast<float*>(&sum[0][i / 16][0])[i % 16] = z;
        }
        __syncthreads();
    }

    using S = Stream<F, A, 1, 1, RT, WAY, true>;
    __shared__ __attribute__((aligned(16))) uint8_t ring[W][S::LDS];
    S st(c.inner, c.h, 2 * h_rows(c.t, c.e, c.top) * c.pitch, ring[wave]);
    struct Source : S::Source {
        Buffer scale;
    } src;
    const int per = st.steps, all = per * count;
    const int part = slice * W + wave, parts = slices * W;
    const int lo = uniform((int)((int64_t)all * part / parts)), n = uniform((int)((int64_t)all * (part + 1) / parts)) - lo;
    auto enter = [&](int a) {
        const int expert = uniform(active[a]), rows = uniform(start[a + 1]) - uniform(start[a]), G = uniform(group[a]);
        const int64_t row = (int64_t)expert * c.hidden + n0;
        st.weights(src, 0, c.down.q, c.down.scale, row, c.e * c.hidden);
        if constexpr (!F::kBlockScales)
            src.scale = Buffer(static_cast<const float*>(c.down.scale) + row, 4 * (c.e * c.hidden - row));
        st.rows(src, rows, [&](int i) { return (G + (i < rows ? i / 4 : 0)) * 4 * c.pitch; });
    };
    int la = uniform(lo / per), lp = lo - la * per, ca = la, cp = lp;  // the loads' expert and step, the products'
    // the channels' scales where the expert's sums are added up, after step lp
    auto load_scale = [&](bool on) {
        u32x4 v{0, 0, 0, 0};
        if constexpr (!F::kBlockScales)
            v = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(src.scale.rsrc, 16 * g, src.scale.at(on, 0), 0));
        return v;
    };
    u32x4 scale_bits{0, 0, 0, 0};
    if (n > 0) {
        enter(la);
        scale_bits = load_scale(lp + 1 == per || n == 1);
        st.load(src, lp, true);
    }
    f32x4 acc[1][RT];
#pragma unroll
    for (int u = 0; u < RT; ++u)
        acc[0][u] = f32x4{0.0f};
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const bool more = i + 1 < n;
        if (++lp == per && more) {
            lp = 0;
            enter(++la);
        }
        const u32x4 scale_next = load_scale(more && (lp + 1 == per || i + 2 == n));
        st.consume(cp, src, lp, more, acc);
        if (++cp == per || !more) {
            const int first = uniform(start[ca]), rows = uniform(start[ca + 1]) - first;
            const f32x4 scale = F::kBlockScales ? f32x4{1.0f, 1.0f, 1.0f, 1.0f} : __builtin_bit_cast(f32x4, scale_bits);
            // lane (r, g): channels 4 g .. 4 g + 3 of row r; an expert has a token once
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                if (16 * u + r < rows) {
                    const int row = first + 16 * u + r;
                    f32x4& to = sum[wave][TOKENS == 1 ? 0 : token[row]][g];
                    const f32x4 v = acc[0][u];
                    const float w = weight[row];
                    f32x4 z = to;
                    z.x = __builtin_fmaf(w, scale.x * v.x, z.x);
                    z.y = __builtin_fmaf(w, scale.y * v.y, z.y);
                    z.z = __builtin_fmaf(w, scale.z * v.z, z.z);
                    z.w = __builtin_fmaf(w, scale.w * v.w, z.w);
                    to = z;
                }
                acc[0][u] = f32x4{0.0f};
            }
            wave_sync();
            cp = 0;
            ++ca;
        }
        scale_bits = scale_next;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < (int)c.t * 16; i += NT) {
        const int tok = i / 16, ch = i % 16;
        float z = reinterpret_cast<const float*>(&sum[0][tok][0])[ch];
#pragma unroll
        for (int v = 1; v < W; ++v)
            z += reinterpret_cast<const float*>(&sum[v][tok][0])[ch];
        if (slices > 1)
            __hip_atomic_store(c.parts + (int64_t)blockIdx.x * c.t * 16 + i, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else if (n0 + ch < c.hidden)
            static_cast<uint16_t*>(c.out)[tok * c.hidden + n0 + ch] = rounded<A>(z);
    }
    if (slices == 1)
        return;
    wait_loads_at_most<0>();  // and stores
    __syncthreads();
    if (tid == 0) {
        last = __hip_atomic_fetch_add(&c.arrived[tile], 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT) ==
               (uint32_t)slices - 1;
        if (last)
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    }
    __syncthreads();
    if (!last)
        return;
#pragma unroll 1
    for (int i = tid; i < (int)c.t * 16; i += NT) {
        const float* from = c.parts + (int64_t)tile * slices * c.t * 16 + i;
        float z = 0.0f;
#pragma unroll 4
        for (int v = 0; v < slices; ++v)
            z += __hip_atomic_load(from + v * c.t * 16, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (n0 + i % 16 < c.hidden)
            static_cast<uint16_t*>(c.out)[i / 16 * c.hidden + n0 + i % 16] = rounded<A>(z);
    }
}

// ------------------------------------------------------------------ plans
constexpr int kUpGroups = 1024, kUpWaves = 4, kDownWaves = 8;

// Workgroups to the second launch's 16 channels: one where those alone take most CUs, else up to
// as many as there are CUs for.
int64_t most_slices(int64_t hidden)
{
    const int64_t tiles = output_tiles(hidden);
    return tiles > 160 ? 1 : std::min<int64_t>(8, (256 + tiles - 1) / tiles);
}

template <typename F, typename A, int RC, int W, Way WAY>
hipError_t run_up(const LayerCall& c, hipStream_t stream)
{
    const int64_t TN = (c.inner + 15) / 16, most = most_entries(c.t, c.e, c.top);
    const int64_t items = TN * most;
    return launch(layer_up_kernel<F, A, RC, W, WAY>, dim3((unsigned)(items < kUpGroups ? items : kUpGroups)),
                  dim3(W * kWave), stream, c, TN);
}

template <typename F, typename A, int RC, int W, Way WAY>
hipError_t run_down(const LayerCall& c, hipStream_t stream)
{
    // a wave's share is two steps at least
    const int64_t steps = std::min(c.e, c.t * c.top) * ((c.inner + 2 * F::kUnit - 1) / (2 * F::kUnit));
    const int64_t slices = std::max<int64_t>(1, std::min(most_slices(c.hidden), steps / (2 * W)));
    return launch(layer_down_kernel<F, A, RC, W, WAY>, dim3((unsigned)(output_tiles(c.hidden) * slices)), dim3(W * kWave),
                  stream, c, (int)slices);
}

// How rows of weights and of x lie: LDS takes those at 16-byte boundaries, and scales at
// dwords'.
template <typename F>
Way way_of(const LayerWeights& w, const void* x, int64_t x_bytes, int64_t k)
{
    const uintptr_t rows = reinterpret_cast<uintptr_t>(w.q) | reinterpret_cast<uintptr_t>(x) | (uintptr_t)x_bytes |
                           (uintptr_t)F::row_bytes(k);
    const uintptr_t scales = F::kBlockScales ? reinterpret_cast<uintptr_t>(w.scale) | (uintptr_t)F::row_scales(k) : 0;
    return (rows & 15) == 0 && (scales & 3) == 0 ? Way::LDS : ((rows & 3) == 0 ? Way::ROWS : Way::SHIFTED);
}

template <typename F, typename A, int RC>
hipError_t run_both(const LayerCall& c, hipStream_t stream)
{
    const Way up = way_of<F>(c.up, c.x, 2 * c.hidden, c.hidden), down = way_of<F>(c.down, nullptr, 0, c.inner);
    const hipError_t st = up == Way::LDS    ? run_up<F, A, RC, kUpWaves, Way::LDS>(c, stream)
                          : up == Way::ROWS ? run_up<F, A, RC, kUpWaves, Way::ROWS>(c, stream)
                                            : run_up<F, A, RC, kUpWaves, Way::SHIFTED>(c, stream);
    if (st != hipSuccess)
        return st;
    return down == Way::LDS    ? run_down<F, A, RC, kDownWaves, Way::LDS>(c, stream)
           : down == Way::ROWS ? run_down<F, A, RC, kDownWaves, Way::ROWS>(c, stream)
                               : run_down<F, A, RC, kDownWaves, Way::SHIFTED>(c, stream);
}

template <typename F, typename A>
hipError_t launch_typed(const LayerCall& c, hipStream_t stream)
{
    if (c.t == 1)
        return run_both<F, A, 0>(c, stream);
    return c.t <= 16 ? run_both<F, A, 1>(c, stream) : run_both<F, A, 2>(c, stream);
}

int64_t plan_numbers(int64_t t, int64_t e, int64_t top)
{
    return 2 + 3 * most_entries(t, e, top) + kPlanNumbers * t * top;
}

int64_t h_pitch(int64_t inner)
{
    return (inner + 63) / 64 * 64;
}

}  // namespace

size_t layer_workspace_bytes(int64_t t, int64_t e, int64_t top, int64_t hidden, int64_t inner)
{
    return (size_t)(h_rows(t, e, top) * h_pitch(inner) * 2 +
                    4 * (plan_numbers(t, e, top) +
                         (most_slices(hidden) > 1 ? output_tiles(hidden) * (1 + most_slices(hidden) * t * 16) : 0)));
}

hipError_t launch_layer(LayerCall c, bool fp4, Act act, void* ws, hipStream_t stream)
{
    c.pitch = h_pitch(c.inner);
    c.h = static_cast<uint16_t*>(ws);
    c.plan = reinterpret_cast<int32_t*>(c.h + h_rows(c.t, c.e, c.top) * c.pitch);
    c.arrived = nullptr;
    c.parts = nullptr;
    if (most_slices(c.hidden) > 1) {
        c.arrived = reinterpret_cast<uint32_t*>(c.plan + plan_numbers(c.t, c.e, c.top));
        c.parts = reinterpret_cast<float*>(c.arrived + output_tiles(c.hidden));
    }
    if (fp4)
        return act == Act::BF16 ? launch_typed<Fp4, Bf16>(c, stream) : launch_typed<Fp4, F16>(c, stream);
    return act == Act::BF16 ? launch_typed<E4m3, Bf16>(c, stream) : launch_typed<E4m3, F16>(c, stream);
}

}  // namespace fp8w
