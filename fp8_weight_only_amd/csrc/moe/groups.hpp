// Row tiles of ragged groups: which expert and which rows a workgroup's tile is.
#pragma once

#include "device.hpp"

namespace fp8w {

struct RowTile {
    int expert;  // e: rows without an expert (positions from offsets[e] on); -1: no such tile
    int row;     // first position
    int rows;    // 1 .. BM
};

__device__ __forceinline__ int clamp_row(int v, int lo, int m)
{
    v = v < lo ? lo : v;
    return v > m ? m : v;
}

// Sum of v over this lane and those below it: DPP shifts within rows of 16
// lanes, then row totals broadcast upwards. Six dependent vector instructions;
// the same through LDS permutes took about a microsecond per tile lookup.
__device__ __forceinline__ int wave_prefix(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
    return v;
}

// Finds row tiles from the offsets, one wave at a time (every wave of a
// workgroup does the same). Group i < e has rows offsets[i] .. offsets[i + 1],
// group e the rows from offsets[e] to m. Offsets are taken clamped to 0 .. m and
// to their group's start, so whatever they hold no row outside the call is
// touched. Lane l holds groups 64 c + l of four runs c at once, whose loads are
// in flight together (e <= 255: the offsets are read once, in one trip).
template <int BM>
struct TileFinder {
    static constexpr int C = 4;
    const int* offsets;
    int e, m;
    int lo[C], rows[C], incl[C];

    __device__ __forceinline__ TileFinder(const int32_t* o, int e_, int m_) : offsets(o), e(e_), m(m_)
    {
        load(0);
    }

    __device__ __forceinline__ void load(int base)
    {
        const int lane = threadIdx.x & (kWave - 1);
        int a[C], b[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = base + 64 * c + lane;
            a[c] = offsets[i < e ? i : e];
            b[c] = offsets[i + 1 < e ? i + 1 : e];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = base + 64 * c + lane;
            lo[c] = clamp_row(a[c], 0, m);
            const int hi = i < e ? clamp_row(b[c], lo[c], m) : m;
            rows[c] = i <= e ? hi - lo[c] : 0;
            incl[c] = wave_prefix((rows[c] + BM - 1) / BM);
        }
    }

    __device__ __forceinline__ int run_total(int c) const { return __builtin_amdgcn_readlane(incl[c], 63); }

    // Tiles of all groups (the same in every lane).
    __device__ __forceinline__ int total()
    {
        int t = 0;
        for (int base = 0;; base += 64 * C) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                t += run_total(c);
            if (base + 64 * C > e)
                break;
            load(base + 64 * C);
        }
        if (e >= 64 * C)
            load(0);
        return t;
    }

    __device__ __forceinline__ RowTile find(int want)
    {
        RowTile r{-1, 0, 0};
        for (int base = 0;; base += 64 * C) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint64_t past = __ballot(incl[c] > want);
                if (past) {
                    const int w = (int)__builtin_ctzll(past);
                    const int all = __builtin_amdgcn_readlane(rows[c], w);
                    const int before = __builtin_amdgcn_readlane(incl[c], w) - (all + BM - 1) / BM;
                    const int first = (want - before) * BM;
                    r.expert = base + 64 * c + w;
                    r.row = __builtin_amdgcn_readlane(lo[c], w) + first;
                    r.rows = all - first < BM ? all - first : BM;
                    return r;
                }
                want -= run_total(c);
            }
            if (base + 64 * C > e)
                return r;
            load(base + 64 * C);
        }
    }
};

}  // namespace fp8w
