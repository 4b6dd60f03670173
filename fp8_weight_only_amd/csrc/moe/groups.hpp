// Row tiles of ragged groups: which expert and which rows a workgroup's tile is.
#pragma once

#include "device.hpp"

namespace fp8w {

struct RowTile {
    int expert;    // e: rows without an expert (positions from offsets[e] on); -1: no such tile
    int64_t row;   // first position
    int rows;      // 1 .. BM
    int64_t total; // tiles of all groups
};

// Offsets are taken as they are, clamped to 0 .. m and to a group's own start,
// so whatever they hold no row outside the call is touched.
__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t lo, int64_t m)
{
    v = v < lo ? lo : v;
    return v > m ? m : v;
}

// The wave's 64 lanes each take one expert of a run of 64, count its tiles, and
// add them up over the lanes; the caller's `pick(total)` turns the number of all
// tiles into the tile it wants (the same in every lane).
template <int BM, typename F>
__device__ __forceinline__ RowTile find_row_tile(const int32_t* __restrict__ offsets, int e, int64_t m, F pick)
{
    const int lane = threadIdx.x & (kWave - 1);
    auto tiles_at = [&](int i, int64_t& lo, int64_t& rows) {
        lo = rows = 0;
        if (i <= e) {
            lo = clamp_row(offsets[i], 0, m);
            const int64_t hi = i < e ? clamp_row(offsets[i + 1], lo, m) : m;
            rows = hi - lo;
        }
        return (int)((rows + BM - 1) / BM);
    };
    int64_t total = 0;
    for (int base = 0; base <= e; base += kWave) {
        int64_t lo, rows;
        int c = tiles_at(base + lane, lo, rows);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            c += __shfl_xor(c, off, kWave);
        total += c;
    }
    RowTile r{-1, 0, 0, total};
    const int64_t want = pick(total);
    if (want < 0 || want >= total)
        return r;
    int64_t run = 0;
    for (int base = 0; base <= e; base += kWave) {
        int64_t lo, rows;
        const int own = tiles_at(base + lane, lo, rows);
        int incl = own;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int v = __shfl_up(incl, off, kWave);
            incl += lane >= off ? v : 0;
        }
        const uint64_t past = __ballot(run + incl > want);
        if (past) {
            const int w = (int)__builtin_ctzll(past);
            const int64_t first = (want - run - (__shfl(incl, w, kWave) - __shfl(own, w, kWave))) * BM;
            r.expert = base + w;
            r.row = __shfl(lo, w, kWave) + first;
            const int64_t left = __shfl(rows, w, kWave) - first;
            r.rows = (int)(left < BM ? left : BM);
            return r;
        }
        run += __shfl(incl, kWave - 1, kWave);
    }
    return r;
}

}  // namespace fp8w
