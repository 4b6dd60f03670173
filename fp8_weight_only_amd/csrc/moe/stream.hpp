// Products of few rows: weights straight from memory into the matrix cores'
// operand registers, for e4m3 and for 4-bit codes.
//
// v_mfma_f32_16x16x32 wants row lane % 16 in a lane, so four neighbouring lanes hold
// four rows. Loaded that way a 16-byte load touches four cache lines per quad of lanes
// and takes 65 cycles of its CU's address unit, 16 bytes a cycle, whatever the caches
// hold; where a quad's lanes read 64 consecutive bytes it takes 17. 4-bit weights with
// their scales and activations are bound by that. So aligned weights go through LDS
// (LdsStream: loaded row by row, read as operands); rows that direct loads into LDS
// cannot take, and calls too small for it to matter, are loaded as they are used
// (RowStream).
//
// Both hold one step of k in flight while the one before is multiplied; a step may be
// another expert's, or another tile's of channels. Which k meet in one instruction does
// not matter as long as both operands agree.
#pragma once

#include <type_traits>

#include "../ring.hpp"
#include "fp4.hpp"
#include "offset.hpp"

namespace fp8w {

struct E4m3 {
    static constexpr bool kBlockScales = false;
    static constexpr int kUnit = 64;  // k of 64 bytes of a row: a 16-byte chunk in each of the four groups of 16 lanes
    __host__ __device__ static int64_t row_bytes(int64_t k) { return k; }
    __host__ __device__ static int64_t row_scales(int64_t) { return 1; }
    // eight of a chunk's weights
    template <typename A>
    __device__ __forceinline__ static u32x4 values(u32x4 v, int part, float)
    {
        const u32x2 a = A::decode4(part ? v.z : v.x), b = A::decode4(part ? v.w : v.y);
        return u32x4{a.x, a.y, b.x, b.y};
    }
    // a chunk's first n weights
    __device__ __forceinline__ static u32x4 first(u32x4 v, int n);
};

struct Fp4 {
    static constexpr bool kBlockScales = true;  // a chunk is one block
    static constexpr int kUnit = 128;
    __host__ __device__ static int64_t row_bytes(int64_t k) { return (k + 1) / 2; }
    __host__ __device__ static int64_t row_scales(int64_t k) { return (k + 31) / 32; }
    template <typename A>
    __device__ __forceinline__ static u32x4 values(u32x4 v, int part, float scale)
    {
        return decode_fp4<A>(part == 0 ? v.x : (part == 1 ? v.y : (part == 2 ? v.z : v.w)), scale);
    }
    __device__ __forceinline__ static u32x4 first(u32x4 v, int n) { return first_codes(v, n); }
};

// A buffer for loads that are the same in all lanes but for a 32-bit offset: reads
// past its end give zeros and touch no memory (each dword for itself, measured too),
// as long as their scalar offset is not past it (offset.hpp).
struct Buffer {
    __amdgpu_buffer_rsrc_t rsrc;  // from the dword boundary at or before the data
    int bytes, rest;              // the data start `rest` behind it

    Buffer() = default;
    __device__ __forceinline__ Buffer(const void* p, int64_t size)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(uniform(p));
        rest = (int)(at & 3);
        // whole dwords, up to the one that holds the last byte
        const int64_t all = size > 0 ? (size + rest + 3) & ~(int64_t)3 : 0;
        bytes = all < 0x70000000 ? (int)all : 0x70000000;  // offsets past it stay ints
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at - rest), 0, bytes, 0x00020000);
    }
    // the scalar offset of a load: the end when it is not on
    __device__ __forceinline__ int at(bool on, int off) const { return buffer_offset(on, off, bytes); }
    __device__ __forceinline__ int at(bool on, int off, int row, int row_bytes) const
    {
        return buffer_offset(on, off, row, row_bytes, bytes);
    }
};

// The first n bytes of 16 (n <= 0: none).
__device__ __forceinline__ u32x4 first_bytes(u32x4 v, int n)
{
    uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = n - 4 * i;
        d[i] = m >= 4 ? d[i] : (m > 0 ? d[i] & ((1u << (8 * m)) - 1) : 0);
    }
    return u32x4{d[0], d[1], d[2], d[3]};
}

__device__ __forceinline__ u32x4 E4m3::first(u32x4 v, int n)
{
    return first_bytes(v, n);
}

// NT tiles of 16 weight rows, in NB buffers of as many each, times RC tiles of 16
// activation rows, from any byte on (SHIFT), else from dwords. lane % 16 is a lane's row.
//
// Rows at any byte come as the dwords that hold them, put together by byte shifts. The dword
// behind a lane's 16 bytes is the first of the lane's that has the next 16, and only the
// step's last is loaded by itself: a load of a dword costs the address unit as much as one of 16 bytes
// (13 tokens over 60 e4m3 experts of [1026, 1030] and [1030, 513]: 17.8 and 25.8 us, with a load each
// 20.1 and 28.0).
//
// X4: x is kept in groups of four rows, eight values of each in turn, as the layer's
// second launch reads what its first wrote: a quad's lanes then read 64 consecutive
// bytes as they are.
//
// A step of K is in registers; consume() takes it out and requests the next. Loads
// that are not on give zeros.
template <typename F, typename A, int NT, int NB, int RC, bool SHIFT, bool X4>
struct RowStream {
    static constexpr int TILES = NT / NB, U = 2, K = U * F::kUnit, P = F::kUnit / 32, LDS = 16;
    static_assert(NT % NB == 0, "as many tiles in each buffer");
    int64_t k;
    int steps;  // those of k, a masked one among them
    int r, g;
    int woff[TILES], soff[TILES];
    Buffer x;

    // Where a step's operands come from: the codes and scales from a weight row on, and
    // this lane's rows of x. The same in all lanes but for xoff.
    struct Source {
        Buffer w[NB], s[NB];
        int xoff[RC];
        bool xon[RC];  // some row of this tile is wanted
    };
    static constexpr bool XSHIFT = SHIFT && !X4;
    u32x4 w[NT][U], xs[RC][U][P];
    uint32_t wshift[SHIFT ? NT : 0], wlast[SHIFT ? NT : 0], xshift[XSHIFT ? RC : 0], xlast[XSHIFT ? RC : 0];
    uint8_t s[F::kBlockScales ? NT : 0][U];

    __device__ __forceinline__ RowStream(int64_t k_, const void* x_, int64_t x_bytes, uint8_t*) : k(k_), x(x_, x_bytes)
    {
        steps = (int)((k + K - 1) / K);
        r = threadIdx.x & 15;
        g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            woff[t] = (16 * t + r) * (int)F::row_bytes(k) + 16 * g;
            soff[t] = (16 * t + r) * (int)F::row_scales(k) + g;
        }
    }
    // Buffer i: from weight row `row` of `rows`. Rows past the last give zeros or others'
    // values, for channels that are not stored.
    __device__ __forceinline__ void weights(Source& src, int i, const uint8_t* q, const void* scale, int64_t row,
                                            int64_t rows) const
    {
        src.w[i] = Buffer(q + row * F::row_bytes(k), (rows - row) * F::row_bytes(k));
        if constexpr (F::kBlockScales)
            src.s[i] = Buffer(static_cast<const uint8_t*>(scale) + row * F::row_scales(k),
                              (rows - row) * F::row_scales(k));
    }
    // The rows of x: at(i) is the first value of row i of the tiles (X4: of the group of
    // four that it is in); the first `rows` are wanted.
    template <typename Fn>
    __device__ __forceinline__ void rows(Source& src, int rows, Fn&& at) const
    {
#pragma unroll
        for (int u = 0; u < RC; ++u) {
            src.xon[u] = 16 * u < rows;
            src.xoff[u] = (int)(2 * at(16 * u + r)) + (X4 ? 8 : 2) * (F::kUnit / 4) * g + (X4 ? 16 * (r & 3) : 0);
        }
    }
    __device__ __forceinline__ void load(const Source& src, int step, bool on)
    {
        constexpr int BY = X4 ? 8 : 2;
        if constexpr (F::kBlockScales)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < U; ++h) {
                    const Buffer& of = src.s[t / TILES];
                    s[t][h] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(of.rsrc, soff[t % TILES] + of.rest + 4 * h,
                                                                           of.at(on, 4 * U * step), 0);
                }
        auto load16 = [](const Buffer& from, int off, int scalar_off) {
            return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from.rsrc, off, scalar_off, 0));
        };
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const Buffer& from = src.w[t / TILES];
            int off = woff[t % TILES];
            const int at = from.at(on, 64 * U * step);
            if constexpr (SHIFT) {
                off += from.rest;
                wshift[t] = (uint32_t)off & 3u;
                off -= (int)wshift[t];
                wlast[t] = 0;
                if (g == 3)
                    wlast[t] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(from.rsrc, off + 64 * (U - 1) + 16, at, 0);
            }
#pragma unroll
            for (int h = 0; h < U; ++h)
                w[t][h] = load16(from, off + 64 * h, at);
        }
#pragma unroll
        for (int u = 0; u < RC; ++u) {
            int off = src.xoff[u];
            const int at = x.at(on && src.xon[u], BY * K * step);
            if constexpr (XSHIFT) {
                off += x.rest;
                xshift[u] = (uint32_t)off & 3u;
                off -= (int)xshift[u];
                xlast[u] = 0;
                if (g == 3)
                    xlast[u] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
                        x.rsrc, off + BY * F::kUnit * (U - 1) + 16 * P, at, 0);
            }
#pragma unroll
            for (int h = 0; h < U; ++h)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    xs[u][h][p] = load16(x, off + BY * (F::kUnit * h + 8 * p), at);
        }
    }
    // The dword behind each unit's bytes of this lane: first[h] is the unit's first, last the one behind the step.
    __device__ __forceinline__ void behind(const uint32_t (&first)[U], uint32_t last, uint32_t (&e)[U]) const
    {
        const int from = 4 * ((int)(threadIdx.x + 16) & 63);
#pragma unroll
        for (int h = 0; h < U; ++h) {
            const uint32_t give = g == 0 && h + 1 < U ? first[h + 1 < U ? h + 1 : h] : first[h];
            const uint32_t got = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)give);
            e[h] = g == 3 && h + 1 == U ? last : got;
        }
    }
    __device__ __forceinline__ static u32x4 shifted(u32x4 v, uint32_t e, uint32_t by)
    {
        return u32x4{__builtin_amdgcn_alignbyte(v.y, v.x, by), __builtin_amdgcn_alignbyte(v.z, v.y, by),
                     __builtin_amdgcn_alignbyte(v.w, v.z, by), __builtin_amdgcn_alignbyte(e, v.w, by)};
    }
    // Adds the loaded step's products, step `step` of k, and loads step `next` of src.
    __device__ __forceinline__ void consume(int step, const Source& src, int next, bool on, f32x4 (&acc)[NT][RC])
    {
        u32x4 v[NT][U], xv[RC][U][P];
        float scale[NT][U];
#pragma unroll
        for (int h = 0; h < U; ++h) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                v[t][h] = w[t][h];
                scale[t][h] = 1.0f;
                if constexpr (F::kBlockScales)
                    scale[t][h] = fp4_scale(s[t][h]);
            }
#pragma unroll
            for (int u = 0; u < RC; ++u)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    xv[u][h][p] = xs[u][h][p];
        }
        if constexpr (SHIFT)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t first[U], e[U];
#pragma unroll
                for (int h = 0; h < U; ++h)
                    first[h] = v[t][h].x;
                behind(first, wlast[t], e);
#pragma unroll
                for (int h = 0; h < U; ++h)
                    v[t][h] = shifted(v[t][h], e[h], wshift[t]);
            }
        if constexpr (XSHIFT)
#pragma unroll
            for (int u = 0; u < RC; ++u) {
                uint32_t first[U], e[U];
#pragma unroll
                for (int h = 0; h < U; ++h)
                    first[h] = xv[u][h][0].x;
                behind(first, xlast[u], e);
#pragma unroll
                for (int h = 0; h < U; ++h)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint32_t next_dword = p + 1 < P ? xv[u][h][p + 1 < P ? p + 1 : p].x : e[h];
                        xv[u][h][p] = shifted(xv[u][h][p], next_dword, xshift[u]);
                    }
            }
        load(src, next, on);
        if ((int64_t)K * (step + 1) > k) {  // what lies behind a row's end is the next row's
#pragma unroll
            for (int h = 0; h < U; ++h) {
                const int left = (int)(k - (int64_t)K * step) - F::kUnit * h - F::kUnit / 4 * g;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    v[t][h] = F::first(v[t][h], left);
                    scale[t][h] = left > 0 ? scale[t][h] : 1.0f;
                }
#pragma unroll
                for (int u = 0; u < RC; ++u)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        xv[u][h][p] = first_bytes(xv[u][h][p], 2 * left - 16 * p);
            }
        }
#pragma unroll
        for (int h = 0; h < U; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 a = F::template values<A>(v[t][h], p, scale[t][h]);
#pragma unroll
                    for (int u = 0; u < RC; ++u)
                        acc[t][u] = A::mfma(a, xv[u][h][p], acc[t][u]);
                }
    }
};

// The same on rows at 16-byte boundaries (scales at dwords'), which go through LDS by
// direct loads, four rows of 256 bytes each, and come out as operands: no registers for
// what is in flight, and no transposes.
//
// In LDS a weight row has its 16 chunks of 16 bytes in the place (chunk / 4 + row) % 4,
// within it (chunk ^ row / 4) % 4: the 16 lanes of a read's phase, 16 rows and the same
// chunk, then meet all banks once, and a quad of a load stays in its 64 bytes.
//
// A step's weights are taken into registers when its turn comes, so its place takes the
// next step's. The activations come as they are needed, lane % 16 their row (X4: as
// above): a quad's four rows are four lines then, shared by NT tiles of weights.
template <typename F, typename A, int NT, int NB, int RC, bool X4>
struct LdsStream {
    static constexpr int TILES = NT / NB, UNIT = F::kUnit, K = 4 * UNIT, P = UNIT / 32;
    static constexpr int WBYTES = NT * 4096, LDS = WBYTES + (F::kBlockScales ? NT * 256 : 0);  // of a wave
    static_assert(NT % NB == 0, "as many tiles in each buffer");
    int64_t k;
    int steps, row_bytes, row_scales;
    int r, g;
    int woff, soff;  // this lane's part of a load, rows 0 .. 3
    uint8_t* lds;
    Buffer x;

    struct Source {
        Buffer w[NB], s[NB];
        int xoff[RC];
        bool xon[RC];
    };
    u32x4 xs[RC][4][P];

    __device__ __forceinline__ LdsStream(int64_t k_, const void* x_, int64_t x_bytes, uint8_t* lds_)
        : k(k_), lds(lds_), x(x_, x_bytes)
    {
        const int lane = threadIdx.x & 63;
        steps = (int)((k + K - 1) / K);
        row_bytes = (int)F::row_bytes(k);
        row_scales = (int)F::row_scales(k);
        r = lane & 15;
        g = lane >> 4;
        woff = g * row_bytes;
        soff = (lane >> 2) * row_scales + 4 * (lane & 3);
    }
    __device__ __forceinline__ void weights(Source& src, int i, const uint8_t* q, const void* scale, int64_t row,
                                            int64_t rows) const
    {
        src.w[i] = Buffer(q + row * F::row_bytes(k), (rows - row) * F::row_bytes(k));
        if constexpr (F::kBlockScales)
            src.s[i] = Buffer(static_cast<const uint8_t*>(scale) + row * F::row_scales(k),
                              (rows - row) * F::row_scales(k));
    }
    template <typename Fn>
    __device__ __forceinline__ void rows(Source& src, int rows, Fn&& at) const
    {
#pragma unroll
        for (int u = 0; u < RC; ++u) {
            src.xon[u] = 16 * u < rows;
            src.xoff[u] = (int)(2 * at(16 * u + r)) + (X4 ? 8 : 2) * (UNIT / 4) * g + (X4 ? 16 * (r & 3) : 0);
        }
    }
    // Rows 4 q .. 4 q + 3 of every tile, and their scales. Nothing moves across the empty
    // statements: the wait in consume() counts what is requested behind these.
    __device__ __forceinline__ void load_weights(const Source& src, int step, bool on) const
    {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const Buffer& from = src.w[t / TILES];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // lane: row 4 q + g, place r
                const int chunk = 4 * ((r / 4 - g) & 3) + ((r ^ q) & 3);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from.rsrc, FP8W_LDS(lds + 4096 * t + 1024 * q), 16,
                                                         woff + 16 * chunk,
                                                         from.at(on, 256 * step, 16 * (t % TILES) + 4 * q, row_bytes), 0, 0);
            }
        }
        if constexpr (F::kBlockScales)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const Buffer& of = src.s[t / TILES];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(of.rsrc, FP8W_LDS(lds + WBYTES + 256 * t), 4, soff,
                                                         of.at(on, 16 * step, 16 * (t % TILES), row_scales), 0, 0);
            }
        asm volatile("" ::: "memory");
    }
    __device__ __forceinline__ void load_x(const Source& src, int j, int step, bool on)
    {
        constexpr int BY = X4 ? 8 : 2;
#pragma unroll
        for (int u = 0; u < RC; ++u)
#pragma unroll
            for (int p = 0; p < P; ++p)
                xs[u][j][p] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(x.rsrc, src.xoff[u] + BY * (UNIT * j + 8 * p),
                                                                 x.at(on && src.xon[u], BY * K * step), 0));
    }
    __device__ __forceinline__ void load(const Source& src, int step, bool on)
    {
        load_weights(src, step, on);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            load_x(src, j, step, on);
    }
    __device__ __forceinline__ void consume(int step, const Source& src, int next, bool on,
                                            f32x4 (&acc)[NT][RC])
    {
        // behind this step's weights its activations were requested, 4 P RC loads
        asm volatile("" ::: "memory");
        wait_loads_at_most<4 * P * RC>();
        u32x4 chunk[NT][4], scales[NT];
        const uint32_t base = (uint32_t)reinterpret_cast<uintptr_t>(FP8W_LDS(lds));
        const uint32_t row = base + 256 * r + 16 * ((g ^ (r >> 2)) & 3);
        const uint32_t a0 = row + 64 * (r & 3), a1 = row + 64 * ((r + 1) & 3), a2 = row + 64 * ((r + 2) & 3),
                       a3 = row + 64 * ((r + 3) & 3);
        // in assembly: the compiler would wait for every load into LDS before a read of it
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (F::kBlockScales)
                asm volatile("ds_read_b128 %0, %5 offset:%10\n\tds_read_b128 %1, %6 offset:%10\n\t"
                             "ds_read_b128 %2, %7 offset:%10\n\tds_read_b128 %3, %8 offset:%10\n\t"
                             "ds_read_b128 %4, %9 offset:%11\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(chunk[t][0]), "=&v"(chunk[t][1]), "=&v"(chunk[t][2]), "=&v"(chunk[t][3]),
                               "=&v"(scales[t])
                             : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "v"(base + 16 * r), "n"(4096 * t),
                               "n"(WBYTES + 256 * t)
                             : "memory");
            else
                asm volatile("ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
                             "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\t"
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(chunk[t][0]), "=&v"(chunk[t][1]), "=&v"(chunk[t][2]), "=&v"(chunk[t][3])
                             : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(4096 * t)
                             : "memory");
        }
        load_weights(src, next, on);
        const bool masked = (int64_t)K * (step + 1) > k;  // what lies behind a row's end is the next row's
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 xv[RC][P], v[NT];
            float scale[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                v[t] = chunk[t][j];
                scale[t] = 1.0f;
                if constexpr (F::kBlockScales) {
                    const u32x4 s = scales[t];
                    scale[t] = fp4_scale(((j == 0 ? s.x : (j == 1 ? s.y : (j == 2 ? s.z : s.w))) >> (8 * g)) & 255u);
                }
            }
#pragma unroll
            for (int u = 0; u < RC; ++u)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    xv[u][p] = xs[u][j][p];
            if (masked) {
                const int left = (int)(k - (int64_t)K * step) - UNIT * j - UNIT / 4 * g;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    v[t] = F::first(v[t], left);
                    scale[t] = left > 0 ? scale[t] : 1.0f;
                }
#pragma unroll
                for (int u = 0; u < RC; ++u)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        xv[u][p] = first_bytes(xv[u][p], 2 * left - 16 * p);
            }
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 w = F::template values<A>(v[t], p, scale[t]);
#pragma unroll
                    for (int u = 0; u < RC; ++u)
                        acc[t][u] = A::mfma(w, xv[u][p], acc[t][u]);
                }
            load_x(src, j, next, on);
        }
    }
};

// How a call's rows lie.
enum class Way { LDS, ROWS, SHIFTED };

template <typename F, typename A, int NT, int NB, int RC, Way WAY, bool X4>
using Stream = std::conditional_t<WAY == Way::LDS, LdsStream<F, A, NT, NB, RC, X4>,
                                  RowStream<F, A, NT, NB, RC, WAY == Way::SHIFTED, X4>>;

}  // namespace fp8w
