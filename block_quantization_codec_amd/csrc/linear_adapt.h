// linear_adapt.h - what a row's low-rank adapter adds to a product on block codes.
//
//   y[m][n]  += sum_r low[m][r] B[g][n][r]     low = s_g x A_g^T
//   dx[m][k] += sum_r low[m][r] A[g][r][k]     low = s_g dy B_g         g = ids[m]
//
// The product's own kernels add it to their sums, before the result's one rounding:
// a pass of its own would read and write the result again, and round it twice.
//
// Rows of a tile may have different adapters. In tiles of many rows up to four bf16
// adapters are multiplied in turn, low set to zero in the rows that have another. Zero
// times an infinity or a NaN is a NaN, so each adapter's elements are looked at as they are
// loaded: if one that only some of the tile's rows have holds such an element in the
// wave's columns, and in tiles of more adapters, of binary32 ones or of few rows, the
// rows of each adapter are gathered and multiplied by themselves. So nothing of an adapter
// reaches another's rows. (Nor does a sum that overflows: it is its own row's.)
//
// Precision: low is binary32 and enters as bf16 parts, like binary32 activations:
// two of them where the product takes activations and weights as one each, from bf16 to bf16
// (16 bits: the first leaves less than 2^-7 of low, and the second's rounding at most 2^-16 of it,
// against the 2^-8 of a bf16 result), three otherwise; a bf16 adapter is one part, a binary32 one three.
#pragma once

#include "linear_device.h"

namespace zpp {

typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// Two values as P bf16 pairs; of two parts, the first is cut off (which cannot
// overflow) and the second rounded (NaN beside an infinite first).
template <int P>
__device__ __forceinline__ void low_parts(float a, float b, uint32_t (&w)[P]) {
    if constexpr (P == 2) {
        w[0] = pack_hi(a, b);
        w[1] = pack_rn(a - as_f(w[0] << 16), b - as_f(w[0] & 0xFFFF0000u));
    } else {
        to_parts<P>(a, b, w);
    }
}

// Eight binary32 values as parts of an operand.
template <int P>
__device__ __forceinline__ void operand_of(const float (&v)[8], u32x4 (&a)[P]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t w[P];
        low_parts<P>(v[2 * d], v[2 * d + 1], w);
#pragma unroll
        for (int x = 0; x < P; ++x) a[x][d] = w[x];
    }
}

// Whether row `row` has an adapter, and which.
__device__ __forceinline__ bool adapter_of(const LinArgs &p, int64_t row, int &id) {
    id = p.ids ? p.ids[min(row, p.rows - 1)] : 0;
    return row < p.rows && static_cast<uint32_t>(id) < static_cast<uint32_t>(p.adapters);
}

// Indices r .. r + 7 of a row of low: any of the row's past the rank.
__device__ __forceinline__ void load_low(const LinArgs &p, int64_t row, int r, f32x4 (&v)[2]) {
    const float *from = p.low + min(row, p.rows - 1) * p.rank + min(r, p.rank - 8);
    v[0] = ld<f32x4>(from), v[1] = ld<f32x4>(from + 4);
}

// As operand parts: zeros unless `in`.
template <int P>
__device__ __forceinline__ void low_operand(const f32x4 (&v)[2], bool in, u32x4 (&a)[P]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = in ? v[i / 4][i % 4] : 0.0f;
    operand_of<P>(f, a);
}

// The adapter's operands for NT tiles of columns, indices r .. r + 7: zeros past
// the rank. Tile t's column is col + t (NEAR) or col + 16 t.
template <bool GRAD, bool NEAR, int PB, int NT>
__device__ __forceinline__ void load_up(const LinArgs &p, int64_t g, int64_t col, int r, u32x4 (&b)[NT][PB]) {
    const bool in = r < p.rank;
    if constexpr (GRAD) {  // [rank][in]: four neighbouring columns of eight rows, turned
        static_assert(NEAR && NT == 4);
        const int64_t c = min(col, p.n_in - 4), base = (g * p.rank + min(r, p.rank - 8)) * p.n_in + c;
        if constexpr (PB == 3) {
            f32x4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = ld<f32x4>(static_cast<const float *>(p.up) + base + i * p.n_in);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float o[8] = {v[0][t], v[1][t], v[2][t], v[3][t], v[4][t], v[5][t], v[6][t], v[7][t]};
                operand_of<PB>(o, b[t]);
            }
        } else {
            u32x2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = ld<u32x2>(static_cast<const uint16_t *>(p.up) + base + i * p.n_in);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    b[t][0][d] = __builtin_amdgcn_perm(v[2 * d + 1][t / 2], v[2 * d][t / 2],
                                                       t % 2 == 0 ? 0x05040100u : 0x07060302u);
        }
    } else {  // [out][rank]
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t c = min(col + (NEAR ? t : 16 * t), p.n_out - 1);
            const int64_t base = (g * p.n_out + c) * p.rank + min(r, p.rank - 8);
            if constexpr (PB == 3) {
                const float *from = static_cast<const float *>(p.up) + base;
                const f32x4 x = ld<f32x4>(from), y = ld<f32x4>(from + 4);
                const float o[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                operand_of<PB>(o, b[t]);
            } else {
                b[t][0] = ld<u32x4>(static_cast<const uint16_t *>(p.up) + base);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < PB; ++x)
#pragma unroll
            for (int d = 0; d < 4; ++d) b[t][x][d] = in ? b[t][x][d] : 0u;
}

// The numbers of match's set bits, in order, one a lane: lane n has the n-th's. They move
// between lanes without memory: one more array in LDS, and the compiler would wait in the
// tiled products' loops for all of the loads into theirs (twice the time).
__device__ __forceinline__ int list_bits(uint64_t match) {
    const int lane = threadIdx.x & (kWave - 1);
    const uint64_t below = (1ull << lane) - 1;
    // the other lanes' numbers go behind: every lane sends, and every lane gets one
    const int at = match >> lane & 1 ? __popcll(match & below) : __popcll(match) + __popcll(~match & below);
    return __builtin_amdgcn_ds_permute(at * 4, lane);
}

// Entry n of such a list, n of the lane's own.
__device__ __forceinline__ int listed(int list, int n) { return __builtin_amdgcn_ds_bpermute(n * 4, list); }

// What ROWS (up to 64) rows from `row0` on get from their adapters in the wave's NT
// tiles of columns, into LDS of the wave's own: held[row][columns], 16 NT a row, tile
// t's at 16 t + (lane & 15), or, NEAR, at 4 (lane & 15) + t. Rows without an adapter get
// zeros. Of the rows' adapters, in the order of their first rows, it takes every
// `parts`-th from `part` on; the others' rows get zeros too.
//
// The rows of an adapter, wherever they stand, are the matrix instruction's rows. NB
// adapters at a time: their operands' loads, each a trip to memory where every row
// has an adapter of its own, are under way together, S steps of 32 ranks of each. One by one, 48 rows of 28672 x
// 8192 with 32 adapters of rank 64 took 75 us more than without adapters.
template <bool GRAD, bool NEAR, int PC, int PB, int NT, int ROWS, int NB, int S>
__device__ __forceinline__ void adapter_gather(const LinArgs &p, int64_t row0, int64_t col, int part, int parts,
                                               float *held) {
    static_assert(ROWS <= kWave && ROWS % 16 == 0);
    const int lane = threadIdx.x & (kWave - 1), q = lane >> 4, j = lane & 15;
#pragma unroll
    for (int i = 0; i < ROWS * NT / 16; ++i)
        reinterpret_cast<f32x4 *>(held)[i * kWave + lane] = f32x4{0, 0, 0, 0};
    int id;
    const bool has = adapter_of(p, row0 + lane, id) && lane < ROWS;
    uint64_t pending = __ballot(has);
    int n = 0;
    while (pending != 0) {
        int g[NB], count[NB], list[NB], most = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            g[b] = b == 0 ? 0 : g[0];
            count[b] = list[b] = 0;
            while (pending != 0 && count[b] == 0) {
                const int c = __builtin_amdgcn_readlane(id, __builtin_ctzll(pending));
                const uint64_t match = __ballot(has && id == c);
                pending &= ~match;
                if (n++ % parts != part) continue;
                g[b] = c;
                count[b] = __popcll(match);
                list[b] = list_bits(match);
            }
            most = max(most, count[b]);
        }
        for (int l0 = 0; l0 < most; l0 += 16) {
            int64_t row[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
                row[b] = row0 + listed(list[b], l0 + j < count[b] ? l0 + j : 0);
            f32x4 e[NB][NT];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t) e[b][t] = f32x4{0, 0, 0, 0};
            for (int r0 = 0; r0 < p.rank; r0 += 32 * S) {
                f32x4 low[S][NB][2];
                u32x4 up[S][NB][NT][PB];
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        load_up<GRAD, NEAR, PB, NT>(p, g[b], col, r0 + 32 * s + 8 * q, up[s][b]);
                        load_low(p, row[b], r0 + 32 * s + 8 * q, low[s][b]);
                    }
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        u32x4 a[PC];
                        low_operand<PC>(low[s][b], r0 + 32 * s + 8 * q < p.rank, a);
#pragma unroll
                        for (int t = 0; t < NT; ++t) e[b][t] = mfma_parts<PC, PB>(a, up[s][b][t], e[b][t]);
                    }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = l0 + 4 * q + i, to_row = listed(list[b], at & (kWave - 1));
                    if (at >= count[b]) continue;
                    float *to = held + to_row * (16 * NT);
                    if constexpr (NEAR) {
                        static_assert(NT == 4);
                        *reinterpret_cast<f32x4 *>(to + 4 * j) = f32x4{e[b][0][i], e[b][1][i], e[b][2][i], e[b][3][i]};
                    } else {
#pragma unroll
                        for (int t = 0; t < NT; ++t) to[16 * t + j] = e[b][t][i];
                    }
                }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <bool GRAD, bool NEAR, int PC, int NT, int ROWS, int NB, int S>
__device__ __forceinline__ void adapter_rows(const LinArgs &p, int64_t row0, int64_t col, int part, int parts,
                                             float *held) {
    if (p.up_f32)  // three parts each: half as many at a time fit
        adapter_gather<GRAD, NEAR, 3, 3, NT, ROWS, (NB + 1) / 2, 1>(p, row0, col, part, parts, held);
    else
        adapter_gather<GRAD, NEAR, PC, 1, NT, ROWS, NB, S>(p, row0, col, part, parts, held);
}

// low[m][r .. r + 7] . B[g][n][r .. r + 7] of one result, by one lane; zero past the rank.
struct AdapterPiece {
    f32x4 low[2];
    u32x4 up[2];

    __device__ __forceinline__ void load(const LinArgs &p, int64_t g, int64_t row, int64_t col, int r) {
        const float *from = p.low + row * p.rank + r;
        low[0] = ld<f32x4>(from), low[1] = ld<f32x4>(from + 4);
        const int64_t base = (g * p.n_out + col) * p.rank + r;
        if (p.up_f32) {
            const float *b = static_cast<const float *>(p.up) + base;
            up[0] = ld<u32x4>(b), up[1] = ld<u32x4>(b + 4);
        } else {
            up[0] = ld<u32x4>(static_cast<const uint16_t *>(p.up) + base);
        }
    }

    __device__ __forceinline__ float dot(const LinArgs &p) const {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float b = p.up_f32 ? as_f(up[i / 4][i % 4]) : i % 2 == 0 ? bf16_lo(up[0][i / 2]) : bf16_hi(up[0][i / 2]);
            v = __builtin_fmaf(low[i / 4][i % 4], b, v);
        }
        return v;
    }
};

}  // namespace zpp
