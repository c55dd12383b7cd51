// linear_tile.h - y = x W^T and dx = dy W on block codes, many rows at once:
// a tiled matrix product that converts the codes in registers.
//
//   y[m][n]  = sum_k x[m][k]  W[n][k]      (contraction over in_features)
//   dx[m][k] = sum_n dy[m][n] W[n][k]      (contraction over out_features)
//   W[n][k]  = code[n*K + k] * s[(n*K + k) / B]
//
// A workgroup of 4 waves computes 16*MT rows x 256 columns; each wave has 64
// columns of all the rows, so every code is read and converted by exactly one
// wave of the workgroup, straight from global memory into the layout of the
// matrix instruction's B operand, and never passes through LDS. What the
// waves share, the 16*MT x 64 tile of the activations, is double-buffered in
// LDS, in 128-byte rows whose 16-byte pieces are XOR-ed with the row number
// so that the 16 rows of an operand read fall on different banks.
//
// Within a step of 64 contraction indices, lane quarter q owns indices
// 16q .. 16q+15 (matrix instruction s takes 16q + 8s + j): any order of the
// contraction is right as long as both operands use it, and this one makes a
// lane's codes of a row contiguous. Columns are dealt the same way: lane
// (l & 15) owns columns 4 (l & 15) + t of the wave's 64, t = 0..3 the tile, so
// that a lane stores 4 neighbouring results, and, in the gradient, reads the
// 4 neighbouring codes of a row in one load.
//
// Precision. PA and PB are the numbers of bf16 parts of the activations and
// of the weights. bf16 activations are one part, exactly; binary32 ones are
// three (24 bits, exactly). Weights are RN_bf16(code * s) for bf16 results
// (the value zpp_dequantize_blocks gives a caller who multiplies in bf16; its
// rounding, 2^-9 relative at most per product and independent over the
// contraction, stays below the rounding of the result itself), and three
// parts of RN(code * s) for binary32 results. Sums are binary32 throughout.
#pragma once

#include "linear_device.h"

namespace zpp {

constexpr int kStep = 64;      // contraction indices per step
constexpr int kTileCols = 256; // columns per workgroup

// 16 bytes of zeros for pieces past the end of the contraction.
__device__ __attribute__((aligned(16))) const uint32_t g_lin_zeros[4] = {0, 0, 0, 0};

// Byte offset of 16-byte piece c of row r in a tile of 128-byte rows.
__device__ __forceinline__ int lds_piece(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// The tile a workgroup computes. An XCD takes a contiguous run of tiles; 8
// rows of tiles run down before the next column, so that the 32 tiles an XCD
// works on at once share both activations and codes in its L2.
struct LinPlace {
    int64_t split, m0, col;
};

__device__ __forceinline__ LinPlace lin_place(const LinArgs &p, int rows) {
    // A launch has fewer than 2^24 workgroups. Divisions leave their results in
    // vector registers; read back, they and all that follows from them are scalar.
    auto div = [](uint32_t a, uint32_t b) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(a / b)); };
    const uint32_t id = static_cast<uint32_t>(xcd_block(blockIdx.x, gridDim.x));
    const uint32_t row_tiles = static_cast<uint32_t>(p.row_tiles), col_tiles = static_cast<uint32_t>(p.col_tiles);
    const uint32_t split = div(id, row_tiles * col_tiles), tile = id - split * (row_tiles * col_tiles);
    const uint32_t g = div(tile, 8 * col_tiles), in_g = min(8u, row_tiles - g * 8), at = tile - g * 8 * col_tiles;
    const uint32_t col = div(at, in_g), row = g * 8 + (at - col * in_g);
    return LinPlace{split, static_cast<int64_t>(row) * rows, col};
}

template <bool GRAD, int BITS, int PA, int PB, int MT, bool ASYNC>
struct LinTile {
    static constexpr int kRows = 16 * MT;
    static constexpr int kPlane = kRows * 128;  // bytes of one part's tile
    static constexpr int kPieces = (kRows * 8 + kBlockThreads - 1) / kBlockThreads;  // 16-byte pieces per thread

    // The codes and scales of one step, as loaded.
    struct Raw {
        uint32_t w[GRAD ? 16 : (BITS == 4 ? 8 : 16)];
        float s[GRAD ? 16 : 4];
    };

    static __device__ __forceinline__ void load_raw(const LinArgs &p, int64_t col, int q, int64_t c0, Raw &r) {
        if constexpr (!GRAD) {
            const int64_t k = c0 + q * 16;
            const bool ok = k < p.n_in;  // in_features is a multiple of 32: all 16 or none
            const int64_t kk = ok ? k : 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t n = min(col + t, p.n_out - 1);
                const int64_t e = n * p.n_in + kk;
                if constexpr (BITS == 4) {
                    const u32x2 v = ld<u32x2>(p.codes + e / 2);
#pragma unroll
                    for (int i = 0; i < 2; ++i) r.w[2 * t + i] = ok ? v[i] : 0;
                } else {
                    const u32x4 v = ld<u32x4>(p.codes + e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r.w[4 * t + i] = ok ? v[i] : 0;
                }
                const float sc = p.scales[e >> p.log2b];
                r.s[t] = ok ? sc : 0.0f;
            }
        } else {
            const int64_t k = min(col, p.n_in - 4);  // in_features is a multiple of 32: all 4 columns or none
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t n = c0 + q * 16 + i;
                const bool ok = n < p.n_out;
                const int64_t e = (ok ? n : 0) * p.n_in + k;
                const uint32_t v = BITS == 4 ? static_cast<uint32_t>(ld<uint16_t>(p.codes + e / 2))
                                             : ld<uint32_t>(p.codes + e);
                r.w[i] = ok ? v : 0;
                const float sc = p.scales[e >> p.log2b];
                r.s[i] = ok ? sc : 0.0f;
            }
        }
    }

    // Weight of column tile t at index i of the lane's 16 (times 1/16 for 4-bit codes).
    static __device__ __forceinline__ float weight(const Raw &r, int t, int i) {
        if constexpr (GRAD) return code_f32<BITS>(r.w[i], t) * r.s[i];
        constexpr int per = 32 / BITS;
        return code_f32<BITS>(r.w[t * (16 / per) + i / per], i % per) * r.s[t];
    }

    using Frag = u32x4[PB];

    // Dword d of the B operands of instruction s, tile t.
    static __device__ __forceinline__ void convert(const Raw &r, int s, int t, int d, Frag &f) {
        uint32_t w[PB];
        to_parts<PB>(weight(r, t, 8 * s + 2 * d), weight(r, t, 8 * s + 2 * d + 1), w);
#pragma unroll
        for (int i = 0; i < PB; ++i) f[i][d] = w[i];
    }

    // ---- the activations' tile ----

    // Straight from global memory to LDS; every wave's instruction fills 8 rows.
    static __device__ __forceinline__ void stage_async(const LinArgs &p, int64_t m0, int64_t c0, int64_t c_len,
                                                       uint8_t *tile) {
        const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
        const uint16_t *a = static_cast<const uint16_t *>(p.a);
#pragma unroll
        for (int i = 0; i < (2 * MT + 3) / 4; ++i) {
            const int g = i * 4 + w;  // group of 8 rows
            if (2 * MT % 4 != 0 && g >= 2 * MT) break;
            const int r = g * 8 + (lane >> 3);
            const int c = (lane & 7) ^ (r & 7);
            const int64_t row = min(m0 + r, p.rows - 1);
            const int64_t k = c0 + c * 8;
            const void *src = k < c_len ? static_cast<const void *>(a + row * p.lda + k) : g_lin_zeros;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                             (__attribute__((address_space(3))) void *)(tile + g * 1024), 16, 0, 0);
        }
    }

    using Held = uint32_t[kPieces][PA == 3 ? 8 : 4];

    // Through registers: any row stride, any contraction length, both types.
    static __device__ __forceinline__ void stage_load(const LinArgs &p, int64_t m0, int64_t c0, int64_t c_len,
                                                      bool vec, Held &h) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int id = i * kBlockThreads + threadIdx.x;
            if (id >= kRows * 8) break;
            const int64_t row = min(m0 + id / 8, p.rows - 1);
            const int64_t k = c0 + (id & 7) * 8;
            if constexpr (PA == 3) {
                const float *a = static_cast<const float *>(p.a) + row * p.lda + k;
                if (vec && k + 8 <= c_len) {
                    const u32x4 u = ld<u32x4>(a), v = ld<u32x4>(a + 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[i][j] = u[j], h[i][4 + j] = v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] = k + j < c_len ? as_u(a[j]) : 0;
                }
            } else {
                const uint16_t *a = static_cast<const uint16_t *>(p.a) + row * p.lda + k;
                if (vec && k + 8 <= c_len) {
                    const u32x4 u = ld<u32x4>(a);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[i][j] = u[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[i][j] = (k + 2 * j < c_len ? a[2 * j] : 0u) |
                                  (k + 2 * j + 1 < c_len ? static_cast<uint32_t>(a[2 * j + 1]) << 16 : 0u);
                }
            }
        }
    }

    static __device__ __forceinline__ void stage_store(const Held &h, uint8_t *tile) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int id = i * kBlockThreads + threadIdx.x;
            if (id >= kRows * 8) break;
            const int at = lds_piece(id / 8, id & 7);
            u32x4 v[PA];
            if constexpr (PA == 3) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[3];
                    to_parts<3>(as_f(h[i][2 * j]), as_f(h[i][2 * j + 1]), w);
#pragma unroll
                    for (int a = 0; a < 3; ++a) v[a][j] = w[a];
                }
            } else {
                v[0] = u32x4{h[i][0], h[i][1], h[i][2], h[i][3]};
            }
#pragma unroll
            for (int a = 0; a < PA; ++a) *reinterpret_cast<u32x4 *>(tile + a * kPlane + at) = v[a];
        }
    }

    static __device__ __forceinline__ void store4(const LinArgs &p, int64_t len, int64_t row, int64_t col,
                                                  const float (&v)[4], int64_t split) {
        if (p.splits > 1) {  // columns of the sums are padded to whole fours
            const int64_t ldp = (len + 3) & ~INT64_C(3);
            if (col < ldp)
                st<f32x4>(p.partial + (split * p.rows + row) * ldp + col, f32x4{v[0], v[1], v[2], v[3]});
            return;
        }
        if (p.out_f32) {
            float *o = static_cast<float *>(p.out) + row * p.ldo + col;
            if ((p.ldo & 3) == 0 && col + 4 <= len) {
                st<f32x4>(o, f32x4{v[0], v[1], v[2], v[3]});
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (col + t < len) o[t] = v[t];
            }
        } else {
            uint16_t *o = static_cast<uint16_t *>(p.out) + row * p.ldo + col;
            const uint32_t a = pack_rn(v[0], v[1]), b = pack_rn(v[2], v[3]);
            if ((p.ldo & 3) == 0 && col + 4 <= len) {
                st<u32x2>(o, u32x2{a, b});
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (col + t < len) o[t] = static_cast<uint16_t>((t < 2 ? a : b) >> (16 * (t & 1)));
            }
        }
    }
};

template <bool GRAD, int BITS, int PA, int PB, int MT, bool ASYNC>
__global__ __launch_bounds__(kBlockThreads, 1) void linear_tile_kernel(LinArgs p) {
    using T = LinTile<GRAD, BITS, PA, PB, MT, ASYNC>;
    __shared__ __attribute__((aligned(128))) uint8_t tiles[2][PA * T::kPlane];

    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
    const int q = lane >> 4;
    const int64_t c_len = GRAD ? p.n_out : p.n_in, len = GRAD ? p.n_in : p.n_out;

    const LinPlace place = lin_place(p, T::kRows);
    const int64_t split = place.split, m0 = place.m0;
    const int64_t col = place.col * kTileCols + w * 64 + (lane & 15) * 4;

    const int64_t steps = (c_len + kStep - 1) / kStep;
    const int64_t s0 = split * p.split_steps, s1 = min(steps, s0 + p.split_steps);
    const bool vec = PA == 3 ? (p.lda & 3) == 0 : (p.lda & 7) == 0;

    f32x4 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0, 0, 0, 0};

    typename T::Raw raw;
    typename T::Frag b[2][4];
    typename T::Held held;

    // The pipeline: codes two steps ahead in registers, converted one step
    // ahead among the matrix instructions; activations one step ahead in LDS.
    if constexpr (ASYNC) {
        T::stage_async(p, m0, s0 * kStep, c_len, tiles[0]);
    } else {
        T::stage_load(p, m0, s0 * kStep, c_len, vec, held);
        T::stage_store(held, tiles[0]);
    }
    T::load_raw(p, col, q, s0 * kStep, raw);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) T::convert(raw, s, t, d, b[s][t]);
    T::load_raw(p, col, q, (s0 + 1) * kStep, raw);  // past the end: zeros
    if constexpr (ASYNC) wait_loads();
    __syncthreads();

    for (int64_t i = s0; i < s1; ++i) {
        const int cur = (i - s0) & 1;
        const uint8_t *tile = tiles[cur];
        typename T::Raw next;
        if (i + 1 < s1) {
            if constexpr (ASYNC)
                T::stage_async(p, m0, (i + 1) * kStep, c_len, tiles[cur ^ 1]);
            else
                T::stage_load(p, m0, (i + 1) * kStep, c_len, vec, held);
        }
        T::load_raw(p, col, q, (i + 2) * kStep, next);
        typename T::Frag bn[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                u32x4 a[PA];
#pragma unroll
                for (int x = 0; x < PA; ++x)
                    a[x] = *reinterpret_cast<const u32x4 *>(tile + x * T::kPlane +
                                                            lds_piece(m * 16 + (lane & 15), q * 2 + s));
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[m][t] = mfma_parts<PA, PB>(a, b[s][t], acc[m][t]);
                // the next step's codes, a share of their 32 dwords after each row of tiles
#pragma unroll
                for (int d = 32 * (s * MT + m) / (2 * MT); d < 32 * (s * MT + m + 1) / (2 * MT); ++d)
                    T::convert(raw, d / 16, d / 4 % 4, d % 4, bn[d / 16][d / 4 % 4]);
            }
        }
        if constexpr (!ASYNC) {
            if (i + 1 < s1) T::stage_store(held, tiles[cur ^ 1]);
        }
        raw = next;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < PB; ++x) b[s][t][x] = bn[s][t][x];
        // this wave's loads into LDS have landed; after the barrier every wave's have
        if constexpr (ASYNC) wait_loads();
        __syncthreads();
    }

#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = m0 + m * 16 + 4 * q + i;
            if (row >= p.rows) continue;
            float v[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] = acc[m][t][i] * kCodeScale<BITS>;
            T::store4(p, len, row, col, v, split);
        }
    }
}

template <bool GRAD, int BITS, int PA, int PB, int MT, bool ASYNC>
hipError_t launch_linear_tile_one(const LinArgs &p, hipStream_t stream) {
    const int64_t grid = p.row_tiles * p.col_tiles * p.splits;
    linear_tile_kernel<GRAD, BITS, PA, PB, MT, ASYNC><<<static_cast<unsigned>(grid), kBlockThreads, 0, stream>>>(p);
    return hipGetLastError();
}

// The kernels of one direction and code width: mode 1 is bf16 to bf16 where
// linear_big.h cannot (activations that are not whole 16-byte pieces, which
// only the gradient's can be, or row strides past 32-bit offsets), 2 bf16 to
// binary32, 3 binary32 activations. mt is the plan's.
template <bool GRAD, int BITS>
hipError_t launch_linear_tile_as(const LinArgs &p, int mode, int mt, hipStream_t stream) {
    if (mode == 3) {
        if (mt == 8) return launch_linear_tile_one<GRAD, BITS, 3, 3, 8, false>(p, stream);
        if (mt == 4) return launch_linear_tile_one<GRAD, BITS, 3, 3, 4, false>(p, stream);
        return launch_linear_tile_one<GRAD, BITS, 3, 3, 1, false>(p, stream);
    }
    if (mode == 2) {
        if (mt == 8) return launch_linear_tile_one<GRAD, BITS, 1, 3, 8, false>(p, stream);
        if (mt == 4) return launch_linear_tile_one<GRAD, BITS, 1, 3, 4, false>(p, stream);
        return launch_linear_tile_one<GRAD, BITS, 1, 3, 1, false>(p, stream);
    }
    if (mt == 16) return launch_linear_tile_one<GRAD, BITS, 1, 1, 16, false>(p, stream);
    if (mt == 8) return launch_linear_tile_one<GRAD, BITS, 1, 1, 8, false>(p, stream);
    if (mt == 4) return launch_linear_tile_one<GRAD, BITS, 1, 1, 4, false>(p, stream);
    return launch_linear_tile_one<GRAD, BITS, 1, 1, 1, false>(p, stream);
}

}  // namespace zpp
