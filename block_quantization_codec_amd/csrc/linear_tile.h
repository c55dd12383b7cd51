// linear_tile.h - what the tiled products on block codes share: the order of
// the tiles, the layout of activations in LDS and how they get there, and the
// stores of results.
#pragma once

#include "linear_device.h"

namespace zpp {

constexpr int kStep = 64;      // contraction indices per step
constexpr int kTileCols = 256; // columns per workgroup (linear_big.h)

// 16 bytes of zeros for pieces past the end of the contraction.
__device__ __attribute__((aligned(16))) const uint32_t g_lin_zeros[4] = {0, 0, 0, 0};

// Byte offset of 16-byte piece c of row r in a tile of 128-byte rows (64
// indices): pieces are XOR-ed with the row number, so that the 16 rows of an
// operand read fall on different banks.
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

// A tile of 16*MT rows x 64 activations in LDS, in PA planes of bf16 parts.
template <int PA, int MT>
struct LinTile {
    static constexpr int kRows = 16 * MT;
    static constexpr int kPlane = kRows * 128;  // bytes of one part's tile
    static constexpr int kPieces = (kRows * 8 + kBlockThreads - 1) / kBlockThreads;  // 16-byte pieces per thread

    // Straight from global memory to LDS; every wave's instruction fills 8 rows.
    // Where this lane's pieces lie in their rows, found once:
    struct Rows {
        const uint16_t *at[(2 * MT + 3) / 4];
    };

    static __device__ __forceinline__ Rows rows(const LinArgs &p, int64_t m0) {
        const int lane = threadIdx.x & (kWave - 1), r = wave_in_block() * 8 + (lane >> 3);
        Rows o;
#pragma unroll
        for (int i = 0; i < (2 * MT + 3) / 4; ++i)
            o.at[i] = static_cast<const uint16_t *>(p.a) + min(m0 + i * 32 + r, p.rows - 1) * p.lda +
                      ((lane & 7) ^ (r & 7)) * 8;
        return o;
    }

    static __device__ __forceinline__ void stage_async(const Rows &rows, int64_t c0, int64_t c_len, uint8_t *tile) {
        const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
        const int c = (lane & 7) ^ (lane >> 3);
        const bool in = c * 8 < c_len - c0;
#pragma unroll
        for (int i = 0; i < (2 * MT + 3) / 4; ++i) {
            const int g = i * 4 + w;  // group of 8 rows
            if (2 * MT % 4 != 0 && g >= 2 * MT) break;
            const uint16_t *src = in ? rows.at[i] + c0 : reinterpret_cast<const uint16_t *>(g_lin_zeros);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                             (__attribute__((address_space(3))) void *)(tile + g * 1024), 16, 0, 0);
        }
    }

    using Held = uint32_t[kPieces][8];

    // binary32 activations, through registers. Rows and their length are whole
    // 16-byte pieces, and the length whole 8 elements.
    static __device__ __forceinline__ void stage_load(const LinArgs &p, int64_t m0, int64_t c0, int64_t c_len,
                                                      Held &h) {
        static_assert(PA == 3);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int id = i * kBlockThreads + threadIdx.x;
            if (id >= kRows * 8) break;
            const int64_t row = min(m0 + id / 8, p.rows - 1);
            const int64_t k = c0 + (id & 7) * 8;
            const float *a = static_cast<const float *>(p.a) + row * p.lda + k;
            u32x4 u = {0, 0, 0, 0}, v = {0, 0, 0, 0};
            if (k < c_len) u = ld<u32x4>(a), v = ld<u32x4>(a + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] = u[j], h[i][4 + j] = v[j];
        }
    }

    static __device__ __forceinline__ void stage_store(const Held &h, uint8_t *tile) {
        static_assert(PA == 3);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int id = i * kBlockThreads + threadIdx.x;
            if (id >= kRows * 8) break;
            const int at = lds_piece(id / 8, id & 7);
            u32x4 v[PA];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[3];
                to_parts<3>(as_f(h[i][2 * j]), as_f(h[i][2 * j + 1]), w);
#pragma unroll
                for (int a = 0; a < 3; ++a) v[a][j] = w[a];
            }
#pragma unroll
            for (int a = 0; a < PA; ++a) *reinterpret_cast<u32x4 *>(tile + a * kPlane + at) = v[a];
        }
    }
};

// 4 neighbouring results of a row, or a split's sums of them.
__device__ __forceinline__ void store4(const LinArgs &p, int64_t len, int64_t row, int64_t col,
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

}  // namespace zpp
