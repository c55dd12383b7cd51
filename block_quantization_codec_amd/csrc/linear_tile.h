// linear_tile.h - what the tiled products on block codes share: the order of
// the tiles, the layout of activations in LDS and how they get there, and the
// stores of results.
#pragma once

#include <type_traits>

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

// Divisions leave their results in vector registers; read back, they and all that
// follows from them are scalar. (A launch has fewer than 2^24 workgroups.)
__device__ __forceinline__ uint32_t scalar_div(uint32_t a, uint32_t b) {
    return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(a / b));
}

// Tile number `tile` of `row_tiles` rows of tiles of `rows` rows.
__device__ __forceinline__ LinPlace lin_tile(const LinArgs &p, int rows, uint32_t tile, uint32_t row_tiles) {
    const uint32_t col_tiles = static_cast<uint32_t>(p.col_tiles);
    const uint32_t g = scalar_div(tile, 8 * col_tiles), in_g = min(8u, row_tiles - g * 8), at = tile - g * 8 * col_tiles;
    const uint32_t col = scalar_div(at, in_g), row = g * 8 + (at - col * in_g);
    return LinPlace{0, static_cast<int64_t>(row) * rows, col};
}

// `grid` workgroups, a launch's or its first ones, cover `row_tiles` rows of tiles of `rows` rows.
__device__ __forceinline__ LinPlace lin_place_of(const LinArgs &p, int rows, uint32_t grid, uint32_t row_tiles) {
    const uint32_t id = static_cast<uint32_t>(xcd_block(blockIdx.x, grid));
    const uint32_t tiles = row_tiles * static_cast<uint32_t>(p.col_tiles);
    const uint32_t split = scalar_div(id, tiles);
    LinPlace place = lin_tile(p, rows, id - split * tiles, row_tiles);
    place.split = split;
    return place;
}

__device__ __forceinline__ LinPlace lin_place(const LinArgs &p, int rows) {
    return lin_place_of(p, rows, gridDim.x, static_cast<uint32_t>(p.row_tiles));
}

// Inclusive sums along the wave's lanes.
__device__ __forceinline__ uint32_t scan_add(uint32_t v) {
    auto moved = [](uint32_t from, auto ctrl, auto rows) {  // lanes without a source take 0
        return static_cast<uint32_t>(
            __builtin_amdgcn_update_dpp(0, static_cast<int>(from), ctrl.value, rows.value, 0xF, true));
    };
    using std::integral_constant;
    using All = integral_constant<int, 0xF>;
    v += moved(v, integral_constant<int, 0x111>{}, All{});  // row_shr 1, 2, 4, 8: within rows of 16
    v += moved(v, integral_constant<int, 0x112>{}, All{});
    v += moved(v, integral_constant<int, 0x114>{}, All{});
    v += moved(v, integral_constant<int, 0x118>{}, All{});
    v += moved(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // lane 15 to row 1, 47 to row 3
    v += moved(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // lane 31 to rows 2 and 3
    return v;
}

// A launch over groups: which group a tile's rows are of follows from the offsets, which
// only the device knows. Every wave counts the groups' tiles, 64 groups at a time.
// Offsets are taken within the launch's rows and tiles, whatever they hold.
struct GroupRows {
    int begin, count;
    uint32_t tiles;
};

__device__ __forceinline__ GroupRows group_rows(const LinArgs &p, int tile_rows, int e) {
    auto clip = [&](int32_t v) {
        return static_cast<int>(min(max(static_cast<int64_t>(v) - p.row0, INT64_C(0)), p.rows));
    };
    const int at = min(e, p.groups - 1);
    GroupRows o;
    o.begin = clip(p.offsets[at]);
    o.count = e < p.groups ? max(clip(p.offsets[at + 1]) - o.begin, 0) : 0;
    o.tiles = static_cast<uint32_t>(min((o.count + tile_rows - 1) / tile_rows, static_cast<int>(p.row_tiles)));
    return o;
}

__device__ __forceinline__ uint32_t last_lane(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// The groups' rows of tiles, together.
__device__ __forceinline__ uint32_t group_tiles(const LinArgs &p, int tile_rows) {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t total = 0;
    for (int e = 0; e < p.groups; e += kWave)
        total = min(total + last_lane(scan_add(group_rows(p, tile_rows, e + lane).tiles)),
                    static_cast<uint32_t>(p.row_tiles));
    return total;
}

// The group that row of tiles `tile` is of: `p` becomes its own product, m0 is the tile's
// first row in it, `first` the group's first row of the launch's.
template <int BITS, int ELEM>
__device__ __forceinline__ bool group_at(LinArgs &p, int tile_rows, uint32_t tile, int64_t &m0, int64_t &first) {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t before = 0;
    for (int e = 0; e < p.groups; e += kWave) {
        const GroupRows o = group_rows(p, tile_rows, e + lane);
        const uint32_t own = o.tiles, upto = before + scan_add(own);
        const uint64_t past = __ballot(upto > tile);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            auto read = [&](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l)); };
            const int64_t group = e + l, weights = p.n_out * p.n_in;
            first = read(static_cast<uint32_t>(o.begin));
            m0 = static_cast<int64_t>(tile - (read(upto) - read(own))) * tile_rows;
            p.a = static_cast<const uint8_t *>(p.a) + first * p.lda * ELEM;
            p.rows = read(static_cast<uint32_t>(o.count));
            p.codes += group * (weights * BITS / 8);
            p.scales += group * (weights >> p.log2b);
            p.out = static_cast<uint8_t *>(p.out) + first * p.ldo * (p.out_f32 ? 4 : 2);
            return true;
        }
        before = last_lane(upto);
    }
    return false;
}

// A workgroup's tile, the contraction in p.splits parts. Workgroups past the groups' tiles have
// nothing to do, and the others are dealt out as if the launch had no more.
template <int BITS, int ELEM>
__device__ __forceinline__ bool group_place(LinArgs &p, int tile_rows, int64_t len, LinPlace &place) {
    const uint32_t total = group_tiles(p, tile_rows);
    const uint32_t grid = total * static_cast<uint32_t>(p.col_tiles * p.splits);
    if (blockIdx.x >= grid) return false;
    place = lin_place_of(p, 1, grid, total);
    int64_t first;
    if (!group_at<BITS, ELEM>(p, tile_rows, static_cast<uint32_t>(place.m0), place.m0, first)) return false;
    p.partial += first * ((len + 3) & ~INT64_C(3));
    return true;
}

// The tiles in rounds of one a CU: whole rounds take the whole contraction a tile, those
// that are left over, which would leave CUs idle for as long, take it in parts. How
// many follows from what is left, which only the device knows: the least steps, the
// parts' writing, reading and joining counted too. 8 groups with 4096 rows of 11008 x 4096,
// backward: 407 us, 463 with the contraction in 2 parts for every tile.
constexpr uint32_t kRound = 256;  // CUs
constexpr uint32_t kParts = 512;  // tiles of parts, at most

struct LinTail {
    uint32_t whole, left;  // tiles
    uint32_t splits;       // of those that are left; 1: they are no different
    uint32_t steps;        // of a part
};

__host__ __device__ __forceinline__ LinTail lin_tail(uint32_t tiles, uint32_t steps, uint32_t join_steps) {
    LinTail o{tiles / kRound * kRound, tiles % kRound, 1, steps};
    if (o.left == 0 || join_steps == 0) return o;
    uint32_t least = steps;
    auto consider = [&](uint32_t want) {
        if (want < 2 || want > steps / 3 || want * o.left > kParts) return;
        const uint32_t each = ((steps + want - 1) / want + 1) & ~1u;  // the pipeline takes steps in pairs
        const uint32_t n = (steps + each - 1) / each, parts = n * o.left;
        const uint32_t cost = (parts + kRound - 1) / kRound * each + join_steps * parts / kRound;
        if (cost < least) least = cost, o.splits = n, o.steps = each;
    };
    for (uint32_t want = 2; want <= 4; ++want) consider(want);
    consider(kRound / o.left);
    consider(kRound / o.left / 2);
    return o;
}

__device__ __forceinline__ LinTail group_tail(const LinArgs &p, uint32_t row_tiles) {
    LinTail o = lin_tail(row_tiles * static_cast<uint32_t>(p.col_tiles), static_cast<uint32_t>(p.split_steps),
                         static_cast<uint32_t>(p.join_steps));
    o.splits = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(o.splits));
    o.steps = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(o.steps));
    return o;
}

// A workgroup's tile; `p` becomes the group's own product, in as many parts as the tile has.
// A part's sums lie at [part][tile that is left][row of the tile][kTileCols].
template <int BITS, int ELEM>
__device__ __forceinline__ bool group_place_tail(LinArgs &p, int tile_rows, LinPlace &place) {
    const uint32_t total = group_tiles(p, tile_rows);
    const LinTail t = group_tail(p, total);
    const uint32_t whole = t.splits == 1 ? t.whole + t.left : t.whole, parts = t.splits == 1 ? 0 : t.left * t.splits;
    if (blockIdx.x >= whole + parts) return false;
    uint32_t tile, split = 0, left = 0;
    const bool part = blockIdx.x >= whole;
    if (part) {
        const uint32_t id = static_cast<uint32_t>(xcd_block(blockIdx.x - whole, parts));
        split = scalar_div(id, t.left);
        left = id - split * t.left;
        tile = whole + left;
    } else {
        tile = static_cast<uint32_t>(xcd_block(blockIdx.x, whole));
    }
    place = lin_tile(p, 1, tile, total);
    place.split = split;
    int64_t first;
    if (!group_at<BITS, ELEM>(p, tile_rows, static_cast<uint32_t>(place.m0), place.m0, first)) return false;
    p.splits = 1;
    if (part) {
        p.splits = static_cast<int>(t.splits);
        p.split_steps = t.steps;
        p.split_rows = static_cast<int64_t>(t.left) * tile_rows;
        p.partial += (static_cast<int64_t>(left) * tile_rows - place.m0 - place.col) * kTileCols;
    }
    return true;
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

// 4 neighbouring results of a row, or a split's sums of them. LDP: between rows of those, if it is
// not the result's width.
template <int LDP = 0>
__device__ __forceinline__ void store4(const LinArgs &p, int64_t len, int64_t row, int64_t col,
                                              const float (&v)[4], int64_t split) {
    if (p.splits > 1) {  // columns of the sums are padded to whole fours
        const int64_t width = (len + 3) & ~INT64_C(3), ldp = LDP ? LDP : width;
        if (col < width)
            st<f32x4>(p.partial + (split * p.split_rows + row) * ldp + col, f32x4{v[0], v[1], v[2], v[3]});
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
