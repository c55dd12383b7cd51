// linear.hip - which kernels a linear product on block codes takes, the packing
// of activations that the tiled ones cannot read, and the sum of the parts of a
// split contraction.
#include <algorithm>
#include <cmath>

#include "../../include/zpp.h"
#include "linear_tile.h"

namespace zpp {

hipError_t launch_linear_few(const LinArgs &p, int bits, bool a_f32, hipStream_t stream);
hipError_t launch_linear_mid(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream);
hipError_t launch_linear_big_fwd4(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_big_fwd8(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_big_grad4(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_big_grad8(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_mid_group(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream);
hipError_t launch_linear_big_group_fwd4(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_big_group_fwd8(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_big_group_grad4(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_big_group_grad8(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_mid_adapt(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream);
hipError_t launch_linear_adapt_fwd4(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_adapt_fwd8(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_adapt_grad4(const LinArgs &p, int parts, int mt, hipStream_t stream);
hipError_t launch_linear_adapt_grad8(const LinArgs &p, int parts, int mt, hipStream_t stream);

namespace {

constexpr int64_t kCus = 256;       // MI355X
constexpr int64_t kFewRows = 4;     // forward: at most this many rows stream the codes, x in registers,
constexpr int64_t kMidRows = 64;    // at most this many always with x in LDS
constexpr int64_t kMaxTiles = 1 << 23;  // workgroups of one launch

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

enum class Way { few, mid, tile };

struct Plan {
    Way way;
    int mt;       // rows of 16 per workgroup
    int splits;   // parts of the contraction
    int64_t split_steps;
    int64_t rows; // rows of one launch
    int64_t groups; // and groups
    int join_steps; // groups in tiles: what a round's parts cost, in steps (linear_tile.h)
    int parts;      // tiles: of the operands (linear_big.h, launch_linear_big_as)
};

// Rows of tiles that `rows` rows make; in groups, each has a last tile of its own, on
// average half full (and a group of few rows is one tile).
int64_t row_tiles(int64_t rows, int64_t groups, int64_t tile) {
    if (groups == 0) return ceil_div(rows, tile);
    const int64_t held = std::min(rows, groups);
    return std::max(held, rows / tile + held / 2);
}

// What the parts of a split contraction cost, in microseconds: their writing,
// reading and joining (5.5 bytes a nanosecond and 4 us).
double join_time(int64_t splits, int64_t rows, int64_t len) {
    return splits > 1 ? 4.0 + static_cast<double>(splits * rows * len) * 8 / 5.5e6 : 0;
}

// What a call by the middle kernel takes, in microseconds: steps of 256 indices
// times the time of one in the CU that holds most workgroups, and the join. One
// workgroup alone leaves the CU idle in its waits; more share its issue. Three
// parts of 64 rows fill LDS, one workgroup a CU. 333 rows of 4096 x 11008 int4:
// 61 us in 4 parts (66 estimated), 71 in 2 (77), 65 in 5 (71); 16 of 8192 x 28672
// int8: 57 in 8 (51), 61 in 12 (54).
double mid_time(bool in_f32, int mt, int64_t tiles, int64_t splits, int64_t split_steps, int64_t rows, int64_t len) {
    const double n = static_cast<double>(ceil_div(tiles * splits, kCus));
    const double cu = in_f32 && mt == 4 ? 6.5 * n : std::max(2.2, 1.5 * n) * (in_f32 ? 2 : 1);
    return static_cast<double>(split_steps) * cu + join_time(splits, rows, len);
}

// What a tiled call takes, in microseconds, with workgroups of mt rows of 16
// and the contraction in `splits` parts: rounds of workgroups over the CUs
// times steps times a step's time, and the join. A step takes, with the
// operands' parts (rows of the table: 1 and 1, 1 and 3, 3 and 3, 1 and 2), measured at
// 128 to 4096 rows of 8192 x 8192 and 11008 x 4096 weights (1 and 2: 1.27 and 1.43 times as long as
// 1 and 1, 16 and 64 rows of 8192 x 65536):
double step_time(int parts, int mt) {
    static constexpr double step_us[4][4] = {{0.92, 1.05, 1.10, 1.60}, {1.50, 1.90, 3.20, 0}, {1.60, 3.20, 4.80, 0},
                                             {1.17, 1.50, 0, 0}};
    return step_us[parts][mt == 1 ? 0 : mt == 4 ? 1 : mt == 8 ? 2 : 3];
}

double tile_time(int parts, int mt, int64_t splits, int64_t rows, int64_t len, int64_t split_steps) {
    const double tiles = static_cast<double>(ceil_div(rows, 16 * mt) * ceil_div(len, 256) * splits);
    // Workgroups that share a CU take about as long as one after the other.
    const double rounds = std::ceil(tiles / kCus);
    return rounds * static_cast<double>(split_steps) * step_time(parts, mt) + join_time(splits, rows, len);
}

// The same for rows in groups, of which only the tiles past whole rounds are in parts.
// join_steps: what kRound tiles' parts take in the kernel and the join, in steps; 0 where a round is too
// short for the join's launch, unless the sizes alone say that there will be parts.
double group_time(int parts, int mt, int64_t rows, int64_t groups, int64_t len, int64_t steps, int &join_steps) {
    const double step = step_time(parts, mt), part_us = 16.0 * mt * kTileCols * 8 / 5.5e6;
    const int64_t tiles = row_tiles(rows, groups, 16 * mt) * ceil_div(len, kTileCols);
    join_steps = std::max(static_cast<int>(std::ceil(kRound * part_us / step)), 1);
    const LinTail t = lin_tail(static_cast<uint32_t>(std::min(tiles, kMaxTiles)), static_cast<uint32_t>(steps),
                               static_cast<uint32_t>(join_steps));
    if (t.splits == 1 && (steps < 6 || static_cast<double>(steps) * step < 40)) join_steps = 0;
    const int64_t last = ceil_div(static_cast<int64_t>(t.left) * t.splits, kRound) * t.steps;
    return static_cast<double>(tiles / kRound * steps + last) * step +
           (t.splits > 1 ? 4.0 + t.left * t.splits * part_us : 0);
}

// How many rows, and groups, one launch takes: kMaxTiles workgroups.
void bound_launch(Plan &p, int64_t groups, int64_t col_tiles) {
    int64_t tiles = std::max<int64_t>(kMaxTiles / col_tiles / p.splits, 2);
    if (groups > 0) {  // each group may have one tile more than its share
        p.groups = std::min(groups, tiles / 2);
        tiles -= p.groups;
    }
    p.rows = tiles * 16 * p.mt;
}

// The way of the least time. Measured on the way: 128 rows of 8192 x 8192 int4,
// 39 us as 128-row tiles in 8 parts (34 estimated) against 48 as 256-row tiles
// in 8, 50 as 64-row tiles in 4 and 135 or more unsplit; 100 rows of 28672 x
// 8192 int4, 92 us as 128-row tiles in 2 parts (83), 122 in 3 (119) and 139 as
// 64-row tiles unsplit (134); 1024 rows of 8192 x 8192, 132 us as 256-row tiles in
// 2 (130) against 146 as 128-row tiles unsplit (141).
//
// A forward product of up to 64 rows, and from bf16 to binary32 of any number,
// multiplies by the exact codes: with binary32 results that is one part of the
// weights in place of three (333 rows of 4096 x 11008 int8: 74 us so, 155 with
// three parts in tiles). Other products do so where the estimate is below the
// tiles' (with a binary32 x, the tiles' and their packing's: 10 bytes read and
// written an element, and a launch of 3 us; with bf16, by a twelfth: of 120 shapes
// whose estimates lie within a quarter of each other, all but two are faster so, or
// equal, from there on, and most are slower below). Exact codes against tiles, bf16,
// int4: 70 rows of 1024 x 8192, 14 us against 20; 200 of 1024 x 4096, 15 against
// 22; 80 of 8192 x 2048, 21 against 25; 256 of 8192 x 8192, 62 against 58; 400 of
// 11008 x 4096, 78 against 71. binary32: 4019 rows of 512 x 928 int8, 30 us against
// 45; 200 of 4096 x 11008 int8, 131 against 115.
//
// Rows in groups (groups > 0) take the same kernels but the stream of few rows.
//
// From bf16 to bf16, tiles multiply by weights rounded to bf16: an error of the size of the result's
// own rounding, and with few results the two add up unevenly (to 1.4 times the result's rounding
// on average, to 2.1 times in a call of one row). So gradients of up to kMidRows rows, in groups or with adapters, take
// the weights in two parts, off by 2^-16; forward, as many rows multiply by exact codes. It costs, int4: one row of
// 8192 x 8192 with an adapter 56 us in place of 51, 8 rows over 8 matrices of 11008 x 4096 127 in place of 104;
// 2048 rows over 64 of those would take 861 in place of 607.
Plan make_plan(bool grad, bool in_f32, bool out_f32, int64_t rows, int64_t groups, int64_t n_out, int64_t n_in,
               bool adapted) {
    Plan p{};
    // rows of one matrix, as far as the sizes say
    const int64_t each_rows = groups == 0 ? rows : ceil_div(rows, std::min(rows, groups));
    if (!grad && groups == 0 && rows <= kFewRows) {
        p.way = Way::few;
        p.rows = rows;
        p.splits = 1;
        return p;
    }
    Plan mid{};
    double mid_us = 0;
    if (!grad) {
        mid.way = Way::mid;
        mid.mt = each_rows <= 16 ? 1 : each_rows <= 32 ? 2 : 4;
        const int64_t steps = ceil_div(n_in, 128 * kMidChunks), col_tiles = ceil_div(n_out, 64 * kMidTiles);
        const int64_t tiles = col_tiles * row_tiles(rows, groups, 16 * mid.mt);
        for (const int64_t want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
            if (want > steps) break;
            const int64_t each = ceil_div(steps, want), n = ceil_div(steps, each);
            const double t = mid_time(in_f32, mid.mt, tiles, n, each, rows, n_out);
            if (mid.splits == 0 || t < mid_us) {
                mid_us = t;
                mid.splits = static_cast<int>(n);
                mid.split_steps = each;
            }
        }
        bound_launch(mid, groups, col_tiles);
        if (each_rows <= kMidRows || (out_f32 && !in_f32)) return mid;
    }
    p.way = Way::tile;
    const int64_t c_len = grad ? n_out : n_in, len = grad ? n_in : n_out;
    const int64_t col_tiles = ceil_div(len, 256), steps = ceil_div(c_len, 64);
    const bool few = grad && rows <= kMidRows && (groups > 0 || adapted);
    const int parts = p.parts = in_f32 ? 2 : out_f32 ? 1 : few ? 3 : 0;
    double least = 0;
    for (const int mt : {16, 8, 4, 1}) {
        if (step_time(parts, mt) == 0) continue;
        if (groups > 0) {
            int join_steps;
            const double t = group_time(parts, mt, rows, groups, len, steps, join_steps);
            if (p.mt == 0 || t < least) least = t, p.mt = mt, p.splits = 1, p.split_steps = steps, p.join_steps = join_steps;
            continue;
        }
        for (const int64_t want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
            if (want > 1 && want > steps / 3) break;
            // the pipeline takes steps in pairs
            const int64_t each = want == 1 ? steps : ceil_div(ceil_div(steps, want), 2) * 2, n = ceil_div(steps, each);
            const double t = tile_time(parts, mt, n, rows, len, each);
            if (p.mt == 0 || t < least) {
                least = t;
                p.mt = mt;
                p.splits = static_cast<int>(n);
                p.split_steps = each;
            }
        }
    }
    if (in_f32) least += 3.0 + static_cast<double>(rows * c_len) * 10 / 5.5e6;
    if (mid.mt != 0 && mid_us * (in_f32 ? 1.0 : 1.08) < least) return mid;
    bound_launch(p, groups, col_tiles);
    return p;
}

// out[r][c] = sum of the parts, in order, 4 columns a thread. GROUPED: of rows
// `first` to `last` of the whole call's, where row0 is this launch's first, alone.
template <bool GROUPED>
__global__ __launch_bounds__(kBlockThreads) void linear_join_kernel(const float *__restrict__ partial, int splits,
                                                                    int64_t rows, int64_t len, void *out,
                                                                    int64_t ldo, int out_f32,
                                                                    const int32_t *__restrict__ first,
                                                                    const int32_t *__restrict__ last, int64_t row0) {
    const int64_t ldp = (len + 3) & ~INT64_C(3), per = ldp / 4;
    int64_t r_first = 0, r_last = 0;
    if constexpr (GROUPED) r_first = *first - row0, r_last = *last - row0;
    const int64_t n = static_cast<int64_t>(gridDim.x) * kBlockThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlockThreads + threadIdx.x; i < rows * per; i += n) {
        const int64_t r = i / per, c = (i - r * per) * 4;
        if (GROUPED && (r < r_first || r >= r_last)) continue;
        f32x4 v = {0, 0, 0, 0};
        const float *from = partial + r * ldp + c;
        int s = 0;
        for (; s + 8 <= splits; s += 8) {  // eight loads in flight
            f32x4 part[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) part[j] = ld<f32x4>(from + (s + j) * rows * ldp);
#pragma unroll
            for (int j = 0; j < 8; ++j) v += part[j];
        }
#pragma unroll 4
        for (; s < splits; ++s) v += ld<f32x4>(from + s * rows * ldp);
        const bool whole = (ldo & 3) == 0 && c + 4 <= len;
        if (out_f32) {
            float *o = static_cast<float *>(out) + r * ldo + c;
            if (whole) {
                st<f32x4>(o, v);
            } else {
                for (int t = 0; t < 4; ++t)
                    if (c + t < len) o[t] = v[t];
            }
        } else {
            uint16_t *o = static_cast<uint16_t *>(out) + r * ldo + c;
            const uint32_t a = pack_rn(v[0], v[1]), b = pack_rn(v[2], v[3]);
            if (whole) {
                st<u32x2>(o, u32x2{a, b});
            } else {
                for (int t = 0; t < 4; ++t)
                    if (c + t < len) o[t] = static_cast<uint16_t>((t < 2 ? a : b) >> (16 * (t & 1)));
            }
        }
    }
}

// The same for groups in tiles: of the tiles that are in parts (linear_tile.h), 16 rows a workgroup.
__global__ __launch_bounds__(kBlockThreads) void linear_join_tail_kernel(LinArgs p, int tile_rows, int64_t len) {
    const uint32_t total = group_tiles(p, tile_rows);
    const LinTail t = group_tail(p, total);
    if (t.splits == 1) return;
    const uint32_t slabs = static_cast<uint32_t>(tile_rows) / 16, left = scalar_div(blockIdx.x, slabs);
    if (left >= t.left) return;
    LinPlace place = lin_tile(p, 1, t.whole + left, total);
    int64_t first;
    if (!group_at<8, 2>(p, tile_rows, static_cast<uint32_t>(place.m0), place.m0, first)) return;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t row = (blockIdx.x - left * slabs) * 16 + wave_in_block() * 4, col = place.col * kTileCols + 4 * lane;
    const float *from = p.partial + (static_cast<int64_t>(left) * tile_rows + row) * kTileCols + 4 * lane;
    const int64_t next = static_cast<int64_t>(t.left) * tile_rows * kTileCols;
    if (place.m0 + row >= p.rows || col >= len) return;
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f32x4{0, 0, 0, 0};
#pragma unroll 2
    for (uint32_t s = 0; s < t.splits; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows past the group's last lie in the tile's part all the same
            v[i] += ld<f32x4>(from + s * next + i * kTileCols);
    }
    p.splits = 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float o[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
        if (place.m0 + row + i < p.rows) store4(p, len, place.m0 + row + i, col, o, 0);
    }
}

// Activations as the tiled kernels read them: PA planes of bf16 parts, rows of
// whole steps, zeros past the end. 8 elements a thread. `vec`: rows lie on
// 16-byte pieces.
template <int PA>
__global__ __launch_bounds__(kBlockThreads) void linear_pack_kernel(const void *__restrict__ a, int64_t lda,
                                                                    int64_t rows, int64_t len, int64_t ldp, bool vec,
                                                                    uint16_t *__restrict__ out) {
    const int64_t per = ldp / 8, n = static_cast<int64_t>(gridDim.x) * kBlockThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlockThreads + threadIdx.x; i < rows * per; i += n) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        u32x4 v[PA];
        if constexpr (PA == 3) {
            const uint32_t *from = static_cast<const uint32_t *>(a) + r * lda + c;
            uint32_t f[8];
            if (vec && c + 8 <= len) {
                const u32x4 lo = ld<u32x4>(from), hi = ld<u32x4>(from + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = lo[j], f[4 + j] = hi[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = c + j < len ? from[j] : 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[3];
                to_parts<3>(as_f(f[2 * j]), as_f(f[2 * j + 1]), w);
#pragma unroll
                for (int x = 0; x < 3; ++x) v[x][j] = w[x];
            }
        } else {
            const uint16_t *from = static_cast<const uint16_t *>(a) + r * lda + c;
            if (vec && c + 8 <= len) {
                v[0] = ld<u32x4>(from);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[0][j] = (c + 2 * j < len ? from[2 * j] : 0u) |
                              (c + 2 * j + 1 < len ? static_cast<uint32_t>(from[2 * j + 1]) << 16 : 0u);
            }
        }
#pragma unroll
        for (int x = 0; x < PA; ++x) st<u32x4>(out + (x * rows + r) * ldp + c, v[x]);
    }
}

// The tiled kernels read bf16 rows on 16-byte pieces, of strides that 32-bit
// offsets of 256 rows can take; anything else is packed first.
bool needs_pack(const Plan &p, bool in_f32, int64_t lda, int64_t c_len) {
    return p.way == Way::tile && (in_f32 || lda % 8 != 0 || c_len % 8 != 0 || lda > (INT64_C(1) << 22));
}

int64_t packed_bytes(const Plan &p, bool in_f32, int64_t rows, int64_t c_len) {
    return ceil_div(c_len, 64) * 64 * std::min(rows, p.rows) * 2 * (in_f32 ? 3 : 1);
}

}  // namespace

int64_t linear_workspace(bool grad, bool in_f32, int64_t lda, bool out_f32, int64_t rows, int64_t groups,
                         int64_t n_out, int64_t n_in, bool adapted) {
    if (rows == 0) return 0;
    const Plan p = make_plan(grad, in_f32, out_f32, rows, groups, n_out, n_in, adapted);
    const int64_t c_len = grad ? n_out : n_in, len = grad ? n_in : n_out;
    int64_t bytes = needs_pack(p, in_f32, lda, c_len) ? packed_bytes(p, in_f32, rows, c_len) : 0;
    if (p.splits > 1) bytes += p.splits * std::min(rows, p.rows) * ((len + 3) & ~INT64_C(3)) * 4;
    if (p.join_steps > 0)
        bytes += std::min<int64_t>(kParts, (ceil_div(std::min(rows, p.rows), 16 * p.mt) + std::min(groups, p.groups)) *
                                               ceil_div(len, kTileCols) * p.split_steps) *
                 16 * p.mt * kTileCols * 4;
    return bytes;
}

hipError_t launch_linear(bool grad, const void *a, bool in_f32, int64_t lda, int64_t rows, const int32_t *offsets,
                         int64_t groups, const void *codes, const float *scales, int bits, int64_t n_out, int64_t n_in,
                         int log2b, void *out, bool out_f32, int64_t ldo, void *workspace, hipStream_t stream,
                         const LinAdapters *ad, const float *low) {
    const Plan plan = make_plan(grad, in_f32, out_f32, rows, groups, n_out, n_in, ad != nullptr);
    const int64_t c_len = grad ? n_out : n_in, len = grad ? n_in : n_out;
    const bool pack = needs_pack(plan, in_f32, lda, c_len);
    for (int64_t r0 = 0; r0 < rows; r0 += plan.rows) {
        LinArgs p{};
        p.a = static_cast<const uint8_t *>(a) + r0 * lda * (in_f32 ? 4 : 2);
        p.lda = lda;
        p.rows = p.split_rows = std::min(rows - r0, plan.rows);
        p.codes = static_cast<const uint8_t *>(codes);
        p.scales = scales;
        p.n_out = n_out;
        p.n_in = n_in;
        p.log2b = log2b;
        p.out = static_cast<uint8_t *>(out) + r0 * ldo * (out_f32 ? 4 : 2);
        p.ldo = ldo;
        p.out_f32 = out_f32;
        p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                              (pack ? packed_bytes(plan, in_f32, rows, c_len) : 0));
        p.splits = plan.splits;
        p.split_steps = plan.split_steps;
        p.join_steps = plan.join_steps;
        p.row0 = r0;
        if (ad) {
            p.low = low + r0 * ad->rank;
            p.up = grad ? ad->a : ad->b;
            p.up_f32 = ad->f32;
            p.ids = ad->ids ? ad->ids + r0 : nullptr;
            p.rank = static_cast<int>(ad->rank);
            p.adapters = static_cast<int>(ad->adapters);
        }
        hipError_t e = hipSuccess;
        if (pack) {
            const int64_t ldp = ceil_div(c_len, 64) * 64;
            const unsigned grid = static_cast<unsigned>(
                std::min<int64_t>(ceil_div(p.rows * ldp / 8, kBlockThreads), 1 << 16));
            uint16_t *to = static_cast<uint16_t *>(workspace);
            if (in_f32)
                linear_pack_kernel<3><<<grid, kBlockThreads, 0, stream>>>(p.a, lda, p.rows, c_len, ldp, lda % 4 == 0, to);
            else
                linear_pack_kernel<1><<<grid, kBlockThreads, 0, stream>>>(p.a, lda, p.rows, c_len, ldp, lda % 8 == 0, to);
            if (e = hipGetLastError(); e != hipSuccess) return e;
            p.a = to;
            p.lda = ldp;
            p.plane = p.rows * ldp;
        }
        p.row_tiles = ceil_div(p.rows, 16 * std::max(plan.mt, 1));
        p.col_tiles = plan.way == Way::mid ? ceil_div(n_out, 64 * kMidTiles) : ceil_div(len, 256);
        const int parts = plan.parts;
        if (groups > 0) {
            for (int64_t g0 = 0; g0 < groups; g0 += plan.groups) {
                LinArgs q = p;
                q.offsets = offsets + g0;
                q.groups = static_cast<int>(std::min(groups - g0, plan.groups));
                q.row_tiles += q.groups;
                q.codes += g0 * (n_out * n_in * bits / 8);
                q.scales += g0 * (n_out * n_in >> log2b);
                if (plan.way == Way::mid)
                    e = launch_linear_mid_group(q, bits, in_f32, plan.mt, stream);
                else if (grad)
                    e = bits == 4 ? launch_linear_big_group_grad4(q, parts, plan.mt, stream)
                                  : launch_linear_big_group_grad8(q, parts, plan.mt, stream);
                else
                    e = bits == 4 ? launch_linear_big_group_fwd4(q, parts, plan.mt, stream)
                                  : launch_linear_big_group_fwd8(q, parts, plan.mt, stream);
                if (e == hipSuccess && q.join_steps > 0) {
                    linear_join_tail_kernel<<<static_cast<unsigned>((kRound - 1) * plan.mt), kBlockThreads, 0, stream>>>(
                        q, 16 * plan.mt, len);
                    e = hipGetLastError();
                }
                if (e != hipSuccess) return e;
            }
        } else if (plan.way == Way::few) {
            e = launch_linear_few(p, bits, in_f32, stream);
        } else if (plan.way == Way::mid) {
            e = ad ? launch_linear_mid_adapt(p, bits, in_f32, plan.mt, stream)
                   : launch_linear_mid(p, bits, in_f32, plan.mt, stream);
        } else if (ad && grad) {
            e = bits == 4 ? launch_linear_adapt_grad4(p, parts, plan.mt, stream)
                          : launch_linear_adapt_grad8(p, parts, plan.mt, stream);
        } else if (ad) {
            e = bits == 4 ? launch_linear_adapt_fwd4(p, parts, plan.mt, stream)
                          : launch_linear_adapt_fwd8(p, parts, plan.mt, stream);
        } else if (grad) {
            e = bits == 4 ? launch_linear_big_grad4(p, parts, plan.mt, stream)
                          : launch_linear_big_grad8(p, parts, plan.mt, stream);
        } else {
            e = bits == 4 ? launch_linear_big_fwd4(p, parts, plan.mt, stream)
                          : launch_linear_big_fwd8(p, parts, plan.mt, stream);
        }
        if (e != hipSuccess) return e;
        if (plan.splits > 1) {
            const int64_t threads = p.rows * ((len + 3) / 4);
            const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ceil_div(threads, kBlockThreads), 1 << 16));
            if (groups > 0)
                linear_join_kernel<true><<<grid, kBlockThreads, 0, stream>>>(
                    p.partial, p.splits, p.rows, len, p.out, ldo, out_f32, offsets, offsets + groups, r0);
            else
                linear_join_kernel<false><<<grid, kBlockThreads, 0, stream>>>(
                    p.partial, p.splits, p.rows, len, p.out, ldo, out_f32, nullptr, nullptr, 0);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace zpp
