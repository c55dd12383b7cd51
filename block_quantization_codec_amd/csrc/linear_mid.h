// linear_mid.h - y = x W^T on block codes for 5 to 64 rows of x, and for more
// where linear.hip finds it faster than tiles: the stream over the codes of
// linear_few.hip, with the activations in LDS.
//
// With more than a few rows, every wave reading x for itself takes as much of
// the path from L2 as the codes do (measured at 16 rows: a third more time).
// Here the 4 waves of a workgroup have 16*NT features each and share the tile
// of x that they multiply by, double-buffered in LDS like the activations of
// linear_tile.h; few workgroups then cover the features, so the contraction is
// split over workgroups to fill the GPU and a second kernel joins the parts.
//
// 16 rows of 8192 x 28672 int8: 57 us, 4.2 TB/s of codes, near what the memory
// gives; 64 rows of 28672 x 8192 int4: 61 to 65 us, and 333 of 4096 x 11008 int8 to
// binary32: 68 to 75 us, where conversion and matrix instructions of the two
// waves that a SIMD holds take the time (conversion is shared by 64 rows only).
// Where the pieces of x lie is found once: found in every step it took 8% more.
// Reading the operands from LDS an instruction ahead gained nothing.
#pragma once

#include "linear_adapt.h"
#include "linear_codes.h"
#include "linear_tile.h"

namespace zpp {

template <int BITS, int PA, int NT, int MT, int U, bool WIDE, LinMode MODE>
__global__ __launch_bounds__(kBlockThreads, MODE == LinMode::adapted ? 2 : 1) void linear_mid_kernel(LinArgs p) {
    constexpr bool ASYNC = PA == 1;
    using C = CodeStream<BITS, NT, U, WIDE>;
    using T = LinTile<PA, MT>;
    constexpr int kTile = PA * T::kPlane;
    __shared__ __attribute__((aligned(128))) uint8_t tiles[2][2 * U][kTile];

    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
    const uint32_t q = lane >> 4;
    LinPlace place;
    if constexpr (MODE == LinMode::grouped) {
        if (!group_place<BITS, PA == 3 ? 4 : 2>(p, T::kRows, p.n_out, place)) return;
    } else {
        place = lin_place(p, T::kRows);
    }
    const int64_t split = place.split, m0 = place.m0;
    const int64_t n0 = (place.col * 4 + w) * (16 * NT);
    // a wave past the last feature works on it, and stores nothing
    const typename C::At at = C::place(p, min(n0, p.n_out - 1));

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0, 0, 0, 0};

    constexpr int64_t kAll = U * kChunk, kStepOf = kMidChunks * kChunk;
    const int64_t k0 = split * p.split_steps * kStepOf, k1 = min(p.n_in, k0 + p.split_steps * kStepOf);
    typename C::Chunks c;
    typename T::Held held[2 * U];

    [[maybe_unused]] const typename T::Rows rows = T::rows(p, m0);
    auto fetch = [&](int64_t k, int buf) {
#pragma unroll
        for (int h = 0; h < 2 * U; ++h) {
            if constexpr (ASYNC)
                T::stage_async(rows, k + h * 64, p.n_in, tiles[buf][h]);
            else
                T::stage_load(p, m0, k + h * 64, p.n_in, held[h]);
        }
    };
    auto land = [&](int buf) {
        if constexpr (!ASYNC) {
#pragma unroll
            for (int h = 0; h < 2 * U; ++h) T::stage_store(held[h], tiles[buf][h]);
        }
    };

    fetch(k0, 0);
    C::load(p, at, k0, c);
    land(0);
    int cur = 0;
    for (int64_t k = k0; k < k1; k += kAll, cur ^= 1) {
        if constexpr (ASYNC) wait_loads();
        __syncthreads();
        typename C::Chunks next;
        const bool more = k + kAll < k1;
        if (more) {
            fetch(k + kAll, cur ^ 1);
            C::load(p, at, k + kAll, next);
        }
        float scale[C::kS][NT][4];
        C::scales(p, k, c, scale);
        typename C::template Sums<MT> sum;
#pragma unroll
        for (int i = 0; i < 4 * U; ++i) {
            const uint32_t at_k = C::index(q, i % 4);
            const uint8_t *tile = tiles[cur][2 * (i / 4)] + (at_k >> 6) * kTile;
            u32x4 a[MT][PA];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int piece = lds_piece(m * 16 + (lane & 15), (at_k & 63) >> 3);
#pragma unroll
                for (int x = 0; x < PA; ++x) a[m][x] = *reinterpret_cast<const u32x4 *>(tile + x * T::kPlane + piece);
            }
            C::template step<PA, MT>(c, i / 4, i % 4, scale, a, sum, acc);
        }
        if (more) {
            land(cur ^ 1);
            c = next;
        }
    }

    auto store = [&](int64_t row, int64_t col, float v) {
        if (p.splits > 1)
            p.partial[(split * p.split_rows + row) * ((p.n_out + 3) & ~INT64_C(3)) + col] = v;
        else if (p.out_f32)
            static_cast<float *>(p.out)[row * p.ldo + col] = v;
        else
            static_cast<uint16_t *>(p.out)[row * p.ldo + col] = static_cast<uint16_t>(pack_rn(v, 0.0f));
    };
    // Adapters: each part of the contraction takes its share of them.
    [[maybe_unused]] float *given = nullptr;
    if constexpr (MODE == LinMode::adapted) {
        static_assert(NT == 2 && sizeof(tiles) >= 4 * T::kRows * NT * 16 * 4);
        __syncthreads();  // no wave reads activations any more
        given = reinterpret_cast<float *>(&tiles[0][0][0] + w * (T::kRows * NT * 16 * 4));
        adapter_rows<false, false, 3, NT, T::kRows, 4, 2>(p, m0, n0 + (lane & 15), static_cast<int>(split), p.splits, given);
    }
    auto more = [&](int m, int t, int i) {
        if constexpr (MODE == LinMode::adapted)
            return given[(m * 16 + 4 * q + i) * (16 * NT) + 16 * t + (lane & 15)];
        else
            return 0.0f;
    };
    uint32_t again = 0;  // of the lane's results, those out of range: stored once more at the end
    static_assert(NT * MT * 4 <= 32, "a bit each");
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t col = n0 + t * 16 + (lane & 15);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = m0 + m * 16 + 4 * q + i;
                if (row >= p.rows || col >= p.n_out) continue;
                const float v = acc[t][m][i] * kCodeScale<BITS>;
                again |= out_of_range(v) ? 1u << ((t * MT + m) * 4 + i) : 0u;
                if constexpr (MODE == LinMode::adapted)
                    store(row, col, v + more(m, t, i));
                else
                    store(row, col, v);
            }
    }
    for (; again != 0; again &= again - 1) {
        const int b = __builtin_ctz(again), t = b / (4 * MT), m = b / 4 % MT;
        const int64_t row = m0 + m * 16 + 4 * q + b % 4, col = n0 + t * 16 + (lane & 15);
        float v = scaled_sum<BITS, PA>(p, row, col, k0, k1);
        if constexpr (MODE == LinMode::adapted) v += more(m, t, b % 4);
        store(row, col, v);
    }
}

template <LinMode MODE, int BITS, int PA, int MT>
hipError_t launch_mid_as(const LinArgs &p, bool wide, hipStream_t stream) {
    constexpr int U = PA == 1 ? kMidChunks : 1;  // three parts of 64 rows fill LDS as they are
    const unsigned grid = static_cast<unsigned>(p.row_tiles * p.col_tiles * p.splits);
    if (wide)
        linear_mid_kernel<BITS, PA, kMidTiles, MT, U, true, MODE><<<grid, kBlockThreads, 0, stream>>>(p);
    else
        linear_mid_kernel<BITS, PA, kMidTiles, MT, U, false, MODE><<<grid, kBlockThreads, 0, stream>>>(p);
    return hipGetLastError();
}

template <LinMode MODE, int BITS, int PA>
hipError_t launch_mid_rows(const LinArgs &p, bool wide, int mt, hipStream_t stream) {
    if (mt == 1) return launch_mid_as<MODE, BITS, PA, 1>(p, wide, stream);
    if (mt == 2) return launch_mid_as<MODE, BITS, PA, 2>(p, wide, stream);
    return launch_mid_as<MODE, BITS, PA, 4>(p, wide, stream);
}

template <LinMode MODE>
hipError_t launch_mid(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream) {
    const bool wide = p.log2b >= 7 && p.n_in % kChunk == 0;
    if (bits == 4)
        return a_f32 ? launch_mid_rows<MODE, 4, 3>(p, wide, mt, stream) : launch_mid_rows<MODE, 4, 1>(p, wide, mt, stream);
    return a_f32 ? launch_mid_rows<MODE, 8, 3>(p, wide, mt, stream) : launch_mid_rows<MODE, 8, 1>(p, wide, mt, stream);
}

}  // namespace zpp
