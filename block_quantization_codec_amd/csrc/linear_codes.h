// linear_codes.h - codes read exactly, for the products that multiply by the
// codes themselves and apply the scales to sums (few rows of activations).
//
//   y[m][n] = sum over chunks of k of s[n, chunk] * sum_k x[m][k] code[n][k]
//
// Codes are exact in bf16, so the inner sums have no rounding but the binary32
// accumulation, and the scale multiplies each chunk's sum in binary32.
// 4-bit codes are converted one by one: pairs made by bit operations alone carry
// an offset, whose sum with a large activation leaves little of the others' even
// where the code there is zero, and they saved 3% of the time of one row.
//
// A wave reads NT tiles of 16 output features, U chunks of 128 indices at a
// time. WIDE: every chunk lies in one block (block >= 128 and in_features a
// multiple of 128), so a lane takes 16-byte pieces and each feature one scale
// a chunk. Otherwise blocks may end at any multiple of 32: lanes take 8
// neighbouring codes of each 32 and there is a scale for each 32.
//
// Sums before their scale reach 2^14 times the largest activation, so from 2^114
// on they can be infinite (or NaN) where the result is not; such a result is
// computed again, each weight scaled first (scaled_sum). Once infinite a sum
// stays infinite or NaN, so finite results need no other look.
#pragma once

#include "linear_device.h"

namespace zpp {

constexpr int kChunk = 128;

// One scale a lane, of row (lane & 15) and of the quarter's chunk, to four
// scales of the row, the same in all quarters.
__device__ __forceinline__ void spread(float v, float (&s)[4]) {
    const auto h = __builtin_amdgcn_permlane16_swap(as_u(v), as_u(v), false, false);  // quarters 0 0 2 2, 1 1 3 3
    const auto a = __builtin_amdgcn_permlane32_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(h[1], h[1], false, false);
    s[0] = as_f(a[0]), s[1] = as_f(b[0]), s[2] = as_f(a[1]), s[3] = as_f(b[1]);
}

// 8 activations (as loaded: 16 bytes of bf16, 32 of binary32) as bf16 parts.
template <int PA>
__device__ __forceinline__ void parts_of(const u32x4 (&v)[PA == 3 ? 2 : 1], u32x4 (&x)[PA]) {
    if constexpr (PA == 3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[3];
            to_parts<3>(as_f(v[j / 2][2 * (j % 2)]), as_f(v[j / 2][2 * (j % 2) + 1]), w);
#pragma unroll
            for (int a = 0; a < 3; ++a) x[a][j] = w[a];
        }
    } else {
        x[0] = v[0];
    }
}

template <int BITS, int NT, int U, bool WIDE>
struct CodeStream {
    static constexpr int kUnit = WIDE ? 7 : 5;    // log2 of the indices of one scale
    static constexpr int kS = WIDE ? (U + 3) / 4 : U;  // loads of scales, four a load
    static constexpr int kW = BITS == 4 ? 4 : 8;  // dwords of a chunk's codes

    // What stays the same over the chunks. Bases are the same in every lane of
    // the wave; lanes add 32-bit offsets.
    struct At {
        const uint8_t *codes;
        const float *scales;
        uint32_t code[NT], unit[NT];
        int shift;
    };

    // For the wave's features n0 .. n0 + 16 NT - 1 (n0 < out_features).
    static __device__ __forceinline__ At place(const LinArgs &p, int64_t n0) {
        const int lane = threadIdx.x & (kWave - 1), q = lane >> 4;
        At a;
        const int64_t units = p.n_in >> kUnit, first = n0 * units;
        a.shift = p.log2b - kUnit;
        a.codes = p.codes + n0 * p.n_in * BITS / 8;
        a.scales = p.scales + (first >> a.shift);
        const uint32_t rem = static_cast<uint32_t>(first & ((INT64_C(1) << a.shift) - 1));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t n =
                static_cast<uint32_t>(min(static_cast<int64_t>(t * 16 + (lane & 15)), p.n_out - 1 - n0));
            // 16 bytes a quarter in each 64-byte run; 8 codes a quarter of each 32. Up to 32 rows of 2^22 codes.
            static_assert(NT <= 2, "offsets are 32-bit");
            a.code[t] = n * static_cast<uint32_t>(p.n_in * BITS / 8) + q * (WIDE ? 16 : BITS);
            a.unit[t] = rem + n * static_cast<uint32_t>(units);
        }
        return a;
    }

    // Where in a chunk the lane's 8 indices of instruction s begin.
    static __device__ __forceinline__ uint32_t index(uint32_t q, uint32_t s) {
        if constexpr (!WIDE) return s * 32 + q * 8;
        return BITS == 4 ? q * 32 + s * 8 : (s >> 1) * 64 + q * 16 + (s & 1) * 8;
    }

    // U chunks of one wave, as loaded.
    struct Chunks {
        uint32_t w[U][NT][kW];
        float s[kS][NT];
    };

    // A chunk, or 32-index step of one, past the end is the last one again;
    // scales() gives it a scale of zero.
    static __device__ __forceinline__ void load(const LinArgs &p, const At &a, int64_t k0, Chunks &c) {
        const uint32_t q = (threadIdx.x & (kWave - 1)) >> 4;
        const uint32_t n_in = static_cast<uint32_t>(p.n_in), k = static_cast<uint32_t>(k0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (WIDE) {
                const uint8_t *codes = a.codes + static_cast<int64_t>(min(k + u * kChunk, n_in - kChunk)) * BITS / 8;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int h = 0; h < BITS / 4; ++h) {
                        const u32x4 v = ld<u32x4>(codes + 64 * h + a.code[t]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) c.w[u][t][4 * h + i] = v[i];
                    }
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint8_t *codes =
                        a.codes + static_cast<int64_t>(min(k + u * kChunk + s * 32, n_in - 32)) * BITS / 8;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if constexpr (BITS == 4) {
                            c.w[u][t][s] = ld<uint32_t>(codes + a.code[t]);
                        } else {
                            const u32x2 v = ld<u32x2>(codes + a.code[t]);
                            c.w[u][t][2 * s] = v[0], c.w[u][t][2 * s + 1] = v[1];
                        }
                    }
                }
            }
        }
        // each quarter loads another chunk's scales (WIDE), or another 32-index step's
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const uint32_t unit = min((k >> kUnit) + i * 4 + q, (n_in >> kUnit) - 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) c.s[i][t] = a.scales[(a.unit[t] + unit) >> a.shift];
        }
    }

    // The scales of the chunks' units, in every quarter.
    static __device__ __forceinline__ void scales(const LinArgs &p, int64_t k0, const Chunks &c,
                                                  float (&scale)[kS][NT][4]) {
        const uint32_t left = k0 < p.n_in ? static_cast<uint32_t>(p.n_in - k0) >> kUnit : 0;
#pragma unroll
        for (int i = 0; i < kS; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                spread(c.s[i][t], scale[i][t]);
#pragma unroll
                for (int u = 0; u < 4; ++u) scale[i][t][u] = i * 4 + u < left ? scale[i][t][u] : 0.0f;
            }
    }

    // A chunk's sums before they are scaled.
    template <int MT>
    struct Sums {
        f32x4 v[NT][MT];
    };

    // Instruction s of chunk u for all the rows, whose operands are a; acc takes
    // each sum at the end of its scale's indices.
    template <int PA, int MT>
    static __device__ __forceinline__ void step(const Chunks &c, int u, int s, const float (&scale)[kS][NT][4],
                                                const u32x4 (&a)[MT][PA], Sums<MT> &sum, f32x4 (&acc)[NT][MT]) {
        const f32x4 zero = {0, 0, 0, 0};
        const bool first = !WIDE || s == 0, last = !WIDE || s == 3;
        u32x4 b[NT][1];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int per = 32 / BITS;
                const int i = 8 * s + 2 * j;
                b[t][0][j] = pack_hi(code_f32<BITS>(c.w[u][t][i / per], i % per),
                                     code_f32<BITS>(c.w[u][t][i / per], i % per + 1));
            }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                sum.v[t][m] = mfma_parts<PA, 1>(a[m], b[t], first ? zero : sum.v[t][m]);
                if (!last) continue;
                const float f = WIDE ? scale[u / 4][t][u % 4] : scale[u][t][s];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t][m][i] = __builtin_fmaf(sum.v[t][m][i], f, acc[t][m][i]);
            }
        }
    }
};

// Whether a result has to be computed again.
__device__ __forceinline__ bool out_of_range(float v) { return !(__builtin_fabsf(v) <= 3.402823466e38f); }

// sum over k in [k0, k1) of x[row][k] * RN(code * scale), one lane's by itself: 32
// indices, which have one scale, at a time, as long as the sum is finite. 0.2 to
// 0.4 ms for the results of a few rows of 28672 x 8192.
template <int BITS, int PA>
__device__ __forceinline__ float scaled_sum(const LinArgs &p, int64_t row, int64_t col, int64_t k0, int64_t k1) {
    float v = 0.0f;
    for (int64_t k = k0; k < k1 && !out_of_range(v); k += 32) {
        const int64_t e = col * p.n_in + k;
        const float scale = p.scales[e >> p.log2b];
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {  // 8 indices
            const uint8_t *codes = p.codes + (e + 8 * j) * BITS / 8;
            const uint8_t *x = static_cast<const uint8_t *>(p.a) + (row * p.lda + k + 8 * j) * (PA == 3 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = code_f32<BITS>(ld<uint32_t>(codes + 4 * (i * BITS / 32)), i % (32 / BITS));
                const float a = PA == 3 ? ld<float>(x + 4 * i) : as_f(static_cast<uint32_t>(ld<uint16_t>(x + 2 * i)) << 16);
                v = __builtin_fmaf(a, c * kCodeScale<BITS> * scale, v);
            }
        }
    }
    return v;
}

}  // namespace zpp
