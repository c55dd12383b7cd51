// linear_few.hip - y = x W^T on block codes for few rows of x (decoding): a
// stream over the codes.
//
//   y[m][n] = sum over chunks of k of s[n, chunk] * sum_k x[m][k] code[n][k]
//
// The codes are exact in bf16, so the inner sums have no rounding but the
// binary32 accumulation, and the scale multiplies each chunk's sum in
// binary32. binary32 activations go through the matrix instructions as three
// bf16 parts (exactly).
//
// Every code is read once from HBM by one wave, 16 bytes a lane, and used for
// up to 16*MT rows; with one row the matrix instruction still costs less than
// multiply-adds would: the conversion to bf16 pairs is about 1.6 instructions
// a code for any number of rows. A wave has NT tiles of 16 output features;
// the WK waves of a workgroup take chunks of 128 indices in turn and join
// their sums in LDS at the end, in wave order.
//
// WIDE: every 128-index chunk lies in one block (block >= 128 and in_features
// a multiple of 128), so a lane takes 32 neighbouring codes and one scale a
// chunk. Otherwise blocks may end at any multiple of 32: lanes take 8
// neighbouring codes of each 32 and a scale for each 32.
#include "linear_device.h"

namespace zpp {
namespace {

constexpr int kChunk = 128;

template <int BITS, int PA, int NT, int MT, bool WIDE>
struct Few {
    // One chunk of one wave, as loaded.
    struct Chunk {
        uint32_t w[NT][BITS == 4 ? 4 : 8];
        float s[NT][WIDE ? 1 : 4];
        u32x4 x[MT][4][PA == 3 ? 2 : 1];
    };

    static __device__ __forceinline__ void load(const LinArgs &p, int64_t n0, int64_t kc, Chunk &c) {
        const int lane = threadIdx.x & (kWave - 1), q = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t n = min(n0 + t * 16 + (lane & 15), p.n_out - 1);
            const int64_t row = n * p.n_in;
            if constexpr (WIDE) {
                const bool ok = kc < p.n_in;
                const int64_t e = row + (ok ? kc : 0) + q * 32;
#pragma unroll
                for (int h = 0; h < BITS / 4; ++h) {
                    const u32x4 v = ld_stream<u32x4>(p.codes + e * BITS / 8 + 16 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) c.w[t][4 * h + i] = v[i];
                }
                const float sc = p.scales[e >> p.log2b];
                c.s[t][0] = ok ? sc : 0.0f;
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int64_t k = kc + s * 32;
                    const bool ok = k < p.n_in;
                    const int64_t e = row + (ok ? k : 0) + q * 8;
                    if constexpr (BITS == 4) {
                        c.w[t][s] = ld<uint32_t>(p.codes + e / 2);
                    } else {
                        const u32x2 v = ld<u32x2>(p.codes + e);
                        c.w[t][2 * s] = v[0], c.w[t][2 * s + 1] = v[1];
                    }
                    const float sc = p.scales[e >> p.log2b];
                    c.s[t][s] = ok ? sc : 0.0f;
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int64_t row = min(static_cast<int64_t>(m * 16 + (lane & 15)), p.rows - 1);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int64_t k = kc + (WIDE ? q * 32 + s * 8 : s * 32 + q * 8);
                const bool ok = k < p.n_in;
                const uint8_t *at = static_cast<const uint8_t *>(p.a) + (row * p.lda + (ok ? k : 0)) * (PA == 3 ? 4 : 2);
#pragma unroll
                for (int h = 0; h < (PA == 3 ? 2 : 1); ++h) {
                    const u32x4 v = ld<u32x4>(at + 16 * h);
                    c.x[m][s][h] = ok ? v : u32x4{0, 0, 0, 0};
                }
            }
        }
    }

    static __device__ __forceinline__ void use(const Chunk &c, f32x4 (&acc)[NT][MT]) {
        f32x4 sum[NT][MT];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            u32x4 x[MT][PA];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if constexpr (PA == 1) {
                    x[m][0] = c.x[m][s][0];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[3];
                        to_parts<3>(as_f(c.x[m][s][j / 2][2 * (j % 2)]), as_f(c.x[m][s][j / 2][2 * (j % 2) + 1]), w);
#pragma unroll
                        for (int a = 0; a < 3; ++a) x[m][a][j] = w[a];
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 b[1];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    constexpr int per = 32 / BITS;
                    const int i = 8 * s + 2 * j;
                    b[0][j] = pack_hi(code_f32<BITS>(c.w[t][i / per], i % per),
                                      code_f32<BITS>(c.w[t][(i + 1) / per], (i + 1) % per));
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const bool first = !WIDE || s == 0;
                    sum[t][m] = mfma_parts<PA, 1>(x[m], b, first ? f32x4{0, 0, 0, 0} : sum[t][m]);
                    if (!WIDE || s == 3) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[t][m][i] = __builtin_fmaf(sum[t][m][i], c.s[t][WIDE ? 0 : s], acc[t][m][i]);
                    }
                }
            }
        }
    }
};

template <int BITS, int PA, int NT, int MT, bool WIDE, int WK, int U>
__global__ __launch_bounds__(WK *kWave) void linear_few_kernel(LinArgs p) {
    using F = Few<BITS, PA, NT, MT, WIDE>;
    constexpr int kSums = NT * MT * 256;  // of one wave
    __shared__ float sums[WK][kSums];
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
    const int64_t n0 = xcd_block(blockIdx.x, gridDim.x) * (16 * NT);

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0, 0, 0, 0};

    const int64_t chunks = (p.n_in + kChunk - 1) / kChunk;
    for (int64_t i = w; i < chunks; i += U * WK) {
        typename F::Chunk c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) F::load(p, n0, (i + u * WK) * kChunk, c[u]);  // past the end: zeros
#pragma unroll
        for (int u = 0; u < U; ++u) F::use(c[u], acc);
    }

#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[w][((t * MT + m) * 4 + i) * 64 + lane] = acc[t][m][i];
    __syncthreads();
    for (int o = threadIdx.x; o < kSums; o += WK * kWave) {
        const int l = o & 63, i = o >> 6 & 3, m = (o >> 8) % MT, t = (o >> 8) / MT;
        const int64_t row = m * 16 + 4 * (l >> 4) + i, col = n0 + t * 16 + (l & 15);
        if (row >= p.rows || col >= p.n_out) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WK; ++k) v += sums[k][o];
        v *= kCodeScale<BITS>;
        if (p.out_f32)
            static_cast<float *>(p.out)[row * p.ldo + col] = v;
        else
            static_cast<uint16_t *>(p.out)[row * p.ldo + col] = static_cast<uint16_t>(pack_rn(v, 0.0f));
    }
}

template <int BITS, int PA, int NT, int MT, int WK, int U>
hipError_t launch_as(const LinArgs &p, bool wide, hipStream_t stream) {
    const unsigned grid = static_cast<unsigned>((p.n_out + 16 * NT - 1) / (16 * NT));
    if (wide)
        linear_few_kernel<BITS, PA, NT, MT, true, WK, U><<<grid, WK * kWave, 0, stream>>>(p);
    else
        linear_few_kernel<BITS, PA, NT, MT, false, WK, U><<<grid, WK * kWave, 0, stream>>>(p);
    return hipGetLastError();
}

template <int BITS, int PA>
hipError_t launch_rows(const LinArgs &p, bool wide, hipStream_t stream) {
    if (p.rows <= 16) return launch_as<BITS, PA, 2, 1, 8, PA == 1 ? 2 : 1>(p, wide, stream);
    if (p.rows <= 32) return launch_as<BITS, PA, 2, 2, 8, 1>(p, wide, stream);
    return launch_as<BITS, PA, 2, 4, 4, 1>(p, wide, stream);
}

}  // namespace

hipError_t launch_linear_few(const LinArgs &p, int bits, bool a_f32, hipStream_t stream) {
    const bool wide = p.log2b >= 7 && p.n_in % kChunk == 0;
    if (bits == 4) return a_f32 ? launch_rows<4, 3>(p, wide, stream) : launch_rows<4, 1>(p, wide, stream);
    return a_f32 ? launch_rows<8, 3>(p, wide, stream) : launch_rows<8, 1>(p, wide, stream);
}

}  // namespace zpp
