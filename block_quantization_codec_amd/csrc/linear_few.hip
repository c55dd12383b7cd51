// linear_few.hip - y = x W^T on block codes for one to four rows of x
// (decoding): a stream over the codes.
//
// Every code is read once from HBM by one wave, 16 bytes a lane, and used for
// all rows; even with one row the matrix instruction costs less than
// multiply-adds would: some 1.6 instructions a code make 4-bit codes bf16
// pairs, for any number of rows. A wave has NT tiles of 16 output features;
// the WK waves of a workgroup take U chunks of 128 indices in turn and join
// their sums in LDS at the end, in wave order.
//
// One row of 28672 x 8192 int4: 28 to 28.5 us, 4.4 TB/s of codes and scales, vector
// instructions issued for 0.65 of the time (4 rows: 38 us); 1024 x 8192: 6.0 us, of which the launch, a load's round trip and the join
// are most.
// x in registers and rotated into place takes one load for 16 instructions'
// operands: loaded for each, x took as much of the path from L2 as the codes
// and the first case 54 us. Non-temporal loads gained nothing.
#include "linear_codes.h"

namespace zpp {
namespace {

// A row's lane i takes lane (i + c) mod 16's value.
template <int C>
__device__ __forceinline__ uint32_t rotate(uint32_t v) {
    if constexpr (C % 16 == 0) return v;
    return dpp_u32<0x120 + (16 - C % 16) % 16>(v);
}

template <int C, int PA>
__device__ __forceinline__ void rotate_parts(const u32x4 (&v)[PA], u32x4 (&o)[PA]) {
#pragma unroll
    for (int a = 0; a < PA; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[a][j] = rotate<C>(v[a][j]);
}

// RM is the number of rows of x that lie in one operand (a power of two below
// 16): the lanes of a quarter load 16 / RM operands' pieces at once, and each
// operand is a rotation of them.
template <int BITS, int PA, int NT, int RM, int U, bool WIDE>
struct Few {
    using C = CodeStream<BITS, NT, U, WIDE>;
    static constexpr int kPer = 16 / RM;                  // operands of one load of x
    static constexpr int kX = (4 * U + kPer - 1) / kPer;  // loads of x
    using Raw = u32x4[kX][PA == 3 ? 2 : 1];

    // Operand i = l * kPer + (lane & 15) / RM is instruction i % 4 of chunk i / 4.
    static __device__ __forceinline__ void load_x(const LinArgs &p, const uint8_t *row, int64_t k0, Raw &x) {
        const uint32_t lane = threadIdx.x & (kWave - 1), q = lane >> 4, j = lane & 15;
        const uint32_t n_in = static_cast<uint32_t>(p.n_in), k = static_cast<uint32_t>(k0);
#pragma unroll
        for (int l = 0; l < kX; ++l) {
            const uint32_t i = l * kPer + j / RM, u = i / 4, s = i % 4;
            const uint32_t at = k + u * kChunk + C::index(q, s);
            // past the end the codes are the last ones again, with scales of zero: any x of the row will do
            const uint8_t *from = row + min(at, n_in - 8) * (PA == 3 ? 4 : 2);
#pragma unroll
            for (int h = 0; h < (PA == 3 ? 2 : 1); ++h) x[l][h] = ld<u32x4>(from + 16 * h);
        }
    }

    template <int I>
    static __device__ __forceinline__ void use_from(const u32x4 (&x)[kX][PA], const typename C::Chunks &c,
                                                    const float (&scale)[C::kS][NT][4], f32x4 (&acc)[NT][1]) {
        u32x4 a[4][1][PA];
        rotate_parts<I % kPer * RM, PA>(x[I / kPer], a[0][0]);
        rotate_parts<(I + 1) % kPer * RM, PA>(x[(I + 1) / kPer], a[1][0]);
        rotate_parts<(I + 2) % kPer * RM, PA>(x[(I + 2) / kPer], a[2][0]);
        rotate_parts<(I + 3) % kPer * RM, PA>(x[(I + 3) / kPer], a[3][0]);
        typename C::template Sums<1> sum;
#pragma unroll
        for (int s = 0; s < 4; ++s) C::template step<PA, 1>(c, I / 4, s, scale, a[s], sum, acc);
        if constexpr (I + 4 < 4 * U) use_from<I + 4>(x, c, scale, acc);
    }
};

template <int BITS, int PA, int NT, int RM, int U, bool WIDE, int WK>
__global__ __launch_bounds__(WK *kWave) void linear_few_kernel(LinArgs p) {
    using F = Few<BITS, PA, NT, RM, U, WIDE>;
    using C = typename F::C;
    __shared__ float sums[WK][NT * 256];
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
    const int64_t n0 = xcd_block(blockIdx.x, gridDim.x) * (16 * NT);
    const typename C::At at = C::place(p, n0);
    const uint8_t *row = static_cast<const uint8_t *>(p.a) +
                         min(static_cast<int64_t>(lane % RM), p.rows - 1) * p.lda * (PA == 3 ? 4 : 2);

    f32x4 acc[NT][1];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = f32x4{0, 0, 0, 0};

    // a wave's U chunks are neighbours: their codes fill whole cache lines
    for (int64_t k = static_cast<int64_t>(w) * U * kChunk; k < p.n_in; k += U * WK * kChunk) {
        typename C::Chunks c;
        typename F::Raw raw;
        C::load(p, at, k, c);
        F::load_x(p, row, k, raw);
        float scale[C::kS][NT][4];
        C::scales(p, k, c, scale);
        u32x4 x[F::kX][PA];
#pragma unroll
        for (int l = 0; l < F::kX; ++l) parts_of<PA>(raw[l], x[l]);
        F::template use_from<0>(x, c, scale, acc);
    }

    // rows 0..3 of a sum are its quarter 0's
    if (lane < 16) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[w][(t * 4 + i) * 16 + lane] = acc[t][0][i];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < NT * 64; o += WK * kWave) {
        const int64_t row_out = o >> 4 & 3, col = n0 + (o >> 6) * 16 + (o & 15);
        if (row_out >= p.rows || col >= p.n_out) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WK; ++k) v += sums[k][o];
        v *= kCodeScale<BITS>;
        if (out_of_range(v)) v = scaled_sum<BITS, PA>(p, row_out, col, 0, p.n_in);
        if (p.out_f32)
            static_cast<float *>(p.out)[row_out * p.ldo + col] = v;
        else
            static_cast<uint16_t *>(p.out)[row_out * p.ldo + col] = static_cast<uint16_t>(pack_rn(v, 0.0f));
    }
}

template <int BITS, int PA, int RM>
hipError_t launch_as(const LinArgs &p, bool wide, hipStream_t stream) {
    constexpr int NT = 1, U = 4, WK = 8;
    const unsigned grid = static_cast<unsigned>((p.n_out + 16 * NT - 1) / (16 * NT));
    if (wide)
        linear_few_kernel<BITS, PA, NT, RM, U, true, WK><<<grid, WK * kWave, 0, stream>>>(p);
    else
        linear_few_kernel<BITS, PA, NT, RM, U, false, WK><<<grid, WK * kWave, 0, stream>>>(p);
    return hipGetLastError();
}

template <int BITS, int PA>
hipError_t launch_rows(const LinArgs &p, bool wide, hipStream_t stream) {
    if (p.rows == 1) return launch_as<BITS, PA, 1>(p, wide, stream);
    if (p.rows == 2) return launch_as<BITS, PA, 2>(p, wide, stream);
    return launch_as<BITS, PA, 4>(p, wide, stream);
}

}  // namespace

hipError_t launch_linear_few(const LinArgs &p, int bits, bool a_f32, hipStream_t stream) {
    const bool wide = p.log2b >= 7 && p.n_in % kChunk == 0;
    if (bits == 4) return a_f32 ? launch_rows<4, 3>(p, wide, stream) : launch_rows<4, 1>(p, wide, stream);
    return a_f32 ? launch_rows<8, 3>(p, wide, stream) : launch_rows<8, 1>(p, wide, stream);
}

}  // namespace zpp
