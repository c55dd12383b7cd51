// linear_device.h - device helpers of the linear products on block-quantized
// weights (gfx950 matrix instructions, wave64).
#pragma once

#include "zpp_device.h"
#include "zpp_launch.h"

namespace zpp {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// D = A B + C on a 16x16 tile, 32 products deep, binary32 sums. Lane l holds
// A[l & 15][8 (l >> 4) + j] and B[8 (l >> 4) + j][l & 15], j = 0..7, and
// C[4 (l >> 4) + i][l & 15], i = 0..3.
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// Code i of a dword as binary32: the code itself for 8 bits, code / 16 for
// 4 bits (what the one conversion instruction for nibbles gives; exact). The
// factor goes back in, exactly, where the sum is finished: kCodeScale.
template <int BITS>
__device__ __forceinline__ float code_f32(uint32_t w, int i) {
    if constexpr (BITS == 8) return static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    // nibbles come out of whole bytes of w and of w >> 4, which the conversion selects by itself
    const uint32_t v = (i & 1) ? w >> 4 : w;
    return __builtin_amdgcn_cvt_off_f32_i4(static_cast<int>((v >> (8 * (i >> 1))) & 0xFFu));
}
template <int BITS>
constexpr float kCodeScale = BITS == 4 ? 16.0f : 1.0f;

// The high halves of two binary32 values as a bf16 pair (a in the low half):
// truncation, exact for values of at most 8 significant bits.
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
    return __builtin_amdgcn_perm(as_u(b), as_u(a), 0x07060302u);
}

// Two binary32 values rounded to nearest-even bf16, in one instruction.
__device__ __forceinline__ uint32_t pack_rn(float a, float b) {
    const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// x = hi + mid + lo exactly, each of at most 8 significant bits, by truncation
// (truncating cannot overflow to infinity). An infinite x is all in hi.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    p[0] = as_f(as_u(x) & 0xFFFF0000u);
    const float r = p[0] == x ? 0.0f : x - p[0];
    p[1] = as_f(as_u(r) & 0xFFFF0000u);
    p[2] = r - p[1];
}

// Two values as P bf16 pairs: rounded (P = 1) or split exactly (P = 3).
template <int P>
__device__ __forceinline__ void to_parts(float a, float b, uint32_t (&w)[P]) {
    if constexpr (P == 1) {
        w[0] = pack_rn(a, b);
    } else {
        float pa[3], pb[3];
        split3(a, pa);
        split3(b, pb);
#pragma unroll
        for (int i = 0; i < 3; ++i) w[i] = pack_hi(pa[i], pb[i]);
    }
}

// acc += A B over the parts of both operands. With 3 parts each, the products
// below 2^-24 of the largest are left out (mid*lo, lo*mid, lo*lo).
template <int PA, int PB>
__device__ __forceinline__ f32x4 mfma_parts(const u32x4 (&a)[PA], const u32x4 (&b)[PB], f32x4 c) {
#pragma unroll
    for (int i = PA - 1; i >= 0; --i)
#pragma unroll
        for (int j = PB - 1; j >= 0; --j)
            if (i + j <= 2) c = mfma16(a[i], b[j], c);
    return c;
}

// linear_mid.h's shape: tiles of 16 features a wave, chunks of 128 indices a step.
constexpr int kMidTiles = 2;
constexpr int kMidChunks = 2;

// Waits for this wave's loads, those into LDS among them, all but the last N, in
// a form the compiler counts too (it then waits for none of them again).
template <int N = 0>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "the counter has 6 bits, the upper 2 apart");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N), nothing else
    asm volatile("" ::: "memory");
}

// One product's operands, as the host describes them. a is [rows, C] with C
// the contraction length (in for the product, out for its gradient); the
// result is [rows, L].
struct LinArgs {
    const void *a;
    int64_t lda;
    int64_t rows;
    const uint8_t *codes;
    const float *scales;
    int64_t n_out, n_in;
    int log2b;
    void *out;
    int64_t ldo;
    int out_f32;
    float *partial;       // splits x split_rows x ldp sums when splits > 1
    int64_t split_rows;   // rows of the launch
    int splits;
    int64_t split_steps;  // contraction steps of each split
    int64_t row_tiles, col_tiles;
    int64_t plane;        // elements from one part of packed activations to the next
    // rows in groups, a weight matrix each: group e has rows offsets[e] .. offsets[e + 1] - 1,
    // counted from row0 before the launch's first
    const int32_t *offsets;
    int groups;
    int64_t row0;
    // rows with a low-rank adapter each (linear_adapt.h)
    const float *low;    // [rows][rank]: what the row has become
    const void *up;      // [adapters][out][rank] (y) or [adapters][rank][in] (dx)
    const int32_t *ids;  // [rows]: which adapter, none if it is no number below `adapters`; null: the first, all of them
    int up_f32, rank, adapters;
    int join_steps;  // rows in groups, in tiles (linear_tile.h): what kRound tiles' parts cost, in steps; 0: no parts
};

// What a product's rows multiply by: one matrix, that of the row's group, or one
// matrix and the row's adapter beside it.
enum class LinMode { one, grouped, adapted };

}  // namespace zpp
