// linear_big.h - y = x W^T and dx = dy W on block codes, many rows at once: a
// tiled matrix product that converts the codes in registers.
//
//   y[m][n]  = sum_k x[m][k]  W[n][k]      (contraction over in_features)
//   dx[m][k] = sum_n dy[m][n] W[n][k]      (contraction over out_features)
//   W[n][k]  = code[n*K + k] * s[(n*K + k) / B]
//
// A workgroup of 4 waves computes 16*MT rows x 256 columns; each wave has 64
// columns of all the rows, so every code is read and converted by exactly one
// wave of the workgroup, straight from global memory into the layout of the
// matrix instruction's B operand, and never passes through LDS. What the
// waves share, the activations, lies in LDS.
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
// three (24 bits, exactly; packed beforehand, see linear.hip). Weights are
// RN_bf16(code * s) for bf16 results: the value zpp_dequantize_blocks gives a
// caller who multiplies in bf16. Each is off by at most 2^-8 of itself (equal codes
// of a block alike), so a result by at most 2^-8 of its products' magnitudes and
// usually by about as much as its own rounding: 4096 rows of 8192 -> 28672, 2.4e-3
// of the results' norm in place of 1.7e-3. That is one product in place of the
// three that a caller gets by asking for binary32 results: weights are three parts
// of RN(code * s) where input or result is binary32 (forward, bf16 to binary32
// takes exact codes instead, linear_mid.h), and two of it in the gradients of few rows that
// linear.hip says. Sums are binary32 throughout.
//
// A step is taken in two halves of 32 indices (one matrix instruction deep).
// With 256 rows a wave has the SIMD to itself (256 sums a lane), so nothing but
// its own instructions hides a wait, and everything is asked for early:
//   - activations go straight to LDS, BUFS - 1 steps ahead;
//   - codes and scales are loaded DEPTH - 1 steps before they are converted;
//   - each half converts the next half's B operands between its matrix
//     instructions, 16 / MT dwords after each row of tiles;
//   - A operands are read from LDS rows of tiles ahead, across the ends of
//     halves and steps: the one barrier of a step stands in its middle, after
//     which the next step's activations can be read;
//   - loads are spread over the step: four waves' loads all at once hold up
//     all four.
// The pipeline takes DEPTH steps at a time; steps past the end multiply by
// scales of zero. What is left over of the contraction, less than 64 indices,
// is one guarded step more. Steps are short with few rows, so those go further
// ahead.
//
// 4096 x 8192 by 28672 x 8192 int4, bf16: 1.53 to 1.56 ms, 1.23 to 1.25 PFLOP/s,
// the matrix units busy for 0.57 of the cycles at the clock that the power
// limit leaves (2.1 GHz); a library product of bf16 weights of that size takes
// 1.37 ms. Tried: 128-row tiles (two workgroups a CU: 18% slower, the conversion
// of each code is shared by half the rows), loads of a step in one burst (+13%),
// a barrier that drains the loads (+9%). 4096 x 8192 by 8192 x 8192 int8,
// gradient: 0.46 to 0.48 ms. With few rows one wave a SIMD waits for itself:
// gradient of 512 x 1024 through 1024 x 8192 int4, 24 us in 16 steps.
#pragma once

#include <type_traits>

#include "linear_adapt.h"
#include "linear_tile.h"

namespace zpp {

// acc += A B. PIN keeps the sums in accumulation registers: 256 of them leave
// the compiler's allocator none to move one through, and in the loop it then
// moves them through the others and memory. (Outside the loop, the bf16 kernels of
// 64 to 256 rows copy sums where their paths meet, and those of 128 rows put one
// or two addresses into scratch memory before the loop and fetch them after it.)
// The instruction is written out for that, so the compiler does not know that
// operands written by ordinary instructions have to be two wait states old:
// operands_ready() stands before every run of these, and within a run nothing
// but LDS reads (which are waited for) writes an operand. Nor does it know how
// long the sums have to be left alone: sums_ready().
template <bool PIN>
__device__ __forceinline__ void mfma(u32x4 a, u32x4 b, f32x4 &acc) {
    if constexpr (PIN)
        asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else
        acc = mfma16(a, b, acc);
}

template <bool PIN>
__device__ __forceinline__ void operands_ready() {
    if constexpr (PIN) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 1");
        __builtin_amdgcn_sched_barrier(0);
    }
}

// After a run of mfma<true>, in the same basic block: the eight wait states
// before anything but another product may read or write the sums, a copy that
// the compiler makes where control flow meets among them.
template <bool PIN>
__device__ __forceinline__ void sums_ready() {
    if constexpr (PIN) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 7");
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A barrier that waits for no memory operation of the wave's own: neither the
// loads nor the LDS reads under way have to be over for what it keeps apart.
__device__ __forceinline__ void barrier_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <bool GRAD, int BITS, int PA, int PB, int MT>
struct LinBig {
    static constexpr bool kPin = MT >= 4;
    using Tile = LinTile<PA, MT>;
    static constexpr int kRows = 16 * MT;
    static constexpr int kPlane = Tile::kPlane;
    static constexpr int kBytes = PA * kPlane;        // of a step's activations
    static constexpr int kGroups = (2 * MT + 3) / 4;  // 8-row groups of activations a wave stages, of each part
    static constexpr int kAhead = MT >= 16 ? 7 : MT >= 4 ? 3 : 0;  // rows of tiles that A is read ahead
    static constexpr int kRing = MT >= 16 ? 8 : MT >= 4 ? 4 : 1;
    // Buffers of activations: up to 8, within 144 KB of LDS (72 KB where two
    // workgroups share a CU). Sets of codes in registers.
    static constexpr int kBufs = PA == 3 ? (MT == 8 ? 3 : MT == 4 ? 4 : 8) : MT >= 8 ? 4 : 8;
    static constexpr int kDepth = MT >= 8 || (PB > 1 && MT == 4) ? 2 : 4;

    // Codes of 16 indices of a lane's 4 columns; scales of the 4 columns (y),
    // or of index (lane & 15) in both 32-column halves (dx).
    struct Raw {
        uint32_t w[GRAD ? 16 : (BITS == 4 ? 8 : 16)];
        float s[GRAD ? 2 : 4];
    };

    // Bases are the same in every lane of a wave; lanes add 32-bit offsets.
    // Scales are counted in units of 32 weights, relative to a base.
    struct At {
        const uint8_t *a;  // activations from the tile's first row on
        int64_t plane;     // bytes from one part to the next
        uint32_t piece[kGroups];
        const uint8_t *codes;
        uint32_t code[GRAD ? 1 : 4], unit[GRAD ? 1 : 4];
        int64_t first;  // the base's unit: of the wave's first row (y), of its first column (dx)
        int64_t units;  // of a row
        uint32_t half;  // dx: from the first 32 columns' unit to the second's (0 at the end)
        int shift;
    };

    static __device__ __forceinline__ At place(const LinArgs &p, int64_t m0, int64_t wave_col) {
        const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
        const uint32_t q = lane >> 4, j = lane & 15;
        At at;
        at.a = static_cast<const uint8_t *>(p.a) + m0 * p.lda * 2;
        at.plane = p.plane * 2;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int r = (i * 4 + w) * 8 + (lane >> 3), c = (lane & 7) ^ (r & 7);
            at.piece[i] = static_cast<uint32_t>(min(static_cast<int64_t>(r), p.rows - 1 - m0) * p.lda * 2) + c * 16;
        }
        at.shift = p.log2b - 5;
        at.units = p.n_in >> 5;
        at.half = 0;
        if constexpr (GRAD) {
            const int64_t c0 = wave_col < p.n_in ? wave_col : 0;
            const uint32_t col = static_cast<uint32_t>(min(static_cast<int64_t>(j * 4), p.n_in - 4 - c0));
            at.codes = p.codes + c0 * BITS / 8;
            at.code[0] = (q * 16 * static_cast<uint32_t>(p.n_in / 4) + col / 4) * (BITS / 2);
            at.first = c0 >> 5;
            at.half = at.first + 1 < at.units ? 1 : 0;
            at.unit[0] = (q * 16 + j) * static_cast<uint32_t>(at.units);
        } else {
            const int64_t n0 = min(wave_col, p.n_out - 1);
            at.codes = p.codes + n0 * p.n_in * BITS / 8;
            at.first = n0 * at.units;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t n = static_cast<uint32_t>(min(static_cast<int64_t>(j * 4 + t), p.n_out - 1 - n0));
                at.code[t] = n * static_cast<uint32_t>(p.n_in * BITS / 8) + q * (2 * BITS);
                at.unit[t] = n * static_cast<uint32_t>(at.units) + (q >> 1);
            }
        }
        return at;
    }

    // Loads I .. END - 1 of the kGroups * PA of a whole step's activations.
    template <int I, int END>
    static __device__ __forceinline__ void stage(const At &at, int64_t step, uint8_t *tile) {
#if defined(__HIP_DEVICE_COMPILE__)
        // A buffer load: its scalar offset takes the step, so that no lane computes
        // an address, and it counts as a global load alone. Offsets are 32-bit; the
        // plan packs activations of longer row strides. 0x27000: plain 32-bit data.
        const int w = wave_in_block();
#pragma unroll
        for (int i = I; i < END; ++i) {
            const int x = i / kGroups, g = i % kGroups * 4 + w;
            if (2 * MT % 4 != 0 && g >= 2 * MT) continue;
            const __amdgpu_buffer_rsrc_t from =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(at.a + x * at.plane), 0, 0xFFFFFFFFu, 0x27000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                from, (__attribute__((address_space(3))) void *)(tile + x * kPlane + g * 1024), 16,
                at.piece[i % kGroups], static_cast<int>(step * 128), 0, 0);
        }
#endif
    }

    // Where a whole step's codes and scales begin.
    struct From {
        const uint8_t *codes;
        const float *scales;
        uint32_t rem;
    };
    static __device__ __forceinline__ From from(const LinArgs &p, const At &at, int64_t step) {
        const int64_t first = at.first + (GRAD ? step * 64 * at.units : step * 2);
        return From{at.codes + (GRAD ? step * 64 * (p.n_in * BITS / 8) : step * (8 * BITS)),
                    p.scales + (first >> at.shift),
                    static_cast<uint32_t>(first & ((INT64_C(1) << at.shift) - 1))};
    }

    // The loads of a step's codes and scales, in the order in which the
    // conversion is done with the registers they go to.
    static constexpr int kLoads = GRAD ? 18 : 8;
    template <int I>
    static __device__ __forceinline__ void load_one(const LinArgs &p, const At &at, const From &f, Raw &r) {
        if constexpr (GRAD && I < 16) {
            const uint8_t *codes = f.codes + I * (p.n_in * BITS / 8);
            if constexpr (BITS == 4)
                r.w[I] = ld<uint16_t>(codes + at.code[0]);
            else
                r.w[I] = ld<uint32_t>(codes + at.code[0]);
        } else if constexpr (GRAD) {
            r.s[I - 16] = f.scales[(at.unit[0] + f.rem + (I - 16) * at.half) >> at.shift];
        } else {
            constexpr int t = I / 2;
            if constexpr (I % 2 == 1) {
                r.s[t] = f.scales[(at.unit[t] + f.rem) >> at.shift];
            } else if constexpr (BITS == 4) {
                const u32x2 v = ld<u32x2>(f.codes + at.code[t]);
#pragma unroll
                for (int i = 0; i < 2; ++i) r.w[2 * t + i] = v[i];
            } else {
                const u32x4 v = ld<u32x4>(f.codes + at.code[t]);
#pragma unroll
                for (int i = 0; i < 4; ++i) r.w[4 * t + i] = v[i];
            }
        }
    }
    template <int I, int END>
    static __device__ __forceinline__ void load_range(const LinArgs &p, const At &at, const From &f, Raw &r) {
        if constexpr (I < END) {
            load_one<I>(p, at, f, r);
            load_range<I + 1, END>(p, at, f, r);
        }
    }

    // The first half of a step converts the second half of its codes; after a
    // register's last use there the step after next is loaded into it. How many
    // of the loads may stand before row of tiles m, and not all at its start:
    // four waves' loads at once hold up all of them.
    static constexpr int loads_before(int m) {
        const int done = 16 * m / MT / 4;  // fours of dwords converted
        if (m < 0) return 0;
        const int free = GRAD ? 8 + 2 * done : 2 * done, share = kLoads * (m + 1) / MT;
        return m >= MT ? kLoads : free < share ? free : share;
    }

    // A guarded step's activations: zeros past the end.
    static __device__ __forceinline__ void stage_last(const LinArgs &p, int64_t m0, int64_t c0, int64_t c_len,
                                                      uint8_t *tile) {
#pragma unroll
        for (int x = 0; x < PA; ++x) {
            LinArgs part = p;
            part.a = static_cast<const uint16_t *>(p.a) + x * p.plane;
            Tile::stage_async(Tile::rows(part, m0), c0, c_len, tile + x * kPlane);
        }
    }

    // A guarded step: indices past the end read valid codes (their activations are zeros).
    static __device__ __forceinline__ void load_last(const LinArgs &p, int64_t wave_col, int64_t c0, Raw &r) {
        const int lane = threadIdx.x & (kWave - 1);
        const int64_t q = lane >> 4, j = lane & 15;
        if constexpr (GRAD) {
            const int64_t col = wave_col < p.n_in ? wave_col : 0, k = min(col + j * 4, p.n_in - 4);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t e = min(c0 + q * 16 + i, p.n_out - 1) * p.n_in + k;
                r.w[i] = BITS == 4 ? static_cast<uint32_t>(ld<uint16_t>(p.codes + e / 2)) : ld<uint32_t>(p.codes + e);
            }
            const int64_t row = min(c0 + q * 16 + j, p.n_out - 1) * p.n_in;
#pragma unroll
            for (int h = 0; h < 2; ++h) r.s[h] = p.scales[(row + min(col + 32 * h, p.n_in - 32)) >> p.log2b];
        } else {
            const int64_t k = min(c0 + q * 16, p.n_in - 16);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t e = min(wave_col + j * 4 + t, p.n_out - 1) * p.n_in + k;
#pragma unroll
                for (int i = 0; i < BITS / 2; ++i) r.w[BITS / 2 * t + i] = ld<uint32_t>(p.codes + e * BITS / 8 + 4 * i);
                r.s[t] = p.scales[e >> p.log2b];
            }
        }
    }

    // A set's scales; zeros for a step past the end.
    using Scales = float[GRAD ? 2 : 4];
    static __device__ __forceinline__ void scales(const Raw &r, bool live, Scales &s) {
#pragma unroll
        for (int i = 0; i < (GRAD ? 2 : 4); ++i) s[i] = live ? r.s[i] : 0.0f;
    }

    // The scale of index I of the lane's 16, in the lane's own half of the columns.
    template <int I>
    static __device__ __forceinline__ float row_scale(const Scales &s) {
        // every lane of a row takes lane I's
        const int lo = __builtin_amdgcn_mov_dpp(static_cast<int>(as_u(s[0])), 0x150 + I, 0xF, 0xF, true);
        const int hi = __builtin_amdgcn_mov_dpp(static_cast<int>(as_u(s[1])), 0x150 + I, 0xF, 0xF, true);
        return as_f(static_cast<uint32_t>((threadIdx.x & 8) ? hi : lo));
    }

    // B operands of a half: parts of four tiles.
    using B = u32x4[PB][4];

    // Dword X of the 16 that half H's four B operands have (of each part), in
    // three pieces that go between matrix instructions: codes to binary32, times
    // the scale, packed. (X / 4, X % 4) is (dword, tile) in the gradient, so that
    // an index's scale is fetched once for four dwords, and (tile, dword)
    // otherwise.
    struct Part {
        float f[2];
    };
    template <int H, int X>
    static __device__ __forceinline__ void widen(const Raw &r, const Scales &s, Part &f, float (&scale)[2]) {
        constexpr int t = GRAD ? X % 4 : X / 4, d = GRAD ? X / 4 : X % 4, i = 8 * H + 2 * d;
        if constexpr (GRAD) {
            f.f[0] = code_f32<BITS>(r.w[i], t);
            f.f[1] = code_f32<BITS>(r.w[i + 1], t);
            if constexpr (t == 0) scale[0] = row_scale<i>(s), scale[1] = row_scale<i + 1>(s);
        } else {
            constexpr int per = 32 / BITS, at = t * (16 / per);
            f.f[0] = code_f32<BITS>(r.w[at + i / per], i % per);
            f.f[1] = code_f32<BITS>(r.w[at + (i + 1) / per], (i + 1) % per);
            scale[0] = scale[1] = s[t];
        }
    }
    template <int X>
    static __device__ __forceinline__ void pack(const Part &f, B &b) {
        constexpr int t = GRAD ? X % 4 : X / 4, d = GRAD ? X / 4 : X % 4;
        uint32_t w[PB];
        low_parts<PB>(f.f[0], f.f[1], w);
#pragma unroll
        for (int i = 0; i < PB; ++i) b[i][t][d] = w[i];
    }

    template <int H, int X, int END>
    static __device__ __forceinline__ void convert_range(const Raw &r, const Scales &s, B &b, float (&scale)[2]) {
        if constexpr (X < END) {
            Part f;
            widen<H, X>(r, s, f, scale);
            f.f[0] *= scale[0], f.f[1] *= scale[1];
            pack<X>(f, b);
            convert_range<H, X + 1, END>(r, s, b, scale);
        }
    }
    template <int H>
    static __device__ __forceinline__ void convert_all(const Raw &r, B &b) {
        Scales s;
        scales(r, true, s);
        float scale[2];
        convert_range<H, 0, 16>(r, s, b, scale);
    }

    using A = u32x4[PA];

    static __device__ __forceinline__ void read_a(const uint8_t *at, int m, A &a) {
#pragma unroll
        for (int x = 0; x < PA; ++x) a[x] = *reinterpret_cast<const u32x4 *>(at + x * kPlane + m * 2048);
    }

    // The products of one row of tiles with tiles T0 .. T1 - 1, the smallest parts
    // first. With three parts each, products below 2^-24 of the largest are left
    // out (mid lo, lo mid, lo lo). Tiles run innermost, and stay so: sums that
    // follow on one another are then instructions apart. `after(k)` stands behind
    // pair k of parts.
    template <int T0, int T1, int K, class F>
    static __device__ __forceinline__ void products_from(const A &a, const B &b, f32x4 (&acc)[4], F &&after) {
        // pairs in order: (2,0) (1,1) (1,0) (0,2) (0,1) (0,0) of three and three parts, the last three of one and three
        constexpr int pairs = PA == 3 ? 6 : PB;
        if constexpr (K < pairs) {
            constexpr int i = PA == 1 ? 0 : K == 0 ? 2 : K < 3 ? 1 : 0;
            constexpr int j = PA == 1 ? PB - 1 - K : K == 0 ? 0 : K < 3 ? 2 - K : 5 - K;
#pragma unroll
            for (int t = T0; t < T1; ++t) mfma<kPin>(a[i], b[j][t], acc[t]);
            after(std::integral_constant<int, K>{});
            if constexpr (PB > 1) __builtin_amdgcn_sched_barrier(0);
            products_from<T0, T1, K + 1>(a, b, acc, after);
        }
    }
    template <int T0, int T1, class F>
    static __device__ __forceinline__ void products(const A &a, const B &b, f32x4 (&acc)[4], F &&after) {
        products_from<T0, T1, 0>(a, b, acc, after);
    }
    template <int T0, int T1>
    static __device__ __forceinline__ void products(const A &a, const B &b, f32x4 (&acc)[4]) {
        products_from<T0, T1, 0>(a, b, acc, [](auto) {});
    }

    // Piece P of row M's share of the conversion.
    template <int HN, int P, int X, int END>
    static __device__ __forceinline__ void piece(const Raw &raw, const Scales &s, B &bn, Part (&f)[16 / MT],
                                                 float (&scale)[16 / MT][2]) {
        if constexpr (X < END) {
            constexpr int i = X % (16 / MT);
            if constexpr (P == 0) {
                if constexpr (GRAD && X % 4 != 0 && i != 0) scale[i][0] = scale[i - 1][0], scale[i][1] = scale[i - 1][1];
                widen<HN, X>(raw, s, f[i], scale[i]);
            } else if constexpr (P == 1) {
                f[i].f[0] *= scale[i][0], f[i].f[1] *= scale[i][1];
            } else {
                pack<X>(f[i], bn);
            }
            piece<HN, P, X + 1, END>(raw, s, bn, f, scale);
        }
    }

    // Rows of tiles M.. of a half: products with b, and the next half's operands
    // bn from raw. `here` and `then` are where the lane's A operands of this half
    // and of the next one lie. The order is fixed as written: a matrix
    // instruction keeps its unit for 16 cycles and the issue for 8 of them, so
    // each is followed by about two instructions of the conversion (a third
    // costs 4 to 5 cycles more). `before(m)` makes the loads that stand before row m.
    template <int HN, int M, class F>
    static __device__ __forceinline__ void rows_from(const uint8_t *here, const uint8_t *then, const B &b,
                                                     const Raw &raw, const Scales &s, B &bn, A (&a)[kRing],
                                                     float (&scale)[16 / MT][2], f32x4 (&acc)[MT][4], F &&before) {
        constexpr int x0 = 16 * M / MT, x1 = 16 * (M + 1) / MT;
        Part f[16 / MT];
        if constexpr (M == 0) operands_ready<kPin>();
        if constexpr (kAhead == 0)
            read_a(here, M, a[0]);
        else if constexpr (M + kAhead < MT)
            read_a(here, M + kAhead, a[(M + kAhead) % kRing]);
        else
            read_a(then, M + kAhead - MT, a[(M + kAhead) % kRing]);
        before(std::integral_constant<int, M>{});
        if constexpr (PB == 1) {
            products<0, 1>(a[M % kRing], b, acc[M]);
            piece<HN, 0, x0, x1>(raw, s, bn, f, scale);
            __builtin_amdgcn_sched_barrier(0);
            products<1, 2>(a[M % kRing], b, acc[M]);
            piece<HN, 1, x0, x1>(raw, s, bn, f, scale);
            __builtin_amdgcn_sched_barrier(0);
            products<2, 3>(a[M % kRing], b, acc[M]);
            piece<HN, 2, x0, x1>(raw, s, bn, f, scale);
            __builtin_amdgcn_sched_barrier(0);
            products<3, 4>(a[M % kRing], b, acc[M]);
            __builtin_amdgcn_sched_barrier(0);
        } else {
            products<0, 4>(a[M % kRing], b, acc[M], [&](auto k) {
                if constexpr (k.value < 3) piece<HN, k.value, x0, x1>(raw, s, bn, f, scale);
                if constexpr (PB == 2 && k.value == 1) piece<HN, 2, x0, x1>(raw, s, bn, f, scale);
            });
        }
        if constexpr (M + 1 < MT) rows_from<HN, M + 1>(here, then, b, raw, s, bn, a, scale, acc, before);
    }

    // Rows of tiles that adapters are added to at once: 64 rows, 32 where half the registers are
    // there, or all of a smaller tile's.
    static constexpr int kTogether = MT == 1 ? 1 : MT < 16 && PA * PB == 1 ? 2 : 4;

    // d += low up of adapter g, for those of kTogether rows of tiles from row `first` on that are
    // in `match`. Low comes by buffer loads, whose range check gives zeros for the other
    // rows, for rows past the end and ranks past the last. Zeros times infinities are NaN: false
    // if the adapter holds any that another row would see.
    template <int PC>
    static __device__ __forceinline__ bool add_adapter(const LinArgs &p, int lane, int64_t first, int64_t col, int g,
                                                       uint64_t match, f32x4 (&d)[kTogether][4]) {
        uint32_t bad = 0;
#if defined(__HIP_DEVICE_COMPILE__)
        constexpr int kRowsOf = kTogether * 16;
        constexpr uint32_t kOut = 1u << 30;
        const int q = lane >> 4, j = lane & 15;
        const int left = static_cast<int>(min(p.rows - first, static_cast<int64_t>(kRowsOf)));
        const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float *>(p.low + first * p.rank), 0, static_cast<uint32_t>(left * p.rank * 4), 0x27000);
        const bool mixed = __popcll(match) != left;
        uint32_t at[kTogether];
#pragma unroll
        for (int m = 0; m < kTogether; ++m)
            at[m] = match >> (m * 16 + j) & 1 ? static_cast<uint32_t>((m * 16 + j) * p.rank * 4) : kOut;
#pragma unroll 1
        for (int r0 = 0; r0 < p.rank; r0 += 32) {
            const int r = r0 + 8 * q;
            const uint32_t plus = r < p.rank ? static_cast<uint32_t>(r * 4) : kOut;
            u32x4 b[4][1], low[kTogether][2];
            load_up<GRAD, true, 1, 4>(p, g, col, r, b);
#pragma unroll
            for (int m = 0; m < kTogether; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    low[m][h] = __builtin_amdgcn_raw_buffer_load_b128(from, at[m] + plus, 16 * h, 0);
            if (mixed) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // an exponent of ones in either half
                        const uint32_t e = ~b[t][0][i];
                        bad |= (e & 0x7F80u) == 0 || (e & 0x7F800000u) == 0 ? 1u : 0u;
                    }
            }
#pragma unroll
            for (int m = 0; m < kTogether; ++m) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = as_f(low[m][i / 4][i % 4]);
                u32x4 a[PC];
                operand_of<PC>(v, a);
#pragma unroll
                for (int t = 0; t < 4; ++t) d[m][t] = mfma_parts<PC, 1>(a, b[t], d[m][t]);
            }
        }
#endif
        return __ballot(bad != 0) == 0;
    }

    // How many adapters kTogether rows of tiles from row `first` on have, up to `most` + 1.
    static __device__ __forceinline__ int count_adapters(const LinArgs &p, int lane, int64_t first, int most) {
        int id, n = 0;
        const bool has = adapter_of(p, first + lane, id) && lane < kTogether * 16;
        for (uint64_t pending = __ballot(has); pending != 0 && n <= most; ++n)
            pending &= ~__ballot(has && id == __builtin_amdgcn_readlane(id, __builtin_ctzll(pending)));
        return n;
    }

    // What the adapters, all of them bf16, add to kTogether rows of tiles from row `first` on, one
    // after the other, each with all the rows; false, and zeros, where an adapter's infinities or
    // NaNs forbid it.
    template <int PC>
    static __device__ __forceinline__ bool add_adapters(const LinArgs &p, int lane, int64_t first, int64_t col,
                                                        f32x4 (&d)[kTogether][4]) {
        int id;
        const bool has = adapter_of(p, first + lane, id) && lane < kTogether * 16;
        uint64_t pending = __ballot(has);
        bool good = true;
#pragma unroll 1
        while (good && pending != 0) {
            const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(pending));
            const uint64_t match = __ballot(has && id == g);
            pending &= ~match;
            good = add_adapter<PC>(p, lane, first, col, g, match, d);
        }
        if (good) return true;
#pragma unroll
        for (int m = 0; m < kTogether; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t) d[m][t] = f32x4{0, 0, 0, 0};
        return false;
    }
};

template <bool GRAD, int BITS, int PA, int PB, int MT, LinMode MODE>
__device__ __forceinline__ void linear_big_tile(const LinArgs &p, const LinPlace &place,
                                                uint8_t (*tiles)[LinBig<GRAD, BITS, PA, PB, MT>::kBytes]) {
    using L = LinBig<GRAD, BITS, PA, PB, MT>;
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
    const int q = lane >> 4;
    const int64_t c_len = GRAD ? p.n_out : p.n_in, len = GRAD ? p.n_in : p.n_out;
    const int64_t m0 = place.m0, wave_col = place.col * kTileCols + w * 64, col = wave_col + (lane & 15) * 4;
    const typename L::At at = L::place(p, m0, wave_col);

    // The split's indices: whole steps in the pipeline, then what is left over.
    const int64_t s0 = place.split * p.split_steps;
    const int64_t c1 = min(c_len, (s0 + p.split_steps) * kStep);
    const int64_t s1 = c1 / kStep;

    f32x4 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0, 0, 0, 0};

    const int a0 = lds_piece(lane & 15, q * 2), a1 = lds_piece(lane & 15, q * 2 + 1);  // of halves 0 and 1
    typename L::A a[L::kRing];
    typename L::B b0, b1;

    if (s0 < s1) {
        constexpr int G = L::kGroups * PA, N = L::kLoads, D = L::kDepth;
        typename L::Raw raw[D];
        float scale[16 / MT][2];
        // steps past the end are the last one again
        auto clamp = [&](int64_t i) { return min(i, s1 - 1); };
#pragma unroll
        for (int i = 0; i < L::kBufs - 1; ++i) L::template stage<0, G>(at, clamp(s0 + i), tiles[i]);
#pragma unroll
        for (int i = 0; i < D; ++i) L::template load_range<0, N>(p, at, L::from(p, at, clamp(s0 + i)), raw[i]);
        L::template convert_all<0>(raw[0], b0);
        wait_loads();
        __syncthreads();
        // byte offsets of this step's activations, the next one's and those asked for
        int o0 = 0, o1 = L::kBytes, to = (L::kBufs - 1) * L::kBytes;
        auto next_of = [](int o) { return o + L::kBytes == L::kBufs * L::kBytes ? 0 : o + L::kBytes; };
        if constexpr (L::kAhead > 0) {
#pragma unroll
            for (int m = 0; m < L::kAhead; ++m) L::read_a(tiles[0] + a0, m, a[m]);
        }
        auto step = [&](int64_t i, typename L::Raw &now, const typename L::Raw &next) {
            const uint8_t *t0 = &tiles[0][0] + o0, *t1 = &tiles[0][0] + o1;
            const typename L::From f = L::from(p, at, clamp(i + D));
            typename L::Scales s;
            L::scales(now, i < s1, s);
            auto load = [&](auto m) {
                L::template load_range<L::loads_before(m.value - 1), L::loads_before(m.value)>(p, at, f, now);
            };
            L::template rows_from<1, 0>(t0 + a0, t0 + a1, b0, now, s, b1, a, scale, acc, load);
            load(std::integral_constant<int, MT>{});
            // Every wave's share of the next step's activations has landed once all
            // are past the barrier, and no wave reads the step before this one any
            // more. Newer than that share are the shares of the kBufs - 3 steps after
            // it and kBufs - 2 steps' codes, four loads or more each.
            wait_loads<(L::kBufs - 3) * G + (L::kBufs - 2) * 4>();
            barrier_only();
            L::scales(next, i + 1 < s1, s);
            auto stage = [&](auto m) {
                L::template stage<G * m.value / MT, G *(m.value + 1) / MT>(at, clamp(i + L::kBufs - 1),
                                                                           &tiles[0][0] + to);
            };
            L::template rows_from<0, 0>(t0 + a1, t1 + a0, b1, next, s, b0, a, scale, acc, stage);
            o0 = o1, o1 = next_of(o1), to = next_of(to);
        };
        for (int64_t i = s0; i < s1; i += D) {
            step(i, raw[0], raw[1 % D]);
            step(i + 1, raw[1 % D], raw[2 % D]);
            if constexpr (D == 4) {
                step(i + 2, raw[2], raw[3]);
                step(i + 3, raw[3], raw[0]);
            }
            sums_ready<L::kPin>();
        }
        wait_loads();
    }

    if (s1 * kStep < c1) {
        typename L::Raw r;
        __syncthreads();
        L::stage_last(p, m0, s1 * kStep, c_len, tiles[0]);
        L::load_last(p, wave_col, s1 * kStep, r);
        L::template convert_all<0>(r, b0);
        L::template convert_all<1>(r, b1);
        wait_loads();
        __syncthreads();
        operands_ready<L::kPin>();
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            typename L::A x, y;
            L::read_a(tiles[0] + a0, m, x);
            L::read_a(tiles[0] + a1, m, y);
            L::template products<0, 4>(x, b0, acc[m]);
            L::template products<0, 4>(y, b1, acc[m]);
        }
        sums_ready<L::kPin>();
    }

    if constexpr (MODE == LinMode::adapted) {
        // Some rows at a time, through LDS, from which a loop stores them. (Written out for all the sums, so that they stay where
        // they are: in a loop that moves them up, they were moved in the products' loop too.)
        constexpr int kTogether = L::kTogether, PC = PA * PB == 1 ? 2 : 3, kMany = 4;
        static_assert(L::kBufs * L::kBytes >= 4 * kTogether * 16 * 64 * 4 && MT % kTogether == 0);
        float *const held = reinterpret_cast<float *>(&tiles[0][0] + w * (kTogether * 16 * 64 * 4));
        __syncthreads();  // no wave reads activations any more
        // The lane as the compiler cannot know it before: what follows from it is not worked out ahead
        // of the loop, where no register is left to keep it in.
        int lane = threadIdx.x & (kWave - 1);
        asm volatile("" : "+v"(lane));
        const int q = lane >> 4;
        const int64_t col = wave_col + (lane & 15) * 4;
        // Rows of tiles M0 .. M0 + kTogether - 1 of the sums, which are rows from `first` on.
        auto finish = [&](auto at, int64_t first) {
            constexpr int M0 = at.value;
            f32x4 d[kTogether][4];
            bool apart = false;
#pragma unroll
            for (int m = 0; m < kTogether; ++m)
#pragma unroll
                for (int t = 0; t < 4; ++t) d[m][t] = f32x4{0, 0, 0, 0};
            // Many adapters: rows gathered, each part of the contraction a share of them. Few: with
            // the first part.
            const int kinds = L::count_adapters(p, lane, first, kMany);
            int part = 0, parts = 1;
            if (kinds > kMany || (kinds > 0 && p.up_f32)) {
                apart = true;
                part = static_cast<int>(place.split), parts = p.splits;
            } else if (kinds > 0 && place.split == 0) {
                apart = !L::template add_adapters<PC>(p, lane, first, col, d);
            }
            if (apart) adapter_rows<GRAD, true, PC, 4, kTogether * 16, 2, 1>(p, first, col, part, parts, held);
#pragma unroll
            for (int m = 0; m < kTogether; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 v = f32x4{acc[M0 + m][0][i], acc[M0 + m][1][i], acc[M0 + m][2][i], acc[M0 + m][3][i]};
                    v = v * kCodeScale<BITS> + f32x4{d[m][0][i], d[m][1][i], d[m][2][i], d[m][3][i]};
                    f32x4 *to = reinterpret_cast<f32x4 *>(held + (m * 16 + 4 * q + i) * 64 + 4 * (lane & 15));
                    if (apart) v += *to;
                    *to = v;
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll 4
            for (int r = 0; r < kTogether * 16; r += 4) {
                const int64_t row = first + r + q;
                const f32x4 s = *reinterpret_cast<const f32x4 *>(held + (r + q) * 64 + 4 * (lane & 15));
                const float v[4] = {s[0], s[1], s[2], s[3]};
                if (row < p.rows) store4(p, len, row, col, v, place.split);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        finish(std::integral_constant<int, 0>{}, m0);
        if constexpr (MT > kTogether) {
            if (m0 + kTogether * 16 < p.rows) finish(std::integral_constant<int, kTogether>{}, m0 + kTogether * 16);
        }
        if constexpr (MT > 2 * kTogether) {
            if (m0 + 2 * kTogether * 16 < p.rows)
                finish(std::integral_constant<int, 2 * kTogether>{}, m0 + 2 * kTogether * 16);
            if (m0 + 3 * kTogether * 16 < p.rows)
                finish(std::integral_constant<int, 3 * kTogether>{}, m0 + 3 * kTogether * 16);
        }
        static_assert(MT == kTogether || MT == 2 * kTogether || MT == 4 * kTogether);
        return;
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
            store4<MODE == LinMode::grouped ? kTileCols : 0>(p, len, row, col, v, place.split);
        }
    }
}

template <bool GRAD, int BITS, int PA, int PB, int MT, LinMode MODE>
__global__ __launch_bounds__(kBlockThreads, MT == 16 || (PB > 1 && MT >= 4) ? 1 : 2) void linear_big_kernel(
    LinArgs p) {
    using L = LinBig<GRAD, BITS, PA, PB, MT>;
    __shared__ __attribute__((aligned(128))) uint8_t tiles[L::kBufs][L::kBytes];
    LinPlace place;
    if constexpr (MODE == LinMode::grouped) {
        if (!group_place_tail<BITS, 2>(p, L::kRows, place)) return;
        // A group's last tile is half empty or more as often as not. 16 groups of 300 rows, int4, 11008 x
        // 4096: 612 us so, 636 with 256-row tiles alone (a step's codes cost as much in either).
        if constexpr (MT == 16) {
            using S = LinBig<GRAD, BITS, PA, PB, 8>;
            static_assert(S::kBufs * S::kBytes <= L::kBufs * L::kBytes);
            if (p.rows - place.m0 <= S::kRows) {
                linear_big_tile<GRAD, BITS, PA, PB, 8, MODE>(p, place, reinterpret_cast<uint8_t(*)[S::kBytes]>(&tiles[0][0]));
                return;
            }
        }
    } else {
        place = lin_place(p, L::kRows);
    }
    linear_big_tile<GRAD, BITS, PA, PB, MT, MODE>(p, place, tiles);
}

template <LinMode MODE, bool GRAD, int BITS, int PA, int PB, int MT>
hipError_t launch_linear_big_one(const LinArgs &p, hipStream_t stream) {
    const int64_t grid = p.row_tiles * p.col_tiles * p.splits + (MODE == LinMode::grouped && p.join_steps ? kParts : 0);
    linear_big_kernel<GRAD, BITS, PA, PB, MT, MODE><<<static_cast<unsigned>(grid), kBlockThreads, 0, stream>>>(p);
    return hipGetLastError();
}

// parts 0: bf16 to bf16; 1: bf16 to binary32; 2: binary32 activations; 3: bf16 to bf16, few rows. mt is the plan's.
template <LinMode MODE, bool GRAD, int BITS>
hipError_t launch_linear_big_as(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    if (parts == 2) {
        if (mt == 8) return launch_linear_big_one<MODE, GRAD, BITS, 3, 3, 8>(p, stream);
        if (mt == 4) return launch_linear_big_one<MODE, GRAD, BITS, 3, 3, 4>(p, stream);
        return launch_linear_big_one<MODE, GRAD, BITS, 3, 3, 1>(p, stream);
    }
    if constexpr (GRAD) {  // forward, the exact codes do better (linear_mid.h)
        if (parts == 1) {
            if (mt == 8) return launch_linear_big_one<MODE, GRAD, BITS, 1, 3, 8>(p, stream);
            if (mt == 4) return launch_linear_big_one<MODE, GRAD, BITS, 1, 3, 4>(p, stream);
            return launch_linear_big_one<MODE, GRAD, BITS, 1, 3, 1>(p, stream);
        }
    }
    if constexpr (GRAD && MODE != LinMode::one) {
        if (parts == 3)
            return mt == 4 ? launch_linear_big_one<MODE, GRAD, BITS, 1, 2, 4>(p, stream)
                           : launch_linear_big_one<MODE, GRAD, BITS, 1, 2, 1>(p, stream);
    }
    if (mt == 16) return launch_linear_big_one<MODE, GRAD, BITS, 1, 1, 16>(p, stream);
    if (mt == 8) return launch_linear_big_one<MODE, GRAD, BITS, 1, 1, 8>(p, stream);
    if (mt == 4) return launch_linear_big_one<MODE, GRAD, BITS, 1, 1, 4>(p, stream);
    return launch_linear_big_one<MODE, GRAD, BITS, 1, 1, 1>(p, stream);
}

}  // namespace zpp
