// norm_device.h - what the norms' kernels share: sums over the threads of a
// row, and rows, weights and shares of weight gradients in 16-byte pieces.
#pragma once

#include "zpp_device.h"

namespace zpp {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float add_dpp(float v, uint32_t o) { return v + as_f(o); }

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v = add_dpp(v, dpp_u32<0xB1>(as_u(v)));
    v = add_dpp(v, dpp_u32<0x4E>(as_u(v)));
    v = add_dpp(v, dpp_u32<0x141>(as_u(v)));
    v = add_dpp(v, dpp_u32<0x140>(as_u(v)));
    auto p = __builtin_amdgcn_permlane16_swap(as_u(v), as_u(v), false, false);
    v = as_f(p[0]) + as_f(p[1]);
    p = __builtin_amdgcn_permlane32_swap(as_u(v), as_u(v), false, false);
    return as_f(p[0]) + as_f(p[1]);
}

// Sums of N values over the T threads of a unit, in every thread. `lds` holds
// 2 * N * (T / 64) floats, used in turn, so one barrier a call is enough: a
// slot is written again only after the barrier of the call between.
template <int T, int N>
__device__ __forceinline__ void unit_sum(float (&v)[N], float *lds, int &turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (T > kWave) {
        constexpr int W = T / kWave;
        float *at = lds + turn * N * W;
        turn ^= 1;
        const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[i * W + w] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) s += at[i * W + k];
            v[i] = s;
        }
    }
}

// Rows whose elements lie on 16-byte pieces are WHOLE: every V elements of a row
// are one aligned access. Other rows are read and written in the same pieces,
// at the addresses they have, but for a last one that would pass the row's end,
// which goes element by element.
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));  // 16 bytes at any element of either type

// V elements from element e on, packed; `left` (> 0) are in the row.
template <bool F32, int V, bool WHOLE>
__device__ __forceinline__ void load_packed(const void *base, int64_t e, int64_t left, uint32_t *w) {
    static_assert(V == (F32 ? 4 : 8), "16 bytes");
    if (WHOLE || left >= V) {
        const uint8_t *p = static_cast<const uint8_t *>(base) + e * (F32 ? 4 : 2);
        const u32x4 v = WHOLE ? *reinterpret_cast<const u32x4 *>(p) : *reinterpret_cast<const u32x4_at2 *>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (F32) {
                w[j] = j < left ? static_cast<const uint32_t *>(base)[e + j] : 0u;
            } else {
                const uint16_t *p = static_cast<const uint16_t *>(base) + e;
                w[j] = (2 * j < left ? p[2 * j] : 0u) | (2 * j + 1 < left ? static_cast<uint32_t>(p[2 * j + 1]) << 16 : 0u);
            }
        }
    }
}

template <bool F32>
__device__ __forceinline__ float unpack(const uint32_t *w, int j) {
    if constexpr (F32)
        return as_f(w[j]);
    else
        return j % 2 == 0 ? bf16_lo(w[j / 2]) : bf16_hi(w[j / 2]);
}

template <bool F32, int V, bool WHOLE>
__device__ __forceinline__ void load_v(const void *base, int64_t e, int64_t left, float (&f)[V]) {
    uint32_t w[4];
    load_packed<F32, V, WHOLE>(base, e, left, w);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = unpack<F32>(w, j);
}

template <bool F32, int V, bool WHOLE>
__device__ __forceinline__ void store_v(void *base, int64_t e, int64_t left, const float (&f)[V]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = F32 ? as_u(f[F32 ? j : 0]) : pack_bf16x2(f[F32 ? 0 : 2 * j], f[F32 ? 0 : 2 * j + 1]);
    if (WHOLE || left >= V) {
        uint8_t *p = static_cast<uint8_t *>(base) + e * (F32 ? 4 : 2);
        if constexpr (WHOLE)
            st_out<u32x4>(p, v);
        else
            *reinterpret_cast<u32x4_at2 *>(p) = v;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j >= left) break;
            if constexpr (F32)
                static_cast<uint32_t *>(base)[e + j] = v[j];
            else
                static_cast<uint16_t *>(base)[e + j] = static_cast<uint16_t>(v[j / 2] >> (16 * (j % 2)));
        }
    }
}

// V elements of a weight vector of either type from column c on (a multiple of
// V below the width); a missing vector's are `none`.
template <int V, bool WHOLE>
__device__ __forceinline__ void load_w(const void *w, bool f32, int64_t c, int64_t width, float none, float (&o)[V]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = none;
    } else if (!WHOLE && c + V > width) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            o[j] = 0.0f;
            if (c + j < width)
                o[j] = f32 ? static_cast<const float *>(w)[c + j] : bf16_lo(static_cast<const uint16_t *>(w)[c + j]);
        }
    } else if (f32) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const f32x4 v = ld<f32x4>(static_cast<const float *>(w) + c + j);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[j + k] = v[k];
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const u32x2 v = ld<u32x2>(static_cast<const uint16_t *>(w) + c + j);
            o[j] = bf16_lo(v[0]), o[j + 1] = bf16_hi(v[0]), o[j + 2] = bf16_lo(v[1]), o[j + 3] = bf16_hi(v[1]);
        }
    }
}

// V of a share's sums, of which `left` are in the row.
template <int V, bool WHOLE>
__device__ __forceinline__ void store_share(float *o, int64_t left, const float (&v)[V]) {
    if (WHOLE || left >= V) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
            *reinterpret_cast<f32x4_at4 *>(o + j) = f32x4{v[j], v[j + 1], v[j + 2], v[j + 3]};
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) o[j] = v[j];
    }
}

// What a thread holds of a row, as loaded: N chunks of V elements, chunk i at
// column (i T + thread) V. Rows are loaded one ahead, so they stay packed.
template <bool F32, bool WHOLE, int T, int N>
struct Held {
    static constexpr int V = F32 ? 4 : 8;
    uint32_t w[N][4];

    static __device__ __forceinline__ int64_t column(int i) {
        return (static_cast<int64_t>(i) * T + threadIdx.x % T) * V;
    }

    // Whether element j of chunk i is in the row.
    static __device__ __forceinline__ bool in(int i, int j, int64_t width) {
        return column(i) + (WHOLE ? 0 : j) < width;
    }

    // Columns past the width are zeros.
    __device__ __forceinline__ void load(const void *base, int64_t e, int64_t width) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = column(i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = 0;
            if (c < width) load_packed<F32, V, WHOLE>(base, e + c, width - c, w[i]);
        }
    }

    __device__ __forceinline__ float at(int i, int j) const { return unpack<F32>(w[i], j); }
};

constexpr int group(int T) { return T < 256 ? 256 : T; }  // threads of a workgroup

// C vectors' gradients (dw, or dw and db) from the units' shares: a workgroup has
// 32 columns and 32 runs of units, each summed in order, then the runs in order.
// 512 shares of 2 x 8192 columns: 7 us, 5 TB/s.
constexpr int kRuns = 32;

template <int C>
__global__ __launch_bounds__(32 * kRuns) void norm_join_kernel(const float *__restrict__ partial, int64_t units,
                                                               int64_t width, void *dw, void *db, bool w_f32) {
    __shared__ float lds[kRuns][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // over dw's columns, then db's
    const int64_t per = (units + kRuns - 1) / kRuns, u1 = min(units, (run + 1) * per);
    float s = 0.0f;
    if (i < C * width) {
#pragma unroll 8
        for (int64_t u = run * per; u < u1; ++u) s += partial[u * C * width + i];
    }
    lds[run][lane] = s;
    __syncthreads();
    if (run != 0 || i >= C * width) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kRuns; ++k) s += lds[k][lane];
    void *o = i < width ? dw : db;
    const int64_t c = i < width ? i : i - width;
    if (!o) return;
    if (w_f32)
        static_cast<float *>(o)[c] = s;
    else
        static_cast<uint16_t *>(o)[c] = static_cast<uint16_t>(pack_bf16x2(s, 0.0f));
}

template <int C>
hipError_t launch_norm_join(const float *partial, int64_t units, int64_t width, void *dw, void *db, bool w_f32,
                            hipStream_t stream) {
    norm_join_kernel<C><<<static_cast<unsigned>((C * width + 31) / 32), 32 * kRuns, 0, stream>>>(partial, units, width,
                                                                                                dw, db, w_f32);
    return hipGetLastError();
}

}  // namespace zpp
