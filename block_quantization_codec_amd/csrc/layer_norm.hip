// layer_norm.hip - layer norm over the rows of a matrix, forward and backward.
//
//   mean = sum x / H,  var = sum (x - mean)^2 / H,  rstd = 1 / sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   xh = (x - mean) rstd,  g = dy w
//   dx = rstd (g - sum g / H - xh sum (g xh) / H)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both are streams: one read of every input and one write of every output.
// A unit of T threads (a wave to 16 of them, by the row's width) holds a whole
// row in registers, up to 32 elements a thread, so the variance is the sum of
// squared differences from the mean already known (no cancellation) and
// nothing is read twice; the next row is on its way meanwhile. Units walk over the rows, keeping the weights,
// and in the backward pass their share of dw and db, in registers; the units'
// shares go to the workspace and a second kernel sums them in unit order, so
// the result does not change from run to run. Rows wider than 32,768 elements
// (16,384 backward) are read again for each sum instead; their shares are
// summed in the workspace itself.
//
// All sums are binary32. Rows whose elements lie on 16-byte pieces move as
// such (V elements each); any others element by element, still contiguous
// across the wave.
#include <algorithm>

#include "zpp_device.h"
#include "zpp_launch.h"

namespace zpp {
namespace {

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

// V elements at p, widened.
template <bool F32, int V>
__device__ __forceinline__ void load_v(const void *base, int64_t e, float *f) {
    if constexpr (F32) {
        if constexpr (V == 4) {
            const f32x4 v = ld<f32x4>(static_cast<const float *>(base) + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = v[i];
        } else {
            f[0] = static_cast<const float *>(base)[e];
        }
    } else {
        if constexpr (V == 8) {
            const u32x4 v = ld<u32x4>(static_cast<const uint16_t *>(base) + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(v[i]), f[2 * i + 1] = bf16_hi(v[i]);
        } else {
            f[0] = bf16_lo(static_cast<const uint16_t *>(base)[e]);
        }
    }
}

template <bool F32, int V>
__device__ __forceinline__ void store_v(void *base, int64_t e, const float *f) {
    if constexpr (F32) {
        if constexpr (V == 4)
            st_out<f32x4>(static_cast<float *>(base) + e, f32x4{f[0], f[1], f[2], f[3]});
        else
            st_out<float>(static_cast<float *>(base) + e, f[0]);
    } else {
        if constexpr (V == 8)
            st_out<u32x4>(static_cast<uint16_t *>(base) + e,
                          u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                pack_bf16x2(f[6], f[7])});
        else
            st_out<uint16_t>(static_cast<uint16_t *>(base) + e, static_cast<uint16_t>(pack_bf16x2(f[0], 0.0f)));
    }
}

// One element of a weight vector of either type; missing ones are `none`.
__device__ __forceinline__ float load_w(const void *w, bool f32, int64_t e, float none) {
    if (!w) return none;
    return f32 ? static_cast<const float *>(w)[e] : bf16_lo(static_cast<const uint16_t *>(w)[e]);
}

struct NormArgs {
    const void *x;
    int64_t x_stride;
    const void *dy;
    int64_t dy_stride;
    int64_t rows, width;
    const void *weight, *bias;
    bool w_f32;
    float eps;
    void *y;
    int64_t y_stride;
    float *mean, *rstd;
    float *partial;  // [units][2][width]: each unit's share of dw and db
    int64_t units;
};

// What a thread holds of a row, as loaded: N chunks of V elements, chunk i at
// column (i T + thread) V. Rows are loaded one ahead, so they stay packed.
template <bool F32, int V, int T, int N>
struct Held {
    static constexpr int kW = F32 ? V : (V + 1) / 2;  // dwords of a chunk
    uint32_t w[N][kW];

    static __device__ __forceinline__ int64_t column(int i) {
        return (static_cast<int64_t>(i) * T + threadIdx.x % T) * V;
    }

    // Columns past the width are zeros.
    __device__ __forceinline__ void load(const void *base, int64_t e, int64_t width) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = column(i);
#pragma unroll
            for (int j = 0; j < kW; ++j) w[i][j] = 0;
            if (c >= width) continue;
            if constexpr (V == 1) {
                w[i][0] = F32 ? static_cast<const uint32_t *>(base)[e + c] : static_cast<const uint16_t *>(base)[e + c];
            } else {
                const u32x4 v = ld<u32x4>(static_cast<const uint8_t *>(base) + (e + c) * (F32 ? 4 : 2));
#pragma unroll
                for (int j = 0; j < 4; ++j) w[i][j] = v[j];
            }
        }
    }

    __device__ __forceinline__ float at(int i, int j) const {
        if constexpr (F32)
            return as_f(w[i][j]);
        else
            return V == 1 || j % 2 == 0 ? bf16_lo(w[i][j / 2]) : bf16_hi(w[i][j / 2]);
    }
};

constexpr int group(int T) { return T < 256 ? 256 : T; }  // threads of a workgroup

// HOLD: the weights stay in registers over the rows (else they are read again for each).
template <bool F32, int V, int T, int N, bool HOLD>
__global__ __launch_bounds__(group(T)) void norm_kernel(NormArgs p) {
    using H = Held<F32, V, T, N>;
    constexpr int kUnits = group(T) / T;
    __shared__ float lds[T > kWave ? 2 * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    if (kUnits > 1 && unit >= p.rows) return;
    const float inv = 1.0f / static_cast<float>(p.width);
    float w[HOLD ? N : 1][V], b[HOLD ? N : 1][V];
    H x, next;
    next.load(p.x, unit * p.x_stride, p.width);
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int64_t c = min(H::column(i) + j, p.width - 1);
                w[i][j] = load_w(p.weight, p.w_f32, c, 1.0f);
                b[i][j] = load_w(p.bias, p.w_f32, c, 0.0f);
            }
    }
    for (int64_t r = unit; r < p.rows; r += p.units) {
        if constexpr (!HOLD) asm volatile("" ::: "memory");  // the weights' loads stay in the loop
        x = next;
        if (r + p.units < p.rows) next.load(p.x, (r + p.units) * p.x_stride, p.width);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] += x.at(i, j);
        unit_sum<T>(s, lds, turn);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = H::column(i) < p.width ? x.at(i, j) - mean : 0.0f;
                s[0] = __builtin_fmaf(d, d, s[0]);
            }
        unit_sum<T>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x % T == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = H::column(i);
            if (c >= p.width) continue;
            float y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float wj = HOLD ? w[HOLD ? i : 0][j] : load_w(p.weight, p.w_f32, c + j, 1.0f);
                const float bj = HOLD ? b[HOLD ? i : 0][j] : load_w(p.bias, p.w_f32, c + j, 0.0f);
                y[j] = __builtin_fmaf((x.at(i, j) - mean) * rstd, wj, bj);
            }
            store_v<F32, V>(p.y, r * p.y_stride + c, y);
        }
    }
}

// AHEAD: the next row's loads are made before this row's sums; a workgroup of
// 16 waves has too few registers a lane for that.
template <bool F32, int V, int T, int N, bool AHEAD>
__global__ __launch_bounds__(group(T)) void norm_grad_kernel(NormArgs p) {
    using H = Held<F32, V, T, N>;
    constexpr int kUnits = group(T) / T;
    __shared__ float lds[T > kWave ? 2 * 2 * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    if (kUnits > 1 && unit >= p.units) return;
    const float inv = 1.0f / static_cast<float>(p.width);
    float w[N][V], dw[N][V], db[N][V];
    H x, dy, next_x, next_dy;
    float mean, rstd, next_mean, next_rstd;
    auto fetch = [&](int64_t r) {
        next_x.load(p.x, r * p.x_stride, p.width);
        next_dy.load(p.dy, r * p.dy_stride, p.width);
        next_mean = p.mean[r], next_rstd = p.rstd[r];
    };
    if constexpr (AHEAD) fetch(unit);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = load_w(p.weight, p.w_f32, min(H::column(i) + j, p.width - 1), 1.0f);
            dw[i][j] = db[i][j] = 0.0f;
        }
    for (int64_t r = unit; r < p.rows; r += p.units) {
        if constexpr (!AHEAD) fetch(r);
        x = next_x, dy = next_dy, mean = next_mean, rstd = next_rstd;
        if (AHEAD && r + p.units < p.rows) fetch(r + p.units);
        // columns past the width have dy = 0: they add nothing (x = 0 there, so xh is finite as mean and rstd are)
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (x.at(i, j) - mean) * rstd, d = dy.at(i, j), g = d * w[i][j];
                dw[i][j] = __builtin_fmaf(d, xh, dw[i][j]);
                db[i][j] += d;
                s[0] += g;
                s[1] = __builtin_fmaf(g, H::column(i) < p.width ? xh : 0.0f, s[1]);
            }
        }
        unit_sum<T>(s, lds, turn);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = H::column(i);
            if (c >= p.width) continue;
            float dx[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (x.at(i, j) - mean) * rstd;
                dx[j] = (dy.at(i, j) * w[i][j] - m0 - xh * m1) * rstd;
            }
            store_v<F32, V>(p.y, r * p.y_stride + c, dx);
        }
    }
    float *mine = p.partial + unit * 2 * p.width;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = H::column(i);
        if (c >= p.width) continue;
        if constexpr (V > 1) {  // the width is a multiple of V, so both shares are 16-byte aligned
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                st<f32x4>(mine + c + j, f32x4{dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]});
                st<f32x4>(mine + p.width + c + j, f32x4{db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]});
            }
        } else {
            mine[c] = dw[i][0];
            mine[p.width + c] = db[i][0];
        }
    }
}

constexpr int kLong = 1024;  // threads of a unit for rows beyond the registers

template <bool F32, int V>
__global__ __launch_bounds__(kLong) void norm_long_kernel(NormArgs p) {
    __shared__ float lds[2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    for (int64_t r = blockIdx.x; r < p.rows; r += p.units) {
        const int64_t x0 = r * p.x_stride, y0 = r * p.y_stride;
        float s[1] = {0.0f}, v[V];
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V>(p.x, x0 + c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] += v[j];
        }
        unit_sum<kLong>(s, lds, turn);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V>(p.x, x0 + c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] = __builtin_fmaf(v[j] - mean, v[j] - mean, s[0]);
        }
        unit_sum<kLong>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V>(p.x, x0 + c, v);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = __builtin_fmaf((v[j] - mean) * rstd, load_w(p.weight, p.w_f32, c + j, 1.0f),
                                      load_w(p.bias, p.w_f32, c + j, 0.0f));
            store_v<F32, V>(p.y, y0 + c, v);
        }
    }
}

template <bool F32, int V>
__global__ __launch_bounds__(kLong) void norm_grad_long_kernel(NormArgs p) {
    __shared__ float lds[2 * 2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    float *mine = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.width;
    for (int64_t r = blockIdx.x; r < p.rows; r += p.units) {
        const int64_t x0 = r * p.x_stride, d0 = r * p.dy_stride, y0 = r * p.y_stride;
        const float mean = p.mean[r], rstd = p.rstd[r];
        const bool first = r == static_cast<int64_t>(blockIdx.x);
        float s[2] = {0.0f, 0.0f}, x[V], dy[V];
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V>(p.x, x0 + c, x);
            load_v<F32, V>(p.dy, d0 + c, dy);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[j] = (x[j] - mean) * rstd;
                // a thread's columns of the unit's shares are its own
                mine[c + j] = __builtin_fmaf(dy[j], x[j], first ? 0.0f : mine[c + j]);
                mine[p.width + c + j] = dy[j] + (first ? 0.0f : mine[p.width + c + j]);
                dy[j] *= load_w(p.weight, p.w_f32, c + j, 1.0f);
                s[0] += dy[j];
                s[1] = __builtin_fmaf(dy[j], x[j], s[1]);
            }
        }
        unit_sum<kLong>(s, lds, turn);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V>(p.x, x0 + c, x);
            load_v<F32, V>(p.dy, d0 + c, dy);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                dy[j] *= load_w(p.weight, p.w_f32, c + j, 1.0f);
                x[j] = (dy[j] - m0 - (x[j] - mean) * rstd * m1) * rstd;
            }
            store_v<F32, V>(p.y, y0 + c, x);
        }
    }
}

// dw and db from the units' shares: a workgroup has 32 columns and 8 runs of
// units, each summed in order, then the runs in order.
__global__ __launch_bounds__(kBlockThreads) void norm_join_kernel(const float *__restrict__ partial, int64_t units,
                                                                  int64_t width, void *dw, void *db, bool w_f32) {
    __shared__ float lds[8][32];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // over dw's columns, then db's
    const int64_t per = (units + 7) / 8;
    float s = 0.0f;
    if (i < 2 * width)
        for (int64_t u = run * per; u < min(units, (run + 1) * per); ++u) s += partial[u * 2 * width + i];
    lds[run][lane] = s;
    __syncthreads();
    if (run != 0 || i >= 2 * width) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += lds[k][lane];
    void *o = i < width ? dw : db;
    const int64_t c = i < width ? i : i - width;
    if (!o) return;
    if (w_f32)
        static_cast<float *>(o)[c] = s;
    else
        static_cast<uint16_t *>(o)[c] = static_cast<uint16_t>(pack_bf16x2(s, 0.0f));
}

constexpr int64_t kMaxHeld = 32768, kMaxGradHeld = 16384;  // widest rows in registers

// Units of the backward pass: two workgroups a CU, so that one's loads run
// under the other's sums; every unit more is two rows of binary32 sums to write
// and read again.
int64_t grad_units(int64_t rows, int64_t width) {
    if (width > kMaxGradHeld) return std::min<int64_t>(rows, 256);
    if (width <= 512) return std::min<int64_t>(rows, 2048);
    return std::min<int64_t>(rows, 512);
}

// Threads of a unit and elements a thread holds: as few as hold the row.
template <bool F32, int V>
hipError_t launch_norm(NormArgs p, hipStream_t stream) {
    const int64_t h = p.width;
    auto go = [&](auto kernel, int units_of_group, int threads, int64_t most) {
        p.units = std::min<int64_t>((p.rows + units_of_group - 1) / units_of_group, most / units_of_group) * units_of_group;
        kernel<<<static_cast<unsigned>(p.units / units_of_group), threads, 0, stream>>>(p);
    };
    if (h <= 512)
        go(norm_kernel<F32, V, 64, 8 / V, true>, 4, 256, 8192);
    else if (h <= 2048)
        go(norm_kernel<F32, V, 256, 8 / V, true>, 1, 256, 2048);
    else if (h <= 4096)
        go(norm_kernel<F32, V, 256, 16 / V, true>, 1, 256, 2048);
    else if (h <= 8192)
        go(norm_kernel<F32, V, 256, 32 / V, true>, 1, 256, 1024);
    else if (h <= 16384)
        go(norm_kernel<F32, V, 1024, 16 / V, true>, 1, 1024, 512);
    else
        go(norm_kernel<F32, V, 1024, 32 / V, false>, 1, 1024, 512);
    return hipGetLastError();
}

template <bool F32, int V>
hipError_t launch_norm_grad(const NormArgs &p, hipStream_t stream) {
    const int64_t h = p.width;
    const unsigned n = static_cast<unsigned>(p.units);
    if (h <= 512)
        norm_grad_kernel<F32, V, 64, 8 / V, true><<<(n + 3) / 4, 256, 0, stream>>>(p);
    else if (h <= 2048)
        norm_grad_kernel<F32, V, 256, 8 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 4096)
        norm_grad_kernel<F32, V, 256, 16 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 8192)
        norm_grad_kernel<F32, V, 512, 16 / V, true><<<n, 512, 0, stream>>>(p);
    else
        norm_grad_kernel<F32, V, 1024, 16 / V, false><<<n, 1024, 0, stream>>>(p);
    return hipGetLastError();
}

// V elements of a row at a time where they lie on 16-byte pieces, one otherwise.
template <bool F32, int V>
hipError_t launch_norm_any(NormArgs p, bool grad, hipStream_t stream) {
    if (p.width <= (grad ? kMaxGradHeld : kMaxHeld))
        return grad ? launch_norm_grad<F32, V>(p, stream) : launch_norm<F32, V>(p, stream);
    if (!grad) p.units = std::min<int64_t>(p.rows, 512);
    const unsigned n = static_cast<unsigned>(p.units);
    if (grad)
        norm_grad_long_kernel<F32, V><<<n, kLong, 0, stream>>>(p);
    else
        norm_long_kernel<F32, V><<<n, kLong, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_norm_typed(const NormArgs &p, bool grad, bool f32, hipStream_t stream) {
    const int v = f32 ? 4 : 8;
    const bool vec = p.width % v == 0 && p.x_stride % v == 0 && p.y_stride % v == 0 && p.dy_stride % v == 0;
    if (f32) return vec ? launch_norm_any<true, 4>(p, grad, stream) : launch_norm_any<true, 1>(p, grad, stream);
    return vec ? launch_norm_any<false, 8>(p, grad, stream) : launch_norm_any<false, 1>(p, grad, stream);
}

}  // namespace

hipError_t launch_layer_norm(const void *x, bool f32, int64_t x_stride, int64_t rows, int64_t width,
                             const void *weight, const void *bias, bool w_f32, float eps, void *y, int64_t y_stride,
                             float *mean, float *rstd, hipStream_t stream) {
    NormArgs p{};
    p.x = x, p.x_stride = x_stride, p.rows = rows, p.width = width;
    p.weight = weight, p.bias = bias, p.w_f32 = w_f32, p.eps = eps;
    p.y = y, p.y_stride = y_stride, p.mean = mean, p.rstd = rstd;
    return launch_norm_typed(p, false, f32, stream);
}

int64_t layer_norm_grad_workspace(int64_t rows, int64_t width) { return grad_units(rows, width) * 2 * width * 4; }

hipError_t launch_layer_norm_grad(const void *dy, int64_t dy_stride, const void *x, bool f32, int64_t x_stride,
                                  int64_t rows, int64_t width, const void *weight, bool w_f32, const float *mean,
                                  const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias,
                                  void *workspace, hipStream_t stream) {
    NormArgs p{};
    p.x = x, p.x_stride = x_stride, p.dy = dy, p.dy_stride = dy_stride, p.rows = rows, p.width = width;
    p.weight = weight, p.w_f32 = w_f32;
    p.y = dx, p.y_stride = dx_stride;
    p.mean = const_cast<float *>(mean), p.rstd = const_cast<float *>(rstd);
    p.partial = static_cast<float *>(workspace);
    p.units = grad_units(rows, width);
    if (rows > 0) {
        if (const hipError_t e = launch_norm_typed(p, true, f32, stream); e != hipSuccess) return e;
    }
    if (!dweight && !dbias) return hipSuccess;
    // no rows, no units: the sums are zero
    norm_join_kernel<<<static_cast<unsigned>((2 * width + 31) / 32), kBlockThreads, 0, stream>>>(
        p.partial, p.units, width, dweight, dbias, w_f32);
    return hipGetLastError();
}

}  // namespace zpp
