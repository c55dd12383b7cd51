// layer_norm.hip - layer norm over the rows of a matrix, forward and backward.
//
//   mean = sum x / H,  var = sum (x - mean)^2 / H,  rstd = 1 / sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   xh = (x - mean) rstd,  g = dy w
//   dx = rstd (g - sum g / H - xh sum (g xh) / H)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both are streams: one read of every input and one write of every output.
// A unit of T threads (a wave, 4 or 16 of them, by the row's width) holds a
// whole row in registers, up to 32 elements a thread, so the variance is the
// sum of squared differences from the mean already known (no cancellation)
// and nothing is read twice. Units walk over the rows, keeping the weights,
// and in the backward pass their share of dw and db, in registers; the units'
// shares go to the workspace and a second kernel sums them in unit order, so
// the result does not change from run to run. Rows wider than 32,768 elements
// are read again for each sum instead (LONG); their shares are summed in the
// workspace itself.
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

constexpr int kHeld = 32;  // elements of a row a thread holds

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

// The columns a thread of a unit holds: chunk i is V elements at (i T + thread) V.
template <int T, int V>
__device__ __forceinline__ int64_t column(int i) {
    return (static_cast<int64_t>(i) * T + threadIdx.x % T) * V;
}

template <bool F32, int V, int T>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(NormArgs p) {
    constexpr int kThreads = T < 256 ? 256 : T, kUnits = kThreads / T, kN = kHeld / V;
    __shared__ float lds[T > kWave ? 2 * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    const float inv = 1.0f / static_cast<float>(p.width);
    float w[kN][V], b[kN][V];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t c = min(column<T, V>(i) + j, p.width - 1);
            w[i][j] = load_w(p.weight, p.w_f32, c, 1.0f);
            b[i][j] = load_w(p.bias, p.w_f32, c, 0.0f);
        }
    for (int64_t r = unit; r < p.rows; r += p.units) {
        float x[kN][V], s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t c = column<T, V>(i);
#pragma unroll
            for (int j = 0; j < V; ++j) x[i][j] = 0.0f;
            if (c < p.width) load_v<F32, V>(p.x, r * p.x_stride + c, x[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] += x[i][j];
        }
        unit_sum<T>(s, lds, turn);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = column<T, V>(i) < p.width ? x[i][j] - mean : 0.0f;
                s[0] = __builtin_fmaf(d, d, s[0]);
            }
        unit_sum<T>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x % T == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t c = column<T, V>(i);
            if (c >= p.width) continue;
            float y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = __builtin_fmaf((x[i][j] - mean) * rstd, w[i][j], b[i][j]);
            store_v<F32, V>(p.y, r * p.y_stride + c, y);
        }
    }
}

template <bool F32, int V, int T>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_grad_kernel(NormArgs p) {
    constexpr int kThreads = T < 256 ? 256 : T, kUnits = kThreads / T, kN = kHeld / V;
    __shared__ float lds[T > kWave ? 2 * 2 * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    if (kUnits > 1 && unit >= p.units) return;
    const float inv = 1.0f / static_cast<float>(p.width);
    float dw[kN][V], db[kN][V];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.0f;
    for (int64_t r = unit; r < p.rows; r += p.units) {
        float xh[kN][V], dy[kN][V], s[2] = {0.0f, 0.0f};
        const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t c = column<T, V>(i);
#pragma unroll
            for (int j = 0; j < V; ++j) xh[i][j] = dy[i][j] = 0.0f;
            if (c < p.width) {
                load_v<F32, V>(p.x, r * p.x_stride + c, xh[i]);
                load_v<F32, V>(p.dy, r * p.dy_stride + c, dy[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t c = column<T, V>(i);
            if (c >= p.width) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[i][j] = (xh[i][j] - mean) * rstd;
                dw[i][j] = __builtin_fmaf(dy[i][j], xh[i][j], dw[i][j]);
                db[i][j] += dy[i][j];
                dy[i][j] *= load_w(p.weight, p.w_f32, c + j, 1.0f);
                s[0] += dy[i][j];
                s[1] = __builtin_fmaf(dy[i][j], xh[i][j], s[1]);
            }
        }
        unit_sum<T>(s, lds, turn);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t c = column<T, V>(i);
            if (c >= p.width) continue;
            float dx[V];
#pragma unroll
            for (int j = 0; j < V; ++j) dx[j] = (dy[i][j] - m0 - xh[i][j] * m1) * rstd;
            store_v<F32, V>(p.y, r * p.y_stride + c, dx);
        }
    }
    float *mine = p.partial + unit * 2 * p.width;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int64_t c = column<T, V>(i);
        if (c >= p.width) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mine[c + j] = dw[i][j];
            mine[p.width + c + j] = db[i][j];
        }
    }
}

constexpr int kLong = 1024;  // threads of a unit for rows beyond the registers

template <bool F32>
__global__ __launch_bounds__(kLong) void norm_long_kernel(NormArgs p) {
    __shared__ float lds[2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    for (int64_t r = blockIdx.x; r < p.rows; r += p.units) {
        const int64_t x0 = r * p.x_stride, y0 = r * p.y_stride;
        float s[1] = {0.0f}, v;
        for (int64_t c = threadIdx.x; c < p.width; c += kLong) {
            load_v<F32, 1>(p.x, x0 + c, &v);
            s[0] += v;
        }
        unit_sum<kLong>(s, lds, turn);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
        for (int64_t c = threadIdx.x; c < p.width; c += kLong) {
            load_v<F32, 1>(p.x, x0 + c, &v);
            s[0] = __builtin_fmaf(v - mean, v - mean, s[0]);
        }
        unit_sum<kLong>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        for (int64_t c = threadIdx.x; c < p.width; c += kLong) {
            load_v<F32, 1>(p.x, x0 + c, &v);
            v = __builtin_fmaf((v - mean) * rstd, load_w(p.weight, p.w_f32, c, 1.0f),
                               load_w(p.bias, p.w_f32, c, 0.0f));
            store_v<F32, 1>(p.y, y0 + c, &v);
        }
    }
}

template <bool F32>
__global__ __launch_bounds__(kLong) void norm_grad_long_kernel(NormArgs p) {
    __shared__ float lds[2 * 2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    float *mine = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.width;
    for (int64_t r = blockIdx.x; r < p.rows; r += p.units) {
        const int64_t x0 = r * p.x_stride, d0 = r * p.dy_stride, y0 = r * p.y_stride;
        const float mean = p.mean[r], rstd = p.rstd[r];
        const bool first = r == static_cast<int64_t>(blockIdx.x);
        float s[2] = {0.0f, 0.0f}, x, dy;
        for (int64_t c = threadIdx.x; c < p.width; c += kLong) {
            load_v<F32, 1>(p.x, x0 + c, &x);
            load_v<F32, 1>(p.dy, d0 + c, &dy);
            x = (x - mean) * rstd;
            // a thread's columns of the unit's shares are its own
            mine[c] = __builtin_fmaf(dy, x, first ? 0.0f : mine[c]);
            mine[p.width + c] = dy + (first ? 0.0f : mine[p.width + c]);
            dy *= load_w(p.weight, p.w_f32, c, 1.0f);
            s[0] += dy;
            s[1] = __builtin_fmaf(dy, x, s[1]);
        }
        unit_sum<kLong>(s, lds, turn);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
        for (int64_t c = threadIdx.x; c < p.width; c += kLong) {
            load_v<F32, 1>(p.x, x0 + c, &x);
            load_v<F32, 1>(p.dy, d0 + c, &dy);
            dy *= load_w(p.weight, p.w_f32, c, 1.0f);
            x = (dy - m0 - (x - mean) * rstd * m1) * rstd;
            store_v<F32, 1>(p.y, y0 + c, &x);
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

// No rows: dw and db are zero.
constexpr int64_t kMaxUnits = 512;

// Threads of a unit: as few as hold the row.
int unit_threads(int64_t width) { return width <= 64 * kHeld ? 64 : width <= 256 * kHeld ? 256 : 1024; }

int64_t grad_units(int64_t rows, int64_t width) {
    const int64_t most = width > 1024 * kHeld ? 256 : unit_threads(width) == 1024 ? 256 : kMaxUnits;
    return std::min(rows, most);
}

template <bool F32, int V>
hipError_t launch_norm(NormArgs p, hipStream_t stream) {
    const int t = unit_threads(p.width);
    p.units = std::min<int64_t>(p.rows, t == 64 ? 8192 : t == 256 ? 2048 : 512);
    const unsigned grid = static_cast<unsigned>(t == 64 ? (p.units + 3) / 4 : p.units);
    if (t == 64) {
        p.units = grid * 4;
        norm_kernel<F32, V, 64><<<grid, 256, 0, stream>>>(p);
    } else if (t == 256) {
        norm_kernel<F32, V, 256><<<grid, 256, 0, stream>>>(p);
    } else {
        norm_kernel<F32, V, 1024><<<grid, 1024, 0, stream>>>(p);
    }
    return hipGetLastError();
}

template <bool F32, int V>
hipError_t launch_norm_grad(const NormArgs &p, hipStream_t stream) {
    const int t = unit_threads(p.width);
    const unsigned grid = static_cast<unsigned>(t == 64 ? (p.units + 3) / 4 : p.units);
    if (t == 64)
        norm_grad_kernel<F32, V, 64><<<grid, 256, 0, stream>>>(p);
    else if (t == 256)
        norm_grad_kernel<F32, V, 256><<<grid, 256, 0, stream>>>(p);
    else
        norm_grad_kernel<F32, V, 1024><<<grid, 1024, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const void *x, bool f32, int64_t x_stride, int64_t rows, int64_t width,
                             const void *weight, const void *bias, bool w_f32, float eps, void *y, int64_t y_stride,
                             float *mean, float *rstd, hipStream_t stream) {
    NormArgs p{};
    p.x = x, p.x_stride = x_stride, p.rows = rows, p.width = width;
    p.weight = weight, p.bias = bias, p.w_f32 = w_f32, p.eps = eps;
    p.y = y, p.y_stride = y_stride, p.mean = mean, p.rstd = rstd;
    if (width > 1024 * kHeld) {
        p.units = std::min<int64_t>(rows, 512);
        if (f32)
            norm_long_kernel<true><<<static_cast<unsigned>(p.units), kLong, 0, stream>>>(p);
        else
            norm_long_kernel<false><<<static_cast<unsigned>(p.units), kLong, 0, stream>>>(p);
        return hipGetLastError();
    }
    const int v = f32 ? 4 : 8;
    const bool vec = width % v == 0 && x_stride % v == 0 && y_stride % v == 0;
    if (f32) return vec ? launch_norm<true, 4>(p, stream) : launch_norm<true, 1>(p, stream);
    return vec ? launch_norm<false, 8>(p, stream) : launch_norm<false, 1>(p, stream);
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
    hipError_t e = hipSuccess;
    if (rows > 0) {
        const int v = f32 ? 4 : 8;
        const bool vec = width % v == 0 && x_stride % v == 0 && dy_stride % v == 0 && dx_stride % v == 0;
        if (width > 1024 * kHeld) {
            if (f32)
                norm_grad_long_kernel<true><<<static_cast<unsigned>(p.units), kLong, 0, stream>>>(p);
            else
                norm_grad_long_kernel<false><<<static_cast<unsigned>(p.units), kLong, 0, stream>>>(p);
            e = hipGetLastError();
        } else if (f32) {
            e = vec ? launch_norm_grad<true, 4>(p, stream) : launch_norm_grad<true, 1>(p, stream);
        } else {
            e = vec ? launch_norm_grad<false, 8>(p, stream) : launch_norm_grad<false, 1>(p, stream);
        }
    }
    if (e != hipSuccess || (!dweight && !dbias)) return e;
    norm_join_kernel<<<static_cast<unsigned>((2 * width + 31) / 32), kBlockThreads, 0, stream>>>(
        p.partial, p.units, width, dweight, dbias, w_f32);
    return hipGetLastError();
}

}  // namespace zpp
