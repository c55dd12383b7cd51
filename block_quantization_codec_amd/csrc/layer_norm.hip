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
// nothing is read twice; the next row is on its way meanwhile. Units walk over
// the rows, keeping the weights, and in the backward pass their share of dw and
// db, in registers; the units' shares go to the workspace and a second kernel
// sums them in unit order, so the result does not change from run to run. Rows
// wider than 16,384 elements (32,768 of whole bf16 pieces, forward) are read
// again for each sum instead, and the backward pass takes two kernels, one along
// the rows and one down the columns.
//
// bf16, forward and backward (read + write over the time; the join included):
// 8192 x 8192, 48 to 52 us (5.2 to 5.6 TB/s) and 84 to 87 us (4.7); 4001 x 8191, whose
// rows start on no 16-byte piece, 49 (2.7) and 83 (2.4); 2048 x 28672, 49 and 107.
// binary32: 8192 x 4096, 41 to 48 and 78; 1001 x 4099 backward 17 us, of which the join and its
// launch are 4. One row of 8192: 4 us, a launch and two round trips to memory.
//
// All sums are binary32.
#include <algorithm>

#include "norm_device.h"
#include "zpp_launch.h"

namespace zpp {
namespace {

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
    float *sums;     // backward pass of long rows: each row's two means
};

// HOLD: the weights stay in registers over the rows (else they are read again for each).
template <bool F32, bool WHOLE, int T, int N, bool HOLD>
__global__ __launch_bounds__(group(T)) void norm_kernel(NormArgs p) {
    using H = Held<F32, WHOLE, T, N>;
    constexpr int V = H::V;
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
        for (int i = 0; i < N; ++i) {
            const int64_t c = H::column(i) < p.width ? H::column(i) : 0;
            load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w[i]);
            load_w<V, WHOLE>(p.bias, p.w_f32, c, p.width, 0.0f, b[i]);
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
                const float d = H::in(i, j, p.width) ? x.at(i, j) - mean : 0.0f;
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
            constexpr int one = HOLD ? 1 : 0;
            if constexpr (!HOLD) {
                load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w[0]);
                load_w<V, WHOLE>(p.bias, p.w_f32, c, p.width, 0.0f, b[0]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
                y[j] = __builtin_fmaf((x.at(i, j) - mean) * rstd, w[one * i][j], b[one * i][j]);
            store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, y);
        }
    }
}

// AHEAD: the next row's loads are made before this row's sums; a workgroup of
// 16 waves has too few registers a lane for that.
template <bool F32, bool WHOLE, int T, int N, bool AHEAD>
__global__ __launch_bounds__(group(T)) void norm_grad_kernel(NormArgs p) {
    using H = Held<F32, WHOLE, T, N>;
    constexpr int V = H::V;
    constexpr int kUnits = group(T) / T;
    __shared__ float lds[T > kWave ? 2 * 2 * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    const int64_t walk = static_cast<int64_t>(gridDim.x) * kUnits;  // rows from one of the unit's to the next
    const float inv = 1.0f / static_cast<float>(p.width);
    float w[N][V], dw[N][V], db[N][V];
    H x, dy, next_x, next_dy;
    float mean, rstd, next_mean, next_rstd;
    auto fetch = [&](int64_t r) {
        next_x.load(p.x, r * p.x_stride, p.width);
        next_dy.load(p.dy, r * p.dy_stride, p.width);
        next_mean = p.mean[r], next_rstd = p.rstd[r];
    };
    if (AHEAD && unit < p.rows) fetch(unit);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        load_w<V, WHOLE>(p.weight, p.w_f32, H::column(i) < p.width ? H::column(i) : 0, p.width, 1.0f, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.0f;
    }
    for (int64_t r = unit; r < p.rows; r += walk) {
        if constexpr (!AHEAD) fetch(r);
        x = next_x, dy = next_dy, mean = next_mean, rstd = next_rstd;
        if (AHEAD && r + walk < p.rows) fetch(r + walk);
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
                s[1] = __builtin_fmaf(g, H::in(i, j, p.width) ? xh : 0.0f, s[1]);
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
            store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, dx);
        }
    }
    if constexpr (kUnits > 1) {  // the waves' shares, in wave order, are the workgroup's
        __shared__ float share[kUnits][2][N * V][T];
        const int w_in = wave_in_block(), lane = threadIdx.x % T;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                share[w_in][0][i * V + j][lane] = dw[i][j];
                share[w_in][1][i * V + j][lane] = db[i][j];
            }
        __syncthreads();
        if (w_in != 0) return;
#pragma unroll
        for (int u = 1; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dw[i][j] += share[u][0][i * V + j][lane];
                    db[i][j] += share[u][1][i * V + j][lane];
                }
    }
    float *mine = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.width;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = H::column(i);
        if (c >= p.width) continue;
        store_share<V, WHOLE>(mine + c, p.width - c, dw[i]);
        store_share<V, WHOLE>(mine + p.width + c, p.width - c, db[i]);
    }
}

constexpr int kLong = 1024;  // threads of a unit for rows beyond the registers

template <bool F32, bool WHOLE>
__global__ __launch_bounds__(kLong) void norm_long_kernel(NormArgs p) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ float lds[2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    for (int64_t r = blockIdx.x; r < p.rows; r += p.units) {
        const int64_t x0 = r * p.x_stride, y0 = r * p.y_stride;
        float s[1] = {0.0f}, v[V];
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V, WHOLE>(p.x, x0 + c, p.width - c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] += v[j];
        }
        unit_sum<kLong>(s, lds, turn);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V, WHOLE>(p.x, x0 + c, p.width - c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = WHOLE || c + j < p.width ? v[j] - mean : 0.0f;
                s[0] = __builtin_fmaf(d, d, s[0]);
            }
        }
        unit_sum<kLong>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            float w[V], b[V];
            load_v<F32, V, WHOLE>(p.x, x0 + c, p.width - c, v);
            load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w);
            load_w<V, WHOLE>(p.bias, p.w_f32, c, p.width, 0.0f, b);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]);
            store_v<F32, V, WHOLE>(p.y, y0 + c, p.width - c, v);
        }
    }
}

// The backward pass of long rows, in two kernels: first each row's two sums,
// then, by columns, what needs them.
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(kLong) void norm_grad_sums_kernel(NormArgs p) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ float lds[2 * 2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s[2] = {0.0f, 0.0f}, x[V], dy[V], w[V];
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V, WHOLE>(p.x, r * p.x_stride + c, p.width - c, x);
            load_v<F32, V, WHOLE>(p.dy, r * p.dy_stride + c, p.width - c, dy);
            load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float g = dy[j] * w[j];
                s[0] += g;
                s[1] = __builtin_fmaf(g, WHOLE || c + j < p.width ? (x[j] - mean) * rstd : 0.0f, s[1]);
            }
        }
        unit_sum<kLong>(s, lds, turn);
        if (threadIdx.x == 0) {
            p.sums[2 * r] = s[0] * inv;
            p.sums[2 * r + 1] = s[1] * inv;
        }
    }
}

// A workgroup has 256 V columns of every p.units-th row; its share of dw and db
// is those rows'.
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(256) void norm_grad_columns_kernel(NormArgs p) {
    constexpr int V = F32 ? 4 : 8;
    const int64_t strips = (p.width + 256 * V - 1) / (256 * V);
    const int64_t unit = blockIdx.x / strips, c = ((blockIdx.x % strips) * 256 + threadIdx.x) * V;
    if (c >= p.width) return;
    float w[V], dw[V], db[V];
    load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.0f;
#pragma unroll 4
    for (int64_t r = unit; r < p.rows; r += p.units) {
        const float mean = p.mean[r], rstd = p.rstd[r], m0 = p.sums[2 * r], m1 = p.sums[2 * r + 1];
        float x[V], dy[V];
        load_v<F32, V, WHOLE>(p.x, r * p.x_stride + c, p.width - c, x);
        load_v<F32, V, WHOLE>(p.dy, r * p.dy_stride + c, p.width - c, dy);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (x[j] - mean) * rstd;
            dw[j] = __builtin_fmaf(dy[j], xh, dw[j]);
            db[j] += dy[j];
            x[j] = (dy[j] * w[j] - m0 - xh * m1) * rstd;
        }
        store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, x);
    }
    float *mine = p.partial + unit * 2 * p.width + c;
    store_share<V, WHOLE>(mine, p.width - c, dw);
    store_share<V, WHOLE>(mine + p.width, p.width - c, db);
}

constexpr int64_t kMaxGradHeld = 16384;  // widest rows in registers
// Forward, twice that where the registers suffice.
template <bool F32, bool WHOLE>
constexpr int64_t kMaxHeld = !F32 && WHOLE ? 32768 : 16384;

// Shares of the backward pass (workgroups): as many as a CU holds, so that one's
// loads run under another's sums, but 16 rows a share as long as that leaves
// every CU one, because a share is two rows of binary32 sums to write and to
// read again.
int64_t grad_units(int64_t rows, int64_t width) {
    if (width > kMaxGradHeld) return std::min<int64_t>((rows + 15) / 16, 128);
    const int64_t most = width <= 2048 ? 2048 : width <= 4096 ? 768 : width <= 8192 ? 512 : 256;
    const int64_t of = width <= 512 ? 4 : 1;  // rows a workgroup has at a time
    return std::min({(rows + of - 1) / of, most, std::max<int64_t>(rows / 16, 256)});
}

// Threads of a unit and elements a thread holds: as few as hold the row. Units
// are as many as the GPU holds at once, so that each keeps its weights for all
// its rows.
template <bool F32, bool WHOLE>
hipError_t launch_norm(NormArgs p, hipStream_t stream) {
    constexpr int V = F32 ? 4 : 8;
    const int64_t h = p.width;
    auto go = [&](auto kernel, int units_of_group, int threads, int64_t most) {
        p.units = std::min<int64_t>((p.rows + units_of_group - 1) / units_of_group, most / units_of_group) * units_of_group;
        kernel<<<static_cast<unsigned>(p.units / units_of_group), threads, 0, stream>>>(p);
    };
    if (h <= 512)
        go(norm_kernel<F32, WHOLE, 64, 8 / V, true>, 4, 256, 8192);
    else if (h <= 2048)
        go(norm_kernel<F32, WHOLE, 256, 8 / V, true>, 1, 256, 2048);
    else if (h <= 4096)
        go(norm_kernel<F32, WHOLE, 256, 16 / V, true>, 1, 256, 2048);
    else if (h <= 8192)
        go(norm_kernel<F32, WHOLE, 256, 32 / V, true>, 1, 256, 1024);
    else if (h <= 16384)
        go(norm_kernel<F32, WHOLE, 1024, 16 / V, true>, 1, 1024, 512);
    else if constexpr (kMaxHeld<F32, WHOLE> > 16384)
        go(norm_kernel<F32, WHOLE, 1024, 32 / V, false>, 1, 1024, 512);
    return hipGetLastError();
}

template <bool F32, bool WHOLE>
hipError_t launch_norm_grad(const NormArgs &p, hipStream_t stream) {
    constexpr int V = F32 ? 4 : 8;
    const int64_t h = p.width;
    const unsigned n = static_cast<unsigned>(p.units);
    if (h <= 512)
        norm_grad_kernel<F32, WHOLE, 64, 8 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 2048)
        norm_grad_kernel<F32, WHOLE, 256, 8 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 4096)
        norm_grad_kernel<F32, WHOLE, 256, 16 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 8192)
        norm_grad_kernel<F32, WHOLE, 512, 16 / V, true><<<n, 512, 0, stream>>>(p);
    else
        norm_grad_kernel<F32, WHOLE, 1024, 16 / V, false><<<n, 1024, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool F32, bool WHOLE>
hipError_t launch_norm_any(NormArgs p, bool grad, hipStream_t stream) {
    if (p.width <= (grad ? kMaxGradHeld : kMaxHeld<F32, WHOLE>))
        return grad ? launch_norm_grad<F32, WHOLE>(p, stream) : launch_norm<F32, WHOLE>(p, stream);
    const unsigned n = static_cast<unsigned>(std::min<int64_t>(p.rows, 512));
    if (!grad) {
        p.units = n;
        norm_long_kernel<F32, WHOLE><<<n, kLong, 0, stream>>>(p);
        return hipGetLastError();
    }
    norm_grad_sums_kernel<F32, WHOLE><<<n, kLong, 0, stream>>>(p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    constexpr int V = F32 ? 4 : 8;
    const int64_t strips = (p.width + 256 * V - 1) / (256 * V);
    norm_grad_columns_kernel<F32, WHOLE><<<static_cast<unsigned>(strips * p.units), 256, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_norm_typed(const NormArgs &p, bool grad, bool f32, hipStream_t stream) {
    const int v = f32 ? 4 : 8;
    const bool whole = p.width % v == 0 && p.x_stride % v == 0 && p.y_stride % v == 0 && p.dy_stride % v == 0;
    if (f32) return whole ? launch_norm_any<true, true>(p, grad, stream) : launch_norm_any<true, false>(p, grad, stream);
    return whole ? launch_norm_any<false, true>(p, grad, stream) : launch_norm_any<false, false>(p, grad, stream);
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

// The shares and, for long rows, the rows' sums after them.
int64_t layer_norm_grad_workspace(int64_t rows, int64_t width) {
    return (grad_units(rows, width) * 2 * width + (width > kMaxGradHeld ? 2 * rows : 0)) * 4;
}

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
    p.sums = p.partial + p.units * 2 * width;
    if (rows > 0) {
        if (const hipError_t e = launch_norm_typed(p, true, f32, stream); e != hipSuccess) return e;
    }
    if (!dweight && !dbias) return hipSuccess;
    // no rows, no units: the sums are zero
    return launch_norm_join<2>(p.partial, p.units, width, dweight, dbias, w_f32, stream);
}

}  // namespace zpp
