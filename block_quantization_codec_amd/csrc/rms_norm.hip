// rms_norm.hip - root-mean-square norm over the rows of a matrix, with the
// residual's addition before it and block quantization behind it, and its
// backward pass.
//
//   h    = RN(x + residual) (x itself without one), kept in x's type
//   rstd = 1 / sqrt(sum h^2 / H + eps)
//   y    = h rstd w;  codes, scales = the block quantization of y in binary32
//   xh = h rstd,  g = dy w
//   dx = rstd (g - xh sum (g xh) / H) + dsum,  dw = sum over rows of dy xh
//
// The norm is that of the h that is kept, rounded once, so that the backward
// pass, which reads it, differentiates what was computed. The codes are those of y
// before its own rounding: no second rounding in the values they stand for, and
// no more work, because y is in registers anyway.
//
// Streams like layer_norm.hip's: a unit of T threads holds a row in registers,
// the next row on its way; units walk over the rows with the weights, and in
// the backward pass their share of dw, in registers. Wider rows are read again.
//
// Memory bounds them: 8192 x 8192 bf16 with a residual to 8-bit codes, 471 MB read
// and written in 83 us (5.7 TB/s; a copy of that size 6.5); backward with dsum, 537 MB in 92
// us (5.9 TB/s) and 4 us for the join of dw. A binary32 row of 1001 x 4099 lies on no 16
// bytes: 11 us for 49 MB. One row of 8192 is a launch and latency.
#include <algorithm>

#include "norm_device.h"
#include "zpp_launch.h"

namespace zpp {
namespace {

struct RmsArgs {
    const void *x, *res;  // backward pass: x is h, res is dsum
    int64_t x_stride, res_stride;
    const void *dy;
    int64_t dy_stride;
    int64_t rows, width;
    const void *weight;
    bool w_f32;
    float eps;
    void *sum;
    int64_t sum_stride;
    void *y;
    int64_t y_stride;
    uint8_t *codes;
    float *scales;
    int bits, log2b;
    float *rstd;
    float *partial;  // [units][width]: each unit's share of dw
    int64_t units;
    float *sums;     // backward pass of long rows: each row's mean
};

// RN(a + b) of packed elements, packed.
template <bool F32>
__device__ __forceinline__ void add_packed(uint32_t (&a)[4], const uint32_t (&b)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        a[j] = F32 ? as_u(as_f(a[j]) + as_f(b[j]))
                   : pack_bf16x2(bf16_lo(a[j]) + bf16_lo(b[j]), bf16_hi(a[j]) + bf16_hi(b[j]));
}

template <bool F32, int V, bool WHOLE>
__device__ __forceinline__ void store_packed(void *base, int64_t e, int64_t left, const uint32_t (&w)[4]) {
    if (WHOLE || left >= V) {
        uint8_t *p = static_cast<uint8_t *>(base) + e * (F32 ? 4 : 2);
        const u32x4 v = {w[0], w[1], w[2], w[3]};
        if constexpr (WHOLE)
            st_out<u32x4>(p, v);
        else
            *reinterpret_cast<u32x4_at2 *>(p) = v;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j >= left) break;
            if constexpr (F32)
                static_cast<uint32_t *>(base)[e + j] = w[j];
            else
                static_cast<uint16_t *>(base)[e + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
        }
    }
}

// Maximum over aligned groups of `lanes` lanes (a power of two, 2 to 64), in each.
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lanes) {
    v = max(v, dpp_u32<0xB1>(v));
    if (lanes >= 4) v = max(v, dpp_u32<0x4E>(v));
    if (lanes >= 8) v = max(v, dpp_u32<0x141>(v));
    if (lanes >= 16) v = max(v, dpp_u32<0x140>(v));
    if (lanes >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(static_cast<uint32_t>(p[0]), static_cast<uint32_t>(p[1]));
    }
    if (lanes >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(static_cast<uint32_t>(p[0]), static_cast<uint32_t>(p[1]));
    }
    return v;
}

// Codes of V neighbouring values from element e on, and, by the block's first
// lane, its scale. `m`: the bits of the block's largest magnitude.
template <int BITS, int V>
__device__ __forceinline__ void quantize_v(const RmsArgs &p, int64_t e, const float (&v)[V], uint32_t m) {
    const float s = block_scale<Codes<BITS>::QMAX>(as_f(m));
    float r[V];
    round_codes<V, BITS>(v, s, r);
    uint8_t *to = p.codes + e * BITS / 8;
    if constexpr (V * BITS >= 32) {
        uint32_t w[V * BITS / 32];
        pack_codes<V, BITS>(r, w);
        if constexpr (V * BITS == 64)
            st_out<u32x2>(to, u32x2{w[0], w[1]});
        else
            st_out<uint32_t>(to, w[0]);
    } else {  // four nibbles in offset binary
        const uint32_t a = (as_u(r[1]) << 4) | (as_u(r[0]) & 0xFu), b = (as_u(r[3]) << 4) | (as_u(r[2]) & 0xFu);
        st_out<uint16_t>(to, static_cast<uint16_t>(__builtin_amdgcn_perm(b, a, 0x0C0C0400u) ^ 0x8888u));
    }
    if ((e & ((INT64_C(1) << p.log2b) - 1)) == 0) p.scales[e >> p.log2b] = s;
}

template <int V>
__device__ __forceinline__ uint32_t absmax_bits(const float (&v)[V]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) m = max(m, as_u(v[j]) & 0x7FFFFFFFu);
    return m;
}

// A thread's N chunks of y as codes; every thread of the unit calls it, since a
// block's maximum is its lanes'. A block is V lanes' worth of a chunk or more:
// past 64 lanes it takes neighbouring waves' and chunks', whose maxima meet in
// `lds` (N T / 64 words). One barrier: the caller has another before the next call.
template <int T, int N, int V>
__device__ __forceinline__ void quantize_chunks(const RmsArgs &p, int64_t row, const float (&y)[N][V], uint32_t *lds) {
    const int lanes = (1 << p.log2b) / V;
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = lanes_max(absmax_bits<V>(y[i]), min(lanes, kWave));
    if (lanes > kWave) {
        const int per = lanes / kWave;  // waves' runs of 64 V columns in a block
        if constexpr (T == kWave) {
            uint32_t all[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                all[i] = 0;
#pragma unroll
                for (int k = 0; k < N; ++k) all[i] = k / per == i / per ? max(all[i], m[k]) : all[i];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = all[i];
        } else {
            constexpr int W = T / kWave;
            const int w = wave_in_block() % W;
            if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) lds[i * W + w] = m[i];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int first = (i * W + w) / per * per;
                m[i] = 0;
                for (int k = 0; k < per; ++k)
                    if (first + k < N * W) m[i] = max(m[i], lds[first + k]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * T + threadIdx.x % T) * V;
        if (c >= p.width) continue;
        if (p.bits == 8)
            quantize_v<8, V>(p, row * p.width + c, y[i], m[i]);
        else
            quantize_v<4, V>(p, row * p.width + c, y[i], m[i]);
    }
}

// The weights stay in registers over the rows.
template <bool F32, bool WHOLE, int T, int N, bool QUANT>
__global__ __launch_bounds__(group(T)) void rms_kernel(RmsArgs p) {
    using H = Held<F32, WHOLE, T, N>;
    constexpr int V = H::V;
    constexpr int kUnits = group(T) / T;
    __shared__ float lds[T > kWave ? 2 * (T / kWave) : 1];
    __shared__ uint32_t maxima[QUANT && T > kWave ? N * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    if (kUnits > 1 && unit >= p.rows) return;
    const float inv = 1.0f / static_cast<float>(p.width);
    float w[N][V];
    H x, next, next_res;
    auto fetch = [&](int64_t r) {
        next.load(p.x, r * p.x_stride, p.width);
        if (p.res) next_res.load(p.res, r * p.res_stride, p.width);
    };
    fetch(unit);
#pragma unroll
    for (int i = 0; i < N; ++i)
        load_w<V, WHOLE>(p.weight, p.w_f32, H::column(i) < p.width ? H::column(i) : 0, p.width, 1.0f, w[i]);
    for (int64_t r = unit; r < p.rows; r += p.units) {
        x = next;
        if (p.res) {
#pragma unroll
            for (int i = 0; i < N; ++i) add_packed<F32>(x.w[i], next_res.w[i]);
        }
        if (r + p.units < p.rows) fetch(r + p.units);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] = __builtin_fmaf(x.at(i, j), x.at(i, j), s[0]);
        if (p.sum) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t c = H::column(i);
                if (c < p.width) store_packed<F32, V, WHOLE>(p.sum, r * p.sum_stride + c, p.width - c, x.w[i]);
            }
        }
        unit_sum<T>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x % T == 0) p.rstd[r] = rstd;
        float y[QUANT ? N : 1][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = H::column(i);
            constexpr int own = QUANT ? 1 : 0;
#pragma unroll
            for (int j = 0; j < V; ++j) y[own * i][j] = x.at(i, j) * rstd * w[i][j];
            if (p.y && c < p.width) store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, y[own * i]);
        }
        if constexpr (QUANT) quantize_chunks<T, N, V>(p, r, y, maxima);
    }
}

// AHEAD: the next row's loads are made before this row's sums; a workgroup of
// 16 waves has too few registers a lane for that.
template <bool F32, bool WHOLE, int T, int N, bool AHEAD>
__global__ __launch_bounds__(group(T)) void rms_grad_kernel(RmsArgs p) {
    using H = Held<F32, WHOLE, T, N>;
    constexpr int V = H::V;
    constexpr int kUnits = group(T) / T;
    __shared__ float lds[T > kWave ? 2 * (T / kWave) : 1];
    int turn = 0;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (kUnits > 1 ? wave_in_block() : 0);
    const int64_t walk = static_cast<int64_t>(gridDim.x) * kUnits;  // rows from one of the unit's to the next
    const float inv = 1.0f / static_cast<float>(p.width);
    float w[N][V], dw[N][V];
    H h, dy, ds, next_h, next_dy, next_ds;
    float rstd, next_rstd;
    auto fetch = [&](int64_t r) {
        next_h.load(p.x, r * p.x_stride, p.width);
        next_dy.load(p.dy, r * p.dy_stride, p.width);
        if (p.res) next_ds.load(p.res, r * p.res_stride, p.width);
        next_rstd = p.rstd[r];
    };
    if (!p.res) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) next_ds.w[i][j] = 0;
    }
    if (AHEAD && unit < p.rows) fetch(unit);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        load_w<V, WHOLE>(p.weight, p.w_f32, H::column(i) < p.width ? H::column(i) : 0, p.width, 1.0f, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.0f;
    }
    for (int64_t r = unit; r < p.rows; r += walk) {
        if constexpr (!AHEAD) fetch(r);
        h = next_h, dy = next_dy, ds = next_ds, rstd = next_rstd;
        if (AHEAD && r + walk < p.rows) fetch(r + walk);
        // columns past the width have h = dy = 0: they add nothing
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = h.at(i, j) * rstd, d = dy.at(i, j), g = d * w[i][j];
                dw[i][j] = __builtin_fmaf(d, xh, dw[i][j]);
                s[0] = __builtin_fmaf(g, H::in(i, j, p.width) ? xh : 0.0f, s[0]);
            }
        unit_sum<T>(s, lds, turn);
        const float m = s[0] * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = H::column(i);
            if (c >= p.width) continue;
            float dx[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = h.at(i, j) * rstd;
                dx[j] = (dy.at(i, j) * w[i][j] - xh * m) * rstd + ds.at(i, j);
            }
            store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, dx);
        }
    }
    if constexpr (kUnits > 1) {  // the waves' shares, in wave order, are the workgroup's
        __shared__ float share[kUnits][N * V][T];
        const int w_in = wave_in_block(), lane = threadIdx.x % T;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) share[w_in][i * V + j][lane] = dw[i][j];
        __syncthreads();
        if (w_in != 0) return;
#pragma unroll
        for (int u = 1; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) dw[i][j] += share[u][i * V + j][lane];
    }
    float *mine = p.partial + static_cast<int64_t>(blockIdx.x) * p.width;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = H::column(i);
        if (c < p.width) store_share<V, WHOLE>(mine + c, p.width - c, dw[i]);
    }
}

constexpr int kLong = 1024;  // threads of a unit for rows beyond the registers

// A row that is read twice: for its sum of squares, and for its results.
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(kLong) void rms_long_kernel(RmsArgs p) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ float lds[2 * (kLong / kWave)];
    __shared__ uint32_t maxima[2][kLong / kWave];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    for (int64_t r = blockIdx.x; r < p.rows; r += p.units) {
        // V elements of h, zeros past the row's end
        auto load = [&](int64_t c, uint32_t(&v)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = 0;
            if (c >= p.width) return;
            load_packed<F32, V, WHOLE>(p.x, r * p.x_stride + c, p.width - c, v);
            if (!p.res) return;
            uint32_t o[4];
            load_packed<F32, V, WHOLE>(p.res, r * p.res_stride + c, p.width - c, o);
            add_packed<F32>(v, o);
        };
        float s[1] = {0.0f};
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            uint32_t v[4];
            load(c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] = __builtin_fmaf(unpack<F32>(v, j), unpack<F32>(v, j), s[0]);
            if (p.sum) store_packed<F32, V, WHOLE>(p.sum, r * p.sum_stride + c, p.width - c, v);
        }
        unit_sum<kLong>(s, lds, turn);
        const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv + p.eps);
        if (threadIdx.x == 0) p.rstd[r] = rstd;
        // all threads take every round: a block's maximum is its lanes'
        int at = 0;
        for (int64_t c0 = 0; c0 < p.width; c0 += kLong * V, at ^= 1) {
            const int64_t c = c0 + threadIdx.x * V;
            uint32_t v[4];
            float w[V], y[V];
            load(c, v);
            load_w<V, WHOLE>(p.weight, p.w_f32, c < p.width ? c : 0, p.width, 1.0f, w);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = unpack<F32>(v, j) * rstd * w[j];
            if (p.y && c < p.width) store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, y);
            if (!p.codes) continue;
            const int lanes = (1 << p.log2b) / V;
            uint32_t m = lanes_max(absmax_bits<V>(y), min(lanes, kWave));
            if (lanes > kWave) {  // a block is at most the workgroup's 1024 lanes
                const int per = lanes / kWave, wave = wave_in_block();
                if ((threadIdx.x & (kWave - 1)) == 0) maxima[at][wave] = m;
                __syncthreads();
                m = 0;
                for (int k = 0; k < per; ++k) m = max(m, maxima[at][wave / per * per + k]);
            }
            if (c >= p.width) continue;
            if (p.bits == 8)
                quantize_v<8, V>(p, r * p.width + c, y, m);
            else
                quantize_v<4, V>(p, r * p.width + c, y, m);
        }
    }
}

// The backward pass of long rows, in two kernels: first each row's mean of
// g xh, then, by columns, what needs it.
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(kLong) void rms_grad_sums_kernel(RmsArgs p) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ float lds[2 * (kLong / kWave)];
    int turn = 0;
    const float inv = 1.0f / static_cast<float>(p.width);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const float rstd = p.rstd[r];
        float s[1] = {0.0f}, h[V], dy[V], w[V];
        for (int64_t c = threadIdx.x * V; c < p.width; c += kLong * V) {
            load_v<F32, V, WHOLE>(p.x, r * p.x_stride + c, p.width - c, h);
            load_v<F32, V, WHOLE>(p.dy, r * p.dy_stride + c, p.width - c, dy);
            load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w);
#pragma unroll
            for (int j = 0; j < V; ++j)
                s[0] = __builtin_fmaf(dy[j] * w[j], WHOLE || c + j < p.width ? h[j] * rstd : 0.0f, s[0]);
        }
        unit_sum<kLong>(s, lds, turn);
        if (threadIdx.x == 0) p.sums[r] = s[0] * inv;
    }
}

// A workgroup has 256 V columns of every p.units-th row; its share of dw is
// those rows'.
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(256) void rms_grad_columns_kernel(RmsArgs p) {
    constexpr int V = F32 ? 4 : 8;
    const int64_t strips = (p.width + 256 * V - 1) / (256 * V);
    const int64_t unit = blockIdx.x / strips, c = ((blockIdx.x % strips) * 256 + threadIdx.x) * V;
    if (c >= p.width) return;
    float w[V], dw[V];
    load_w<V, WHOLE>(p.weight, p.w_f32, c, p.width, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j) dw[j] = 0.0f;
#pragma unroll 4
    for (int64_t r = unit; r < p.rows; r += p.units) {
        const float rstd = p.rstd[r], m = p.sums[r];
        float h[V], dy[V], ds[V];
        load_v<F32, V, WHOLE>(p.x, r * p.x_stride + c, p.width - c, h);
        load_v<F32, V, WHOLE>(p.dy, r * p.dy_stride + c, p.width - c, dy);
#pragma unroll
        for (int j = 0; j < V; ++j) ds[j] = 0.0f;
        if (p.res) load_v<F32, V, WHOLE>(p.res, r * p.res_stride + c, p.width - c, ds);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = h[j] * rstd;
            dw[j] = __builtin_fmaf(dy[j], xh, dw[j]);
            h[j] = (dy[j] * w[j] - xh * m) * rstd + ds[j];
        }
        store_v<F32, V, WHOLE>(p.y, r * p.y_stride + c, p.width - c, h);
    }
    store_share<V, WHOLE>(p.partial + unit * p.width + c, p.width - c, dw);
}

constexpr int64_t kMaxHeld = 16384;  // widest rows in registers

// Shares of the backward pass (workgroups): as many as keep the memory busy, but 16 rows
// a share as long as that leaves every CU one, because a share is a row of binary32 sums to
// write and to read again. 8192 x 5120 bf16: 65 us with 256 shares, 68 with 512.
int64_t grad_units(int64_t rows, int64_t width) {
    if (width > kMaxHeld) return std::min<int64_t>((rows + 15) / 16, 128);
    const int64_t most = width <= 2048 ? 2048 : width <= 4096 ? 768 : 256;
    const int64_t of = width <= 512 ? 4 : 1;  // rows a workgroup has at a time
    return std::min({(rows + of - 1) / of, most, std::max<int64_t>(rows / 16, 256)});
}

// Threads of a unit and elements a thread holds: as few as hold the row. Units are as
// many as the GPU holds at once or some more, so that each keeps its weights for its
// rows. 8192 x 8192 bf16 to 8-bit codes: 86 us with 512 threads and 2048 units, 96 with 256
// threads and 1024 units.
template <bool F32, bool WHOLE, bool QUANT>
hipError_t launch_rms(RmsArgs p, hipStream_t stream) {
    constexpr int V = F32 ? 4 : 8;
    const int64_t h = p.width;
    auto go = [&](auto kernel, int units_of_group, int threads, int64_t most) {
        p.units = std::min<int64_t>((p.rows + units_of_group - 1) / units_of_group, most / units_of_group) * units_of_group;
        kernel<<<static_cast<unsigned>(p.units / units_of_group), threads, 0, stream>>>(p);
    };
    if (h <= 512)
        go(rms_kernel<F32, WHOLE, 64, 8 / V, QUANT>, 4, 256, 8192);
    else if (h <= 2048)
        go(rms_kernel<F32, WHOLE, 256, 8 / V, QUANT>, 1, 256, 2048);
    else if (h <= 4096)
        go(rms_kernel<F32, WHOLE, 256, 16 / V, QUANT>, 1, 256, 4096);
    else if (h <= 8192)
        go(rms_kernel<F32, WHOLE, 512, 16 / V, QUANT>, 1, 512, 2048);
    else
        go(rms_kernel<F32, WHOLE, 1024, 16 / V, QUANT>, 1, 1024, 512);
    return hipGetLastError();
}

template <bool F32, bool WHOLE>
hipError_t launch_rms_grad(const RmsArgs &p, hipStream_t stream) {
    constexpr int V = F32 ? 4 : 8;
    const int64_t h = p.width;
    const unsigned n = static_cast<unsigned>(p.units);
    if (h <= 512)
        rms_grad_kernel<F32, WHOLE, 64, 8 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 2048)
        rms_grad_kernel<F32, WHOLE, 256, 8 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 4096)
        rms_grad_kernel<F32, WHOLE, 256, 16 / V, true><<<n, 256, 0, stream>>>(p);
    else if (h <= 8192)
        rms_grad_kernel<F32, WHOLE, 512, 16 / V, true><<<n, 512, 0, stream>>>(p);
    else
        rms_grad_kernel<F32, WHOLE, 1024, 16 / V, false><<<n, 1024, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool F32, bool WHOLE>
hipError_t launch_rms_any(RmsArgs p, bool grad, hipStream_t stream) {
    if (p.width <= kMaxHeld) {
        if (grad) return launch_rms_grad<F32, WHOLE>(p, stream);
        return p.codes ? launch_rms<F32, WHOLE, true>(p, stream) : launch_rms<F32, WHOLE, false>(p, stream);
    }
    const unsigned n = static_cast<unsigned>(std::min<int64_t>(p.rows, 512));
    if (!grad) {
        p.units = n;
        rms_long_kernel<F32, WHOLE><<<n, kLong, 0, stream>>>(p);
        return hipGetLastError();
    }
    rms_grad_sums_kernel<F32, WHOLE><<<n, kLong, 0, stream>>>(p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    constexpr int V = F32 ? 4 : 8;
    const int64_t strips = (p.width + 256 * V - 1) / (256 * V);
    rms_grad_columns_kernel<F32, WHOLE><<<static_cast<unsigned>(strips * p.units), 256, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_rms_typed(const RmsArgs &p, bool grad, bool f32, hipStream_t stream) {
    const int64_t v = f32 ? 4 : 8, all = p.width | p.x_stride | p.res_stride | p.dy_stride | p.sum_stride | p.y_stride;
    const bool whole = all % v == 0;
    if (f32) return whole ? launch_rms_any<true, true>(p, grad, stream) : launch_rms_any<true, false>(p, grad, stream);
    return whole ? launch_rms_any<false, true>(p, grad, stream) : launch_rms_any<false, false>(p, grad, stream);
}

}  // namespace

hipError_t launch_rms_norm(const void *x, bool f32, int64_t x_stride, const void *residual, int64_t residual_stride,
                           int64_t rows, int64_t width, const void *weight, bool w_f32, float eps, void *sum,
                           int64_t sum_stride, void *y, int64_t y_stride, void *codes, float *scales, int bits,
                           int log2b, float *rstd, hipStream_t stream) {
    RmsArgs p{};
    p.x = x, p.x_stride = x_stride, p.rows = rows, p.width = width;
    p.res = residual, p.res_stride = residual ? residual_stride : 0;
    p.weight = weight, p.w_f32 = w_f32, p.eps = eps;
    p.sum = sum, p.sum_stride = sum ? sum_stride : 0;
    p.y = y, p.y_stride = y ? y_stride : 0;
    p.codes = static_cast<uint8_t *>(codes), p.scales = scales, p.bits = bits, p.log2b = log2b;
    p.rstd = rstd;
    return launch_rms_typed(p, false, f32, stream);
}

// The shares and, for long rows, the rows' means after them.
int64_t rms_norm_grad_workspace(int64_t rows, int64_t width) {
    return (grad_units(rows, width) * width + (width > kMaxHeld ? rows : 0)) * 4;
}

hipError_t launch_rms_norm_grad(const void *dy, int64_t dy_stride, const void *h, bool f32, int64_t h_stride,
                                const void *dsum, int64_t dsum_stride, int64_t rows, int64_t width,
                                const void *weight, bool w_f32, const float *rstd, void *dx, int64_t dx_stride,
                                void *dweight, void *workspace, hipStream_t stream) {
    RmsArgs p{};
    p.x = h, p.x_stride = h_stride, p.dy = dy, p.dy_stride = dy_stride, p.rows = rows, p.width = width;
    p.res = dsum, p.res_stride = dsum ? dsum_stride : 0;
    p.weight = weight, p.w_f32 = w_f32;
    p.y = dx, p.y_stride = dx_stride;
    p.rstd = const_cast<float *>(rstd);
    p.partial = static_cast<float *>(workspace);
    p.units = grad_units(rows, width);
    p.sums = p.partial + p.units * width;
    if (rows > 0) {
        if (const hipError_t e = launch_rms_typed(p, true, f32, stream); e != hipSuccess) return e;
    }
    if (!dweight) return hipSuccess;
    // no rows, no units: the sum is zero
    return launch_norm_join<1>(p.partial, p.units, width, dweight, nullptr, w_f32, stream);
}

}  // namespace zpp
