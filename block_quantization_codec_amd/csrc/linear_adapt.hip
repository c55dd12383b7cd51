// linear_adapt.hip - low-rank adapters beside a product on block codes: what their
// own kernels compute. The product's kernels add the result (linear_adapt.h).
//
//   down:  low[m] = s_g x[m] A_g^T (forward),  s_g dy[m] B_g (backward)     g = ids[m]
//   rows:  dA_g = sum over g's rows of low[m]^T x[m],  dB_g = sum of dy[m]^T low[m]
//
// Both read x or dy once from memory and little else, so they are streams that
// end in matrix instructions: operands go from global memory straight into
// registers, and what is small (the adapters, low) is read again from L2.
//
// Rows are taken 64 at a time. A ballot says which of them have an adapter; those
// rows, wherever they stand, become the matrix instruction's rows (down) or its
// contraction (rows). Rows without an adapter get low = 0 and are in no sum.
//
// Sums are binary32; bf16 factors are exact, binary32 ones enter as three bf16
// parts (low, where everything else is bf16, as two: linear_adapt.h).
#include <algorithm>

#include "linear_adapt.h"

namespace zpp {
namespace {

constexpr int64_t kMaxGroups = 1 << 22;  // workgroups of one launch

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct AdaptArgs {
    const void *x;        // rows of len elements: x (forward, dA), dy (backward, dB)
    int64_t x_stride;
    int64_t rows, len;
    const void *w;        // down: A [adapters][rank][len], or B [adapters][len][rank]
    const int32_t *ids;   // null: every row has the first
    const float *scaling; // null: ones
    int adapters, rank;
    float *low;           // [rows][rank]
    float *partial;       // parts of low, or of the adapters' gradients
    int splits;
    int64_t split_steps;  // down: steps of 64 of each part; rows: chunks of 64 rows
    int64_t chunks, slots, ranks;
};

__device__ __forceinline__ bool has_adapter(const AdaptArgs &p, int64_t row, int &id) {
    const bool in = row < p.rows;
    id = p.ids ? p.ids[in ? row : 0] : 0;
    return in && static_cast<uint32_t>(id) < static_cast<uint32_t>(p.adapters);
}

// ---- down -------------------------------------------------------------------------

// 16 elements of a row from k on as operand parts of two matrix instructions:
// zeros past the end. `whole`: all 16 are in the row.
template <bool F32>
__device__ __forceinline__ void load16(const void *base, int64_t e, int64_t left, u32x4 (&b)[2][F32 ? 3 : 1]) {
    if constexpr (F32) {
        float f[16];
        const float *from = static_cast<const float *>(base) + e;
        if (left >= 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 v = *reinterpret_cast<const u32x4_at4 *>(from + 4 * i);
#pragma unroll
                for (int c = 0; c < 4; ++c) f[4 * i + c] = as_f(v[c]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = i < left ? from[i] : 0.0f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float v[8] = {f[8 * h], f[8 * h + 1], f[8 * h + 2], f[8 * h + 3],
                                f[8 * h + 4], f[8 * h + 5], f[8 * h + 6], f[8 * h + 7]};
            operand_of<3>(v, b[h]);
        }
    } else {
        const uint16_t *from = static_cast<const uint16_t *>(base) + e;
        if (left >= 16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) b[h][0] = *reinterpret_cast<const u32x4_any *>(from + 8 * h);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int i = 8 * h + 2 * d;
                    b[h][0][d] = (i < left ? from[i] : 0u) | (i + 1 < left ? static_cast<uint32_t>(from[i + 1]) << 16 : 0u);
                }
        }
    }
}

// The adapter's operands of the step's two matrix instructions, four tiles of
// ranks each: tile t's rank is r + t. The lane has contraction indices k .. k + 15.
template <bool GRAD, bool F32>
__device__ __forceinline__ void load_w(const AdaptArgs &p, int64_t g, int r, int64_t k, u32x4 (&b)[4][2][F32 ? 3 : 1]) {
    constexpr int P = F32 ? 3 : 1;
    if constexpr (!GRAD) {  // [rank][len]: the lane's indices lie side by side
#pragma unroll
        for (int t = 0; t < 4; ++t)
            load16<F32>(p.w, (g * p.rank + min(r + t, p.rank - 1)) * p.len + min(k, p.len), p.len - k, b[t]);
    } else {  // [len][rank]: four neighbouring ranks of 16 rows, turned
        const int64_t base = g * p.len * p.rank + min(r, p.rank - 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (F32) {
                f32x4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t n = k + 8 * h + i;
                    v[i] = ld<f32x4>(static_cast<const float *>(p.w) + base + min(n, p.len - 1) * p.rank);
                    if (n >= p.len) v[i] = f32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float o[8] = {v[0][t], v[1][t], v[2][t], v[3][t], v[4][t], v[5][t], v[6][t], v[7][t]};
                    operand_of<P>(o, b[t][h]);
                }
            } else {
                u32x2 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t n = k + 8 * h + i;
                    v[i] = ld<u32x2>(static_cast<const uint16_t *>(p.w) + base + min(n, p.len - 1) * p.rank);
                    if (n >= p.len) v[i] = u32x2{0, 0};
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        b[t][h][0][d] = __builtin_amdgcn_perm(v[2 * d + 1][t / 2], v[2 * d][t / 2],
                                                              t % 2 == 0 ? 0x05040100u : 0x07060302u);
            }
        }
    }
}

// One adapter's rows of a chunk (16 MT of them at most) by 64 of its ranks: the
// workgroup's 4 waves take steps of 64 indices in turn and join their sums in LDS.
template <bool GRAD, bool XF32, bool WF32, int MT>
__device__ __forceinline__ void down_rows(const AdaptArgs &p, int64_t chunk, int64_t rank0, int split, int g, int count,
                                          int list, f32x4 *sums) {
    constexpr int PX = XF32 ? 3 : 1, PW = WF32 ? 3 : 1;
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block(), q = lane >> 4, j = lane & 15;
    const int r = static_cast<int>(rank0) + 4 * j;
    int64_t at[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) at[m] = (chunk * 64 + listed(list, min(16 * m + j, count - 1))) * p.x_stride;
    f32x4 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
    const int64_t s0 = split * p.split_steps, s1 = min(s0 + p.split_steps, (p.len + 63) / 64);
#pragma unroll 2
    for (int64_t s = s0 + w; s < s1; s += 4) {
        const int64_t k = s * 64 + 16 * q;
        u32x4 b[4][2][PW];
        load_w<GRAD, WF32>(p, g, r, k, b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            u32x4 a[2][PX];
            load16<XF32>(p.x, at[m] + min(k, p.len), p.len - k, a);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                acc[m][t] = mfma_parts<PX, PW>(a[0], b[t][0], acc[m][t]);
                acc[m][t] = mfma_parts<PX, PW>(a[1], b[t][1], acc[m][t]);
            }
        }
    }
    // Lane (q, j) has rows 4 q + i and ranks 4 j + t: turned into one piece of four ranks a row.
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sums[((m * 4 + i) * 4 + w) * kWave + lane] = f32x4{acc[m][0][i], acc[m][1][i], acc[m][2][i], acc[m][3][i]};
    __syncthreads();
    const float scale = p.scaling ? p.scaling[g] : 1.0f;
    for (int o = w; o < MT * 4; o += 4) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) v += sums[(o * 4 + k) * kWave + lane];
        const int row = o / 4 * 16 + 4 * q + o % 4, in_chunk = listed(list, row);
        if (row >= count || r >= p.rank) continue;
        const int64_t to = (chunk * 64 + in_chunk) * p.rank + r;
        if (p.splits > 1)
            st<f32x4>(p.partial + split * p.rows * p.rank + to, v);
        else
            st<f32x4>(p.low + to, v * scale);
    }
    __syncthreads();
}

// Grid: chunks of 64 rows x slots x runs of 64 ranks x parts of the contraction. Of a
// chunk's adapters, in the order of their first rows, slot s takes each slots-th.
template <bool GRAD, bool XF32, bool WF32>
__global__ __launch_bounds__(kBlockThreads) void adapter_down_kernel(AdaptArgs p) {
    __shared__ f32x4 sums[4 * 4 * 4 * kWave];
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
    auto div = [](uint32_t &a, uint32_t b) {  // a mod b, and a becomes a / b
        const uint32_t d = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(a / b)), m = a - d * b;
        a = d;
        return m;
    };
    uint32_t id = blockIdx.x;
    const int slot = static_cast<int>(div(id, static_cast<uint32_t>(p.slots)));
    const int64_t rank0 = 64 * static_cast<int64_t>(div(id, static_cast<uint32_t>(p.ranks)));
    const int split = static_cast<int>(div(id, static_cast<uint32_t>(p.splits)));
    const int64_t chunk = id, row = chunk * 64 + lane;
    int mine;
    const bool has = has_adapter(p, row, mine);
    if (slot == 0 && w == 0 && row < p.rows && !has) {
        float *to = (p.splits > 1 ? p.partial + split * p.rows * p.rank : p.low) + row * p.rank;
        for (int r = static_cast<int>(rank0); r < min(static_cast<int>(rank0) + 64, p.rank); r += 4)
            st<f32x4>(to + r, f32x4{0, 0, 0, 0});
    }
    uint64_t pending = __ballot(has);
    for (int n = 0; pending != 0; ++n) {
        const int g = __builtin_amdgcn_readlane(mine, __builtin_ctzll(pending));
        const uint64_t match = __ballot(has && mine == g);
        pending &= ~match;
        if (n % static_cast<int>(p.slots) != slot) continue;
        const int count = __popcll(match), list = list_bits(match);
        if (count <= 16)
            down_rows<GRAD, XF32, WF32, 1>(p, chunk, rank0, split, g, count, list, sums);
        else if (count <= 32)
            down_rows<GRAD, XF32, WF32, 2>(p, chunk, rank0, split, g, count, list, sums);
        else
            down_rows<GRAD, XF32, WF32, 4>(p, chunk, rank0, split, g, count, list, sums);
    }
}

// low = s_g times the parts' sum, in order; 4 ranks a thread.
__global__ __launch_bounds__(kBlockThreads) void adapter_join_kernel(AdaptArgs p) {
    const int64_t n = p.rows * p.rank / 4, walk = static_cast<int64_t>(gridDim.x) * kBlockThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlockThreads + threadIdx.x; i < n; i += walk) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll 8
        for (int s = 0; s < p.splits; ++s) v += ld<f32x4>(p.partial + (s * n + i) * 4);
        int id;
        const bool has = has_adapter(p, i * 4 / p.rank, id);
        st<f32x4>(p.low + i * 4, has && p.scaling ? v * p.scaling[id] : v);
    }
}

// How a call's low is shared out: about 768 workgroups of 4 waves, with 4 steps of 64
// or more each; in few rows a chunk's adapters have workgroups of their own.
struct DownPlan {
    int64_t rows;  // of one launch
    int64_t slots, ranks, splits, split_steps;
};

DownPlan down_plan(int64_t rows, int64_t len, int64_t adapters, int64_t rank) {
    DownPlan d{};
    d.rows = std::min<int64_t>(rows, INT64_C(1) << 20);
    const int64_t chunks = ceil_div(d.rows, 64), steps = ceil_div(len, 64);
    d.ranks = ceil_div(rank, 64);
    d.slots = std::max<int64_t>(std::min({adapters, d.rows, 64 / chunks}), 1);
    const int64_t most = std::max<int64_t>(768 / (chunks * d.ranks * d.slots), 1);
    d.split_steps = std::max<int64_t>(ceil_div(ceil_div(steps, most), 4) * 4, 4);
    d.splits = ceil_div(steps, d.split_steps);
    return d;
}

template <bool GRAD>
hipError_t launch_down(AdaptArgs p, bool x_f32, bool w_f32, hipStream_t stream) {
    const DownPlan d = down_plan(p.rows, p.len, p.adapters, p.rank);
    p.slots = d.slots, p.ranks = d.ranks, p.splits = static_cast<int>(d.splits), p.split_steps = d.split_steps;
    const int64_t rows = p.rows;
    const void *x = p.x;
    const int32_t *ids = p.ids;
    float *low = p.low;
    for (int64_t r0 = 0; r0 < rows; r0 += d.rows) {
        p.rows = std::min(rows - r0, d.rows);
        p.x = static_cast<const uint8_t *>(x) + r0 * p.x_stride * (x_f32 ? 4 : 2);
        p.ids = ids ? ids + r0 : nullptr;
        p.low = low + r0 * p.rank;
        const unsigned grid = static_cast<unsigned>(ceil_div(p.rows, 64) * d.slots * d.ranks * d.splits);
        if (x_f32) {
            if (w_f32)
                adapter_down_kernel<GRAD, true, true><<<grid, kBlockThreads, 0, stream>>>(p);
            else
                adapter_down_kernel<GRAD, true, false><<<grid, kBlockThreads, 0, stream>>>(p);
        } else {
            if (w_f32)
                adapter_down_kernel<GRAD, false, true><<<grid, kBlockThreads, 0, stream>>>(p);
            else
                adapter_down_kernel<GRAD, false, false><<<grid, kBlockThreads, 0, stream>>>(p);
        }
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        if (d.splits == 1) continue;
        const int64_t joins = std::min<int64_t>(ceil_div(p.rows * p.rank / 4, kBlockThreads), 1 << 14);
        adapter_join_kernel<<<static_cast<unsigned>(joins), kBlockThreads, 0, stream>>>(p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---- the adapters' gradients --------------------------------------------------------

constexpr int kRowWaves = 8;  // of a workgroup, on the same columns

struct RowsArgs {
    const void *x;       // rows of len elements: x (dA) or dy (dB)
    int64_t x_stride, len;
    const float *low;    // [rows][rank]
    void *out;           // [adapters][rank][len] (dA), [adapters][len][rank] (dB)
    float *partial;
    int64_t tiles;       // of 64 columns; 0: not wanted
};

struct RowsCall {
    RowsArgs of[2];      // dA, dB
    const int32_t *ids;
    int64_t rows;
    int adapters, rank, first;  // first: adapter of this launch
    int splits;
    int64_t split_chunks, ranks;
    int out_f32;
};

// Four neighbouring elements from e on, `left` of them in the row, zeros past it.
template <bool F32>
__device__ __forceinline__ void load4(const void *base, int64_t e, int64_t left, uint32_t (&v)[F32 ? 4 : 2]) {
    if constexpr (F32) {
        const uint32_t *from = static_cast<const uint32_t *>(base) + e;
        if (left >= 4) {
            const u32x4 u = *reinterpret_cast<const u32x4_at4 *>(from);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = u[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i < left ? from[i] : 0u;
        }
    } else {
        const uint16_t *from = static_cast<const uint16_t *>(base) + e;
        if (left >= 4) {
            const u32x2 u = *reinterpret_cast<const u32x2_any *>(from);
            v[0] = u[0], v[1] = u[1];
        } else {
            v[0] = (0 < left ? from[0] : 0u) | (1 < left ? static_cast<uint32_t>(from[1]) << 16 : 0u);
            v[1] = 2 < left ? from[2] : 0u;
        }
    }
}

// One adapter's sums over its rows, 64 ranks x 64 columns a workgroup: the waves
// take chunks of 64 rows in turn. A lane loads, of the 8 rows that are its quarter's
// share of 32, four neighbouring ranks of low and four neighbouring columns of x,
// and turns them: tile t has the lane's rank or column t. The waves' sums meet in LDS.
template <bool F32, int PC>
__global__ __launch_bounds__(kRowWaves *kWave) void adapter_rows_kernel(RowsCall p) {
    constexpr int PX = F32 ? 3 : 1;
    __shared__ f32x4 sums[kRowWaves / 2][16][kWave];
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block(), q = lane >> 4, j = lane & 15;
    auto div = [](uint32_t &a, uint32_t b) {
        const uint32_t d = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(a / b)), m = a - d * b;
        a = d;
        return m;
    };
    uint32_t id = static_cast<uint32_t>(xcd_block(blockIdx.x, gridDim.x));
    const int64_t tiles = p.of[0].tiles + p.of[1].tiles;
    int64_t tile = div(id, static_cast<uint32_t>(tiles));
    const int64_t rank0 = 64 * static_cast<int64_t>(div(id, static_cast<uint32_t>(p.ranks)));
    const int split = static_cast<int>(div(id, static_cast<uint32_t>(p.splits)));
    const int g = p.first + static_cast<int>(id);
    const bool second = tile >= p.of[0].tiles;
    if (second) tile -= p.of[0].tiles;
    const RowsArgs &o = p.of[second ? 1 : 0];
    const int64_t col = tile * 64 + 4 * j;
    const int r = static_cast<int>(rank0) + 4 * j;

    f32x4 acc[4][4];  // [tile of ranks][tile of columns]
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[a][t] = f32x4{0, 0, 0, 0};

    const int64_t c0 = split * p.split_chunks, c1 = min(c0 + p.split_chunks, (p.rows + 63) / 64);
    for (int64_t c = c0 + w; c < c1; c += kRowWaves) {
        const int64_t row = c * 64 + lane;
        const bool in = row < p.rows;
        const int mine = p.ids ? p.ids[in ? row : 0] : 0;
        const uint64_t match = __ballot(in && mine == g);
        if (match == 0) continue;
        const int count = __popcll(match), list = list_bits(match);
        for (int n = 0; n < count; n += 32) {
            f32x4 low[8];
            uint32_t x[8][F32 ? 4 : 2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = n + 8 * q + i;
                const int64_t m = c * 64 + listed(list, min(at, count - 1));
                low[i] = ld<f32x4>(o.low + m * p.rank + min(r, p.rank - 4));
                load4<F32>(o.x, m * o.x_stride + min(col, o.len), o.len - col, x[i]);
                if (at >= count) {  // zeros on both sides: a row past the last is in no sum, whatever it holds
                    low[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < (F32 ? 4 : 2); ++e) x[i][e] = 0;
                }
            }
            u32x4 a[4][PC], b[4][PX];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float v[8] = {low[0][t], low[1][t], low[2][t], low[3][t], low[4][t], low[5][t], low[6][t], low[7][t]};
                operand_of<PC>(v, a[t]);
                if constexpr (F32) {
                    const float u[8] = {as_f(x[0][t]), as_f(x[1][t]), as_f(x[2][t]), as_f(x[3][t]),
                                        as_f(x[4][t]), as_f(x[5][t]), as_f(x[6][t]), as_f(x[7][t])};
                    operand_of<PX>(u, b[t]);
                } else {
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        b[t][0][d] = __builtin_amdgcn_perm(x[2 * d + 1][t / 2], x[2 * d][t / 2],
                                                           t % 2 == 0 ? 0x05040100u : 0x07060302u);
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[s][t] = mfma_parts<PC, PX>(a[s], b[t], acc[s][t]);
        }
    }

    // The upper half of the waves hand their sums to the lower half, until wave 0 has them all.
#pragma unroll
    for (int half = kRowWaves / 2; half > 0; half /= 2) {
        __syncthreads();
        if (w >= half && w < 2 * half) {
#pragma unroll
            for (int s = 0; s < 16; ++s) sums[w - half][s][lane] = acc[s / 4][s % 4];
        }
        __syncthreads();
        if (w < half) {
#pragma unroll
            for (int s = 0; s < 16; ++s) acc[s / 4][s % 4] += sums[w][s][lane];
        }
    }
    if (w != 0) return;
    // Lane (q, j) has ranks rank0 + 16 q + 4 i + s and columns col + t.
    const int64_t all = static_cast<int64_t>(p.rank) * o.len, base = g * all;
    float *part = p.splits > 1 ? o.partial + split * p.adapters * all : nullptr;
    auto store = [&](int64_t at, const f32x4 &v, int64_t left) {
        if (part || p.out_f32) {
            float *to = (part ? part : static_cast<float *>(o.out)) + at;
            if (left >= 4) {
                typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
                *reinterpret_cast<f32x4_at4 *>(to) = v;
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < left) to[t] = v[t];
            }
        } else {
            uint16_t *to = static_cast<uint16_t *>(o.out) + at;
            const uint32_t lo = pack_rn(v[0], v[1]), hi = pack_rn(v[2], v[3]);
            if (left >= 4) {
                *reinterpret_cast<u32x2_any *>(to) = u32x2{lo, hi};
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < left) to[t] = static_cast<uint16_t>((t < 2 ? lo : hi) >> (16 * (t & 1)));
            }
        }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rr = static_cast<int>(rank0) + 16 * q + 4 * i;
        if (rr >= p.rank) continue;
        if (!second) {  // [rank][len]
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (col < o.len)
                    store(base + (rr + s) * o.len + col, f32x4{acc[s][0][i], acc[s][1][i], acc[s][2][i], acc[s][3][i]},
                          o.len - col);
        } else {  // [len][rank]
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (col + t < o.len)
                    store(base + (col + t) * p.rank + rr, f32x4{acc[0][t][i], acc[1][t][i], acc[2][t][i], acc[3][t][i]}, 4);
        }
    }
}

// The parts' sum, in order, 4 elements a thread.
__global__ __launch_bounds__(kBlockThreads) void adapter_rows_join_kernel(const float *__restrict__ partial, int splits,
                                                                          int64_t n, void *out, int out_f32) {
    const int64_t walk = static_cast<int64_t>(gridDim.x) * kBlockThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlockThreads + threadIdx.x; i < n / 4; i += walk) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll 8
        for (int s = 0; s < splits; ++s) v += ld<f32x4>(partial + s * n + i * 4);
        if (out_f32)
            st<f32x4>(static_cast<float *>(out) + i * 4, v);
        else
            st<u32x2>(static_cast<uint16_t *>(out) + i * 4, u32x2{pack_rn(v[0], v[1]), pack_rn(v[2], v[3])});
    }
}

// Parts of the rows: as many as give 256 workgroups, of 8 chunks of 64 rows or more.
int64_t rows_splits(int64_t rows, int64_t tiles, int64_t adapters, int64_t rank) {
    const int64_t chunks = ceil_div(rows, 64), others = tiles * adapters * ceil_div(rank, 64);
    const int64_t want = std::max<int64_t>(256 / std::max<int64_t>(others, 1), 1);
    const int64_t each = std::max<int64_t>(ceil_div(ceil_div(chunks, want), kRowWaves) * kRowWaves, kRowWaves);
    return std::max<int64_t>(ceil_div(chunks, each), 1);
}

int64_t align16(int64_t bytes) { return (bytes + 15) & ~INT64_C(15); }

int64_t down_workspace(int64_t rows, int64_t len, int64_t adapters, int64_t rank) {
    const DownPlan d = down_plan(rows, len, adapters, rank);
    return d.splits > 1 ? d.splits * d.rows * rank * 4 : 0;
}

hipError_t launch_down_any(bool grad, const void *x, bool x_f32, int64_t x_stride, int64_t rows, int64_t len,
                           const void *w, const LinAdapters &ad, float *low, void *workspace, hipStream_t stream) {
    AdaptArgs p{};
    p.x = x, p.x_stride = x_stride, p.rows = rows, p.len = len;
    p.w = w, p.ids = ad.ids, p.scaling = ad.scaling;
    p.adapters = static_cast<int>(ad.adapters), p.rank = static_cast<int>(ad.rank);
    p.low = low, p.partial = static_cast<float *>(workspace);
    return grad ? launch_down<true>(p, x_f32, ad.f32, stream) : launch_down<false>(p, x_f32, ad.f32, stream);
}

int64_t rows_workspace(int64_t rows, int64_t n_out, int64_t n_in, int64_t adapters, int64_t rank) {
    const int64_t splits = rows_splits(rows, ceil_div(n_in, 64) + ceil_div(n_out, 64), adapters, rank);
    return splits > 1 ? align16(splits * adapters * rank * n_in * 4) + align16(splits * adapters * rank * n_out * 4) : 0;
}

hipError_t launch_adapter_rows(const void *x, int64_t x_stride, const float *up, void *da, const void *dy,
                               int64_t dy_stride, const float *reduced, void *db, bool f32, bool w_f32, int64_t rows,
                               int64_t n_out, int64_t n_in, int64_t adapters, int64_t rank, const int32_t *ids,
                               void *workspace, hipStream_t stream) {
    RowsCall p{};
    // planned for both, so that each comes out the same without the other
    const int64_t tiles = ceil_div(n_in, 64) + ceil_div(n_out, 64);
    p.splits = static_cast<int>(rows_splits(rows, tiles, adapters, rank));
    p.split_chunks = ceil_div(ceil_div(rows, 64), p.splits);
    float *second = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                              align16(p.splits * adapters * rank * n_in * 4));
    p.of[0] = RowsArgs{x, x_stride, n_in, up, da, static_cast<float *>(workspace), da ? ceil_div(n_in, 64) : 0};
    p.of[1] = RowsArgs{dy, dy_stride, n_out, reduced, db, second, db ? ceil_div(n_out, 64) : 0};
    p.ids = ids, p.rows = rows, p.adapters = static_cast<int>(adapters), p.rank = static_cast<int>(rank);
    p.ranks = ceil_div(rank, 64), p.out_f32 = w_f32;
    const int64_t each = (p.of[0].tiles + p.of[1].tiles) * p.ranks * p.splits;
    const int64_t at_once = std::max<int64_t>(kMaxGroups / each, 1);
    for (int64_t g0 = 0; g0 < adapters; g0 += at_once) {
        p.first = static_cast<int>(g0);
        const unsigned grid = static_cast<unsigned>(each * std::min(adapters - g0, at_once));
        if (f32)
            adapter_rows_kernel<true, 3><<<grid, kRowWaves * kWave, 0, stream>>>(p);
        else if (w_f32)
            adapter_rows_kernel<false, 3><<<grid, kRowWaves * kWave, 0, stream>>>(p);
        else
            adapter_rows_kernel<false, 2><<<grid, kRowWaves * kWave, 0, stream>>>(p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (p.splits == 1) return hipSuccess;
    for (const RowsArgs &o : p.of) {
        if (o.tiles == 0) continue;
        const int64_t n = adapters * rank * o.len;
        const int64_t joins = std::min<int64_t>(ceil_div(n / 4, kBlockThreads), 1 << 14);
        adapter_rows_join_kernel<<<static_cast<unsigned>(joins), kBlockThreads, 0, stream>>>(o.partial, p.splits, n,
                                                                                            o.out, w_f32);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t linear_adapters_workspace(bool grad, bool in_f32, int64_t lda, bool out_f32, int64_t rows, int64_t n_out,
                                  int64_t n_in, int64_t adapters, int64_t rank) {
    int64_t most = 0;
    if (rows > 0)
        most = std::max(linear_workspace(grad, in_f32, lda, out_f32, rows, 0, n_out, n_in),
                        down_workspace(rows, grad ? n_out : n_in, adapters, rank));
    if (!grad) return align16(most);
    // low of the backward pass, then what one step after the other uses
    return align16(rows * rank * 4) + align16(std::max(most, rows_workspace(rows, n_out, n_in, adapters, rank)));
}

hipError_t launch_linear_adapters(const void *x, bool in_f32, int64_t x_stride, int64_t rows, const void *codes,
                                  const float *scales, int bits, int64_t n_out, int64_t n_in, int log2b,
                                  const LinAdapters &ad, float *reduced, void *y, bool out_f32, int64_t y_stride,
                                  void *workspace, hipStream_t stream) {
    if (const hipError_t e = launch_down_any(false, x, in_f32, x_stride, rows, n_in, ad.a, ad, reduced, workspace, stream);
        e != hipSuccess)
        return e;
    return launch_linear(false, x, in_f32, x_stride, rows, nullptr, 0, codes, scales, bits, n_out, n_in, log2b, y, out_f32,
                         y_stride, workspace, stream, &ad, reduced);
}

hipError_t launch_linear_adapters_grad(const void *dy, bool in_f32, int64_t dy_stride, const void *x, int64_t x_stride,
                                       const float *reduced, int64_t rows, const void *codes, const float *scales,
                                       int bits, int64_t n_out, int64_t n_in, int log2b, const LinAdapters &ad,
                                       void *dx, bool out_f32, int64_t dx_stride, void *da, void *db, void *workspace,
                                       hipStream_t stream) {
    float *low = static_cast<float *>(workspace);
    void *rest = static_cast<uint8_t *>(workspace) + align16(rows * ad.rank * 4);
    if (rows > 0) {
        hipError_t e = launch_down_any(true, dy, in_f32, dy_stride, rows, n_out, ad.b, ad, low, rest, stream);
        if (e != hipSuccess) return e;
        e = launch_linear(true, dy, in_f32, dy_stride, rows, nullptr, 0, codes, scales, bits, n_out, n_in, log2b, dx,
                          out_f32, dx_stride, rest, stream, &ad, low);
        if (e != hipSuccess) return e;
    }
    if (!da && !db) return hipSuccess;
    return launch_adapter_rows(x, x_stride, low, da, dy, dy_stride, reduced, db, in_f32, ad.f32, rows, n_out, n_in,
                               ad.adapters, ad.rank, ad.ids, rest, stream);
}

}  // namespace zpp
