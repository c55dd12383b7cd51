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
// parts (low, in the sums of bf16 rows for bf16 adapters, as two, off by 2^-16: linear_adapt.h).
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

// What a lane loads of a step of 64 contraction indices, of which it has k .. k + 15:
// of the rows of MT tiles, and of four ranks (forward: their 16 elements each;
// backward: four neighbouring ranks of 16 rows, to be turned).
template <bool GRAD, bool XF32, bool WF32, int MT>
struct Step {
    static constexpr int kX = XF32 ? 4 : 2, kW = (WF32 ? 2 : 1) * 2;
    u32x4 x[MT][kX];
    u32x4 w[4][kW];

    // 16 elements of a row from `base` on, of which the first `left` are in it.
    template <bool F32, bool WHOLE, class Off>
    static __device__ __forceinline__ void load16(const void *base, Off e, int64_t left, u32x4 *v) {
        if constexpr (F32) {
            const uint32_t *from = static_cast<const uint32_t *>(base) + e;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (WHOLE) {
                    v[i] = *reinterpret_cast<const u32x4_at4 *>(from + 4 * i);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[i][c] = 4 * i + c < left ? from[4 * i + c] : 0u;
                }
            }
        } else {
            const uint16_t *from = static_cast<const uint16_t *>(base) + e;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (WHOLE) {
                    v[h] = *reinterpret_cast<const u32x4_any *>(from + 8 * h);
                } else {
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int i = 8 * h + 2 * d;
                        v[h][d] = (i < left ? from[i] : 0u) | (i + 1 < left ? static_cast<uint32_t>(from[i + 1]) << 16 : 0u);
                    }
                }
            }
        }
    }

    // Step s of 64 indices; WHOLE: all of them are below len. x and w are those of the
    // chunk's first row and of the adapter; a lane adds its offsets (Off: 32 bits where
    // they suffice) to what is the same in all lanes.
    template <bool WHOLE, class Off>
    __device__ __forceinline__ void load(const AdaptArgs &p, const uint8_t *rows, const uint8_t *adapter,
                                         const Off (&at)[MT], int r, int64_t s) {
        const int k = 16 * static_cast<int>(threadIdx.x >> 4 & 3);  // the lane's first index of the step's
        const int64_t left = p.len - s * 64 - k;
        if constexpr (!GRAD) {
            const uint8_t *from = adapter + s * 64 * (WF32 ? 4 : 2);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                load16<WF32, WHOLE>(from, static_cast<Off>(min(r + t, p.rank - 1)) * static_cast<Off>(p.len) + k, left, w[t]);
        } else {
            const uint8_t *from = adapter + s * 64 * p.rank * (WF32 ? 4 : 2);
            const uint32_t rr = static_cast<uint32_t>(min(r, p.rank - 4)), rank = static_cast<uint32_t>(p.rank);
            const uint32_t first = k * rank + rr;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool in = WHOLE || i < left;  // zeros past the end, whatever stands there
                // the last one again past the end (of len, so not before this step's first)
                const int64_t last = p.len - 1 - s * 64;
                const uint32_t e = WHOLE ? first : static_cast<uint32_t>(min(static_cast<int64_t>(k + i), last)) * rank + rr;
                const uint8_t *row = from + (WHOLE ? i * rank * (WF32 ? 4u : 2u) : 0u);
                if constexpr (WF32) {
                    const u32x4 v = ld<u32x4>(reinterpret_cast<const float *>(row) + e);
                    w16(i) = in ? v : u32x4{0, 0, 0, 0};
                } else {
                    const u32x2 v = ld<u32x2>(reinterpret_cast<const uint16_t *>(row) + e);
                    w[i / 4][i % 4 / 2][i % 2 * 2] = in ? v[0] : 0u;
                    w[i / 4][i % 4 / 2][i % 2 * 2 + 1] = in ? v[1] : 0u;
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) load16<XF32, WHOLE>(rows + s * 64 * (XF32 ? 4 : 2), at[m] + k, left, x[m]);
    }

    __device__ __forceinline__ u32x4 &w16(int i) { return w[i / 4][i % 4]; }

    // Half H of 16 elements as an operand's parts.
    template <bool F32, int H>
    static __device__ __forceinline__ void half(const u32x4 *v, u32x4 (&o)[F32 ? 3 : 1]) {
        if constexpr (F32) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = as_f(v[2 * H + i / 4][i % 4]);
            operand_of<3>(f, o);
        } else {
            o[0] = v[H];
        }
    }

    // Tile t of ranks, half H of the indices.
    template <int H>
    __device__ __forceinline__ void rank_tile(int t, u32x4 (&o)[WF32 ? 3 : 1]) const {
        if constexpr (!GRAD) {
            half<WF32, H>(w[t], o);
        } else if constexpr (WF32) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = as_f(w[(8 * H + i) / 4][i % 4][t]);
            operand_of<3>(f, o);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                // rows 8 H + 2 d and the next: elements t of two pairs of dwords
                const int i = 8 * H + 2 * d;
                const u32x4 &v = w[i / 4][i % 4 / 2];
                o[0][d] = __builtin_amdgcn_perm(v[2 + t / 2], v[t / 2], t % 2 == 0 ? 0x05040100u : 0x07060302u);
            }
        }
    }

    template <int H>
    __device__ __forceinline__ void use_half(f32x4 (&acc)[MT][4]) const {
        constexpr int PX = XF32 ? 3 : 1, PW = WF32 ? 3 : 1;
        u32x4 b[4][PW];
#pragma unroll
        for (int t = 0; t < 4; ++t) rank_tile<H>(t, b[t]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            u32x4 a[PX];
            half<XF32, H>(x[m], a);
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[m][t] = mfma_parts<PX, PW>(a, b[t], acc[m][t]);
        }
    }

    __device__ __forceinline__ void use(f32x4 (&acc)[MT][4]) const {
        use_half<0>(acc);
        use_half<1>(acc);
    }
};

// One adapter's rows of a chunk (16 MT of them at most) by 64 of its ranks: the
// workgroup's 4 waves take steps of 64 indices in turn, the next one's loads under
// way, and join their sums in LDS.
template <bool GRAD, bool XF32, bool WF32, int MT, class Off>
__device__ __forceinline__ void down_rows(const AdaptArgs &p, int64_t chunk, int64_t rank0, int split, int g, int count,
                                          int list, f32x4 *sums) {
    using S = Step<GRAD, XF32, WF32, MT>;
    constexpr bool AHEAD = !XF32 && !WF32;  // binary32 steps fill the registers
    const int lane = threadIdx.x & (kWave - 1), w = wave_in_block(), q = lane >> 4, j = lane & 15;
    const int r = static_cast<int>(rank0) + 4 * j;
    const float scale = p.scaling && p.splits == 1 ? p.scaling[g] : 1.0f;
    const uint8_t *rows = static_cast<const uint8_t *>(p.x) + chunk * 64 * p.x_stride * (XF32 ? 4 : 2);
    const uint8_t *adapter = static_cast<const uint8_t *>(p.w) + static_cast<int64_t>(g) * p.rank * p.len * (WF32 ? 4 : 2);
    Off at[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) at[m] = static_cast<Off>(listed(list, min(16 * m + j, count - 1))) * static_cast<Off>(p.x_stride);
    f32x4 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
    const int64_t s0 = split * p.split_steps + w, s1 = min((split + 1) * p.split_steps, p.len / 64);
    if constexpr (AHEAD && !GRAD) {  // less code, which is fetched anew in every launch, than in turn
        S now, next;
        if (s0 < s1) now.template load<true>(p, rows, adapter, at, r, s0);
        for (int64_t s = s0; s < s1; s += 4) {
            if (s + 4 < s1) next.template load<true>(p, rows, adapter, at, r, s + 4);
            now.use(acc);
            now = next;
        }
    } else if constexpr (AHEAD) {
        S a, b;
        if (s0 < s1) a.template load<true>(p, rows, adapter, at, r, s0);
        for (int64_t s = s0; s < s1; s += 8) {
            if (s + 4 < s1) b.template load<true>(p, rows, adapter, at, r, s + 4);
            a.use(acc);
            if (s + 4 >= s1) break;
            if (s + 8 < s1) a.template load<true>(p, rows, adapter, at, r, s + 8);
            b.use(acc);
        }
    } else {
        for (int64_t s = s0; s < s1; s += 4) {
            S a;
            a.template load<true>(p, rows, adapter, at, r, s);
            a.use(acc);
        }
    }
    // what is left, less than 64 indices, is the last part's, and the wave's whose turn it is
    if (const int64_t s = p.len / 64; p.len % 64 != 0 && s / p.split_steps == split && s % 4 == w) {
        S last;
        last.template load<false>(p, rows, adapter, at, r, s);
        last.use(acc);
    }
    // Lane (q, j) has rows 4 q + i and ranks 4 j + t: turned into one piece of four ranks a row.
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sums[((m * 4 + i) * 4 + w) * kWave + lane] = f32x4{acc[m][0][i], acc[m][1][i], acc[m][2][i], acc[m][3][i]};
    __syncthreads();
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
//
// Latency bounds it: a wave's steps are few (4 to 8 of 64 indices), each a trip to
// memory for 16 to 32 matrix instructions. 4096 rows of 8192 with one bf16 adapter of rank
// 64: 25 us (67 MB, 2.7 TB/s) and 4 for the join; 48 rows with 32 such adapters: 16 us.
template <bool GRAD, bool XF32, bool WF32>
__global__ __launch_bounds__(kBlockThreads, XF32 || WF32 ? 1 : 2) void adapter_down_kernel(AdaptArgs p) {
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
        auto go = [&](auto off) {
            using Off = decltype(off);
            if (count <= 16)
                down_rows<GRAD, XF32, WF32, 1, Off>(p, chunk, rank0, split, g, count, list, sums);
            else if (count <= 32)
                down_rows<GRAD, XF32, WF32, 2, Off>(p, chunk, rank0, split, g, count, list, sums);
            else
                down_rows<GRAD, XF32, WF32, 4, Off>(p, chunk, rank0, split, g, count, list, sums);
        };
        // in elements, and four bytes each: 64 rows of x, and an adapter's
        if (GRAD && p.x_stride < (1 << 24) && p.rank * p.len < (1 << 30))
            go(uint32_t{});
        else
            go(int64_t{});
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

// How a call's low is shared out: up to 512 workgroups of 4 waves (two a CU), with 4 steps
// of 64 or more each; in few rows a chunk's adapters have workgroups of their own.
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
    const int64_t most = std::max<int64_t>(512 / (chunks * d.ranks * d.slots), 1);
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

constexpr int kRowWaves = 8;    // of a workgroup, on the same columns
constexpr int kAloneWaves = 4;  // each on its own

struct RowsArgs {
    const void *x;       // rows of len elements: x (dA) or dy (dB)
    int64_t x_stride, len;
    const float *low;    // [rows][rank]
    void *out;           // [adapters][rank][len] (dA), [adapters][len][rank] (dB)
    float *partial;
    int64_t tiles;       // of 64 columns (4 of them, ALONE); 0: not wanted
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

// 32 of an adapter's rows: which they are, and what a lane loads of the 8 that are its
// quarter's, four neighbouring columns of x and four neighbouring ranks of low.
template <bool F32>
struct RowsOfX {
    static constexpr int kX = F32 ? 4 : 2;
    int64_t row0;        // of their chunk
    int list, n, count;  // rows row0 + list[n] .. of `count` that the chunk has
    uint32_t x[8][kX];

    // The lane's first row; and its i-th, i rows on where the chunk has all of its rows.
    __device__ __forceinline__ uint32_t first() const { return n + 8 * (threadIdx.x >> 4 & 3); }
    __device__ __forceinline__ uint32_t row(int i) const {
        return static_cast<uint32_t>(listed(list, min(static_cast<int>(first()) + i, count - 1)));
    }

    // FAST: the columns are all in the row, and 64 rows' offsets fit 32 bits.
    template <bool FAST>
    __device__ __forceinline__ void load(const RowsArgs &o, int64_t col) {
        const uint8_t *rows = static_cast<const uint8_t *>(o.x) + row0 * o.x_stride * (F32 ? 4 : 2);
        const uint32_t stride = static_cast<uint32_t>(o.x_stride) * (F32 ? 4 : 2);
        const uint32_t at_col = static_cast<uint32_t>(col) * (F32 ? 4 : 2);
        auto piece = [&](int i, const uint8_t *from, uint32_t at) {
            if constexpr (F32) {
                const u32x4 v = *reinterpret_cast<const u32x4_at4 *>(from + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = v[e];
            } else {
                const u32x2 v = *reinterpret_cast<const u32x2_any *>(from + at);
                x[i][0] = v[0], x[i][1] = v[1];
            }
        };
        if (FAST && count == 64) {
            const uint32_t at = first() * stride + at_col;
#pragma unroll
            for (int i = 0; i < 8; ++i) piece(i, rows + i * static_cast<uint64_t>(stride), at);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (FAST)
                    piece(i, rows, row(i) * stride + at_col);
                else
                    load4<F32>(rows, row(i) * o.x_stride + min(col, o.len), o.len - col, x[i]);
            }
        }
    }

    __device__ __forceinline__ void load_low(const RowsArgs &o, int rank, int r, f32x4 (&low)[8]) const {
        const float *lows = o.low + row0 * rank;
        const uint32_t at = static_cast<uint32_t>(min(r, rank - 4)), stride = static_cast<uint32_t>(rank);
        if (count == 64) {
            const uint32_t from = first() * stride + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) low[i] = ld<f32x4>(lows + i * stride + from);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) low[i] = ld<f32x4>(lows + (row(i) * stride + at));
        }
    }

    // Turned: tile t has the lane's rank or column t.
    template <int PC>
    __device__ __forceinline__ void use(f32x4 (&low)[8], f32x4 (&acc)[4][4]) {
        constexpr int PX = F32 ? 3 : 1;
        if (n + 32 > count) {  // zeros past the last, on both sides: such a row is in no sum, whatever it holds
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = n + 8 * static_cast<int>(threadIdx.x >> 4 & 3) + i < count;
#pragma unroll
                for (int e = 0; e < 4; ++e) low[i][e] = in ? low[i][e] : 0.0f;
#pragma unroll
                for (int e = 0; e < kX; ++e) x[i][e] = in ? x[i][e] : 0u;
            }
        }
        u32x4 b[4][PX];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if constexpr (F32) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = as_f(x[i][t]);
                operand_of<PX>(f, b[t]);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    b[t][0][d] = __builtin_amdgcn_perm(x[2 * d + 1][t / 2], x[2 * d][t / 2],
                                                       t % 2 == 0 ? 0x05040100u : 0x07060302u);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float f[8];
            u32x4 a[PC];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = low[i][s];
            operand_of<PC>(f, a);
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[s][t] = mfma_parts<PC, PX>(a, b[t], acc[s][t]);
        }
    }
};

// The sums of one wave over chunks c, c + step, ... below c1. The next 32 rows' loads are under
// way while these are multiplied (AHEAD: two sets of binary32 rows do not fit, and few rows have
// no next; two steps ahead gained nothing), and the ids of the next chunk.
template <bool F32, int PC, bool FAST, bool AHEAD>
__device__ __forceinline__ void adapter_sums(const RowsCall &p, const RowsArgs &o, int g, int64_t c, int64_t step,
                                             int64_t c1, int r, int64_t col, f32x4 (&acc)[4][4]) {
    using S = RowsOfX<F32>;
    const int lane = threadIdx.x & (kWave - 1);
    auto id_of = [&](int64_t c) {
        const int64_t row = c * 64 + lane;
        if (row >= p.rows) return -1;
        return p.ids ? p.ids[row] : 0;
    };
    int ids = c < c1 ? id_of(c) : -1;
    // The 32 rows of the adapter behind those of `s`, into `to`: false if there are none.
    auto advance = [&](const S &s, S &to, f32x4(&low)[8]) {
        to.row0 = s.row0, to.list = s.list, to.n = s.n + 32, to.count = s.count;
        while (to.n >= to.count) {
            if (c >= c1) return false;
            const uint64_t match = __ballot(ids == g);
            to.row0 = c * 64;
            c += step;
            ids = c < c1 ? id_of(c) : -1;
            to.n = 0;
            to.count = __popcll(match);
            to.list = list_bits(match);
        }
        to.template load<FAST>(o, col);
        to.load_low(o, p.rank, r, low);
        return true;
    };
    S s0, s1;
    f32x4 low0[8], low1[8];
    s0.row0 = 0, s0.list = s0.n = s0.count = 0;
    if constexpr (!AHEAD) {
        while (advance(s0, s0, low0)) s0.template use<PC>(low0, acc);
        return;
    }
    if (!advance(s0, s0, low0)) return;
    for (;;) {  // in turn: copied from one to the other, they were a fifth of the instructions
        const bool more1 = advance(s0, s1, low1);
        s0.template use<PC>(low0, acc);
        if (!more1) return;
        const bool more0 = advance(s1, s0, low0);
        s1.template use<PC>(low1, acc);
        if (!more0) return;
    }
}

// One adapter's sums over its rows, 64 ranks x 64 columns a workgroup: the waves
// take chunks of 64 rows in turn, and their sums meet in LDS. ALONE, where there are
// enough sums for a wave each: a wave has all the rows of its own 64 columns, of the 256 of
// a workgroup, and nothing to join. Latency bounds it too: 4096 rows of 8192 and 8192 columns,
// rank 64: 44 us (134 MB, 3.0 TB/s; 32 with x and dy in the caches, 38 without loads of
// low; loads two steps ahead gained nothing). ALONE: 64 rows with 64 adapters of rank 16, 8192 x 8192,
// 52 us in place of 382.
template <bool F32, int PC, bool ALONE>
__global__ __launch_bounds__(ALONE ? kAloneWaves *kWave : kRowWaves *kWave, 2) void adapter_rows_kernel(RowsCall p) {
    [[maybe_unused]] __shared__ f32x4 sums[ALONE ? 1 : kRowWaves / 2][ALONE ? 1 : 16][kWave];
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
    if constexpr (ALONE) {
        tile = tile * kAloneWaves + w;
        if (tile * 64 >= o.len) return;
    }
    const int64_t col = tile * 64 + 4 * j;
    const int r = static_cast<int>(rank0) + 4 * j;

    f32x4 acc[4][4];  // [tile of ranks][tile of columns]
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[a][t] = f32x4{0, 0, 0, 0};

    const int64_t c0 = split * p.split_chunks, c1 = min(c0 + p.split_chunks, (p.rows + 63) / 64);
    if (tile * 64 + 64 <= o.len && o.x_stride < (1 << 22))
        adapter_sums<F32, PC, true, !F32 && !ALONE>(p, o, g, ALONE ? c0 : c0 + w, ALONE ? 1 : kRowWaves, c1, r, col, acc);
    else
        adapter_sums<F32, PC, false, !F32 && !ALONE>(p, o, g, ALONE ? c0 : c0 + w, ALONE ? 1 : kRowWaves, c1, r, col, acc);

    if constexpr (!ALONE) {
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
    }
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

// How a call's sums are shared out: a wave each (alone), or a workgroup each with the rows in parts, as
// many as give 256 workgroups, of 8 chunks of 64 rows or more.
//
// The estimated time decides, in microseconds: rounds of the waves (2048) or workgroups (256) that the GPU
// holds at once, times the chunks that a wave walks, at 0.26 a chunk and 3.3 more if all of its rows are the
// adapter's, and 5 to begin and to join. Alone against shared, bf16, measured: 4096 rows of 8192 and 8192 columns, one
// adapter of rank 64, 214 us against 50, 16 of them 77 against 147, 128 of rank 16 250 against 887; 8192 and 28672
// columns, one of rank 256, 434 against 296 with 4096 rows, 63 against 86 with 512; 192 rows of 8192 and 8192, one of
// rank 64, 16.1 against 12.5, four 11.8 against 33.5. Of 70 such cases the estimate was wrong in two, by 3 and 4%.
struct RowsPlan {
    bool alone;
    int64_t splits;  // parts of the rows
};

RowsPlan rows_plan(int64_t rows, int64_t tiles, int64_t adapters, int64_t rank) {
    const int64_t chunks = ceil_div(rows, 64), sums = tiles * adapters * ceil_div(rank, 64);
    const int64_t want = std::max<int64_t>(256 / sums, 1);
    const int64_t each = std::max<int64_t>(ceil_div(ceil_div(chunks, want), kRowWaves) * kRowWaves, kRowWaves);
    const int64_t splits = std::max<int64_t>(ceil_div(chunks, each), 1);
    const double chunk_us = 0.26 + 3.3 / static_cast<double>(adapters);
    auto time = [&](int64_t rounds, int64_t walked) {
        return static_cast<double>(rounds) * (static_cast<double>(walked) * chunk_us + 5);
    };
    if (time(ceil_div(sums, 2048), chunks) <= time(ceil_div(sums * splits, 256), ceil_div(chunks, kRowWaves * splits)))
        return RowsPlan{true, 1};
    return RowsPlan{false, splits};
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
    const int64_t splits = rows_plan(rows, ceil_div(n_in, 64) + ceil_div(n_out, 64), adapters, rank).splits;
    return splits > 1 ? align16(splits * adapters * rank * n_in * 4) + align16(splits * adapters * rank * n_out * 4) : 0;
}

hipError_t launch_adapter_rows(const void *x, int64_t x_stride, const float *up, void *da, const void *dy,
                               int64_t dy_stride, const float *reduced, void *db, bool f32, bool w_f32, int64_t rows,
                               int64_t n_out, int64_t n_in, int64_t adapters, int64_t rank, const int32_t *ids,
                               void *workspace, hipStream_t stream) {
    RowsCall p{};
    // planned for both, so that each comes out the same without the other
    const RowsPlan plan = rows_plan(rows, ceil_div(n_in, 64) + ceil_div(n_out, 64), adapters, rank);
    p.splits = static_cast<int>(plan.splits);
    p.split_chunks = ceil_div(ceil_div(rows, 64), p.splits);
    float *second = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                              align16(p.splits * adapters * rank * n_in * 4));
    const bool alone = plan.alone;
    const int64_t columns = alone ? 64 * kAloneWaves : 64;
    p.of[0] = RowsArgs{x, x_stride, n_in, up, da, static_cast<float *>(workspace), da ? ceil_div(n_in, columns) : 0};
    p.of[1] = RowsArgs{dy, dy_stride, n_out, reduced, db, second, db ? ceil_div(n_out, columns) : 0};
    p.ids = ids, p.rows = rows, p.adapters = static_cast<int>(adapters), p.rank = static_cast<int>(rank);
    p.ranks = ceil_div(rank, 64), p.out_f32 = w_f32;
    const int64_t each = (p.of[0].tiles + p.of[1].tiles) * p.ranks * p.splits;
    const int64_t at_once = std::max<int64_t>(kMaxGroups / each, 1);
    for (int64_t g0 = 0; g0 < adapters; g0 += at_once) {
        p.first = static_cast<int>(g0);
        const unsigned grid = static_cast<unsigned>(each * std::min(adapters - g0, at_once));
        auto go = [&](auto kernel, auto lonely) {
            (alone ? lonely : kernel)<<<grid, (alone ? kAloneWaves : kRowWaves) * kWave, 0, stream>>>(p);
        };
        if (f32)
            go(adapter_rows_kernel<true, 3, false>, adapter_rows_kernel<true, 3, true>);
        else if (w_f32)
            go(adapter_rows_kernel<false, 3, false>, adapter_rows_kernel<false, 3, true>);
        else
            go(adapter_rows_kernel<false, 2, false>, adapter_rows_kernel<false, 2, true>);
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
        most = std::max(linear_workspace(grad, in_f32, lda, out_f32, rows, 0, n_out, n_in, true),
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
