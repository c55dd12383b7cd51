// zpp_launch.h - internal launchers, one per kernel family. Arguments are
// already validated by the C ABI layer; each returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zpp {

hipError_t launch_quantize(const void *x, bool f32_in, int64_t numel, int log2b, int bits, void *codes,
                           float *scales, hipStream_t stream);

hipError_t launch_quantize_reordered(const void *x, bool f32_in, int64_t slice_elems, int n_nodes, int gpus_per_node,
                                     int first_slice, int n_slices, int log2b, int bits, void *codes, float *scales,
                                     hipStream_t stream);

hipError_t launch_dequantize(const void *codes, const float *scales, int bits, int64_t numel, int log2b,
                             void *y, bool f32_out, hipStream_t stream);

hipError_t launch_reorder(const void *in, void *out, int64_t slice_bytes, int n_nodes, int gpus_per_node,
                          hipStream_t stream);

hipError_t launch_drr(const void *codes_in, int64_t codes_stride, const float *scales_in, int64_t scales_stride,
                      int n_inputs, int bits_in, int64_t numel, int log2b, void *codes_out, float *scales_out,
                      int bits_out, float *sum_out, hipStream_t stream);

hipError_t launch_drr_split(const void *codes_in, int64_t codes_stride, const float *scales_in,
                            int64_t scales_stride, int n_inputs, int bits_in, int64_t numel, int log2b,
                            int64_t keep_begin, int64_t keep_len, void *codes_send, float *scales_send,
                            void *codes_keep, float *scales_keep, int bits_out, hipStream_t stream);

hipError_t launch_drr_average(const void *codes_in, int64_t codes_stride, const float *scales_in,
                              int64_t scales_stride, int n_inputs, int bits_in, int64_t numel, int log2b,
                              int divisor, float *avg_out, hipStream_t stream);

// Low-rank adapters: a [adapters][rank][n_in] and b [adapters][n_out][rank], of binary32 or bf16; ids may be null (the
// first for every row), scaling too (ones).
struct LinAdapters {
    const void *a, *b;
    bool f32;
    int64_t adapters, rank;
    const int32_t *ids;
    const float *scaling;
};

// y = x W^T (grad false: a is x, rows of n_in) or dx = dy W (grad true: a is dy, rows of n_out). With groups > 0,
// rows offsets[e] .. offsets[e + 1] - 1 (device memory) by the e-th of as many matrices. With `ad` (and no groups),
// low times the row's adapter's b (y) or a (dx) is added.
hipError_t launch_linear(bool grad, const void *a, bool in_f32, int64_t lda, int64_t rows, const int32_t *offsets,
                         int64_t groups, const void *codes, const float *scales, int bits, int64_t n_out, int64_t n_in,
                         int log2b, void *out, bool out_f32, int64_t ldo, void *workspace, hipStream_t stream,
                         const LinAdapters *ad = nullptr, const float *low = nullptr);
int64_t linear_workspace(bool grad, bool in_f32, int64_t lda, bool out_f32, int64_t rows, int64_t groups,
                         int64_t n_out, int64_t n_in, bool adapted = false);

// reduced: [rows][rank], s x A^T of each row's adapter. da and db may be null.
hipError_t launch_linear_adapters(const void *x, bool in_f32, int64_t x_stride, int64_t rows, const void *codes,
                                  const float *scales, int bits, int64_t n_out, int64_t n_in, int log2b,
                                  const LinAdapters &ad, float *reduced, void *y, bool out_f32, int64_t y_stride,
                                  void *workspace, hipStream_t stream);
hipError_t launch_linear_adapters_grad(const void *dy, bool in_f32, int64_t dy_stride, const void *x, int64_t x_stride,
                                       const float *reduced, int64_t rows, const void *codes, const float *scales,
                                       int bits, int64_t n_out, int64_t n_in, int log2b, const LinAdapters &ad,
                                       void *dx, bool out_f32, int64_t dx_stride, void *da, void *db, void *workspace,
                                       hipStream_t stream);
int64_t linear_adapters_workspace(bool grad, bool in_f32, int64_t lda, bool out_f32, int64_t rows, int64_t n_out,
                                  int64_t n_in, int64_t adapters, int64_t rank);

hipError_t launch_layer_norm(const void *x, bool f32, int64_t x_stride, int64_t rows, int64_t width,
                             const void *weight, const void *bias, bool w_f32, float eps, void *y, int64_t y_stride,
                             float *mean, float *rstd, hipStream_t stream);
hipError_t launch_layer_norm_grad(const void *dy, int64_t dy_stride, const void *x, bool f32, int64_t x_stride,
                                  int64_t rows, int64_t width, const void *weight, bool w_f32, const float *mean,
                                  const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias,
                                  void *workspace, hipStream_t stream);
int64_t layer_norm_grad_workspace(int64_t rows, int64_t width);

// residual, sum, y and codes may be null (bits 0 without codes).
hipError_t launch_rms_norm(const void *x, bool f32, int64_t x_stride, const void *residual, int64_t residual_stride,
                           int64_t rows, int64_t width, const void *weight, bool w_f32, float eps, void *sum,
                           int64_t sum_stride, void *y, int64_t y_stride, void *codes, float *scales, int bits,
                           int log2b, float *rstd, hipStream_t stream);
hipError_t launch_rms_norm_grad(const void *dy, int64_t dy_stride, const void *h, bool f32, int64_t h_stride,
                                const void *dsum, int64_t dsum_stride, int64_t rows, int64_t width,
                                const void *weight, bool w_f32, const float *rstd, void *dx, int64_t dx_stride,
                                void *dweight, void *workspace, hipStream_t stream);
int64_t rms_norm_grad_workspace(int64_t rows, int64_t width);

}  // namespace zpp
