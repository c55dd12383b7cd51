/*
 * zpp.h - C ABI of the ZeRO++ block-quantization codec on AMD Instinct MI355X
 * (gfx950, CDNA4).
 *
 * The library is the per-GPU arithmetic of ZeRO++'s communication reduction:
 * block quantization of weights before the forward all-gather (qwZ), the
 * gather-side dequantization, and the gradient path of qgZ (tensor-slice
 * reordering, one-shot 4-bit quantization, and the dequantize-reduce-
 * requantize step between the two hops of its hierarchical all-to-all).
 * Next to it stand the operators that use those weights on the GPU that holds
 * their codes: linear products and their input gradient straight from codes
 * and scales, layer norm, RMS norm (with a residual's addition and codes of its
 * result), low-rank adapters beside a product, and products of rows grouped by
 * weight matrix, all forward and backward.
 * It moves no data between GPUs: the caller's collectives do that.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every data pointer is a DEVICE pointer (memory the current GPU can
 *   address: hipMalloc'd on it or on a peer it can access, or
 *   hipHostMalloc'd pinned host memory). Ordinary host memory, and another
 *   GPU's memory without peer access, are rejected with ZPP_ERR_POINTER.
 * - Every call is asynchronous on `stream` (a hipStream_t; NULL means the
 *   null stream). The call validates all arguments on the host first; if any
 *   check fails it returns an error code, launches nothing and leaves every
 *   output untouched. Faults during execution surface at the caller's next
 *   synchronization of the stream, as with any HIP kernel. Right before
 *   its launch a call reads and clears the calling thread's pending HIP
 *   error (hipGetLastError), so an error left there by an earlier call does
 *   not survive it; a rejected launch returns ZPP_ERR_LAUNCH and leaves no
 *   error pending. The hop reductions launch once per 2^29 output elements;
 *   if a later launch is rejected, the earlier ones still run, so after
 *   ZPP_ERR_LAUNCH the outputs are unspecified (likewise of a linear call, or
 *   a norm's backward pass, which may take two launches or more).
 * - The caller allocates and owns every buffer; the library allocates
 *   nothing, keeps no per-call state and may be called from several threads
 *   and streams at once. Outputs must not overlap inputs or each other
 *   (ZPP_ERR_OVERLAP); inputs may overlap each other.
 * - Block quantization layout (structure of arrays): for `numel` elements
 *   and block size B, block b holds elements [b*B, (b+1)*B). `codes` holds
 *   numel*bits/8 bytes: 8-bit codes are two's-complement bytes; 4-bit codes
 *   are two's-complement nibbles, element 2i in the low nibble of byte i.
 *   `scales` holds numel/B binary32 scales s_b (the scale itself, not its
 *   inverse). An element's value is code * s_b.
 * - B is a power of two in [ZPP_MIN_BLOCK, ZPP_MAX_BLOCK]; 0 <= numel <=
 *   ZPP_MAX_NUMEL and numel % B == 0 (callers pad; zero padding changes no
 *   scale and no sum). numel == 0 is a no-op returning ZPP_OK.
 * - Alignment: element data and code pointers 16-byte aligned, scale
 *   pointers 4-byte aligned (ZPP_ERR_ALIGN otherwise).
 *
 * Sources (pages as published, by title and section):
 *   [QWZ] "Quantized LLM Training at Scale with ZeRO++", section "The Three
 *         Pillars of ZeRO++", pillar 1 (QWZ): weights are quantized chunk by
 *         chunk (block quantization) and all-gathered as 8-bit values.
 *   [QGZ] same page and section, pillar 3 (QGZ): one-shot gradient
 *         quantization, two-hop all-to-all (intra-node exchange and
 *         reduction, then inter-node exchange), tensor-slice reordering
 *         before any communication; gradient volume cut to a quarter.
 *   [RS]  "ZeRO Stage 2: Gradient Partitioning": after the reduce-scatter,
 *         GPU i holds the reduced gradient of shard i.
 *   [ZPP2] "ZeRO-1/2/3", section "ZeRO++": quantized weights may be 8- or
 *         4-bit.
 *   [AVG] "ZeRO Stage 2: Gradient Partitioning", the numbered steps of the
 *         stage-2 flow, step 2: the reduce-scatter averages the gradients
 *         over all GPUs, and GPU i keeps the average of shard i.
 * Quantization rule (the pages name block quantization but print no
 * formula; this is the symmetric absmax reading the library implements):
 *   a_b = max |x| over block b;  s_b = a_b / Q rounded once to binary32,
 *   Q = 127 for 8-bit and 7 for 4-bit codes; code = round-half-even of the
 *   correctly rounded binary32 quotient x / s_b, clamped to [-Q, Q];
 *   a block whose scale is 0 gets all-zero codes.
 */
#ifndef ZPP_H
#define ZPP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZPP_ABI_VERSION 2
#define ZPP_MIN_BLOCK 32
#define ZPP_MAX_BLOCK 4096
#define ZPP_MAX_INPUTS 4096
#define ZPP_MAX_DIVISOR 16777216 /* 2^24: every divisor up to it is exact in binary32 */
#define ZPP_MAX_FEATURES 4194304 /* 2^22: the longest row of a weight matrix or of a norm */
#define ZPP_MAX_ROWS 1073741824  /* 2^30: the most rows of one linear or norm call */
#define ZPP_MAX_GROUPS 4096      /* the most weight matrices of one grouped linear call, and adapters of another */
#define ZPP_MAX_RANK 256         /* the largest rank of an adapter */
/* 2^40: the largest element count, input stride (bytes for codes, floats
 * for scales), and reordered buffer (elements, or bytes / 4) accepted; far
 * beyond any GPU's memory, it keeps every byte range of a call exact in
 * 64-bit arithmetic (larger values: ZPP_ERR_ARG). */
#define ZPP_MAX_NUMEL ((int64_t)1 << 40)

typedef enum zpp_status {
    ZPP_OK = 0,
    ZPP_ERR_NULL = 1,        /* a required pointer is NULL                        */
    ZPP_ERR_ARG = 2,         /* size, block, bit width, count or stride invalid   */
    ZPP_ERR_ALIGN = 3,       /* pointer or stride not aligned as required         */
    ZPP_ERR_UNSUPPORTED = 4, /* valid request the library does not implement      */
    ZPP_ERR_LAUNCH = 5,      /* the HIP runtime reported an error for the launch  */
    /* Beyond the five error kinds above, the library tells apart two more
     * argument errors; they come after ZPP_ERR_LAUNCH so that codes 0-5
     * keep their meaning for callers that know only those. */
    ZPP_ERR_OVERLAP = 6,     /* an output overlaps an input or another output     */
    ZPP_ERR_POINTER = 7      /* a pointer is not memory the GPU can address       */
} zpp_status;

typedef enum zpp_dtype {
    ZPP_BF16 = 1, /* bfloat16 */
    ZPP_FP32 = 2  /* IEEE-754 binary32 */
} zpp_dtype;

/* Element types and status codes cross the ABI as int32_t parameters (one of
 * the enumerators above), so that any value a caller passes is well defined
 * and is refused (ZPP_ERR_ARG, or "unknown zpp_status"). */

/*
 * Block-quantize `numel` elements of `x` to `bits`-bit codes and per-block
 * scales. [QWZ] (8-bit weights before the forward all-gather) and [QGZ]
 * (the one-shot 4-bit gradient quantization before the all-to-all).
 *
 *   x        in   numel elements of x_dtype (ZPP_BF16 or ZPP_FP32), 16-B aligned
 *   numel    in   element count, multiple of `block`, <= ZPP_MAX_NUMEL
 *   block    in   block size B (power of two, 32..4096)
 *   bits     in   8 or 4
 *   codes    out  numel*bits/8 bytes, 16-B aligned
 *   scales   out  numel/block floats, 4-B aligned
 *   stream   in   hipStream_t
 * Non-finite inputs are outside the contract (they cannot fault the GPU,
 * but their codes are unspecified).
 */
zpp_status zpp_quantize_blocks(const void *x, int32_t x_dtype, int64_t numel,
                               int32_t block, int32_t bits, void *codes, float *scales,
                               void *stream);

/*
 * Tensor-slice reordering fused into the one-shot quantization [QGZ] (the
 * page lists kernel fusion among the QGZ optimizations): quantizes the
 * reordered view of x (see zpp_reorder_slices) without writing it out.
 * x holds N = n_nodes * gpus_per_node slices of slice_elems elements in
 * their original order; output slice positions
 * [first_slice, first_slice + n_slices) of the reordered buffer are
 * quantized, and their codes and scales are written contiguously, exactly
 * as zpp_quantize_blocks would write them for those slices of the
 * reordered buffer (blocks never straddle slices). Choosing the range lets a
 * caller quantize the chunk it keeps straight into its receive buffer.
 *
 *   x               in   N * slice_elems elements of x_dtype, 16-B aligned
 *   slice_elems     in   multiple of `block`; N * slice_elems <= ZPP_MAX_NUMEL
 *   n_nodes, gpus_per_node  in  >= 1 each, product <= 65535
 *   first_slice, n_slices   in  0 <= first_slice, first_slice + n_slices <= N
 *   block, bits     in   as zpp_quantize_blocks
 *   codes           out  n_slices * slice_elems * bits / 8 bytes, 16-B aligned
 *   scales          out  n_slices * slice_elems / block floats, 4-B aligned
 *   stream          in   hipStream_t
 */
zpp_status zpp_quantize_reordered(const void *x, int32_t x_dtype, int64_t slice_elems, int32_t n_nodes,
                                  int32_t gpus_per_node, int32_t first_slice, int32_t n_slices, int32_t block,
                                  int32_t bits, void *codes, float *scales, void *stream);

/*
 * Rebuild values from codes and scales: y = code * s_b in binary32, then
 * rounded to nearest-even for ZPP_BF16 output. [QWZ] (the receiver of the
 * 8-bit all-gather needs 16-bit weights to compute with) and [ZPP2].
 *
 *   codes    in   numel*bits/8 bytes, 16-B aligned
 *   scales   in   numel/block floats, 4-B aligned
 *   bits     in   8 or 4 (any code value is accepted, including -128 / -8)
 *   numel    in   element count, multiple of `block`, <= ZPP_MAX_NUMEL
 *   block    in   block size B
 *   y        out  numel elements of y_dtype (ZPP_BF16 or ZPP_FP32), 16-B aligned
 *   stream   in   hipStream_t
 */
zpp_status zpp_dequantize_blocks(const void *codes, const float *scales, int32_t bits,
                                 int64_t numel, int32_t block, void *y, int32_t y_dtype,
                                 void *stream);

/*
 * Tensor-slice reordering before the two-hop exchange [QGZ], so that after
 * hop 1 (contiguous chunk j to local rank j) and hop 2 (sub-chunk k of it
 * to node k) every rank holds its own shard [RS]. The buffer is
 * N = n_nodes * gpus_per_node equal slices of `slice_bytes` bytes; ranks
 * are node-major (rank = node * gpus_per_node + local). Output slice
 * position j*n_nodes + k receives input slice k*gpus_per_node + j.
 * Byte-wise: works on any element type, and commutes with block
 * quantization when every slice is a whole number of blocks.
 *
 *   in, out      in/out  N * slice_bytes bytes each, out-of-place
 *   slice_bytes  in      >= 0; any value (vector width adapts to alignment);
 *                        N * slice_bytes <= 4 * ZPP_MAX_NUMEL
 *   n_nodes, gpus_per_node  in  >= 1 each, product <= 65535
 *   stream       in      hipStream_t
 */
zpp_status zpp_reorder_slices(const void *in, void *out, int64_t slice_bytes, int32_t n_nodes,
                              int32_t gpus_per_node, void *stream);

/*
 * The fused hop step of qgZ [QGZ]: dequantize n_inputs received pieces,
 * sum them in binary32 in ascending input order (each product and each sum
 * rounded on its own: no product is fused into the sum), and either
 * requantize the sum for the next hop (hop 1, intra-node reduction) or emit
 * it as binary32 (hop 2, the owner's reduced shard [RS]). It sums; it does
 * not average.
 *
 *   codes_in            in   input r's codes at codes_in + r*codes_stride_bytes
 *   codes_stride_bytes  in   0..ZPP_MAX_NUMEL, multiple of 16
 *   scales_in           in   input r's scales at scales_in + r*scales_stride
 *   scales_stride       in   0..ZPP_MAX_NUMEL, in floats
 *   n_inputs            in   1..ZPP_MAX_INPUTS
 *   bits_in             in   8 or 4
 *   numel, block        in   elements per input (<= ZPP_MAX_NUMEL) and block size B (same B for
 *                            the inputs and the requantized output)
 *   codes_out, scales_out, bits_out
 *                       out  requantized sum (bits_out 8 or 4), or
 *                            NULL, NULL, 0 to skip requantization
 *   sum_out             out  binary32 sum (numel floats, 16-B aligned), or NULL
 *   stream              in   hipStream_t
 * At least one of the two outputs must be requested (ZPP_ERR_ARG).
 * Any code bytes and any finite scales are accepted; the binary32 sum is
 * exact to the contract for all of them. A sum that overflows to infinity
 * (only possible with scales near the binary32 limit) is outside the
 * contract for requantization: that block's codes and scale are unspecified.
 */
zpp_status zpp_dequant_reduce_requant(const void *codes_in, int64_t codes_stride_bytes,
                                      const float *scales_in, int64_t scales_stride,
                                      int32_t n_inputs, int32_t bits_in, int64_t numel,
                                      int32_t block, void *codes_out, float *scales_out,
                                      int32_t bits_out, float *sum_out, void *stream);

/*
 * The hop-1 step of qgZ [QGZ] with its output split the way the next hop
 * needs it: the same binary32 input-order sum as zpp_dequant_reduce_requant,
 * requantized, with the requantized codes and scales of the elements in
 * [keep_begin, keep_begin + keep_elems) written to codes_keep / scales_keep
 * (the piece this GPU keeps for itself in hop 2: its own sub-chunk, which
 * goes straight into its slot of the hop-2 receive buffer), and those of
 * all other elements written to codes_send / scales_send, in element order
 * with the kept window left out (what the inter-node all-to-all sends). One
 * pass over the inputs; both outputs are exactly the corresponding parts of
 * zpp_dequant_reduce_requant's output.
 *
 *   codes_in, codes_stride_bytes, scales_in, scales_stride, n_inputs,
 *   bits_in, numel, block   in   as zpp_dequant_reduce_requant
 *   keep_begin, keep_elems  in   the kept window, whole blocks:
 *                                0 <= keep_begin <= keep_begin + keep_elems <= numel
 *   codes_send   out  (numel - keep_elems) * bits_out / 8 bytes, 16-B aligned
 *   scales_send  out  (numel - keep_elems) / block floats, 4-B aligned
 *                     (both may be NULL when keep_elems == numel)
 *   codes_keep   out  keep_elems * bits_out / 8 bytes, 16-B aligned
 *   scales_keep  out  keep_elems / block floats, 4-B aligned
 *                     (both may be NULL when keep_elems == 0)
 *   bits_out     in   8 or 4
 *   stream       in   hipStream_t
 * Errors as zpp_dequant_reduce_requant's, and ZPP_ERR_ARG for a window that
 * is not whole blocks or does not lie inside [0, numel); ZPP_ERR_OVERLAP
 * when any two of the four outputs overlap.
 */
zpp_status zpp_dequant_reduce_requant_split(const void *codes_in, int64_t codes_stride_bytes,
                                            const float *scales_in, int64_t scales_stride,
                                            int32_t n_inputs, int32_t bits_in, int64_t numel,
                                            int32_t block, int64_t keep_begin, int64_t keep_elems,
                                            void *codes_send, float *scales_send, void *codes_keep,
                                            float *scales_keep, int32_t bits_out, void *stream);

/*
 * The final hop of qgZ writing the optimizer-ready shard [QGZ][AVG]: the same
 * input-order binary32 sum as zpp_dequant_reduce_requant, then divided by
 * `divisor`, the number of GPUs whose gradients the sum holds (for the
 * two-hop exchange, n_nodes * gpus_per_node, not n_inputs), with one
 * correctly rounded binary32 division per element. A power-of-two divisor
 * only lowers the exponent (exact unless the result is subnormal).
 *
 *   codes_in, codes_stride_bytes, scales_in, scales_stride, n_inputs,
 *   bits_in, numel, block   in   as zpp_dequant_reduce_requant
 *   divisor             in   1..ZPP_MAX_DIVISOR (1 gives the plain sum)
 *   avg_out             out  numel floats, 16-B aligned
 *   stream              in   hipStream_t
 */
zpp_status zpp_dequant_reduce_average(const void *codes_in, int64_t codes_stride_bytes,
                                      const float *scales_in, int64_t scales_stride,
                                      int32_t n_inputs, int32_t bits_in, int64_t numel,
                                      int32_t block, int32_t divisor, float *avg_out, void *stream);

/*
 * Linear products on block-quantized weights, without rebuilding the weights
 * in memory: the receiver of the quantized all-gather [QWZ][ZPP2] multiplies
 * by the codes it holds. The weight matrix is out_features x in_features,
 * row-major, quantized as one flat buffer of out_features * in_features
 * elements (as zpp_quantize_blocks writes it; blocks may straddle rows):
 *
 *   W[n][k] = code[n*K + k] * scales[(n*K + k) / B],   K = in_features
 *   zpp_linear_blocks:       y[m][n]  = sum over k of x[m][k]  * W[n][k]
 *   zpp_linear_blocks_grad:  dx[m][k] = sum over n of dy[m][n] * W[n][k]
 *
 * the second being the gradient of the first with respect to x. Any number
 * of rows, from one token to a long sequence. Sums are binary32. Where input
 * and output are both ZPP_BF16, the weights may enter the products of more
 * than 64 rows, and enter those of every gradient, as bf16: exactly the values
 * zpp_dequantize_blocks writes as ZPP_BF16, each off by at most 2^-8 of itself.
 * Otherwise nothing is rounded below binary32 but the result, so a caller who
 * wants the weights in full asks for a ZPP_FP32 result (three products instead
 * of one in the gradient). Both statements hold for weights and binary32
 * activations of magnitude 2^-105 and more; smaller ones may enter with an
 * absolute error of up to 2^-128. The number of rows chooses kernels, so a row's
 * result can differ by these roundings between calls of different numbers of
 * rows; calls of the same sizes give the same bits.
 *
 *   x / dy          in   rows of in_features (dy: out_features) elements of x_dtype, 16-B aligned
 *   x_stride        in   elements from one row to the next, >= the row's length; for x a
 *                        multiple of 16 bytes; <= ZPP_MAX_NUMEL
 *   rows            in   0..ZPP_MAX_ROWS; 0 is a no-op returning ZPP_OK
 *   codes, scales   in   as zpp_quantize_blocks writes them for out_features * in_features elements
 *   bits            in   8 or 4 (any code value is accepted)
 *   out_features    in   1..ZPP_MAX_FEATURES
 *   in_features     in   a multiple of 32, 32..ZPP_MAX_FEATURES
 *   block           in   block size B; divides out_features * in_features
 *   y / dx          out  rows of out_features (dx: in_features) elements of y_dtype, 16-B aligned;
 *                        elements between a row's end and the next row are not written
 *   y_stride        in   as x_stride; for dx a multiple of 16 bytes
 *   workspace       in   workspace_bytes of memory for this call alone, 16-B aligned; NULL if 0 bytes
 *                        are needed. Its contents are unspecified before and after.
 *   workspace_bytes in   at least zpp_linear_blocks_workspace(...) (ZPP_ERR_ARG otherwise)
 *   stream          in   hipStream_t
 * A matrix with a row stride counts, for the overlap and range checks, from
 * its first element to its last. An infinite or NaN element of x or dy makes
 * results of its own row infinite or NaN (unspecified which), of no other row.
 */
zpp_status zpp_linear_blocks(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, const void *codes,
                             const float *scales, int32_t bits, int64_t out_features, int64_t in_features,
                             int32_t block, void *y, int32_t y_dtype, int64_t y_stride, void *workspace,
                             int64_t workspace_bytes, void *stream);

zpp_status zpp_linear_blocks_grad(const void *dy, int32_t dy_dtype, int64_t dy_stride, int64_t rows,
                                  const void *codes, const float *scales, int32_t bits, int64_t out_features,
                                  int64_t in_features, int32_t block, void *dx, int32_t dx_dtype, int64_t dx_stride,
                                  void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace that zpp_linear_blocks (grad == 0) or zpp_linear_blocks_grad
 * (grad != 0) needs for these types, sizes and row stride of its input (any
 * stride that is the row's length or more; pass the call's own, because rows on
 * no 16-byte piece, and rows more than 2^22 elements apart, may need more than
 * others): for the sums of a contraction that is split to share out few tiles of
 * results over the GPU, and for a packed copy of activations of binary32 or of
 * such rows. 0 where neither is needed. It depends on the arguments alone, and
 * fewer rows may need more than many; 0 for sizes the calls refuse. */
int64_t zpp_linear_blocks_workspace(int32_t grad, int32_t in_dtype, int64_t in_stride, int32_t out_dtype,
                                    int64_t rows, int64_t out_features, int64_t in_features);

/*
 * Linear products of rows in groups, a block-quantized weight matrix for each (the
 * experts of a layer, of which every row has been given one): `groups` matrices of
 * out_features x in_features lie behind one another, codes and scales alike, as
 * zpp_quantize_blocks writes them for groups * out_features * in_features elements.
 * Row m of group e, offsets[e] <= m < offsets[e + 1], has
 *
 *   zpp_linear_grouped:       y[m][n]  = sum over k of x[m][k]  * W[e][n][k]
 *   zpp_linear_grouped_grad:  dx[m][k] = sum over n of dy[m][n] * W[e][n][k]
 *
 *   offsets         in   groups + 1 int32, 4-B aligned, in device memory: ascending, from 0 to rows. A group may be
 *                        empty; rows before offsets[0] and from offsets[groups] on are in no group, and what the output
 *                        holds for them is left as it is. The library cannot check them before the launch: results of
 *                        offsets that do not ascend are unspecified, but nothing outside of the call's rows is read or
 *                        written, whatever the offsets hold.
 *   groups          in   1..ZPP_MAX_GROUPS; groups * out_features * in_features <= ZPP_MAX_NUMEL
 *   block           in   block size B; divides out_features * in_features
 *   workspace_bytes in   at least zpp_linear_grouped_workspace(...) (ZPP_ERR_ARG otherwise)
 * Everything else is as in zpp_linear_blocks: types, strides, precision (where that speaks of more than 64 rows:
 * where rows / groups is more than 64), and rows that hold infinite or NaN elements. But in the gradient of up to 64
 * rows, all groups together, weights enter with 16 bits or more (off by at most 2^-16) from ZPP_BF16 to ZPP_BF16 too.
 */
zpp_status zpp_linear_grouped(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, const int32_t *offsets,
                              int64_t groups, const void *codes, const float *scales, int32_t bits,
                              int64_t out_features, int64_t in_features, int32_t block, void *y, int32_t y_dtype,
                              int64_t y_stride, void *workspace, int64_t workspace_bytes, void *stream);

zpp_status zpp_linear_grouped_grad(const void *dy, int32_t dy_dtype, int64_t dy_stride, int64_t rows,
                                   const int32_t *offsets, int64_t groups, const void *codes, const float *scales,
                                   int32_t bits, int64_t out_features, int64_t in_features, int32_t block, void *dx,
                                   int32_t dx_dtype, int64_t dx_stride, void *workspace, int64_t workspace_bytes,
                                   void *stream);

/* Bytes of workspace that zpp_linear_grouped (grad == 0) or zpp_linear_grouped_grad
 * (grad != 0) needs, as zpp_linear_blocks_workspace; 0 for sizes the calls refuse. */
int64_t zpp_linear_grouped_workspace(int32_t grad, int32_t in_dtype, int64_t in_stride, int32_t out_dtype,
                                     int64_t rows, int64_t groups, int64_t out_features, int64_t in_features);

/*
 * Linear products on block-quantized weights with a low-rank adapter beside them: a
 * weight that stays as codes serves many requests, and is trained, through adapters. Row
 * m has adapter g = ids[m], a number in [0, adapters), or none (any other number):
 *
 *   reduced[m] = s_g * sum over k of x[m][k] * A[g][.][k]            (zeros without an adapter)
 *   y[m][n]    = sum over k of x[m][k] * W[n][k] + sum over r of reduced[m][r] * B[g][n][r]
 *
 * Rows of one adapter need not be neighbours, though long prompts are faster if they are.
 * The sum is rounded once, to y_dtype. What is said of zpp_linear_blocks holds for x, the
 * codes, y, their strides and the first product's precision. Adapters enter exactly,
 * `reduced` is binary32; where x, y and the adapters are all ZPP_BF16, it enters the
 * second product with 16 bits or more (off by at most 2^-16 of itself). Nothing of an adapter, not its infinities or NaNs
 * either, reaches rows that do not name it.
 *
 *   a         in   adapters x rank x in_features elements of ab_dtype, 16-B aligned, without gaps
 *   b         in   adapters x out_features x rank elements of ab_dtype, 16-B aligned, without gaps
 *   adapters  in   1..ZPP_MAX_GROUPS
 *   rank      in   a multiple of 8, 8..ZPP_MAX_RANK (fill up smaller ones with zeros); adapters * rank times
 *                  out_features, and times in_features, <= ZPP_MAX_NUMEL
 *   ids       in   rows int32, 4-B aligned, in device memory; NULL: every row has adapter 0
 *   scaling   in   adapters floats (s_g), 4-B aligned, in device memory; NULL: ones
 *   reduced   out  rows x rank floats, 16-B aligned: what the backward pass needs
 *   workspace_bytes  in  at least zpp_linear_adapters_workspace(0, ...) (ZPP_ERR_ARG otherwise)
 */
zpp_status zpp_linear_adapters(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, const void *codes,
                               const float *scales, int32_t bits, int64_t out_features, int64_t in_features,
                               int32_t block, const void *a, const void *b, int32_t ab_dtype, int64_t adapters,
                               int64_t rank, const int32_t *ids, const float *scaling, float *reduced, void *y,
                               int32_t y_dtype, int64_t y_stride, void *workspace, int64_t workspace_bytes,
                               void *stream);

/*
 * The backward pass of zpp_linear_adapters: with u[m] = s_g * sum over n of dy[m][n] * B[g][n][.],
 *
 *   dx[m][k]    = sum over n of dy[m][n] * W[n][k] + sum over r of u[m][r] * A[g][r][k]
 *   da[g][r][k] = sum over the rows m of adapter g of u[m][r] * x[m][k]
 *   db[g][n][r] = sum over the rows m of adapter g of dy[m][n] * reduced[m][r]
 *
 * Sums are binary32, in an order fixed by the sizes and the ids, and rounded once: the same
 * inputs give the same bits. An adapter without rows gets zeros. Where dy and the adapters are
 * ZPP_BF16, u and `reduced` enter da and db with 16 bits (off by at most 2^-16 of themselves), and
 * u enters dx so where dx is ZPP_BF16 too and there are more than 64 rows; otherwise in full. Weights enter dx
 * as in zpp_linear_blocks_grad, but of up to 64 rows from ZPP_BF16 to ZPP_BF16 with 16 bits or more (off by at most
 * 2^-16), not as bf16.
 *
 *   dy        in   rows of out_features elements of dy_dtype, as in zpp_linear_blocks_grad
 *   x         in   rows of in_features elements of dy_dtype, 16-B aligned, x_stride (any of in_features or more)
 *                  between rows, as in the forward pass; may be NULL without da; its stride is then ignored
 *   reduced   in   as the forward pass wrote it; may be NULL without db
 *   a, b, ab_dtype, adapters, rank, ids, scaling
 *             in   as in the forward pass
 *   dx        out  rows of in_features elements of dx_dtype, as in zpp_linear_blocks_grad
 *   da        out  adapters x rank x in_features elements of ab_dtype, 16-B aligned, or NULL
 *   db        out  adapters x out_features x rank elements of ab_dtype, 16-B aligned, or NULL
 *   workspace_bytes  in  at least zpp_linear_adapters_workspace(1, ...) (ZPP_ERR_ARG otherwise)
 * With rows == 0, da and db are set to zero (the empty sums).
 */
zpp_status zpp_linear_adapters_grad(const void *dy, int32_t dy_dtype, int64_t dy_stride, const void *x, int64_t x_stride,
                                    const float *reduced, int64_t rows, const void *codes, const float *scales,
                                    int32_t bits, int64_t out_features, int64_t in_features, int32_t block,
                                    const void *a, const void *b, int32_t ab_dtype, int64_t adapters, int64_t rank,
                                    const int32_t *ids, const float *scaling, void *dx, int32_t dx_dtype,
                                    int64_t dx_stride, void *da, void *db, void *workspace, int64_t workspace_bytes,
                                    void *stream);

/* Bytes of workspace that zpp_linear_adapters (grad == 0) or zpp_linear_adapters_grad (grad != 0)
 * needs for these types, sizes and row stride of x (dy); it depends on the arguments alone. 0 for sizes the
 * calls refuse. */
int64_t zpp_linear_adapters_workspace(int32_t grad, int32_t in_dtype, int64_t in_stride, int32_t out_dtype,
                                      int64_t rows, int64_t out_features, int64_t in_features, int64_t adapters,
                                      int64_t rank);

/*
 * Layer norm over each row of `width` elements, as it stands before the
 * projections of a layer:
 *
 *   mean = sum x / width;  rstd = 1 / sqrt(sum (x - mean)^2 / width + eps)
 *   y = (x - mean) * rstd * weight + bias
 *
 *   x         in   rows x width elements of x_dtype, 16-B aligned
 *   x_stride  in   elements from one row to the next, width..ZPP_MAX_NUMEL
 *   rows      in   0..ZPP_MAX_ROWS; 0 is a no-op returning ZPP_OK
 *   width     in   1..ZPP_MAX_FEATURES
 *   weight    in   width elements of w_dtype, 16-B aligned, or NULL (ones)
 *   bias      in   width elements of w_dtype, 16-B aligned, or NULL (zeros)
 *   eps       in   >= 0, finite
 *   y         out  rows x width elements of x_dtype, 16-B aligned, y_stride between rows
 *   mean, rstd  out  rows floats each, 4-B aligned: what the backward pass needs
 *   stream    in   hipStream_t
 * Everything between the loads and the stores is binary32.
 */
zpp_status zpp_layer_norm(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t width,
                          const void *weight, const void *bias, int32_t w_dtype, float eps, void *y,
                          int64_t y_stride, float *mean, float *rstd, void *stream);

/*
 * The backward pass of zpp_layer_norm: with xh = (x - mean) * rstd and
 * g = dy * weight,
 *
 *   dx = rstd * (g - sum g / width - xh * sum (g * xh) / width)
 *   dweight = sum over rows of dy * xh;   dbias = sum over rows of dy
 *
 * The sums over rows are binary32, in an order fixed by the sizes alone, and
 * rounded once to w_dtype: the same inputs give the same bits.
 *
 *   dy, x       in   rows x width elements of x_dtype each, 16-B aligned, with their row strides
 *   weight      in   as in zpp_layer_norm (NULL: ones)
 *   mean, rstd  in   as zpp_layer_norm wrote them
 *   dx          out  rows x width elements of x_dtype, 16-B aligned, dx_stride between rows
 *   dweight     out  width elements of w_dtype, 16-B aligned, or NULL
 *   dbias       out  width elements of w_dtype, 16-B aligned, or NULL
 *   workspace   in   workspace_bytes of memory for this call alone, 16-B aligned (NULL if 0 bytes are needed)
 *   workspace_bytes  in  at least zpp_layer_norm_grad_workspace(rows, width) (ZPP_ERR_ARG otherwise)
 *   stream      in   hipStream_t
 * With rows == 0, dweight and dbias are set to zero (the empty sum).
 */
zpp_status zpp_layer_norm_grad(const void *dy, int64_t dy_stride, const void *x, int32_t x_dtype, int64_t x_stride,
                               int64_t rows, int64_t width, const void *weight, int32_t w_dtype, const float *mean,
                               const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias,
                               void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace zpp_layer_norm_grad needs; 0 for sizes it refuses. */
int64_t zpp_layer_norm_grad_workspace(int64_t rows, int64_t width);

/*
 * Root-mean-square norm over each row of `width` elements, with the addition
 * that comes before it in a layer and the quantization that may come behind it:
 *
 *   h    = x + residual, rounded once to x_dtype (x itself without a residual)
 *   rstd = 1 / sqrt(sum h^2 / width + eps)
 *   y    = h * rstd * weight
 *   codes, scales = the block quantization of the binary32 y (the rule above)
 *
 * The norm is that of the rounded h: of what `sum` holds. The codes are those of
 * y before it is rounded to x_dtype, so with ZPP_FP32 they are exactly what
 * zpp_quantize_blocks writes for y. Any of sum, y and the codes can be left out, but
 * not both y and the codes.
 *
 *   x, residual  in   rows x width elements of x_dtype each, 16-B aligned; residual may be NULL
 *   x_stride, residual_stride, sum_stride, y_stride
 *                in   elements from one row to the next, width..ZPP_MAX_NUMEL (ignored for a NULL matrix)
 *   rows         in   0..ZPP_MAX_ROWS; 0 is a no-op returning ZPP_OK
 *   width        in   1..ZPP_MAX_FEATURES
 *   weight       in   width elements of w_dtype, 16-B aligned, or NULL (ones)
 *   eps          in   >= 0, finite
 *   sum          out  h, 16-B aligned, or NULL; NULL without a residual (ZPP_ERR_ARG otherwise)
 *   y            out  rows x width elements of x_dtype, 16-B aligned, or NULL
 *   codes, scales, bits, block
 *                out  as zpp_quantize_blocks writes them for rows * width elements, row after row without gaps:
 *                     bits 8 or 4, block a block size B that divides width; or NULL, NULL, 0, 0
 *   rstd         out  rows floats, 4-B aligned: what the backward pass needs
 *   stream       in   hipStream_t
 * Everything between the loads and the stores is binary32, but h. Codes and scales of
 * a row that holds infinite or NaN elements are unspecified (those of other rows are not).
 */
zpp_status zpp_rms_norm(const void *x, int32_t x_dtype, int64_t x_stride, const void *residual,
                        int64_t residual_stride, int64_t rows, int64_t width, const void *weight, int32_t w_dtype,
                        float eps, void *sum, int64_t sum_stride, void *y, int64_t y_stride, void *codes,
                        float *scales, int32_t bits, int32_t block, float *rstd, void *stream);

/*
 * The backward pass of zpp_rms_norm: with xh = h * rstd and g = dy * weight,
 *
 *   dx = rstd * (g - xh * sum (g * xh) / width) + dsum
 *   dweight = sum over rows of dy * xh
 *
 * dx is the gradient of x and of residual alike. The sum over rows is binary32, in an
 * order fixed by the sizes alone, and rounded once to w_dtype: the same inputs give the
 * same bits.
 *
 *   dy, h       in   rows x width elements of x_dtype each, 16-B aligned, with their row strides; h is `sum`, or x
 *                    where there was no residual
 *   dsum        in   as dy: the gradient that reaches `sum` by other ways, or NULL (none); its stride is then ignored
 *   weight      in   as in zpp_rms_norm (NULL: ones)
 *   rstd        in   as zpp_rms_norm wrote it
 *   dx          out  rows x width elements of x_dtype, 16-B aligned, dx_stride between rows
 *   dweight     out  width elements of w_dtype, 16-B aligned, or NULL
 *   workspace   in   workspace_bytes of memory for this call alone, 16-B aligned (NULL if 0 bytes are needed)
 *   workspace_bytes  in  at least zpp_rms_norm_grad_workspace(rows, width) (ZPP_ERR_ARG otherwise)
 *   stream      in   hipStream_t
 * With rows == 0, dweight is set to zero (the empty sum).
 */
zpp_status zpp_rms_norm_grad(const void *dy, int64_t dy_stride, const void *h, int32_t x_dtype, int64_t h_stride,
                             const void *dsum, int64_t dsum_stride, int64_t rows, int64_t width, const void *weight,
                             int32_t w_dtype, const float *rstd, void *dx, int64_t dx_stride, void *dweight,
                             void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace zpp_rms_norm_grad needs; 0 for sizes it refuses. */
int64_t zpp_rms_norm_grad_workspace(int64_t rows, int64_t width);

/*
 * Switch the library's HIP-runtime pointer checks on (enabled != 0, the
 * default) or off for the whole process; returns the previous setting (1 or
 * 0). With the checks on, every call asks the HIP runtime, before it
 * launches anything, whether each pointer is memory the current GPU can
 * address (ZPP_ERR_POINTER otherwise) and whether each buffer's byte range
 * lies inside its allocation (ZPP_ERR_ARG otherwise), about 0.2 us of host
 * time per buffer. With them off, those two checks are skipped: the caller
 * guarantees that every pointer it passes is device-addressable and that
 * every buffer is as long as the call's sizes imply, and a call that breaks
 * this faults the GPU instead of returning an error. Every other check (NULL
 * pointers, sizes, block, bit widths, strides, alignment, overlapping
 * outputs) always runs. Safe to call from any thread; calls already past
 * their checks are not affected.
 */
int32_t zpp_set_pointer_checks(int32_t enabled);

/* Static, human-readable name of a status code (a zpp_status value); any
 * other value gives "unknown zpp_status". Never NULL. */
const char *zpp_status_string(int32_t status);

/* ZPP_ABI_VERSION of the loaded library. */
int32_t zpp_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZPP_H */
