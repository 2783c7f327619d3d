/*
 * rbf_ops.h -- C ABI of the scoring-head operators of librbf.so.
 *
 * What stands next to the search: a corpus or a layer held in 8-bit integers
 * (a quarter of the fp32 corpus), its product with a batch of queries or
 * tokens, and a choice drawn from the scores.
 *
 *   quantize_rows_i8_dev   rows to 8-bit integers with one scale a row
 *   matmul_i8_dev          product of two 8-bit matrices with a scale for
 *                          each row of either (token and channel)
 *   linear_i8_dev          both in one call: floating-point rows times 8-bit
 *                          weights
 *   sample_dev             one index a row, drawn from its scores with
 *                          temperature, top-k, top-p and min-p
 *
 * Conventions (those of rbf.h, and:)
 *   - Sizes and strides are element counts; a stride (ld...) is the distance
 *     between the starts of two rows and at least the row's length.
 *   - All data pointers are device pointers on the handle's device, aligned to
 *     their element type. The calls are stream-ordered on the handle's stream:
 *     they enqueue work and return; a tensor that another stream has written or
 *     will reuse is ordered by the caller. One handle serves one call at a time.
 *   - The handle owns its workspace, allocated in rbf_ops_create; a call
 *     allocates nothing. Calls may be captured in a graph; its replays use the
 *     same workspace and are ordered with the handle's other calls by the caller.
 *   - Outputs do not overlap inputs.
 *   - An empty call (zero rows or columns of output) does nothing: RBF_OK.
 */
#ifndef RBF_OPS_H_
#define RBF_OPS_H_

#include "rbf.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct rbf_ops rbf_ops;

typedef enum rbf_dtype {
  RBF_DTYPE_F32 = 0,
  RBF_DTYPE_BF16 = 1,
  RBF_DTYPE_F16 = 2,
  RBF_DTYPE_I32 = 3 /* matmul_i8_dev's output only: the sums themselves */
} rbf_dtype;

/* Largest depth (values of one row) of an 8-bit matrix: every sum of that
 * many products fits 32 bits. */
#define RBF_OPS_MAX_DEPTH 65536
/* Largest row that sample_dev draws from. */
#define RBF_OPS_MAX_VOCAB (1 << 26)

/* Create a handle for products of up to max_rows rows of up to max_depth
 * values (1 .. 2^20 and 1 .. RBF_OPS_MAX_DEPTH; max_rows counts the rows of
 * the first operand, the queries or tokens; the second operand's rows are not
 * limited). Its workspace is max_rows x max_depth 16-bit numbers, and up to
 * 40 MB for partial sums and 32 MB for rows that are put on 16-byte boundaries.
 *   cuda_stream  stream of every call (NULL: the handle creates its own;
 *                cudaStreamLegacy names the default stream)
 * Errors: INVALID_VALUE, OUT_OF_MEMORY, CUDA. */
rbf_status rbf_ops_create(int64_t max_rows, int32_t max_depth, void* cuda_stream, rbf_ops** out);
/* Waits for the handle's stream, then frees everything. NULL is fine. */
rbf_status rbf_ops_destroy(rbf_ops* ops);
/* The handle's device: the one that was current when it was created. A call
 * made while another one is current is refused (INVALID_VALUE). */
int32_t rbf_ops_device(rbf_ops* ops);
/* The handle's stream. */
void* rbf_ops_stream(rbf_ops* ops);
/* The CUDA error behind the last RBF_ERR_CUDA. */
int32_t rbf_ops_last_cuda_error(rbf_ops* ops);
/* Kernels the most recent call enqueued. */
int32_t rbf_ops_last_launches(rbf_ops* ops);
/* Waits for the handle's stream and returns (and clears) what its kernels
 * reported since the last check: RBF_ERR_TIMEOUT if a bounded device-side
 * wait ran out (the outputs of that call are not valid), else RBF_OK. */
rbf_status rbf_ops_check_device_error(rbf_ops* ops);
/* Bound on each device-side wait of the calls that follow, in nanoseconds
 * (default 2e9, at least 1e6: copies in flight have landed by then). A wait is
 * for another part of the same kernel to go one step on, so the bound does not
 * limit how long a call takes. */
rbf_status rbf_ops_set_timeout(rbf_ops* ops, int64_t nanoseconds);
/* The next `count` kernel launches report failure without being issued
 * (tests of the error path; touches no GPU state). 0 clears. */
rbf_status rbf_ops_inject_host_fault(rbf_ops* ops, int32_t count);

/* Rows to 8-bit integers, one scale a row:
 *   scale[i] = t * (1 / 127), with t = max_j |x[i, j]|
 *   q[i, j]  = x[i, j] * ((1 / t) * 127), rounded to nearest (halves to even)
 * in fp32, rounded after each step. A row of zeros has scale 0 and zeros; a row that holds a NaN or an
 * infinity has scale NaN and zeros, so that its products are NaN.
 *   d_x      [rows, cols] of x_dtype (F32, BF16 or F16), stride ld_x
 *   d_q      [rows, cols] int8, stride ld_q (a multiple of 16 from a 16-byte
 *            boundary is what matmul_i8_dev reads fastest)
 *   d_scale  [rows] fp32
 * Errors: INVALID_VALUE, CUDA. */
rbf_status quantize_rows_i8_dev(rbf_ops* ops, const void* d_x, rbf_dtype x_dtype, int64_t ld_x, int64_t rows,
                                int32_t cols, int8_t* d_q, int64_t ld_q, float* d_scale);

/* out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k] + bias[j].
 * The sums are exact (32-bit integers); they are converted to fp32, scaled and
 * rounded once to out_dtype. For RBF_DTYPE_I32 the sums are returned and
 * d_a_scale, d_b_scale and d_bias have to be NULL.
 *   d_a        [m, k] int8, stride ld_a (queries or tokens); m <= max_rows
 *   d_a_scale  [m] fp32 (NULL: 1)
 *   d_b        [n, k] int8, stride ld_b (corpus rows, or a layer's output
 *              channels); fastest from a 16-byte boundary with ld_b a multiple
 *              of 16: other rows are first put on such boundaries, up to 32 MB
 *              at a time, in the handle's workspace (one more launch a part)
 *   d_b_scale  [n] fp32 (NULL: 1)
 *   d_bias     [n] fp32 (NULL: none)
 *   d_out      [m, n] of out_dtype, stride ld_out
 * Up to four tokens of up to 96 KB take one launch (dp4a), more a launch that
 * expands them and the tensor cores' one; the sums are the same.
 * k = 0: the sums are 0. k <= max_depth.
 * Errors: INVALID_VALUE, CUDA; a device-side timeout through
 * rbf_ops_check_device_error. */
rbf_status matmul_i8_dev(rbf_ops* ops, const int8_t* d_a, int64_t ld_a, const float* d_a_scale, const int8_t* d_b,
                         int64_t ld_b, const float* d_b_scale, const float* d_bias, void* d_out, rbf_dtype out_dtype,
                         int64_t ld_out, int64_t m, int64_t n, int32_t k);

/* matmul_i8_dev on the rows of d_x as quantize_rows_i8_dev quantises them:
 * the same result as those two calls, with the 8-bit rows and their scales
 * kept in the workspace.
 *   d_x        [m, k] of x_dtype, stride ld_x
 *   d_w        [n, k] int8, stride ld_w;  d_w_scale [n] (NULL: 1)
 *   d_out      [m, n] of out_dtype (F32, BF16 or F16) */
rbf_status linear_i8_dev(rbf_ops* ops, const void* d_x, rbf_dtype x_dtype, int64_t ld_x, const int8_t* d_w,
                         int64_t ld_w, const float* d_w_scale, const float* d_bias, void* d_out, rbf_dtype out_dtype,
                         int64_t ld_out, int64_t m, int64_t n, int32_t k);

/* Draw one index from each row of scores.
 *
 * With x the row's scores (a NaN counts as -infinity) and T its temperature,
 * index j has the weight 2^((x_j - max x) log2(e) / T), computed in fp32 (log2(e) / T
 * as a finite number above 0: at infinite T every finite score has the weight 1) and
 * held as a whole multiple of 2^-36, so that every sum of weights below is
 * exact and the result depends on no order of summation. In the order of
 * rbf.h (higher score first, on equal scores the lower index):
 *   1. the first top_k indices are kept;
 *   2. of those the fewest whose weights reach top_p of those indices' sum;
 *   3. of those the ones whose weight is at least min_p (of the largest, 1).
 * The first index is always kept. The drawn index is the first one, in
 * index order, at which the running sum of the kept weights exceeds u times
 * their total. An index at -infinity is never drawn; a row that has
 * nothing else (or no columns) gives index -1 and log-probability -infinity.
 *   d_logits       [rows, vocab] of dtype (F32, BF16 or F16), stride ld
 *   d_u            [rows] fp32 random numbers in [0, 1), used to 30 bits
 *                  (others are clamped to it, a NaN is 0)
 *   d_temperature  [rows] fp32 (NULL: 1); not above 0, or NaN: the row's best
 *                  index is taken
 *   d_top_k        [rows] int32 (NULL or below 1: all)
 *   d_top_p        [rows] fp32, used to 30 bits (NULL, 1 and above, or NaN: all)
 *   d_min_p        [rows] fp32 (NULL, 0 and below, or NaN: all)
 *   d_token        [rows] int32
 *   d_logprob      [rows] fp32 (may be NULL): log of the drawn index's share of
 *                  the kept weights
 * vocab <= RBF_OPS_MAX_VOCAB. Errors: INVALID_VALUE, CUDA. */
rbf_status sample_dev(rbf_ops* ops, const void* d_logits, rbf_dtype dtype, int64_t ld, int64_t rows, int32_t vocab,
                      const float* d_u, const float* d_temperature, const int32_t* d_top_k, const float* d_top_p,
                      const float* d_min_p, int32_t* d_token, float* d_logprob);

#ifdef __cplusplus
}
#endif

#endif /* RBF_OPS_H_ */
