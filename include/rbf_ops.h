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
 *   quantize_f8_dev        rows to 8-bit floating point with a scale for each
 *                          128 values of a row, or each block of 128 x 128
 *   matmul_f8_dev          product of two such matrices
 *   verify_dev             several tokens at once: drafted ones checked against
 *                          the target's scores, and the answer after them
 *   distill_dev            loss and gradient of scores against a teacher's best
 *                          logits (a search's result, or a larger model's)
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
  RBF_DTYPE_I32 = 3, /* matmul_i8_dev's output only: the sums themselves */
  RBF_DTYPE_E4M3 = 5, /* 8-bit floating point, largest number 448, no infinities */
  RBF_DTYPE_E5M2 = 6  /* 8-bit floating point, largest number 57344 */
} rbf_dtype;

/* Largest depth (values of one row) of an 8-bit integer matrix: every sum of
 * that many products fits 32 bits. */
#define RBF_OPS_MAX_DEPTH 65536
/* Largest row that sample_dev draws from, and of verify_dev and distill_dev;
 * largest depth of matmul_f8_dev, as a head's gradient has its vocabulary for one. */
#define RBF_OPS_MAX_VOCAB (1 << 26)
/* Most drafted tokens of a sequence of verify_dev. */
#define RBF_OPS_MAX_DRAFTS 1024
/* Most teacher's entries of a row of distill_dev. */
#define RBF_OPS_MAX_TEACHER 1024

/* Create a handle for products of up to max_rows rows of up to max_depth
 * values (1 .. 2^20 and 1 .. RBF_OPS_MAX_DEPTH; max_rows counts the rows of
 * the first operand, the queries or tokens; the second operand's rows are not
 * limited, nor is matmul_f8_dev's depth by max_depth). Its workspace is max_rows x max_depth 16-bit numbers, and up to
 * 40 MB for partial sums, 32 MB for rows that are put on 16-byte boundaries and
 * 0.3 MB (64 bytes a row more) for verify_dev's sums.
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

/* Rows to 8-bit floating point. A block is 128 values of a row (fewer at its
 * end) of block_rows rows (1, or 128; fewer at the end). With t = max |x| over
 * the block and MAX the type's largest number (448 or 57344):
 *   scale = t * (1 / MAX),  q = x * ((1 / t) * MAX), rounded to nearest (halves to even)
 * in fp32, rounded after each step. Where (1 / t) * MAX is above 2^127 it is 2^127
 * and the scale 2^-127. A block of zeros has scale 0 and zeros; a block that holds a
 * NaN or an infinity has scale NaN and zeros, so that its products are NaN.
 *   d_x      [rows, cols] of x_dtype (F32, BF16 or F16), stride ld_x
 *   d_q      [rows, cols] of q_dtype (E4M3 or E5M2), stride ld_q (a multiple of
 *            16 from a 16-byte boundary is what matmul_f8_dev reads fastest)
 *   d_scale  [ceil(rows / block_rows), ceil(cols / 128)] fp32, stride ld_scale
 * Errors: INVALID_VALUE, CUDA. */
rbf_status quantize_f8_dev(rbf_ops* ops, const void* d_x, rbf_dtype x_dtype, int64_t ld_x, int64_t rows, int32_t cols,
                           int32_t block_rows, void* d_q, rbf_dtype q_dtype, int64_t ld_q, float* d_scale,
                           int64_t ld_scale);

/* out[i, j] = sum_c a_scale[i, c] * b_scale[j / block_rows, c] * sum_{k in block c} a[i, k] b[j, k] + bias[j],
 * block c being the values 128 c .. 128 c + 127 of a row. A block's products
 * are summed in fp32; the two scales are multiplied, in fp32, and their
 * product with the sum. So scales whose product leaves fp32's normal numbers
 * (2^-126 .. 2^128) lose bits, or the block, below them, and make it infinite
 * above, NaN where its sum is 0. The blocks' sums with their scales are added
 * in fp32; the result is rounded once to out_dtype. It is the same for every
 * replay. Rows of a and b are read fastest from a 16-byte boundary with a
 * stride that is a multiple of 16: others are first put on such boundaries in
 * the handle's workspace, a's with one more launch, b's up to 32 MB at a time
 * with one more launch each.
 *   d_a        [m, k] of a_dtype (E4M3 or E5M2), stride ld_a; m <= max_rows
 *   d_a_scale  [m, ceil(k / 128)] fp32, stride ld_a_scale
 *   d_b        [n, k] of b_dtype (E4M3 or E5M2), stride ld_b
 *   d_b_scale  [ceil(n / block_rows), ceil(k / 128)] fp32, stride ld_b_scale;
 *              block_rows is 1 or 128
 *   d_bias     [n] fp32 (NULL: none)
 *   d_out      [m, n] of out_dtype (F32, BF16 or F16), stride ld_out
 * A linear layer's gradients are two more calls: for its input's, the output's
 * gradient times the transposed weights, for its weights' the transposed
 * gradient times the transposed input, each quantised along its rows.
 * k = 0: the sums are 0. k <= RBF_OPS_MAX_VOCAB, with (m / 256 + 1)(k / 128 +
 * 1) below 10^9 (m / 32 up to 128 rows). Rows off 16-byte boundaries are
 * refused where the workspace does not hold them on such: all of a's, of k
 * bytes rounded up to 16, in max_rows x max_depth 16-bit numbers; of b's 256
 * in 32 MB (k up to 131,072).
 * Errors: INVALID_VALUE, CUDA; a device-side timeout through
 * rbf_ops_check_device_error. */
rbf_status matmul_f8_dev(rbf_ops* ops, const void* d_a, rbf_dtype a_dtype, int64_t ld_a, const float* d_a_scale,
                         int64_t ld_a_scale, const void* d_b, rbf_dtype b_dtype, int64_t ld_b, const float* d_b_scale,
                         int64_t ld_b_scale, int32_t block_rows, const float* d_bias, void* d_out, rbf_dtype out_dtype,
                         int64_t ld_out, int64_t m, int64_t n, int32_t k);

/* Check the drafted tokens of each sequence against the target's scores.
 *
 * With p_i the softmax of the target's scores at place i divided by the
 * sequence's temperature T, and q_i that of the draft's (without draft scores:
 * all of it on the drafted token), drafted token x_i is accepted if all before
 * it are and u_i q_i(x_i) < p_i(x_i); one outside of [0, vocab) is not. The
 * answer goes on with one more token: at the first place r whose token is not
 * accepted drawn from max(0, p_r - q_r) (from p_r where that is no more than
 * 2^-28 in all, to which the two probabilities are held together), behind the
 * last accepted one from p. It is the first index, in index order, at which the
 * running sum exceeds u times the total. So the tokens are distributed as the
 * target's own. A NaN score counts as -infinity, which has no probability, nor
 * has one of less than 2^-1074 of the row's largest (64 bits hold no such
 * number: a mask of the type's lowest value is one); where +infinity is a row's
 * largest score only the scores that equal it have any. A place whose scores are
 * all -infinity accepts no token and answers -1. At an infinite T every finite
 * score has the same probability. At a T not above 0, or NaN, p has all of it on
 * the first of the best indices, a token is accepted if it is that one, and
 * log-probabilities are 0.
 * Scores that were masked to -infinity stand for any filter of either side.
 *   d_target       [seqs, drafts + 1, vocab] of dtype (F32, BF16 or F16): ld_target
 *                  from place to place, ld_target_seq from sequence to sequence
 *   d_draft        [seqs, drafts, vocab] of dtype, in the same way (NULL: none)
 *   d_draft_token  [seqs, drafts] int32
 *   d_draft_count  [seqs] int32: drafted tokens of a sequence, clamped to 0 ..
 *                  drafts (NULL: drafts); what lies behind them is not read
 *   d_u            [seqs, drafts + 1] fp32 random numbers in [0, 1): one a drafted
 *                  token, and the last of a row for the draw (used to 30 bits, as
 *                  sample_dev's)
 *   d_temperature  [seqs] fp32 (NULL: 1)
 *   d_token        [seqs, drafts + 1] int32: the accepted tokens, the drawn one, -1
 *   d_accepted     [seqs] int32: how many were accepted
 *   d_logprob      [seqs, drafts + 1] fp32 (may be NULL): log p of each of
 *                  d_token's entries, -infinity where that is -1
 * The sums that a token's acceptance depends on are fp32 ones; the drawn
 * index is decided by 64-bit integers that hold each probability to 2^-29 of itself
 * and 2^-60 of the whole. The former depend, in their last bits, on how the rows
 * lie on 16-byte boundaries; a call made again with the same tensors gives the same bits.
 * seqs * (drafts + 1) <= max_rows, drafts <= RBF_OPS_MAX_DRAFTS,
 * vocab <= RBF_OPS_MAX_VOCAB. Errors: INVALID_VALUE, CUDA. */
rbf_status verify_dev(rbf_ops* ops, const void* d_target, int64_t ld_target_seq, int64_t ld_target, const void* d_draft,
                      int64_t ld_draft_seq, int64_t ld_draft, rbf_dtype dtype, int64_t seqs, int32_t drafts,
                      int32_t vocab, const int32_t* d_draft_token, const int32_t* d_draft_count, const float* d_u,
                      const float* d_temperature, int32_t* d_token, int32_t* d_accepted, float* d_logprob);

/* Distillation from a teacher's best logits: the loss of each row and the
 * gradient of the losses' sum with respect to the scores, in one read of them.
 *
 * Of a row: p is the softmax of the k logits / T and, where d_rest is given, of
 * one more entry whose logarithm (of the teacher's remaining mass, at T) that
 * is; q is the softmax of the scores / T, and q_rest its mass outside of the listed indices.
 *   loss = weight * T^2 * (sum_e p_e log(p_e / q_e) + p_rest log(p_rest / q_rest))
 * An entry whose index is outside of [0, vocab) (such as -1, no entry, in a
 * search's list) does not count; entries with the same index add up in the
 * gradient. A listed score of -infinity with p_e above 0 makes the loss infinite.
 * A row of weight 0, without any entry or remaining mass, or whose scores are all
 * -infinity has loss 0 and gradient 0; else a NaN, or +infinity, among its scores
 * or logits makes both NaN. (The weight multiplies both.)
 *   d_scores   [rows, vocab] of dtype (F32, BF16 or F16), stride ld_scores
 *   d_index    [rows, k] int32, stride ld_index
 *   d_teacher  [rows, k] of teacher_dtype (F32, BF16 or F16), stride ld_teacher
 *   d_rest     [rows] fp32 (NULL: no remaining mass)
 *   d_weight   [rows] fp32 (NULL: 1): of a mean 1 / rows, of a backward pass the
 *              loss' gradient
 *   d_loss     [rows] fp32 (NULL: not wanted)
 *   d_grad     [rows, vocab] of dtype, stride ld_grad (NULL: not wanted); d_scores
 *              itself, with its stride, is fine: a score is read before its place is written
 * T = temperature, 2^-20 .. 2^20. k <= RBF_OPS_MAX_TEACHER, vocab <=
 * RBF_OPS_MAX_VOCAB. Errors: INVALID_VALUE, CUDA; a device-side timeout through
 * rbf_ops_check_device_error. */
rbf_status distill_dev(rbf_ops* ops, const void* d_scores, rbf_dtype dtype, int64_t ld_scores, int64_t rows, int32_t vocab,
                       const int32_t* d_index, int64_t ld_index, const void* d_teacher, rbf_dtype teacher_dtype,
                       int64_t ld_teacher, int32_t k, const float* d_rest, const float* d_weight, float temperature,
                       float* d_loss, void* d_grad, int64_t ld_grad);

#ifdef __cplusplus
}
#endif

#endif /* RBF_OPS_H_ */
