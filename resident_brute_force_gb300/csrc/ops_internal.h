// ops_internal.h -- host-side launch interfaces between the translation units
// of the scoring-head operators. Not part of the public ABI (include/rbf_ops.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rbf {

// Element types of floating-point tensors (the values of rbf_dtype).
constexpr int kF32 = 0;
constexpr int kBF16 = 1;
constexpr int kF16 = 2;
constexpr int kI32 = 3;
constexpr int kI8 = 4;  // internal: the tokens of matmul_i8_dev
constexpr int kE4M3 = 5;
constexpr int kE5M2 = 6;

inline int dtype_bytes(int dtype) { return dtype == kF32 || dtype == kI32 ? 4 : 2; }

// Rows to 8-bit integers. The quantised row goes to `q` (int8, stride ld_q) or,
// as fp16 numbers, to `f16` (stride f16_pitch, zero past the row).
struct QuantizeLaunch {
  const void* x = nullptr;
  int dtype = 0;
  int64_t ld_x = 0;
  int64_t rows = 0;
  int cols = 0;
  int8_t* q = nullptr;
  int64_t ld_q = 0;
  void* f16 = nullptr;
  int f16_pitch = 0;
  unsigned* block_l1 = nullptr;  // with f16: the largest sum of |q| over 128 values of a row is put here (atomicMax)
  float* scale = nullptr;
};
cudaError_t launch_quantize_rows(const QuantizeLaunch& a, cudaStream_t stream);

// out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k] + bias[j].
struct MatmulI8Launch {
  const int8_t* a = nullptr;
  int64_t ld_a = 0;
  const float* a_scale = nullptr;
  const int8_t* b = nullptr;
  int64_t ld_b = 0;
  const float* b_scale = nullptr;
  const float* bias = nullptr;
  void* out = nullptr;
  int out_dtype = 0;
  int64_t ld_out = 0;
  int64_t m = 0;
  int64_t n = 0;
  int k = 0;
  bool b_is_new = false;  // b is written by the kernel enqueued just before
};
// Rows of k bytes to rows of `pitch` bytes (a multiple of 16 from k on, whose
// last ones are not set), which start on 16-byte boundaries.
cudaError_t launch_pitch_rows(const int8_t* b, int64_t ld_b, int64_t rows, int k, int8_t* out, int pitch, int num_sms,
                              cudaStream_t stream);
// The result of a depth of zero: 0 times the scales, plus the bias.
cudaError_t launch_matmul_i8_empty(const MatmulI8Launch& a, int num_sms, cudaStream_t stream);

// Up to four tokens, in one launch: 8-bit ones (dtype kI8), or floating-point
// ones that it quantises. a.a and a.ld_a are not used, nor a.a_scale with the
// latter.
constexpr int kFewMaxTokenBytes = 96 * 1024;  // of the 8-bit tokens in shared memory
bool matmul_i8_few_fits(const MatmulI8Launch& a);
cudaError_t launch_matmul_i8_few(const MatmulI8Launch& a, const void* tokens, int64_t ld, int dtype, int num_sms,
                                 cudaStream_t stream);

// The tensor-core product. Its first operand is the workspace's fp16 rows
// (launch_expand_rows or launch_quantize_rows writes them, enqueued just
// before); a.a and a.ld_a are not used.
struct MatmulI8Workspace {
  void* rows_f16 = nullptr;     // [m][matmul_i8_pitch(k)]
  int* partial = nullptr;       // matmul_i8_partial_bytes
  unsigned* arrived = nullptr;  // num_sms counters, zero between launches
  unsigned* block_l1 = nullptr;       // largest sum of |a| over 128 values of a row; its writer found it zero
  unsigned* block_l1_next = nullptr;  // the word of the next call, which the product clears
  int* err = nullptr;
  int num_sms = 0;
  uint64_t timeout_ns = 0;
};
int matmul_i8_pitch(int k);  // fp16 numbers per workspace row
size_t matmul_i8_partial_bytes(int num_sms);
int64_t matmul_i8_tc_rows(int64_t m, int k);  // most rows of b that one launch takes
cudaError_t launch_expand_rows(const int8_t* a, int64_t ld_a, int64_t m, int k, const MatmulI8Workspace& w,
                               cudaStream_t stream);
cudaError_t launch_matmul_i8_tc(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t stream);

struct SampleLaunch {
  const void* logits = nullptr;
  int dtype = 0;
  int64_t ld = 0;
  int64_t rows = 0;
  int vocab = 0;
  const float* u = nullptr;
  const float* temperature = nullptr;
  const int32_t* top_k = nullptr;
  const float* top_p = nullptr;
  const float* min_p = nullptr;
  int32_t* token = nullptr;
  float* logprob = nullptr;
};
cudaError_t launch_sample(const SampleLaunch& a, cudaStream_t stream);

// Rows to 8-bit floating point, a scale for each 128 values of block_rows (1 or 128) rows.
struct QuantizeF8Launch {
  const void* x = nullptr;
  int dtype = 0;
  int64_t ld_x = 0;
  int64_t rows = 0;
  int cols = 0;
  int block_rows = 1;
  void* q = nullptr;
  int q_dtype = 0;
  int64_t ld_q = 0;
  float* scale = nullptr;
  int64_t ld_scale = 0;
};
cudaError_t launch_quantize_f8(const QuantizeF8Launch& a, int num_sms, cudaStream_t stream);

// out[i, j] = sum_c a_scale[i, c] b_scale[j / block_rows, c] sum_{k in block c} a[i, k] b[j, k] + bias[j].
struct MatmulF8Launch {
  const uint8_t* a = nullptr;
  int a_dtype = 0;
  int64_t ld_a = 0;
  const float* a_scale = nullptr;
  int64_t ld_a_scale = 0;
  const uint8_t* b = nullptr;
  int b_dtype = 0;
  int64_t ld_b = 0;
  const float* b_scale = nullptr;
  int64_t ld_b_scale = 0;
  int block_rows = 1;
  const float* bias = nullptr;
  void* out = nullptr;
  int out_dtype = 0;
  int64_t ld_out = 0;
  int64_t m = 0;
  int64_t n = 0;
  int k = 0;
};
// Both operands' rows start on 16-byte boundaries (one row: any stride).
struct MatmulF8Workspace {
  float* partial = nullptr;     // matmul_i8_partial_bytes
  unsigned* arrived = nullptr;  // num_sms counters, zero between launches
  int* err = nullptr;
  int num_sms = 0;
  uint64_t timeout_ns = 0;
};
int64_t matmul_f8_rows(int64_t m, int k);  // most rows of b that one launch takes
cudaError_t launch_matmul_f8(const MatmulF8Launch& a, const MatmulF8Workspace& w, cudaStream_t stream);

// Drafted tokens checked against the target's scores, and the answer after them.
struct VerifyLaunch {
  const void* target = nullptr;  // [seqs, drafts + 1, vocab]
  int64_t ld_target_seq = 0, ld_target = 0;
  const void* draft = nullptr;   // [seqs, drafts, vocab], or none
  int64_t ld_draft_seq = 0, ld_draft = 0;
  int dtype = 0;
  int64_t seqs = 0;
  int drafts = 0;
  int vocab = 0;
  const int32_t* draft_token = nullptr;
  const int32_t* count = nullptr;
  const float* u = nullptr;
  const float* temperature = nullptr;
  int32_t* token = nullptr;
  int32_t* accepted = nullptr;
  float* logprob = nullptr;
};
// What a part of a row says: its largest score and the sum of its weights, or
// the key of its best index.
struct VerifyPart {
  float top, z;
  unsigned long long key;
};
int64_t verify_max_parts(int64_t max_rows, int num_sms);  // for up to 2 max_rows rows: at least two each
// The rows' sums, then the accepted tokens and the draw (enqueued just behind it).
cudaError_t launch_verify_stats(const VerifyLaunch& a, VerifyPart* parts, int64_t max_parts, int num_sms, cudaStream_t stream);
cudaError_t launch_verify_draw(const VerifyLaunch& a, const VerifyPart* parts, int64_t max_parts, int num_sms, cudaStream_t stream);

// Distillation from a teacher's best logits.
struct DistillLaunch {
  const void* scores = nullptr;
  int dtype = 0;
  int64_t ld_scores = 0;
  int64_t rows = 0;
  int vocab = 0;
  const int32_t* index = nullptr;
  int64_t ld_index = 0;
  const void* teacher = nullptr;
  int teacher_dtype = 0;
  int64_t ld_teacher = 0;
  int k = 0;
  const float* rest = nullptr;
  const float* weight = nullptr;
  float temperature = 1.0f;
  float* loss = nullptr;
  void* grad = nullptr;
  int64_t ld_grad = 0;
};
constexpr int kMaxTeacher = 1024;  // entries of a row
cudaError_t launch_distill(const DistillLaunch& a, int* err, uint64_t timeout_ns, int num_sms, cudaStream_t stream);

}  // namespace rbf
