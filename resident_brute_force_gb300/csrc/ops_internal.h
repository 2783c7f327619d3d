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

}  // namespace rbf
