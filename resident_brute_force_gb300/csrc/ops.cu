// ops.cu -- the handle behind include/rbf_ops.h: workspace, argument checks,
// and the order of launches of the scoring-head operators.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "../../include/rbf_ops.h"
#include "ops_internal.h"

using namespace rbf;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 20;

}  // namespace

struct rbf_ops {
  int device = 0;
  int num_sms = 0;
  cudaStream_t stream = nullptr;
  bool own_stream = false;
  int64_t max_rows = 0;
  int max_depth = 0;

  void* rows_f16 = nullptr;      // the product's first operand in fp16, max_rows x matmul_i8_pitch(max_depth)
  float* row_scale = nullptr;    // linear_i8_dev: the rows' scales
  int* partial = nullptr;        // the product's partial sums of shared tiles
  unsigned* arrived = nullptr;   // and their counters
  // Two words, used by turns: a product clears the next one's. A replayed graph
  // uses one of them out of turn; what it then finds is a larger bound, no smaller one.
  unsigned* block_l1 = nullptr;
  int turn = 0;
  VerifyPart* parts = nullptr;   // verify_dev: what parts of rows say, verify_max_parts
  int8_t* staged = nullptr;      // rows of b put on 16-byte boundaries, kStagedBytes
  int* errw = nullptr;           // error bits of the kernels since the last check
  uint64_t timeout_ns = 2000000000ull;  // bound on every device-side wait

  int last_cuda_error = 0;
  int launches = 0;
  int fault_count = 0;
};

namespace {

constexpr size_t kStagedBytes = size_t(32) << 20;  // a part of b that L2 holds between its two kernels

rbf_status cuda_fail(rbf_ops* o, cudaError_t err) {
  o->last_cuda_error = static_cast<int>(err);
  return RBF_ERR_CUDA;
}

#define OPS_LAUNCH(o, call)                                              \
  do {                                                                   \
    if ((o)->fault_count > 0) {                                          \
      --(o)->fault_count;                                                \
      return cuda_fail((o), cudaErrorUnknown);                           \
    }                                                                    \
    const cudaError_t _st = (call);                                      \
    if (_st != cudaSuccess) return cuda_fail((o), _st);                  \
    ++(o)->launches;                                                     \
  } while (0)

// The handle's stream (the default one is each device's own) and its workspace
// belong to its device: no work is enqueued while another one is current.
bool on_its_device(const rbf_ops* o) {
  int current = -1;
  return cudaGetDevice(&current) == cudaSuccess && current == o->device;
}

// The handle's device, current for a wait or a release.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    changed_ = cudaGetDevice(&before_) == cudaSuccess && before_ != device && cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceScope() {
    if (changed_) cudaSetDevice(before_);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;

 private:
  int before_ = 0;
  bool changed_ = false;
};

void release(rbf_ops* o) {
  const DeviceScope scope(o->device);
  if (o->stream) cudaStreamSynchronize(o->stream);
  cudaFree(o->rows_f16);
  cudaFree(o->row_scale);
  cudaFree(o->partial);
  cudaFree(o->arrived);
  cudaFree(o->block_l1);
  cudaFree(o->staged);
  cudaFree(o->parts);
  cudaFree(o->errw);
  if (o->own_stream && o->stream) cudaStreamDestroy(o->stream);
  delete o;
}

bool float_dtype(rbf_dtype t) { return t == RBF_DTYPE_F32 || t == RBF_DTYPE_BF16 || t == RBF_DTYPE_F16; }

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0; }

// A matrix argument: a pointer aligned to its element and a stride of at
// least a row, in which no row's end passes what 64 bits address.
bool matrix_ok(const void* p, int elem, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0 || ld < cols) return false;
  if (rows == 0 || cols == 0) return true;
  if (!p || !aligned(p, elem)) return false;
  return ld <= (INT64_MAX / 8) / std::max<int64_t>(rows, 1);
}

bool f8_dtype(rbf_dtype t) { return t == RBF_DTYPE_E4M3 || t == RBF_DTYPE_E5M2; }

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

bool floats_ok(const void* p) { return !p || aligned(p, 4); }

rbf_status check_matmul(const rbf_ops* o, const MatmulI8Launch& a) {
  if (a.m < 0 || a.n < 0 || a.k < 0 || a.m > o->max_rows || a.n > INT32_MAX || a.k > o->max_depth)
    return RBF_ERR_INVALID_VALUE;
  if (!matrix_ok(a.b, 1, a.n, a.k, a.ld_b)) return RBF_ERR_INVALID_VALUE;
  if (!matrix_ok(a.out, dtype_bytes(a.out_dtype), a.m, a.n, a.ld_out)) return RBF_ERR_INVALID_VALUE;
  if (!floats_ok(a.a_scale) || !floats_ok(a.b_scale) || !floats_ok(a.bias)) return RBF_ERR_INVALID_VALUE;
  return RBF_OK;
}

// The workspace of the next product.
MatmulI8Workspace take_workspace(rbf_ops* o) {
  MatmulI8Workspace w;
  w.rows_f16 = o->rows_f16;
  w.partial = o->partial;
  w.arrived = o->arrived;
  w.block_l1 = o->block_l1 + o->turn;
  o->turn ^= 1;
  w.block_l1_next = o->block_l1 + o->turn;
  w.err = o->errw;
  w.num_sms = o->num_sms;
  w.timeout_ns = o->timeout_ns;
  return w;
}

// The product as its kernels see it, or the first of its parts: as many rows of
// b as a launch takes and, where they do not start on 16-byte boundaries, as the
// room holds in which they are put on them.
MatmulI8Launch first_part(const rbf_ops* o, const MatmulI8Launch& a) {
  MatmulI8Launch f = a;
  f.n = std::min(a.n, matmul_i8_tc_rows(a.m, a.k));
  if (!aligned(a.b, 16) || a.ld_b % 16 != 0) {
    const int pitch = (a.k + 15) / 16 * 16;
    f.b = o->staged;
    f.ld_b = pitch;
    f.n = std::min<int64_t>(f.n, static_cast<int64_t>(kStagedBytes / pitch / 256 * 256));
    f.b_is_new = true;
  }
  return f;
}

// launch(part) for all parts of a.
template <typename F>
rbf_status each_part(rbf_ops* o, const MatmulI8Launch& a, const MatmulI8Launch& first, F&& launch) {
  for (int64_t j = 0; j < a.n; j += first.n) {
    MatmulI8Launch part = first;
    part.n = std::min(first.n, a.n - j);
    part.b_scale = a.b_scale ? a.b_scale + j : nullptr;
    part.bias = a.bias ? a.bias + j : nullptr;
    part.out = static_cast<char*>(a.out) + j * dtype_bytes(a.out_dtype);
    if (first.b_is_new)
      OPS_LAUNCH(o, launch_pitch_rows(a.b + j * a.ld_b, a.ld_b, part.n, a.k, o->staged, static_cast<int>(first.ld_b), o->num_sms,
                                      o->stream));
    else
      part.b = a.b + j * a.ld_b;
    OPS_LAUNCH(o, launch(part));
  }
  return RBF_OK;
}

}  // namespace

extern "C" {

rbf_status rbf_ops_create(int64_t max_rows, int32_t max_depth, void* cuda_stream, rbf_ops** out) {
  if (!out) return RBF_ERR_INVALID_VALUE;
  if (max_rows < 1 || max_rows > kMaxRows || max_depth < 1 || max_depth > RBF_OPS_MAX_DEPTH)
    return RBF_ERR_INVALID_VALUE;
  rbf_ops* o = new (std::nothrow) rbf_ops();
  if (!o) return RBF_ERR_OUT_OF_MEMORY;
  cudaError_t st = cudaGetDevice(&o->device);
  if (st == cudaSuccess) st = cudaDeviceGetAttribute(&o->num_sms, cudaDevAttrMultiProcessorCount, o->device);
  if (st != cudaSuccess) {
    delete o;
    return RBF_ERR_CUDA;
  }
  o->max_rows = max_rows;
  o->max_depth = max_depth;
  if (cuda_stream) {
    o->stream = static_cast<cudaStream_t>(cuda_stream);
  } else {
    if (cudaStreamCreateWithFlags(&o->stream, cudaStreamNonBlocking) != cudaSuccess) {
      delete o;
      return RBF_ERR_CUDA;
    }
    o->own_stream = true;
  }
  const bool ok = cudaMalloc(&o->rows_f16, static_cast<size_t>(max_rows) * matmul_i8_pitch(max_depth) * 2) == cudaSuccess &&
                  cudaMalloc(&o->partial, matmul_i8_partial_bytes(o->num_sms)) == cudaSuccess &&
                  cudaMalloc(&o->arrived, o->num_sms * sizeof(unsigned)) == cudaSuccess &&
                  cudaMalloc(&o->row_scale, static_cast<size_t>(max_rows) * sizeof(float)) == cudaSuccess &&
                  cudaMalloc(&o->block_l1, 2 * sizeof(unsigned)) == cudaSuccess &&
                  cudaMalloc(&o->staged, kStagedBytes) == cudaSuccess &&
                  cudaMalloc(&o->parts, static_cast<size_t>(verify_max_parts(max_rows, o->num_sms)) * sizeof(VerifyPart)) == cudaSuccess &&
                  cudaMalloc(&o->errw, 4 * sizeof(int)) == cudaSuccess;
  if (!ok) {
    cudaGetLastError();
    release(o);
    return RBF_ERR_OUT_OF_MEMORY;
  }
  if (cudaMemsetAsync(o->errw, 0, 4 * sizeof(int), o->stream) != cudaSuccess ||
      cudaMemsetAsync(o->arrived, 0, o->num_sms * sizeof(unsigned), o->stream) != cudaSuccess ||
      cudaMemsetAsync(o->block_l1, 0, 2 * sizeof(unsigned), o->stream) != cudaSuccess ||
      cudaStreamSynchronize(o->stream) != cudaSuccess) {
    release(o);
    return RBF_ERR_CUDA;
  }
  *out = o;
  return RBF_OK;
}

rbf_status rbf_ops_destroy(rbf_ops* o) {
  if (o) release(o);
  return RBF_OK;
}

int32_t rbf_ops_device(rbf_ops* o) { return o ? o->device : -1; }
void* rbf_ops_stream(rbf_ops* o) { return o ? o->stream : nullptr; }
int32_t rbf_ops_last_cuda_error(rbf_ops* o) { return o ? o->last_cuda_error : 0; }
int32_t rbf_ops_last_launches(rbf_ops* o) { return o ? o->launches : 0; }

rbf_status rbf_ops_check_device_error(rbf_ops* o) {
  if (!o) return RBF_ERR_INVALID_VALUE;
  const DeviceScope scope(o->device);
  int e = 0;
  cudaError_t st = cudaMemcpyAsync(&e, o->errw, sizeof(int), cudaMemcpyDeviceToHost, o->stream);
  if (st == cudaSuccess) st = cudaStreamSynchronize(o->stream);
  if (st == cudaSuccess && e != 0) {
    st = cudaMemsetAsync(o->errw, 0, 4 * sizeof(int), o->stream);
    // A launch that gave up may have left counters behind.
    if (st == cudaSuccess) st = cudaMemsetAsync(o->arrived, 0, o->num_sms * sizeof(unsigned), o->stream);
  }
  if (st != cudaSuccess) return cuda_fail(o, st);
  return e ? RBF_ERR_TIMEOUT : RBF_OK;
}

rbf_status rbf_ops_set_timeout(rbf_ops* o, int64_t nanoseconds) {
  if (!o || nanoseconds < 1000000) return RBF_ERR_INVALID_VALUE;
  o->timeout_ns = static_cast<uint64_t>(nanoseconds);
  return RBF_OK;
}

rbf_status rbf_ops_inject_host_fault(rbf_ops* o, int32_t count) {
  if (!o || count < 0) return RBF_ERR_INVALID_VALUE;
  o->fault_count = count;
  return RBF_OK;
}

rbf_status quantize_rows_i8_dev(rbf_ops* o, const void* d_x, rbf_dtype x_dtype, int64_t ld_x, int64_t rows,
                                int32_t cols, int8_t* d_q, int64_t ld_q, float* d_scale) {
  if (!o || !float_dtype(x_dtype) || rows < 0 || cols < 0 || rows > INT32_MAX) return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  if (!matrix_ok(d_x, dtype_bytes(x_dtype), rows, cols, ld_x) || !matrix_ok(d_q, 1, rows, cols, ld_q))
    return RBF_ERR_INVALID_VALUE;
  if (rows == 0) return RBF_OK;
  if (!d_scale || !aligned(d_scale, 4)) return RBF_ERR_INVALID_VALUE;
  QuantizeLaunch a;
  a.x = d_x;
  a.dtype = x_dtype;
  a.ld_x = ld_x;
  a.rows = rows;
  a.cols = cols;
  a.q = d_q;
  a.ld_q = ld_q;
  a.scale = d_scale;
  OPS_LAUNCH(o, launch_quantize_rows(a, o->stream));
  return RBF_OK;
}

rbf_status matmul_i8_dev(rbf_ops* o, const int8_t* d_a, int64_t ld_a, const float* d_a_scale, const int8_t* d_b,
                         int64_t ld_b, const float* d_b_scale, const float* d_bias, void* d_out, rbf_dtype out_dtype,
                         int64_t ld_out, int64_t m, int64_t n, int32_t k) {
  if (!o || !(float_dtype(out_dtype) || out_dtype == RBF_DTYPE_I32)) return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  MatmulI8Launch a;
  a.a = d_a;
  a.ld_a = ld_a;
  a.a_scale = d_a_scale;
  a.b = d_b;
  a.ld_b = ld_b;
  a.b_scale = d_b_scale;
  a.bias = d_bias;
  a.out = d_out;
  a.out_dtype = out_dtype;
  a.ld_out = ld_out;
  a.m = m;
  a.n = n;
  a.k = k;
  if (rbf_status st = check_matmul(o, a)) return st;
  if (!matrix_ok(d_a, 1, m, k, ld_a)) return RBF_ERR_INVALID_VALUE;
  if (out_dtype == RBF_DTYPE_I32 && (d_a_scale || d_b_scale || d_bias)) return RBF_ERR_INVALID_VALUE;
  if (m == 0 || n == 0) return RBF_OK;
  if (k == 0) {
    OPS_LAUNCH(o, launch_matmul_i8_empty(a, o->num_sms, o->stream));
    return RBF_OK;
  }
  const MatmulI8Launch first = first_part(o, a);
  if (matmul_i8_few_fits(first))
    return each_part(o, a, first, [&](const MatmulI8Launch& p) { return launch_matmul_i8_few(p, d_a, ld_a, kI8, o->num_sms, o->stream); });
  const MatmulI8Workspace w = take_workspace(o);
  OPS_LAUNCH(o, launch_expand_rows(d_a, ld_a, m, k, w, o->stream));
  return each_part(o, a, first, [&](const MatmulI8Launch& p) { return launch_matmul_i8_tc(p, w, o->stream); });
}

rbf_status linear_i8_dev(rbf_ops* o, const void* d_x, rbf_dtype x_dtype, int64_t ld_x, const int8_t* d_w,
                         int64_t ld_w, const float* d_w_scale, const float* d_bias, void* d_out, rbf_dtype out_dtype,
                         int64_t ld_out, int64_t m, int64_t n, int32_t k) {
  if (!o || !float_dtype(x_dtype) || !float_dtype(out_dtype)) return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  MatmulI8Launch a;
  a.a = static_cast<const int8_t*>(o->rows_f16);
  a.ld_a = matmul_i8_pitch(k);
  a.a_scale = o->row_scale;
  a.b = d_w;
  a.ld_b = ld_w;
  a.b_scale = d_w_scale;
  a.bias = d_bias;
  a.out = d_out;
  a.out_dtype = out_dtype;
  a.ld_out = ld_out;
  a.m = m;
  a.n = n;
  a.k = k;
  if (rbf_status st = check_matmul(o, a)) return st;
  if (!matrix_ok(d_x, dtype_bytes(x_dtype), m, k, ld_x)) return RBF_ERR_INVALID_VALUE;
  if (m == 0 || n == 0) return RBF_OK;
  if (k == 0) {
    a.a_scale = nullptr;
    OPS_LAUNCH(o, launch_matmul_i8_empty(a, o->num_sms, o->stream));
    return RBF_OK;
  }
  const MatmulI8Launch first = first_part(o, a);
  if (matmul_i8_few_fits(first))
    return each_part(o, a, first, [&](const MatmulI8Launch& p) { return launch_matmul_i8_few(p, d_x, ld_x, x_dtype, o->num_sms, o->stream); });
  QuantizeLaunch q;
  q.x = d_x;
  q.dtype = x_dtype;
  q.ld_x = ld_x;
  q.rows = m;
  q.cols = k;
  q.scale = o->row_scale;
  const MatmulI8Workspace w = take_workspace(o);
  q.f16 = w.rows_f16;
  q.f16_pitch = matmul_i8_pitch(k);
  q.block_l1 = w.block_l1;
  OPS_LAUNCH(o, launch_quantize_rows(q, o->stream));
  return each_part(o, a, first, [&](const MatmulI8Launch& p) { return launch_matmul_i8_tc(p, w, o->stream); });
}

rbf_status sample_dev(rbf_ops* o, const void* d_logits, rbf_dtype dtype, int64_t ld, int64_t rows, int32_t vocab,
                      const float* d_u, const float* d_temperature, const int32_t* d_top_k, const float* d_top_p,
                      const float* d_min_p, int32_t* d_token, float* d_logprob) {
  if (!o || !float_dtype(dtype) || rows < 0 || rows > INT32_MAX || vocab < 0 || vocab > RBF_OPS_MAX_VOCAB)
    return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  if (!matrix_ok(d_logits, dtype_bytes(dtype), rows, vocab, ld)) return RBF_ERR_INVALID_VALUE;
  if (rows == 0) return RBF_OK;
  if (!d_u || !d_token || !floats_ok(d_u) || !floats_ok(d_temperature) || !floats_ok(d_top_k) || !floats_ok(d_top_p) ||
      !floats_ok(d_min_p) || !floats_ok(d_token) || !floats_ok(d_logprob))
    return RBF_ERR_INVALID_VALUE;
  SampleLaunch a;
  a.logits = d_logits;
  a.dtype = dtype;
  a.ld = ld;
  a.rows = rows;
  a.vocab = vocab;
  a.u = d_u;
  a.temperature = d_temperature;
  a.top_k = d_top_k;
  a.top_p = d_top_p;
  a.min_p = d_min_p;
  a.token = d_token;
  a.logprob = d_logprob;
  OPS_LAUNCH(o, launch_sample(a, o->stream));
  return RBF_OK;
}

rbf_status quantize_f8_dev(rbf_ops* o, const void* d_x, rbf_dtype x_dtype, int64_t ld_x, int64_t rows, int32_t cols,
                           int32_t block_rows, void* d_q, rbf_dtype q_dtype, int64_t ld_q, float* d_scale,
                           int64_t ld_scale) {
  if (!o || !float_dtype(x_dtype) || !f8_dtype(q_dtype) || rows < 0 || cols < 0 || rows > INT32_MAX ||
      (block_rows != 1 && block_rows != 128))
    return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  const int64_t scale_rows = block_rows == 1 ? rows : blocks_of(rows);
  if (!matrix_ok(d_x, dtype_bytes(x_dtype), rows, cols, ld_x) || !matrix_ok(d_q, 1, rows, cols, ld_q) ||
      !matrix_ok(d_scale, 4, scale_rows, blocks_of(cols), ld_scale))
    return RBF_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return RBF_OK;
  QuantizeF8Launch a;
  a.x = d_x;
  a.dtype = x_dtype;
  a.ld_x = ld_x;
  a.rows = rows;
  a.cols = cols;
  a.block_rows = block_rows;
  a.q = d_q;
  a.q_dtype = q_dtype;
  a.ld_q = ld_q;
  a.scale = d_scale;
  a.ld_scale = ld_scale;
  OPS_LAUNCH(o, launch_quantize_f8(a, o->num_sms, o->stream));
  return RBF_OK;
}

rbf_status matmul_f8_dev(rbf_ops* o, const void* d_a, rbf_dtype a_dtype, int64_t ld_a, const float* d_a_scale,
                         int64_t ld_a_scale, const void* d_b, rbf_dtype b_dtype, int64_t ld_b, const float* d_b_scale,
                         int64_t ld_b_scale, int32_t block_rows, const float* d_bias, void* d_out, rbf_dtype out_dtype,
                         int64_t ld_out, int64_t m, int64_t n, int32_t k) {
  if (!o || !f8_dtype(a_dtype) || !f8_dtype(b_dtype) || !float_dtype(out_dtype) || (block_rows != 1 && block_rows != 128))
    return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  if (m < 0 || n < 0 || k < 0 || m > o->max_rows || n > INT32_MAX || k > RBF_OPS_MAX_VOCAB) return RBF_ERR_INVALID_VALUE;
  const int64_t b_scale_rows = block_rows == 1 ? n : blocks_of(n);
  if (!matrix_ok(d_a, 1, m, k, ld_a) || !matrix_ok(d_b, 1, n, k, ld_b) ||
      !matrix_ok(d_out, dtype_bytes(out_dtype), m, n, ld_out) || !matrix_ok(d_a_scale, 4, m, blocks_of(k), ld_a_scale) ||
      !matrix_ok(d_b_scale, 4, b_scale_rows, blocks_of(k), ld_b_scale) || !floats_ok(d_bias))
    return RBF_ERR_INVALID_VALUE;
  if (m == 0 || n == 0) return RBF_OK;
  MatmulF8Launch a;
  a.a = static_cast<const uint8_t*>(d_a);
  a.a_dtype = a_dtype;
  a.ld_a = ld_a;
  a.a_scale = d_a_scale;
  a.ld_a_scale = ld_a_scale;
  a.b = static_cast<const uint8_t*>(d_b);
  a.b_dtype = b_dtype;
  a.ld_b = ld_b;
  a.b_scale = d_b_scale;
  a.ld_b_scale = ld_b_scale;
  a.block_rows = block_rows;
  a.bias = d_bias;
  a.out = d_out;
  a.out_dtype = out_dtype;
  a.ld_out = ld_out;
  a.m = m;
  a.n = n;
  a.k = k;
  if (k == 0) {
    MatmulI8Launch none;  // the bias, or zeros
    none.bias = d_bias;
    none.out = d_out;
    none.out_dtype = out_dtype;
    none.ld_out = ld_out;
    none.m = m;
    none.n = n;
    OPS_LAUNCH(o, launch_matmul_i8_empty(none, o->num_sms, o->stream));
    return RBF_OK;
  }
  MatmulF8Workspace w;
  w.partial = reinterpret_cast<float*>(o->partial);
  w.arrived = o->arrived;
  w.err = o->errw;
  w.num_sms = o->num_sms;
  w.timeout_ns = o->timeout_ns;
  const int pitch = (k + 15) / 16 * 16;
  if (m == 1) a.ld_a = pitch;
  // As many rows of b as a launch takes and, where they do not start on 16-byte
  // boundaries, as the room holds in which they are put on them. Rows of a have the
  // other products' room, max_rows x max_depth 16-bit numbers.
  const bool staged_a = !aligned(a.a, 16) || a.ld_a % 16 != 0, staged = !aligned(d_b, 16) || (n > 1 && ld_b % 16 != 0);
  int64_t most = std::min(n, matmul_f8_rows(m, k));
  if (staged) most = std::min<int64_t>(most, static_cast<int64_t>(kStagedBytes / pitch / 256 * 256));
  if (most < 1 || (staged_a && m * pitch > o->max_rows * matmul_i8_pitch(o->max_depth) * 2)) return RBF_ERR_INVALID_VALUE;
  if (staged_a) {
    OPS_LAUNCH(o, launch_pitch_rows(reinterpret_cast<const int8_t*>(a.a), a.ld_a, m, k, static_cast<int8_t*>(o->rows_f16), pitch,
                                    o->num_sms, o->stream));
    a.a = static_cast<const uint8_t*>(o->rows_f16);
    a.ld_a = pitch;
  }
  for (int64_t j = 0; j < n; j += most) {
    MatmulF8Launch part = a;
    part.n = std::min(most, n - j);
    part.b = a.b + j * ld_b;
    part.b_scale = d_b_scale + j / block_rows * ld_b_scale;
    part.bias = d_bias ? d_bias + j : nullptr;
    part.out = static_cast<char*>(d_out) + j * dtype_bytes(out_dtype);
    if (staged) {
      OPS_LAUNCH(o, launch_pitch_rows(reinterpret_cast<const int8_t*>(part.b), ld_b, part.n, k, o->staged, pitch, o->num_sms, o->stream));
      part.b = reinterpret_cast<const uint8_t*>(o->staged);
      part.ld_b = pitch;
    } else if (n == 1) {
      part.ld_b = pitch;
    }
    OPS_LAUNCH(o, launch_matmul_f8(part, w, o->stream));
  }
  return RBF_OK;
}

rbf_status verify_dev(rbf_ops* o, const void* d_target, int64_t ld_target_seq, int64_t ld_target, const void* d_draft,
                      int64_t ld_draft_seq, int64_t ld_draft, rbf_dtype dtype, int64_t seqs, int32_t drafts,
                      int32_t vocab, const int32_t* d_draft_token, const int32_t* d_draft_count, const float* d_u,
                      const float* d_temperature, int32_t* d_token, int32_t* d_accepted, float* d_logprob) {
  if (!o || !float_dtype(dtype) || seqs < 0 || drafts < 0 || drafts > RBF_OPS_MAX_DRAFTS || vocab < 0 ||
      vocab > RBF_OPS_MAX_VOCAB)
    return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  if (seqs > o->max_rows / (drafts + 1)) return RBF_ERR_INVALID_VALUE;
  if (seqs == 0) return RBF_OK;
  const int elem = dtype_bytes(dtype);
  // Places of a sequence are rows, sequences rows of those.
  if (!matrix_ok(d_target, elem, drafts + 1, vocab, ld_target) ||
      !matrix_ok(d_target, elem, seqs, std::min<int64_t>(vocab, 1) * (drafts * ld_target + vocab), ld_target_seq))
    return RBF_ERR_INVALID_VALUE;
  if (d_draft && (!matrix_ok(d_draft, elem, drafts, vocab, ld_draft) ||
                  !matrix_ok(d_draft, elem, seqs, std::min<int64_t>(vocab, 1) * std::min(drafts, 1) * ((drafts - 1) * ld_draft + vocab), ld_draft_seq)))
    return RBF_ERR_INVALID_VALUE;
  if ((drafts > 0 && !d_draft_token) || !d_u || !d_token || !d_accepted || !floats_ok(d_draft_token) ||
      !floats_ok(d_draft_count) || !floats_ok(d_u) || !floats_ok(d_temperature) || !floats_ok(d_token) ||
      !floats_ok(d_accepted) || !floats_ok(d_logprob))
    return RBF_ERR_INVALID_VALUE;
  VerifyLaunch a;
  a.target = d_target;
  a.ld_target_seq = ld_target_seq;
  a.ld_target = ld_target;
  a.draft = drafts > 0 ? d_draft : nullptr;
  a.ld_draft_seq = ld_draft_seq;
  a.ld_draft = ld_draft;
  a.dtype = dtype;
  a.seqs = seqs;
  a.drafts = drafts;
  a.vocab = vocab;
  a.draft_token = d_draft_token;
  a.count = d_draft_count;
  a.u = d_u;
  a.temperature = d_temperature;
  a.token = d_token;
  a.accepted = d_accepted;
  a.logprob = d_logprob;
  OPS_LAUNCH(o, launch_verify_stats(a, o->parts, verify_max_parts(o->max_rows, o->num_sms), o->num_sms, o->stream));
  OPS_LAUNCH(o, launch_verify_draw(a, o->parts, verify_max_parts(o->max_rows, o->num_sms), o->num_sms, o->stream));
  return RBF_OK;
}

rbf_status distill_dev(rbf_ops* o, const void* d_scores, rbf_dtype dtype, int64_t ld_scores, int64_t rows, int32_t vocab,
                       const int32_t* d_index, int64_t ld_index, const void* d_teacher, rbf_dtype teacher_dtype,
                       int64_t ld_teacher, int32_t k, const float* d_rest, const float* d_weight, float temperature,
                       float* d_loss, void* d_grad, int64_t ld_grad) {
  if (!o || !float_dtype(dtype) || !float_dtype(teacher_dtype) || rows < 0 || rows > INT32_MAX || vocab < 0 ||
      vocab > RBF_OPS_MAX_VOCAB || k < 0 || k > RBF_OPS_MAX_TEACHER || !(temperature >= 0x1p-20f && temperature <= 0x1p20f))
    return RBF_ERR_INVALID_VALUE;
  o->launches = 0;
  if (!on_its_device(o)) return RBF_ERR_INVALID_VALUE;
  const int elem = dtype_bytes(dtype);
  if (!matrix_ok(d_scores, elem, rows, vocab, ld_scores) || (d_grad && !matrix_ok(d_grad, elem, rows, vocab, ld_grad)) ||
      !matrix_ok(d_index, 4, rows, k, ld_index) || !matrix_ok(d_teacher, dtype_bytes(teacher_dtype), rows, k, ld_teacher))
    return RBF_ERR_INVALID_VALUE;
  if (!floats_ok(d_rest) || !floats_ok(d_weight) || !floats_ok(d_loss)) return RBF_ERR_INVALID_VALUE;
  if (rows == 0 || (!d_loss && !d_grad)) return RBF_OK;
  DistillLaunch a;
  a.scores = d_scores;
  a.dtype = dtype;
  a.ld_scores = ld_scores;
  a.rows = rows;
  a.vocab = vocab;
  a.index = d_index;
  a.ld_index = ld_index;
  a.teacher = d_teacher;
  a.teacher_dtype = teacher_dtype;
  a.ld_teacher = ld_teacher;
  a.k = k;
  a.rest = d_rest;
  a.weight = d_weight;
  a.temperature = temperature;
  a.loss = d_loss;
  a.grad = d_grad;
  a.ld_grad = ld_grad;
  OPS_LAUNCH(o, launch_distill(a, o->errw, o->timeout_ns, o->num_sms, o->stream));
  return RBF_OK;
}

}  // extern "C"
