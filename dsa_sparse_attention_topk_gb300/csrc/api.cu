// C ABI entry points (include/dsa.h): argument checking, the device status word and
// the per-thread error message.  Every compute step runs in the kernels behind
// dsa_launch.h; nothing here touches tensor data on the host.

#include <atomic>
#include <cstdint>
#include <cstdarg>
#include <cstdio>
#include <cmath>
#include <mutex>
#include <string>

#include "dsa_common.cuh"
#include "dsa_launch.h"

namespace {

__device__ unsigned g_status_word;

thread_local std::string t_last_error;

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(DSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Device address of the status word, looked up once per device with that device current.
unsigned* status_ptr() {
  static std::mutex mu;
  static unsigned* ptrs[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<unsigned*>(p);
  }
  return ptrs[dev];
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// dsa_test_stall_indexer: 0 = normal operation, else the waits' limit in microseconds with
// the indexer's copy producer stalled
std::atomic<int> g_stall_wait_us{0};

void apply_test_hooks(dsa::IndexerArgs& a) {
  const int us = g_stall_wait_us.load(std::memory_order_relaxed);
  if (us > 0) {
    a.wait_ns = static_cast<uint64_t>(us) * 1000ull;
    a.stall_producer = 1;
  }
}

}  // namespace

bool dsa::device_info(DevInfo* out, const char** err) {
  static std::mutex mu;
  static DevInfo cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    *err = "no current CUDA device";
    return false;
  }
  if (dev < 0 || dev >= 64) {
    *err = "device ordinal out of range (the library serves ordinals 0..63)";
    return false;
  }
  std::lock_guard<std::mutex> lock(mu);
  DevInfo& d = cache[dev];
  if (!d.n_sm) {
    DevInfo q;
    if (cudaDeviceGetAttribute(&q.n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&q.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        q.n_sm <= 0) {
      *err = "device attribute query failed";
      return false;
    }
    d = q;
  }
  *out = d;
  return true;
}

extern "C" {

int dsa_version(void) { return 101; }

const char* dsa_last_error(void) { return t_last_error.c_str(); }

int dsa_quant_kv_mxfp8(const void* k_bf16, const int64_t* slot_mapping, int32_t n_tokens,
                       uint8_t* k_cache, int64_t num_slots, void* stream) {
  if (n_tokens < 0) return fail(DSA_ERR_INVALID_ARG, "quant_kv_mxfp8: n_tokens < 0");
  if (n_tokens == 0) return DSA_OK;
  if (!k_bf16 || !slot_mapping || !k_cache) return fail(DSA_ERR_INVALID_ARG, "quant_kv_mxfp8: null pointer");
  if (!aligned(k_bf16, 16) || !aligned(k_cache, 16) || !aligned(slot_mapping, 8))
    return fail(DSA_ERR_INVALID_ARG, "quant_kv_mxfp8: k_bf16/k_cache must be 16-byte aligned");
  if (num_slots <= 0 || num_slots % DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "quant_kv_mxfp8: num_slots must be a positive multiple of 64");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "quant_kv_mxfp8: no CUDA device");
  cudaError_t e = dsa::launch_quant_mxfp8(k_bf16, slot_mapping, n_tokens, k_cache, num_slots, st,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "quant_kv_mxfp8 launch");
}

int dsa_quant_kv_fp8(const void* kv_bf16, const int64_t* slot_mapping, int32_t n_tokens,
                     uint8_t* kv_cache, int64_t num_slots, void* stream) {
  if (n_tokens < 0) return fail(DSA_ERR_INVALID_ARG, "quant_kv_fp8: n_tokens < 0");
  if (n_tokens == 0) return DSA_OK;
  if (!kv_bf16 || !slot_mapping || !kv_cache) return fail(DSA_ERR_INVALID_ARG, "quant_kv_fp8: null pointer");
  if (!aligned(kv_bf16, 16) || !aligned(kv_cache, 16) || !aligned(slot_mapping, 8))
    return fail(DSA_ERR_INVALID_ARG, "quant_kv_fp8: kv_bf16/kv_cache must be 16-byte aligned");
  if (num_slots <= 0 || num_slots % DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "quant_kv_fp8: num_slots must be a positive multiple of 64");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "quant_kv_fp8: no CUDA device");
  cudaError_t e = dsa::launch_quant_fp8(kv_bf16, slot_mapping, n_tokens, kv_cache, num_slots, st,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "quant_kv_fp8 launch");
}

int dsa_quant_kv(const void* k_bf16, const void* kv_bf16, const int64_t* slot_mapping, int32_t n_tokens,
                 uint8_t* k_cache, uint8_t* kv_cache, int64_t num_slots, void* stream) {
  if (n_tokens < 0) return fail(DSA_ERR_INVALID_ARG, "quant_kv: n_tokens < 0");
  if (n_tokens == 0) return DSA_OK;
  if (!k_bf16 || !kv_bf16 || !slot_mapping || !k_cache || !kv_cache)
    return fail(DSA_ERR_INVALID_ARG, "quant_kv: null pointer");
  if (!aligned(k_bf16, 16) || !aligned(kv_bf16, 16) || !aligned(k_cache, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8))
    return fail(DSA_ERR_INVALID_ARG, "quant_kv: rows and caches must be 16-byte aligned");
  if (num_slots <= 0 || num_slots % DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "quant_kv: num_slots must be a positive multiple of 64");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "quant_kv: no CUDA device");
  cudaError_t e = dsa::launch_quant_both(k_bf16, kv_bf16, slot_mapping, n_tokens, k_cache, kv_cache, num_slots, st,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "quant_kv launch");
}

// n elements `stride` apart, none more than 2^40 elements behind the first
static bool spans(int64_t stride, int32_t n) {
  const int64_t most = int64_t{1} << 40;
  return stride >= 0 && stride <= (n > 1 ? most / (n - 1) : most);
}

// [n][h] rows of d elements, of which no two share memory: the strides nest
static bool rows_apart(int64_t stride_t, int n, int64_t stride_h, int h, int d) {
  auto nests = [d](int64_t in, int n_in, int64_t over, int n_over) {
    return (n_in == 1 || in >= d) && (n_over == 1 || over >= (n_in - 1) * in + d);
  };
  return nests(stride_h, h, stride_t, n) || nests(stride_t, n, stride_h, h);
}

int dsa_rope(const void* x, void* out, int32_t dtype, int32_t n, int32_t h, int32_t d, int64_t x_stride_t,
             int64_t x_stride_h, int64_t out_stride_t, int64_t out_stride_h, const int32_t* pos,
             const int64_t* turns, int32_t rot, int32_t offset, int32_t layout, float amplitude,
             int32_t transpose, void* stream) {
  if (n < 0 || h < 0) return fail(DSA_ERR_INVALID_ARG, "rope: negative n or h");
  if (dtype < DSA_DTYPE_BF16 || dtype > DSA_DTYPE_FP32)
    return fail(DSA_ERR_UNSUPPORTED, "rope: dtype must be bf16, fp16 or fp32");
  if (d < 2 || d > 65536) return fail(DSA_ERR_UNSUPPORTED, "rope: d must be 2..65536 (got %d)", d);
  if (rot < 2 || rot % 2 || rot > d || offset < 0 || offset > d - rot)
    return fail(DSA_ERR_INVALID_ARG, "rope: rot must be even and [offset, offset + rot) lie in [0, %d)", d);
  if (layout != DSA_ROPE_INTERLEAVED && layout != DSA_ROPE_HALF)
    return fail(DSA_ERR_INVALID_ARG, "rope: unknown layout %d", layout);
  if (!std::isfinite(amplitude)) return fail(DSA_ERR_INVALID_ARG, "rope: amplitude must be finite");
  if (n == 0 || h == 0) return DSA_OK;
  if (static_cast<int64_t>(n) * h > INT32_MAX)
    return fail(DSA_ERR_UNSUPPORTED, "rope: n * h must be below 2^31");
  if (!x || !out || !pos || !turns) return fail(DSA_ERR_INVALID_ARG, "rope: null pointer");
  const size_t size = dtype == DSA_DTYPE_FP32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(out, size) || !aligned(pos, 4) || !aligned(turns, 8))
    return fail(DSA_ERR_INVALID_ARG, "rope: a pointer is not aligned to its element");
  // (axes of up to 2^40 elements keep every offset far from overflow)
  if (!spans(x_stride_t, n) || !spans(x_stride_h, h) || !spans(out_stride_t, n) || !spans(out_stride_h, h))
    return fail(DSA_ERR_INVALID_ARG, "rope: a stride is negative, or an axis longer than 2^40 elements");
  // strides of an axis of length 1 are never used
  if (n == 1) x_stride_t = out_stride_t = 0;
  if (h == 1) x_stride_h = out_stride_h = 0;
  if (!rows_apart(out_stride_t, n, out_stride_h, h, d))
    return fail(DSA_ERR_INVALID_ARG, "rope: the strides of out let its elements overlap");
  if (x == out && (x_stride_t != out_stride_t || x_stride_h != out_stride_h))
    return fail(DSA_ERR_INVALID_ARG, "rope: in place, x and out need the same strides");
  dsa::RopeArgs a{x, out, dtype, n, h, d, x_stride_t, x_stride_h, out_stride_t, out_stride_h, pos, turns, rot, offset,
                  layout, amplitude, transpose};
  cudaError_t e = dsa::launch_rope(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "rope launch");
}

// What the norm with rotation and its gradient check alike; `who` names the entry.
static int check_norm(const char* who, const dsa::NormArgs& a) {
  if (a.n < 0 || a.h < 0) return fail(DSA_ERR_INVALID_ARG, "%s: negative n or h", who);
  if (a.dtype < DSA_DTYPE_BF16 || a.dtype > DSA_DTYPE_FP32 || a.w_dtype < DSA_DTYPE_BF16 || a.w_dtype > DSA_DTYPE_FP32)
    return fail(DSA_ERR_UNSUPPORTED, "%s: dtypes must be bf16, fp16 or fp32", who);
  if (a.d < 2 || a.d > 1024) return fail(DSA_ERR_UNSUPPORTED, "%s: d must be 2..1024 (got %d)", who, a.d);
  if (a.span < 1 || a.span > a.d) return fail(DSA_ERR_INVALID_ARG, "%s: norm_dim must lie in 1..%d (got %d)", who, a.d, a.span);
  if (a.rot < 2 || a.rot % 2 || a.rot > a.d || a.offset < 0 || a.offset > a.d - a.rot)
    return fail(DSA_ERR_INVALID_ARG, "%s: rot must be even and [offset, offset + rot) lie in [0, %d)", who, a.d);
  if (a.layout != DSA_ROPE_INTERLEAVED && a.layout != DSA_ROPE_HALF)
    return fail(DSA_ERR_INVALID_ARG, "%s: unknown layout %d", who, a.layout);
  if (a.center != 0 && a.center != 1) return fail(DSA_ERR_INVALID_ARG, "%s: center must be 0 or 1", who);
  if (!std::isfinite(a.amplitude) || !std::isfinite(a.eps) || a.eps < 0.f)
    return fail(DSA_ERR_INVALID_ARG, "%s: amplitude must be finite, eps finite and not negative", who);
  if (static_cast<int64_t>(a.n) * a.h > INT32_MAX) return fail(DSA_ERR_UNSUPPORTED, "%s: n * h must be below 2^31", who);
  const size_t wsize = a.w_dtype == DSA_DTYPE_FP32 ? 4 : 2;
  if (!aligned(a.weight, wsize) || !aligned(a.bias, wsize) || !aligned(a.dweight, 4) || !aligned(a.dbias, 4))
    return fail(DSA_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", who);
  if (a.n == 0 || a.h == 0) return DSA_OK;
  if (!a.x || !a.out || !a.pos || !a.turns) return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", who);
  const size_t size = a.dtype == DSA_DTYPE_FP32 ? 4 : 2;
  if (!aligned(a.x, size) || !aligned(a.dy, size) || !aligned(a.out, size) || !aligned(a.pos, 4) || !aligned(a.turns, 8))
    return fail(DSA_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", who);
  if (!spans(a.x_stride_t, a.n) || !spans(a.x_stride_h, a.h) || !spans(a.dy_stride_t, a.n) || !spans(a.dy_stride_h, a.h) ||
      !spans(a.out_stride_t, a.n) || !spans(a.out_stride_h, a.h))
    return fail(DSA_ERR_INVALID_ARG, "%s: a stride is negative, or an axis longer than 2^40 elements", who);
  if (!rows_apart(a.out_stride_t, a.n, a.out_stride_h, a.h, a.d))
    return fail(DSA_ERR_INVALID_ARG, "%s: the strides of the result let its elements overlap", who);
  auto differ = [&](const void* p, int64_t st, int64_t sh) {
    return p == a.out && ((a.n > 1 && st != a.out_stride_t) || (a.h > 1 && sh != a.out_stride_h));
  };
  if (differ(a.x, a.x_stride_t, a.x_stride_h) || differ(a.dy, a.dy_stride_t, a.dy_stride_h))
    return fail(DSA_ERR_INVALID_ARG, "%s: in place, the result needs the strides of what it replaces", who);
  return DSA_OK;
}
// strides of an axis of length 1 are never used
static void drop_unused_strides(dsa::NormArgs& a) {
  if (a.n == 1) a.x_stride_t = a.dy_stride_t = a.out_stride_t = 0;
  if (a.h == 1) a.x_stride_h = a.dy_stride_h = a.out_stride_h = 0;
}

int dsa_norm_rope(const void* x, void* out, int32_t dtype, int32_t n, int32_t h, int32_t d, int64_t x_stride_t,
                  int64_t x_stride_h, int64_t out_stride_t, int64_t out_stride_h, const void* weight, const void* bias,
                  int32_t w_dtype, int32_t norm_dim, int32_t center, float eps, const int32_t* pos, const int64_t* turns,
                  int32_t rot, int32_t offset, int32_t layout, float amplitude, void* stream) {
  dsa::NormArgs a{x, nullptr, out, dtype, n, h, d, x_stride_t, x_stride_h, 0, 0, out_stride_t, out_stride_h, pos, turns, rot,
                  offset, layout, amplitude, norm_dim, center, eps, weight, bias, w_dtype, nullptr, nullptr, nullptr};
  const int rc = check_norm("norm_rope", a);
  if (rc || n == 0 || h == 0) return rc;
  drop_unused_strides(a);
  cudaError_t e = dsa::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "norm_rope launch");
}

size_t dsa_norm_rope_grad_workspace_size(int32_t norm_dim) {
  return norm_dim < 1 || norm_dim > 1024 ? 0 : dsa::norm_grad_workspace_bytes(norm_dim);
}

int dsa_norm_rope_grad(const void* dy, const void* x, void* dx, int32_t dtype, int32_t n, int32_t h, int32_t d,
                       int64_t dy_stride_t, int64_t dy_stride_h, int64_t x_stride_t, int64_t x_stride_h,
                       int64_t dx_stride_t, int64_t dx_stride_h, const void* weight, int32_t w_dtype, int32_t norm_dim,
                       int32_t center, float eps, const int32_t* pos, const int64_t* turns, int32_t rot, int32_t offset,
                       int32_t layout, float amplitude, float* dweight, float* dbias, void* workspace,
                       size_t workspace_bytes, void* stream) {
  dsa::NormArgs a{x, dy, dx, dtype, n, h, d, x_stride_t, x_stride_h, dy_stride_t, dy_stride_h, dx_stride_t, dx_stride_h, pos,
                  turns, rot, offset, layout, amplitude, norm_dim, center, eps, weight, nullptr, w_dtype, dweight, dbias,
                  static_cast<float*>(workspace)};
  const int rc = check_norm("norm_rope_grad", a);
  if (rc) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (n == 0 || h == 0) {  // the sums over no rows
    if (dweight) e = cudaMemsetAsync(dweight, 0, sizeof(float) * norm_dim, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * norm_dim, s);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "norm_rope_grad");
  }
  if (!dy) return fail(DSA_ERR_INVALID_ARG, "norm_rope_grad: null pointer");
  const size_t need = dsa::norm_grad_workspace_bytes(norm_dim);
  if ((dweight || dbias) && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(DSA_ERR_INVALID_ARG, "norm_rope_grad: workspace must be >= %zu bytes and 256-byte aligned", need);
  drop_unused_strides(a);
  e = dsa::launch_norm_rope_grad(a, s);
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "norm_rope_grad launch");
}

static int check_rope_quant(const char* who, const void* k_bf16, int64_t k_stride, const void* kv_bf16, int64_t kv_stride,
                            const int32_t* pos, const int64_t* slot_mapping, int32_t n_tokens, const uint8_t* k_cache,
                            const uint8_t* kv_cache, int64_t num_slots, const int64_t* turns, float amplitude,
                            int32_t k_offset, int32_t k_layout, int32_t kv_layout) {
  if (n_tokens < 0) return fail(DSA_ERR_INVALID_ARG, "%s: n_tokens < 0", who);
  if (k_offset < 0 || k_offset > DSA_INDEX_DIM - 64 || k_offset % 4)
    return fail(DSA_ERR_INVALID_ARG, "%s: k_offset must be a multiple of 4 in 0..64 (got %d)", who, k_offset);
  if ((k_layout != DSA_ROPE_INTERLEAVED && k_layout != DSA_ROPE_HALF) ||
      (kv_layout != DSA_ROPE_INTERLEAVED && kv_layout != DSA_ROPE_HALF))
    return fail(DSA_ERR_INVALID_ARG, "%s: unknown layout", who);
  if (!std::isfinite(amplitude)) return fail(DSA_ERR_INVALID_ARG, "%s: amplitude must be finite", who);
  if (n_tokens == 0) return DSA_OK;
  if (!pos || !slot_mapping || !turns || (!k_bf16 && !kv_bf16) || (k_bf16 && !k_cache) || (kv_bf16 && !kv_cache))
    return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(k_bf16, 8) || !aligned(kv_bf16, 8) || !aligned(k_cache, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8) || !aligned(turns, 8) || !aligned(pos, 4))
    return fail(DSA_ERR_INVALID_ARG, "%s: rows must be 8-byte and caches 16-byte aligned", who);
  if ((k_bf16 && (!spans(k_stride, n_tokens) || k_stride % 4)) ||
      (kv_bf16 && (!spans(kv_stride, n_tokens) || kv_stride % 4)))
    return fail(DSA_ERR_INVALID_ARG, "%s: row strides must be multiples of 4 elements, all rows within 2^40", who);
  if (num_slots <= 0 || num_slots % DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "%s: num_slots must be a positive multiple of 64", who);
  return DSA_OK;
}

int dsa_rope_quant_kv(const void* k_bf16, int64_t k_stride, const void* kv_bf16, int64_t kv_stride,
                      const int32_t* pos, const int64_t* slot_mapping, int32_t n_tokens, uint8_t* k_cache,
                      uint8_t* kv_cache, int64_t num_slots, const int64_t* turns, float amplitude,
                      int32_t k_offset, int32_t k_layout, int32_t kv_layout, void* stream) {
  const int rc = check_rope_quant("rope_quant_kv", k_bf16, k_stride, kv_bf16, kv_stride, pos, slot_mapping, n_tokens, k_cache,
                                  kv_cache, num_slots, turns, amplitude, k_offset, k_layout, kv_layout);
  if (rc || n_tokens == 0) return rc;
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "rope_quant_kv: no CUDA device");
  dsa::RopeQuantArgs a{k_bf16, k_stride, kv_bf16, kv_stride, pos, slot_mapping, n_tokens, k_cache, kv_cache, num_slots,
                       turns, amplitude, k_offset, k_layout, kv_layout, st};
  cudaError_t e = dsa::launch_rope_quant(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "rope_quant_kv launch");
}

static int check_indexer(const char* who, const void* q_bf16, const float* w, int32_t n_q, int32_t h_i,
                         int32_t q_group, const uint8_t* k_cache, int64_t num_pages,
                         const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                         const int32_t* q_seq, const int32_t* q_pos, int32_t n_seq, int32_t max_ctx) {
  if (n_q < 0 || n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "%s: negative n_q or n_seq", who);
  if (h_i < 1 || h_i > 64) return fail(DSA_ERR_UNSUPPORTED, "%s: h_i must be 1..64 (got %d)", who, h_i);
  if (q_group < 1 || q_group > 4) return fail(DSA_ERR_UNSUPPORTED, "%s: q_group must be 1..4", who);
  if (q_group * h_i > 256) return fail(DSA_ERR_UNSUPPORTED, "%s: q_group * h_i must be <= 256", who);
  if (n_q % q_group) return fail(DSA_ERR_INVALID_ARG, "%s: n_q must be a multiple of q_group", who);
  if (max_ctx < 1 || max_ctx > 262144) return fail(DSA_ERR_UNSUPPORTED, "%s: max_ctx must be 1..262144", who);
  if (max_pages < (max_ctx + DSA_PAGE_SIZE - 1) / DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "%s: max_pages < ceil(max_ctx / 64)", who);
  if (num_pages < 1) return fail(DSA_ERR_INVALID_ARG, "%s: num_pages must be >= 1", who);
  if (n_q == 0) return DSA_OK;
  if (!q_bf16 || !w || !k_cache || !page_table || !seq_lens || !q_seq || !q_pos)
    return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(q_bf16, 16) || !aligned(k_cache, 16) || !aligned(w, 4))
    return fail(DSA_ERR_INVALID_ARG, "%s: q_bf16 and k_cache must be 16-byte aligned", who);
  return DSA_OK;
}

int dsa_indexer_topk(const void* q_bf16, const float* w, int32_t n_q, int32_t h_i,
                     int32_t q_group, const uint8_t* k_cache, int64_t num_pages,
                     const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                     const int32_t* q_seq, const int32_t* q_pos, int32_t n_seq,
                     int32_t max_ctx, int32_t topk, int32_t* out_idx, float* out_scores,
                     void* stream) {
  int rc = check_indexer("indexer_topk", q_bf16, w, n_q, h_i, q_group, k_cache, num_pages, page_table,
                         max_pages, seq_lens, q_seq, q_pos, n_seq, max_ctx);
  if (rc) return rc;
  if (topk < 1 || topk > 2048) return fail(DSA_ERR_UNSUPPORTED, "indexer_topk: topk must be 1..2048");
  if (n_q == 0) return DSA_OK;
  if (!out_idx) return fail(DSA_ERR_INVALID_ARG, "indexer_topk: out_idx is null");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "indexer_topk: no CUDA device");
  dsa::IndexerArgs a{q_bf16, w, n_q, h_i, q_group, k_cache, num_pages, page_table, max_pages,
                     seq_lens, q_seq, q_pos, n_seq, max_ctx, topk, out_idx, out_scores, nullptr, st};
  apply_test_hooks(a);
  const char* why = nullptr;
  cudaError_t e = dsa::launch_indexer(a, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "indexer_topk launch");
  return DSA_OK;
}

int dsa_indexer_scores(const void* q_bf16, const float* w, int32_t n_q, int32_t h_i,
                       int32_t q_group, const uint8_t* k_cache, int64_t num_pages,
                       const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                       const int32_t* q_seq, const int32_t* q_pos, int32_t n_seq,
                       int32_t max_ctx, float* out_scores, void* stream) {
  int rc = check_indexer("indexer_scores", q_bf16, w, n_q, h_i, q_group, k_cache, num_pages, page_table,
                         max_pages, seq_lens, q_seq, q_pos, n_seq, max_ctx);
  if (rc) return rc;
  if (n_q == 0) return DSA_OK;
  if (!out_scores) return fail(DSA_ERR_INVALID_ARG, "indexer_scores: out_scores is null");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "indexer_scores: no CUDA device");
  dsa::IndexerArgs a{q_bf16, w, n_q, h_i, q_group, k_cache, num_pages, page_table, max_pages,
                     seq_lens, q_seq, q_pos, n_seq, max_ctx, 1, nullptr, nullptr, out_scores, st};
  apply_test_hooks(a);
  const char* why = nullptr;
  cudaError_t e = dsa::launch_indexer(a, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "indexer_scores launch");
  return DSA_OK;
}

size_t dsa_sparse_attn_workspace_size(int32_t n_q, int32_t h_s, int32_t topk) {
  if (n_q <= 0 || h_s <= 0 || topk <= 0) return 0;
  return dsa::sfa_workspace_bytes(n_q, h_s, topk);
}

int dsa_sparse_attn(const void* q_bf16, int32_t n_q, int32_t h_s, const uint8_t* kv_cache,
                    int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                    const int32_t* seq_lens, const int32_t* q_seq, int32_t n_seq,
                    const int32_t* topk_idx, int32_t topk, float sm_scale, void* out_bf16,
                    float* out_lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (n_q < 0 || n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "sparse_attn: negative n_q or n_seq");
  if (h_s < 1 || h_s > 128) return fail(DSA_ERR_UNSUPPORTED, "sparse_attn: h_s must be 1..128");
  if (topk < 1 || topk > 65536) return fail(DSA_ERR_UNSUPPORTED, "sparse_attn: topk must be 1..65536");
  if (max_pages < 1 || num_pages < 1) return fail(DSA_ERR_INVALID_ARG, "sparse_attn: max_pages and num_pages must be >= 1");
  if (!(sm_scale > 0.f) || sm_scale != sm_scale) return fail(DSA_ERR_INVALID_ARG, "sparse_attn: sm_scale must be positive");
  if (n_q == 0) return DSA_OK;
  if (!q_bf16 || !kv_cache || !page_table || !seq_lens || !q_seq || !topk_idx || !out_bf16)
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn: null pointer");
  if (!aligned(q_bf16, 16) || !aligned(kv_cache, 16) || !aligned(out_bf16, 16))
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn: q, kv_cache and out must be 16-byte aligned");
  const size_t need = dsa::sfa_workspace_bytes(n_q, h_s, topk);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn: workspace must be >= %zu bytes and 256-byte aligned", need);
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "sparse_attn: no CUDA device");
  dsa::SfaArgs a{q_bf16, n_q, h_s, kv_cache, num_pages, page_table, max_pages, seq_lens, q_seq, n_seq,
                 topk_idx, topk, sm_scale, out_bf16, out_lse, workspace, workspace_bytes, st};
  const char* why = nullptr;
  cudaError_t e = dsa::launch_sfa(a, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "sparse_attn launch");
  return DSA_OK;
}

int dsa_decode_step(const void* k_new_bf16, const void* kv_new_bf16, const int64_t* slot_mapping, int32_t n_new,
                    uint8_t* k_cache, uint8_t* kv_cache, int64_t num_pages, const int32_t* page_table,
                    int32_t max_pages, const int32_t* seq_lens, int32_t n_seq, int32_t max_ctx, int32_t n_q,
                    const int32_t* q_seq, const int32_t* q_pos, int32_t q_group, const void* q_idx_bf16,
                    const float* w, int32_t h_i, int32_t topk, int32_t* out_idx, const void* q_sfa_bf16,
                    int32_t h_s, float sm_scale, void* out_bf16, float* out_lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  // every argument is checked before anything is launched
  if (n_new < 0) return fail(DSA_ERR_INVALID_ARG, "decode_step: n_new < 0");
  if (num_pages < 1 || num_pages > INT64_MAX / DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "decode_step: num_pages must be >= 1");
  if (n_new > 0) {
    if (!k_new_bf16 || !kv_new_bf16 || !slot_mapping || !k_cache || !kv_cache)
      return fail(DSA_ERR_INVALID_ARG, "decode_step: null pointer among the new tokens or caches");
    if (!aligned(k_new_bf16, 16) || !aligned(kv_new_bf16, 16) || !aligned(k_cache, 16) || !aligned(kv_cache, 16) ||
        !aligned(slot_mapping, 8))
      return fail(DSA_ERR_INVALID_ARG, "decode_step: rows and caches must be 16-byte aligned");
  }
  int rc = check_indexer("decode_step", q_idx_bf16, w, n_q, h_i, q_group, k_cache, num_pages, page_table,
                         max_pages, seq_lens, q_seq, q_pos, n_seq, max_ctx);
  if (rc) return rc;
  if (topk < 1 || topk > 2048) return fail(DSA_ERR_UNSUPPORTED, "decode_step: topk must be 1..2048");
  if (h_s < 1 || h_s > 128) return fail(DSA_ERR_UNSUPPORTED, "decode_step: h_s must be 1..128");
  if (!(sm_scale > 0.f) || sm_scale != sm_scale) return fail(DSA_ERR_INVALID_ARG, "decode_step: sm_scale must be positive");
  if (n_q > 0) {
    if (!out_idx || !q_sfa_bf16 || !kv_cache || !out_bf16) return fail(DSA_ERR_INVALID_ARG, "decode_step: null pointer");
    if (!aligned(q_sfa_bf16, 16) || !aligned(kv_cache, 16) || !aligned(out_bf16, 16))
      return fail(DSA_ERR_INVALID_ARG, "decode_step: q_sfa, kv_cache and out must be 16-byte aligned");
    const size_t need = dsa::sfa_workspace_bytes(n_q, h_s, topk);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
      return fail(DSA_ERR_INVALID_ARG, "decode_step: workspace must be >= %zu bytes and 256-byte aligned", need);
  }
  if (n_new == 0 && n_q == 0) return DSA_OK;  // nothing to launch
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "decode_step: no CUDA device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // one new token per query row (token i is row i's own token): the indexer writes them
  // itself, each before it loads the page that holds it; otherwise a writer launch first
  const bool fuse = n_new > 0 && n_new == n_q;
  cudaError_t e = cudaSuccess;
  if (!fuse) {
    e = dsa::launch_quant_both(k_new_bf16, kv_new_bf16, slot_mapping, n_new, k_cache, kv_cache,
                               num_pages * DSA_PAGE_SIZE, st, s);
    if (e != cudaSuccess) return cuda_fail(e, "decode_step: cache writer launch");
  }
  if (n_q == 0) return DSA_OK;
  dsa::IndexerArgs ia{q_idx_bf16, w, n_q, h_i, q_group, k_cache, num_pages, page_table, max_pages,
                      seq_lens, q_seq, q_pos, n_seq, max_ctx, topk, out_idx, nullptr, nullptr, st};
  if (fuse) {
    ia.fuse_writes = 1;
    ia.k_new = k_new_bf16;
    ia.kv_new = kv_new_bf16;
    ia.slot_mapping = slot_mapping;
    ia.kv_cache = kv_cache;
    ia.num_slots = num_pages * DSA_PAGE_SIZE;
  } else {
    ia.early_inputs = n_new > 0 ? 1 : 0;  // the writer launched just above precedes the indexer
  }
  apply_test_hooks(ia);
  const char* why = nullptr;
  e = dsa::launch_indexer(ia, s, &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "decode_step: indexer launch");
  dsa::SfaArgs sa{q_sfa_bf16, n_q, h_s, kv_cache, num_pages, page_table, max_pages, seq_lens, q_seq, n_seq,
                  out_idx, topk, sm_scale, out_bf16, out_lse, workspace, workspace_bytes, st};
  e = dsa::launch_sfa(sa, s, &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "decode_step: sparse_attn launch");
  return DSA_OK;
}

int dsa_sparse_attn_noalloc(const void* q_bf16, int32_t n_q, int32_t h_s, const uint8_t* kv_cache,
                            int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                            const int32_t* seq_lens, const int32_t* q_seq, int32_t n_seq,
                            const int32_t* topk_idx, int32_t topk, float sm_scale, void* out_bf16,
                            float* out_lse, void* stream) {
  if (n_q < 0 || n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "sparse_attn_noalloc: negative n_q or n_seq");
  if (h_s < 1 || h_s > 128) return fail(DSA_ERR_UNSUPPORTED, "sparse_attn_noalloc: h_s must be 1..128");
  if (topk < 1 || topk > 65536) return fail(DSA_ERR_UNSUPPORTED, "sparse_attn_noalloc: topk must be 1..65536");
  if (max_pages < 1 || num_pages < 1)
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn_noalloc: max_pages and num_pages must be >= 1");
  if (!(sm_scale > 0.f) || sm_scale != sm_scale)
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn_noalloc: sm_scale must be positive");
  if (n_q == 0) return DSA_OK;
  if (!q_bf16 || !kv_cache || !page_table || !seq_lens || !q_seq || !topk_idx || !out_bf16)
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn_noalloc: null pointer");
  if (!aligned(q_bf16, 16) || !aligned(kv_cache, 16) || !aligned(out_bf16, 16))
    return fail(DSA_ERR_INVALID_ARG, "sparse_attn_noalloc: q, kv_cache and out must be 16-byte aligned");
  const size_t need = dsa::sfa_workspace_bytes(n_q, h_s, topk);
  if (need > static_cast<size_t>(DSA_NOALLOC_SCRATCH_BYTES))
    return fail(DSA_ERR_UNSUPPORTED,
                "sparse_attn_noalloc: n_q=%d, h_s=%d, topk=%d need %zu bytes of scratch, more than the "
                "fixed %zu (use dsa_sparse_attn with a caller-allocated workspace)",
                n_q, h_s, topk, need, static_cast<size_t>(DSA_NOALLOC_SCRATCH_BYTES));
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "sparse_attn_noalloc: no CUDA device");
  dsa::SfaArgs a{q_bf16, n_q, h_s, kv_cache, num_pages, page_table, max_pages, seq_lens, q_seq, n_seq,
                 topk_idx, topk, sm_scale, out_bf16, out_lse, nullptr, 0, st};
  const char* why = nullptr;
  cudaError_t e = dsa::launch_sfa_noalloc(a, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess)
    return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "sparse_attn_noalloc launch");
  return DSA_OK;
}

static bool prefix_sizes_ok(int32_t n_q, int32_t h_s, int32_t n_seq, int32_t prefix_len, int32_t max_ctx) {
  return n_q > 0 && h_s >= 1 && h_s <= 128 && n_seq >= 1 && max_ctx >= 1 && max_ctx <= 1048576 && prefix_len >= 0 &&
         prefix_len <= max_ctx;
}

size_t dsa_prefix_attn_workspace_size(int32_t n_q, int32_t h_s, int32_t n_seq, int32_t prefix_len, int32_t max_ctx) {
  if (!prefix_sizes_ok(n_q, h_s, n_seq, prefix_len, max_ctx)) return 0;
  return dsa::prefix_workspace_bytes(n_q, h_s, n_seq, prefix_len, max_ctx);
}

int dsa_prefix_attn(const void* q_bf16, int32_t n_q, int32_t h_s, const uint8_t* kv_cache, int64_t num_pages,
                    const int32_t* prefix_pages, int32_t prefix_len, const int32_t* page_table, int32_t max_pages,
                    const int32_t* seq_lens, int32_t n_seq, const int32_t* q_seq, const int32_t* q_pos,
                    int32_t max_ctx, float sm_scale, void* out_bf16, float* out_lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (n_q < 0 || n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "prefix_attn: negative n_q or n_seq");
  if (h_s < 1 || h_s > 128) return fail(DSA_ERR_UNSUPPORTED, "prefix_attn: h_s must be 1..128 (got %d)", h_s);
  if (max_ctx < 1 || max_ctx > 1048576) return fail(DSA_ERR_UNSUPPORTED, "prefix_attn: max_ctx must be 1..1048576");
  if (prefix_len < 0 || prefix_len > max_ctx)
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: prefix_len must lie in 0..max_ctx");
  if (num_pages < 1) return fail(DSA_ERR_INVALID_ARG, "prefix_attn: num_pages must be >= 1");
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale))
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: sm_scale must be positive and finite");
  if (n_q == 0) return DSA_OK;
  if (n_seq == 0) return fail(DSA_ERR_INVALID_ARG, "prefix_attn: query rows without sequences");
  const bool tails = max_ctx > prefix_len;
  if (tails && max_pages < (max_ctx + DSA_PAGE_SIZE - 1) / DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: max_pages < ceil(max_ctx / 64)");
  if (!q_bf16 || !kv_cache || !seq_lens || !q_seq || !q_pos || !out_bf16 || (prefix_len && !prefix_pages) ||
      (tails && !page_table) || !workspace)
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: null pointer");
  if (!aligned(q_bf16, 16) || !aligned(kv_cache, 16) || !aligned(out_bf16, 16))
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: q, kv_cache and out must be 16-byte aligned");
  if (!aligned(prefix_pages, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(q_seq, 4) ||
      !aligned(q_pos, 4) || !aligned(out_lse, 4))
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: tables, lengths, rows and out_lse must be 4-byte aligned");
  const size_t need = dsa::prefix_workspace_bytes(n_q, h_s, n_seq, prefix_len, max_ctx);
  if (workspace_bytes < need || !aligned(workspace, 256))
    return fail(DSA_ERR_INVALID_ARG, "prefix_attn: workspace must be >= %zu bytes and 256-byte aligned", need);
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "prefix_attn: no CUDA device");
  dsa::PrefixArgs a{q_bf16, n_q, h_s, kv_cache, num_pages, prefix_pages, prefix_len, page_table, max_pages, seq_lens,
                    n_seq, q_seq, q_pos, max_ctx, sm_scale, out_bf16, out_lse, workspace, st};
  const char* why = nullptr;
  cudaError_t e = dsa::launch_prefix_attn(a, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, "prefix_attn launch");
  return DSA_OK;
}

int dsa_norm_rope_quant_kv(const void* k_bf16, int64_t k_stride, const float* k_weight, const float* k_bias,
                           int32_t k_center, const void* kv_bf16, int64_t kv_stride, const float* kv_weight, float eps,
                           const int32_t* pos, const int64_t* slot_mapping, int32_t n_tokens, uint8_t* k_cache,
                           uint8_t* kv_cache, int64_t num_slots, const int64_t* turns, float amplitude,
                           int32_t k_offset, int32_t k_layout, int32_t kv_layout, void* stream) {
  const int rc = check_rope_quant("norm_rope_quant_kv", k_bf16, k_stride, kv_bf16, kv_stride, pos, slot_mapping, n_tokens,
                                  k_cache, kv_cache, num_slots, turns, amplitude, k_offset, k_layout, kv_layout);
  if (rc) return rc;
  if (k_center != 0 && k_center != 1) return fail(DSA_ERR_INVALID_ARG, "norm_rope_quant_kv: k_center must be 0 or 1");
  if (!std::isfinite(eps) || eps < 0.f)
    return fail(DSA_ERR_INVALID_ARG, "norm_rope_quant_kv: eps must be finite and not negative");
  if (!aligned(k_weight, 16) || !aligned(k_bias, 16) || !aligned(kv_weight, 16))
    return fail(DSA_ERR_INVALID_ARG, "norm_rope_quant_kv: weights and bias must be 16-byte aligned");
  if (n_tokens == 0) return DSA_OK;
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "norm_rope_quant_kv: no CUDA device");
  dsa::NormQuantArgs a{{k_bf16, k_stride, kv_bf16, kv_stride, pos, slot_mapping, n_tokens, k_cache, kv_cache, num_slots,
                        turns, amplitude, k_offset, k_layout, kv_layout, st},
                       k_weight, k_bias, kv_weight, k_center, eps};
  cudaError_t e = dsa::launch_norm_rope_quant(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "norm_rope_quant_kv launch");
}

static bool mass_sizes_ok(int32_t n_q, int32_t h_s) { return n_q >= 1 && n_q <= 65536 && h_s >= 1 && h_s <= 128; }

// What the two kinds of accumulated weights check alike.
static int check_mass(const char* who, const dsa::MassArgs& a, size_t workspace_bytes) {
  if (a.n_q < 0 || a.n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "%s: negative n_q or n_seq", who);
  if (a.h_s < 1 || a.h_s > 128) return fail(DSA_ERR_UNSUPPORTED, "%s: h_s must be 1..128 (got %d)", who, a.h_s);
  // (a walk over more empty sequences could outlast the waits for it)
  if (a.n_q > 65536 || a.n_seq > 65536) return fail(DSA_ERR_UNSUPPORTED, "%s: at most 65536 query rows and sequences a call", who);
  if (a.max_ctx < 1 || a.max_ctx > 1048576) return fail(DSA_ERR_UNSUPPORTED, "%s: max_ctx must be 1..1048576", who);
  if (a.max_pages < (a.max_ctx + DSA_PAGE_SIZE - 1) / DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "%s: max_pages < ceil(max_ctx / 64)", who);
  if (a.num_pages < 1) return fail(DSA_ERR_INVALID_ARG, "%s: num_pages must be >= 1", who);
  if (a.num_pages > 1 << 25) return fail(DSA_ERR_UNSUPPORTED, "%s: at most 2^25 pages", who);
  if (!(a.sm_scale > 0.f) || !std::isfinite(a.sm_scale))
    return fail(DSA_ERR_INVALID_ARG, "%s: sm_scale must be positive and finite", who);
  if (a.mass && (!spans(a.mass_stride, a.n_seq) || (a.n_seq > 1 && a.mass_stride < a.max_ctx)))
    return fail(DSA_ERR_INVALID_ARG, "%s: mass_stride must be max_ctx or more, all rows within 2^40 elements", who);
  if (a.n_q == 0) return DSA_OK;
  if (a.n_seq == 0) return fail(DSA_ERR_INVALID_ARG, "%s: query rows without sequences", who);
  if (!a.q || !a.kv_cache || !a.page_table || !a.seq_lens || !a.q_seq || !a.lse || !a.workspace)
    return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(a.q, 16) || !aligned(a.kv_cache, 16) || !aligned(a.page_table, 4) || !aligned(a.seq_lens, 4) ||
      !aligned(a.q_seq, 4) || !aligned(a.q_pos, 4) || !aligned(a.idx, 4) || !aligned(a.lse, 4) || !aligned(a.mass, 8) ||
      !aligned(a.weights, 4))
    return fail(DSA_ERR_INVALID_ARG, "%s: q and kv_cache must be 16-byte aligned, the others to their elements", who);
  const size_t need = dsa::mass_workspace_bytes(a.n_q, a.h_s, a.n_seq);
  if (workspace_bytes < need || !aligned(a.workspace, 256))
    return fail(DSA_ERR_INVALID_ARG, "%s: workspace must be >= %zu bytes and 256-byte aligned", who, need);
  return DSA_OK;
}
static int run_mass(const char* who, dsa::MassArgs& a, void* stream) {
  if (!(a.status = status_ptr())) return fail(DSA_ERR_CUDA, "%s: no CUDA device", who);
  const char* why = nullptr;
  cudaError_t e = dsa::launch_attn_mass(a, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess) return why ? fail(DSA_ERR_UNSUPPORTED, "%s", why) : cuda_fail(e, who);
  return DSA_OK;
}

size_t dsa_attn_mass_workspace_size(int32_t n_q, int32_t h_s, int32_t n_seq) {
  return mass_sizes_ok(n_q, h_s) && n_seq >= 1 && n_seq <= 65536 ? dsa::mass_workspace_bytes(n_q, h_s, n_seq) : 0;
}

int dsa_attn_mass(const void* q_bf16, int32_t n_q, int32_t h_s, const uint8_t* kv_cache, int64_t num_pages,
                  const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens, int32_t n_seq,
                  const int32_t* q_seq, const int32_t* q_pos, int32_t max_ctx, float sm_scale, const float* lse,
                  int64_t* mass, int64_t mass_stride, void* workspace, size_t workspace_bytes, void* stream) {
  dsa::MassArgs a{q_bf16, n_q, h_s, kv_cache, num_pages, page_table, max_pages, seq_lens, n_seq, q_seq, q_pos, nullptr, 0,
                  max_ctx, sm_scale, lse, mass, mass_stride, nullptr, workspace, nullptr};
  const int rc = check_mass("attn_mass", a, workspace_bytes);
  if (rc || n_q == 0) return rc;
  if (!q_pos || !mass) return fail(DSA_ERR_INVALID_ARG, "attn_mass: null pointer");
  return run_mass("attn_mass", a, stream);
}

int dsa_sparse_attn_mass(const void* q_bf16, int32_t n_q, int32_t h_s, const uint8_t* kv_cache, int64_t num_pages,
                         const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens, int32_t n_seq,
                         const int32_t* q_seq, const int32_t* topk_idx, int32_t topk, int32_t max_ctx, float sm_scale,
                         const float* lse, int64_t* mass, int64_t mass_stride, float* out_weights, void* workspace,
                         size_t workspace_bytes, void* stream) {
  dsa::MassArgs a{q_bf16, n_q, h_s, kv_cache, num_pages, page_table, max_pages, seq_lens, n_seq, q_seq, nullptr, topk_idx, topk,
                  max_ctx, sm_scale, lse, mass, mass_stride, out_weights, workspace, nullptr};
  if (topk < 1 || topk > 65536) return fail(DSA_ERR_UNSUPPORTED, "sparse_attn_mass: topk must be 1..65536");
  const int rc = check_mass("sparse_attn_mass", a, workspace_bytes);
  if (rc || n_q == 0) return rc;
  if (!topk_idx || (!mass && !out_weights)) return fail(DSA_ERR_INVALID_ARG, "sparse_attn_mass: null pointer");
  return run_mass("sparse_attn_mass", a, stream);
}

int dsa_evict_select(const int64_t* mass, int64_t mass_stride, const int32_t* seq_lens, int32_t n_seq, int32_t max_ctx,
                     int32_t budget, int32_t sinks, int32_t recent, int32_t* kept, int32_t* new_lens,
                     int64_t* kept_mass, void* stream) {
  if (n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "evict_select: n_seq < 0");
  if (max_ctx < 1 || max_ctx > 1048576) return fail(DSA_ERR_UNSUPPORTED, "evict_select: max_ctx must be 1..1048576");
  if (budget < 1 || budget > 1048576) return fail(DSA_ERR_UNSUPPORTED, "evict_select: budget must be 1..1048576");
  if (sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > budget)
    return fail(DSA_ERR_INVALID_ARG, "evict_select: sinks and recent must not be negative, nor more than budget together");
  if (n_seq > INT32_MAX / 16) return fail(DSA_ERR_UNSUPPORTED, "evict_select: n_seq must be below 2^27");
  if (n_seq == 0) return DSA_OK;
  if (!spans(mass_stride, n_seq) || (n_seq > 1 && mass_stride < max_ctx))
    return fail(DSA_ERR_INVALID_ARG, "evict_select: mass_stride must be max_ctx or more, all rows within 2^40 elements");
  if (!mass || !seq_lens || !kept || !new_lens) return fail(DSA_ERR_INVALID_ARG, "evict_select: null pointer");
  if (!aligned(mass, 8) || !aligned(kept_mass, 8) || !aligned(seq_lens, 4) || !aligned(kept, 4) || !aligned(new_lens, 4))
    return fail(DSA_ERR_INVALID_ARG, "evict_select: a pointer is not aligned to its element");
  if (static_cast<const int32_t*>(new_lens) < seq_lens + n_seq && seq_lens < new_lens + n_seq)
    return fail(DSA_ERR_INVALID_ARG, "evict_select: new_lens must not share memory with seq_lens");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "evict_select: no CUDA device");
  dsa::EvictSelectArgs a{mass, mass_stride, seq_lens, n_seq, max_ctx, budget, sinks, recent, kept, new_lens, kept_mass, st};
  cudaError_t e = dsa::launch_evict_select(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "evict_select launch");
}

size_t dsa_evict_compact_workspace_size(int32_t n_seq, int32_t budget) {
  return n_seq < 1 || budget < 1 ? 0 : dsa::evict_workspace_bytes(n_seq, budget);
}

int dsa_evict_compact(const int32_t* kept, int32_t n_seq, int32_t budget, const int32_t* page_table, int32_t max_pages,
                      const int32_t* dst_table, int32_t dst_max_pages, uint8_t* k_cache, uint8_t* kv_cache,
                      int64_t num_pages, void* workspace, size_t workspace_bytes, void* stream) {
  if (n_seq < 0) return fail(DSA_ERR_INVALID_ARG, "evict_compact: n_seq < 0");
  if (budget < 1 || budget > 1048576) return fail(DSA_ERR_UNSUPPORTED, "evict_compact: budget must be 1..1048576");
  if (max_pages < 1 || num_pages < 1 || num_pages > INT64_MAX / 65536)
    return fail(DSA_ERR_INVALID_ARG, "evict_compact: max_pages and num_pages must be >= 1");
  if (n_seq == 0) return DSA_OK;
  if (static_cast<int64_t>(n_seq) * budget > int64_t{1} << 35)
    return fail(DSA_ERR_UNSUPPORTED, "evict_compact: n_seq * budget must be 2^35 at most");
  if (!kept || !page_table || (!k_cache && !kv_cache)) return fail(DSA_ERR_INVALID_ARG, "evict_compact: null pointer");
  const bool in_place = !dst_table || dst_table == page_table;
  if (in_place) {
    if (dst_table && dst_max_pages != max_pages)
      return fail(DSA_ERR_INVALID_ARG, "evict_compact: one table with two widths");
    dst_table = page_table;
    dst_max_pages = max_pages;
  }
  if (dst_max_pages < (budget + DSA_PAGE_SIZE - 1) / DSA_PAGE_SIZE)
    return fail(DSA_ERR_INVALID_ARG, "evict_compact: the pages that receive must hold budget positions");
  if (!aligned(kept, 4) || !aligned(page_table, 4) || !aligned(dst_table, 4) || !aligned(k_cache, 16) || !aligned(kv_cache, 16))
    return fail(DSA_ERR_INVALID_ARG, "evict_compact: tables must be 4-byte and caches 16-byte aligned");
  const size_t need = dsa::evict_workspace_bytes(n_seq, budget);
  if (in_place && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(DSA_ERR_INVALID_ARG, "evict_compact: in place, workspace must be >= %zu bytes and 256-byte aligned", need);
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "evict_compact: no CUDA device");
  dsa::EvictCompactArgs a{kept, n_seq, budget, page_table, max_pages, dst_table, dst_max_pages, k_cache, kv_cache, num_pages,
                          static_cast<uint8_t*>(workspace), st};
  cudaError_t e = dsa::launch_evict_compact(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "evict_compact launch");
}

int dsa_topk_merge(const int32_t* cand_idx, const float* cand_scores, const int32_t* part_offsets, int32_t n_parts,
                   int32_t n_q, int32_t k_in, int32_t topk, int32_t* out_idx, float* out_scores,
                   const int32_t* local_lo, const int32_t* local_hi, int32_t* out_local, void* stream) {
  if (n_q < 0) return fail(DSA_ERR_INVALID_ARG, "topk_merge: n_q < 0");
  if (n_parts < 1 || k_in < 1 || topk < 1) return fail(DSA_ERR_INVALID_ARG, "topk_merge: n_parts, k_in and topk must be >= 1");
  if (static_cast<int64_t>(n_parts) * k_in > dsa::kMostMerged)
    return fail(DSA_ERR_UNSUPPORTED, "topk_merge: n_parts * k_in must be <= %d (got %lld)", dsa::kMostMerged,
                static_cast<long long>(n_parts) * k_in);
  if (n_q == 0) return DSA_OK;
  if (!cand_idx || !cand_scores || !out_idx) return fail(DSA_ERR_INVALID_ARG, "topk_merge: null pointer");
  if ((out_local != nullptr) != (local_lo != nullptr && local_hi != nullptr))
    return fail(DSA_ERR_INVALID_ARG, "topk_merge: out_local needs local_lo and local_hi (and they need it)");
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "topk_merge: no CUDA device");
  dsa::TopkMergeArgs a{cand_idx, cand_scores, part_offsets, n_parts, n_q, k_in, topk, out_idx, out_scores,
                       local_lo, local_hi, out_local, st};
  cudaError_t e = dsa::launch_topk_merge(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "topk_merge launch");
}

int dsa_lse_combine(const void* o_parts, const float* lse_parts, int32_t n_parts, int32_t n_q, int32_t h,
                    void* out_bf16, float* out_lse, void* stream) {
  if (n_q < 0) return fail(DSA_ERR_INVALID_ARG, "lse_combine: n_q < 0");
  if (n_parts < 1 || h < 1 || h > 65535) return fail(DSA_ERR_INVALID_ARG, "lse_combine: n_parts >= 1 and h in 1..65535");
  if (n_q == 0) return DSA_OK;
  if (!o_parts || !lse_parts || !out_bf16) return fail(DSA_ERR_INVALID_ARG, "lse_combine: null pointer");
  if (!aligned(o_parts, 8) || !aligned(out_bf16, 8))
    return fail(DSA_ERR_INVALID_ARG, "lse_combine: o_parts and out must be 8-byte aligned");
  cudaError_t e = dsa::launch_lse_combine(o_parts, lse_parts, n_parts, n_q, h, out_bf16, out_lse,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DSA_OK : cuda_fail(e, "lse_combine launch");
}

int dsa_test_prefix_plan(int32_t n_q, int32_t h_s, int32_t n_seq, int32_t prefix_len, int32_t max_ctx, int32_t* plan) {
  if (!prefix_sizes_ok(n_q, h_s, n_seq, prefix_len, max_ctx) || !plan)
    return fail(DSA_ERR_INVALID_ARG, "test_prefix_plan: sizes out of range, or null");
  dsa::prefix_plan_numbers(n_q, h_s, n_seq, prefix_len, max_ctx, plan);
  return DSA_OK;
}

int dsa_test_stall_indexer(int32_t wait_limit_us) {
  if (wait_limit_us < 0 || wait_limit_us > 10000000)
    return fail(DSA_ERR_INVALID_ARG, "test_stall_indexer: wait_limit_us must be 0..10000000");
  g_stall_wait_us.store(wait_limit_us, std::memory_order_relaxed);
  return DSA_OK;
}

int dsa_device_status(void* stream) {
  unsigned* st = status_ptr();
  if (!st) return fail(DSA_ERR_CUDA, "device_status: no CUDA device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, st, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(st, 0, sizeof(unsigned), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "device_status");
  return static_cast<int>(v);
}

}  // extern "C"
