// Shared by the kernels of the shared-prefix attention.
#pragma once

#include "dsa_common.cuh"
#include "dsa_launch.h"

namespace dsa {

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float exp2_approx(float x) {  // relative error ~2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool has_nan_code(uint32_t w) {  // a byte 0x7F or 0xFF among four E4M3 codes
  return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
}

// Positions row t sees: 0 for a row whose sequence or length is out of range (flagged).
__device__ __forceinline__ int prefix_row_limit(const PrefixArgs& a, int t, bool report) {
  const int b = a.q_seq[t];
  if (b < 0 || b >= a.n_seq) {
    if (report) flag(a.status, DSA_STATUS_BAD_SEQ);
    return 0;
  }
  const int len = a.seq_lens[b];
  if (len < 0 || len > a.max_ctx) {
    if (report) flag(a.status, DSA_STATUS_BAD_LEN);
    return 0;
  }
  const int pos = a.q_pos[t];
  return pos < 0 ? 0 : min(pos, len - 1) + 1;
}

// A row's result in one split, for the merge: o = O / l as fp16 times 2^-e, and (reference, sum, e):
// the sum's own exponent joins the reference, so that the merge compares true sizes.  An empty
// split has reference -inf and no output; NaN logits leave no reference, so theirs is 0.
__device__ __forceinline__ float4 split_state(float ref, float l, int e) {
  if (l == 0.f) return make_float4(-INFINITY, 0.f, 0.f, 0.f);
  const int el = l > 0.f && l < INFINITY ? static_cast<int>(__float_as_uint(l) >> 23) - 127 : 0;
  return make_float4(l != l ? 0.f : ref + static_cast<float>(el), l * exp2i(-max(el, -126)), static_cast<float>(e), 0.f);
}
__device__ __forceinline__ float natural_lse(float ref, float l) {
  return l > 0.f || l != l ? (ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// The kernel for few heads (prefix_few.cu): positions lo .. of every query row.  With splits = 1 a
// block takes a row; otherwise `blocks` blocks take equal shares of all rows' steps, which cuts a
// row into at most `splits` parts.  Row t's parts go to the slots slot0 .. slot0 + used[t] of ns;
// directly to the output when ns is 1.
struct FewArgs {
  PrefixArgs a;
  int lo, splits, blocks, slot0, ns;
  __half* o;
  float4* ml;
  int* used;
};
constexpr int kFewHeads = 32;
constexpr int kFewCutRows = 65536;  // with more rows none is cut: 2^16 rows of 2^14 steps are what 31 bits count
cudaError_t launch_prefix_few(const FewArgs& f, cudaStream_t s);

}  // namespace dsa
