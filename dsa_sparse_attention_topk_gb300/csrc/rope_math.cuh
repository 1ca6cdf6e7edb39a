// What the rotary kernels share: the phase of a position at a frequency, its sine and cosine (the
// header of rope.cu says how), element types and vector words, and the writers' conversions.
#pragma once

#include <cuda_fp16.h>

#include "dsa_common.cuh"

namespace dsa {
namespace {

// an unevaluated sum of two floats, |lo| at most half an ulp of hi
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum_ordered(float a, float b) {  // |a| >= |b| or a == 0
  const float h = a + b;
  return {h, (a - h) + b};
}
// position p at a frequency of `turns` 2^-64 turns per position: the nearest quarter turn, and the
// rest, at most an eighth of a turn, in 2^-64 turns
__device__ __forceinline__ int64_t phase_rest(int pos, int64_t turns, uint32_t& quarter) {
  const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(pos)) * static_cast<uint64_t>(turns);
  quarter = static_cast<uint32_t>((p + (1ull << 61)) >> 62);
  return static_cast<int64_t>(p - (static_cast<uint64_t>(quarter) << 62));
}

// cos and sin, times the amplitude
__device__ __forceinline__ float2 phase_cs(int pos, int64_t turns, float amp) {
  uint32_t quarter;
  const int64_t rest64 = phase_rest(pos, turns, quarter);
  // the rest, in 2^-33 turns: |rest| <= 2^30, and what it leaves (of a small angle most of it)
  const int rest = static_cast<int>(rest64 >> 31);
  const float rh = static_cast<float>(rest);
  const float rl = fmaf(static_cast<float>(static_cast<uint32_t>(rest64) & 0x7FFFFFFFu), 4.656612873077393e-10f,
                        static_cast<float>(rest - static_cast<int>(rh)));
  constexpr double kRad = 6.283185307179586476925 / 8589934592.0;  // 2 pi 2^-33
  constexpr float kHi = static_cast<float>(kRad);
  constexpr float kLo = static_cast<float>(kRad - static_cast<double>(kHi));
  const float x = __fmul_rn(rh, kHi);  // (rounded here, whatever it is added to: so below)
  const float xl = fmaf(rh, kHi, -x) + fmaf(rl, kHi, rh * kLo);
  const float z = x * x;
  // sin = x + (x^3 S(z) + xl cos x),  cos = 1 + (-z/2 + z^2 C(z) - rounding of z / 2 - x xl)
  float S = -1.0f / 39916800.0f, C = -1.0f / 3628800.0f;
  S = fmaf(S, z, 1.0f / 362880.0f);
  S = fmaf(S, z, -1.0f / 5040.0f);
  S = fmaf(S, z, 1.0f / 120.0f);
  S = fmaf(S, z, -1.0f / 6.0f);
  C = fmaf(C, z, 1.0f / 40320.0f);
  C = fmaf(C, z, -1.0f / 720.0f);
  C = fmaf(C, z, 1.0f / 24.0f);
  const Two sn = two_sum_ordered(x, fmaf(x * z, S, fmaf(-0.5f * z, xl, xl)));
  const float zl = fmaf(x, x, -z);
  const Two cn = two_sum_ordered(1.0f, fmaf(z * z, C, -0.5f * z) - fmaf(x, xl, 0.5f * zl));
  // a quarter turn: (c, s) -> (-s, c)
  const bool swap = quarter & 1u;
  Two c = swap ? sn : cn, s = swap ? cn : sn;
  const float cf = ((quarter + 1u) & 2u) ? -amp : amp, sf = (quarter & 2u) ? -amp : amp;
  const float ch = __fmul_rn(c.hi, cf), sh = __fmul_rn(s.hi, sf);
  return make_float2(ch + (fmaf(c.hi, cf, -ch) + c.lo * cf), sh + (fmaf(s.hi, sf, -sh) + s.lo * sf));
}

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
  static __device__ float get(__half v) { return __half2float(v); }
  static __device__ __half put(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
  static __device__ float get(float v) { return v; }
  static __device__ float put(float v) { return v; }
};

template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <typename T, int V> union Vec {
  typename Word<V * sizeof(T)>::type u;
  T e[V];
};

// two packed bf16 values -> fp32 (exact)
__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t v) {
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&v);
  return make_float2(__low2float(b), __high2float(b));
}
// largest of the warp's floats; a NaN is ignored unless every lane has one, as in a chain of fmaxf
// (an integer maximum over the bits would do for numbers, but makes a tile of NaN one of zeros)
__device__ __forceinline__ float warp_amax(float v) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(f32x2_to_e4m3x2(a, b)) | (static_cast<uint32_t>(f32x2_to_e4m3x2(c, d)) << 16);
}

}  // namespace
}  // namespace dsa
