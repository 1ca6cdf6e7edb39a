// Rotary positions: queries and keys turned by their positions (dsa_rope), and the cache
// writers with the turn on the way (dsa_rope_quant_kv).
//
// A pair (a, b) of a head's rotary part with frequency f (radians per position) at position
// p becomes  amp * (a cos(p f) - b sin(p f),  a sin(p f) + b cos(p f)).
//
// The angle.  p f is taken modulo a whole turn in 64-bit fixed point: the table holds
// f / 2 pi * 2^64, the integer product with p wraps exactly where the angle does, and its
// top 32 bits are the phase as a signed fraction of a turn.  A far position costs no
// accuracy (the phase is off by at most p * 2^-65 of a turn from the table's rounding and
// 2^-32 from the cut, where p * f in fp32 is off by 2^-24 p f radians), and no double
// arithmetic is needed; sincospif of the fraction is then within an ulp or two.
//
// Both kernels are bound by memory: a rotation is 3 multiply-adds per pair.

#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_launch.h"
#include "quant_tok.cuh"

namespace dsa {
namespace {

// cos and sin (times the amplitude) of position p at a frequency of `turns` 2^-64 turns per
// position
__device__ __forceinline__ float2 phase_cs(int pos, int64_t turns, float amp) {
  const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(pos)) * static_cast<uint64_t>(turns);
  const float half_turns = static_cast<float>(static_cast<int32_t>(p >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(amp * c, amp * s);
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

template <typename T> union Vec {
  uint4 u;
  T e[16 / sizeof(T)];
};

struct RopeGeom {
  int slots;         // work items of one head (vectors, or pairs and single elements)
  int slots_block;   // of them in one block; blockIdx.y picks the block's share
  int lo;            // first element an item covers (the rotary part's start in place, else 0)
};

// A thread owns one 16-byte vector position of a head (with its partner half a rotary part
// further on in the half layout) and takes R consecutive (token, head) rows, so that the
// sines of its pairs are computed once per token and the R loads are in flight together.
template <typename T, bool HALF, int R>
__global__ void __launch_bounds__(256)
rope_vec_kernel(RopeArgs a, RopeGeom g) {
  constexpr int V = 16 / sizeof(T);
  constexpr int P = HALF ? V : V / 2;  // pairs per item
  pdl_launch_dependents();
  pdl_wait();
  const int grp = threadIdx.x / g.slots_block;
  const int slot = blockIdx.y * g.slots_block + threadIdx.x % g.slots_block;
  if (grp >= static_cast<int>(blockDim.x) / g.slots_block || slot >= g.slots) return;
  const int64_t rows = static_cast<int64_t>(a.n) * a.h;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x / g.slots_block) + grp) * R;
  if (r0 >= rows) return;
  int e0 = g.lo + slot * V;
  const int half = a.rot >> 1;
  if (HALF && e0 >= a.offset + half) e0 += half;  // the second halves go with the first
  const bool turn = e0 >= a.offset && e0 < a.offset + (HALF ? half : a.rot);
  const T* xb = static_cast<const T*>(a.x) + e0;
  T* ob = static_cast<T*>(a.out) + e0;

  int t = static_cast<int>(static_cast<uint32_t>(r0) / static_cast<uint32_t>(a.h));
  int hh = static_cast<int>(static_cast<uint32_t>(r0) - static_cast<uint32_t>(t) * static_cast<uint32_t>(a.h));
  const int t0 = t, h0 = hh;
  Vec<T> v[R], w[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k < rows) {
      const T* src = xb + t * a.x_stride_t + hh * a.x_stride_h;
      v[k].u = *reinterpret_cast<const uint4*>(src);
      if (HALF && turn) w[k].u = *reinterpret_cast<const uint4*>(src + half);
    }
    if (++hh == a.h) { hh = 0; ++t; }
  }
  float2 cs[P];
  int have = -1;
  t = t0;
  hh = h0;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k >= rows) break;
    T* dst = ob + t * a.out_stride_t + hh * a.out_stride_h;
    if (turn) {
      if (t != have) {
        const int f0 = HALF ? e0 - a.offset : (e0 - a.offset) >> 1;
        const int pos = a.pos[t];
#pragma unroll
        for (int i = 0; i < P; ++i) cs[i] = phase_cs(pos, a.turns[f0 + i], a.amplitude);
        if (a.transpose) {
#pragma unroll
          for (int i = 0; i < P; ++i) cs[i].y = -cs[i].y;
        }
        have = t;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float p = Elem<T>::get(HALF ? v[k].e[i] : v[k].e[2 * i]);
        const float q = Elem<T>::get(HALF ? w[k].e[i] : v[k].e[2 * i + 1]);
        const T y0 = Elem<T>::put(p * cs[i].x - q * cs[i].y), y1 = Elem<T>::put(p * cs[i].y + q * cs[i].x);
        if (HALF) {
          v[k].e[i] = y0;
          w[k].e[i] = y1;
        } else {
          v[k].e[2 * i] = y0;
          v[k].e[2 * i + 1] = y1;
        }
      }
      if (HALF) *reinterpret_cast<uint4*>(dst + half) = w[k].u;
    }
    *reinterpret_cast<uint4*>(dst) = v[k].u;
    if (++hh == a.h) { hh = 0; ++t; }
  }
}

// Any alignment, stride and size: a work item is one pair or, out of place, one element
// beside the rotary part.
template <typename T>
__global__ void __launch_bounds__(256)
rope_pair_kernel(RopeArgs a, RopeGeom g, int half_layout) {
  pdl_launch_dependents();
  pdl_wait();
  const int grp = threadIdx.x / g.slots_block;
  const int slot = blockIdx.y * g.slots_block + threadIdx.x % g.slots_block;
  if (grp >= static_cast<int>(blockDim.x) / g.slots_block || slot >= g.slots) return;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x / g.slots_block) + grp;
  if (r >= static_cast<int64_t>(a.n) * a.h) return;
  const int t = static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(a.h));
  const int hh = static_cast<int>(r - static_cast<int64_t>(t) * a.h);
  const T* src = static_cast<const T*>(a.x) + t * a.x_stride_t + hh * a.x_stride_h;
  T* dst = static_cast<T*>(a.out) + t * a.out_stride_t + hh * a.out_stride_h;
  const int half = a.rot >> 1;
  if (slot < half) {
    const int i0 = a.offset + (half_layout ? slot : 2 * slot), i1 = half_layout ? i0 + half : i0 + 1;
    float2 cs = phase_cs(a.pos[t], a.turns[slot], a.amplitude);
    if (a.transpose) cs.y = -cs.y;
    const float p = Elem<T>::get(src[i0]), q = Elem<T>::get(src[i1]);
    dst[i0] = Elem<T>::put(p * cs.x - q * cs.y);
    dst[i1] = Elem<T>::put(p * cs.y + q * cs.x);
  } else {
    const int c = slot - half;
    const int e = c < a.offset ? c : c + a.rot;
    dst[e] = src[e];
  }
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool in_place = a.x == a.out, half = a.layout == DSA_ROPE_HALF;
  auto whole = [](int64_t v) { return v % V == 0; };
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                   whole(a.x_stride_t) && whole(a.x_stride_h) && whole(a.out_stride_t) && whole(a.out_stride_h) &&
                   whole(a.offset) && whole(half ? a.rot / 2 : a.rot) && (in_place || whole(a.d));
  const int64_t rows = static_cast<int64_t>(a.n) * a.h;
  RopeGeom g;
  if (vec) {
    g.lo = in_place ? a.offset : 0;
    g.slots = ((in_place ? a.rot : a.d) - (half ? a.rot / 2 : 0)) / V;
  } else {
    g.lo = 0;
    g.slots = in_place ? a.rot / 2 : a.d - a.rot / 2;
  }
  g.slots_block = g.slots < 256 ? g.slots : 256;
  const int groups = 256 / g.slots_block;
  const int threads = (groups * g.slots_block + 31) / 32 * 32;
  // four rows a thread once one row each would fill every SM four times over
  const int R = vec && rows * g.slots >= 4ll * 152 * 2048 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((rows + static_cast<int64_t>(groups) * R - 1) / (static_cast<int64_t>(groups) * R)),
                  static_cast<unsigned>((g.slots + g.slots_block - 1) / g.slots_block));
  if (!vec) return launch_pdl(rope_pair_kernel<T>, grid, dim3(threads), 0, s, 1, a, g, half ? 1 : 0);
  if (half)
    return R == 4 ? launch_pdl(rope_vec_kernel<T, true, 4>, grid, dim3(threads), 0, s, 1, a, g)
                  : launch_pdl(rope_vec_kernel<T, true, 1>, grid, dim3(threads), 0, s, 1, a, g);
  return R == 4 ? launch_pdl(rope_vec_kernel<T, false, 4>, grid, dim3(threads), 0, s, 1, a, g)
                : launch_pdl(rope_vec_kernel<T, false, 1>, grid, dim3(threads), 0, s, 1, a, g);
}

// ---- the cache writers with the rotation on the way ---------------------------------
// One warp per token, as in the plain writers: lane i computes the sine and cosine of
// frequency i of the token's position, and the lanes that hold a pair's values fetch them
// by shuffle.  The rotated values are quantised from fp32: they are never rounded to bf16.
constexpr int kWarpsPerBlock = 8;
constexpr int kRot = 64;

// the k values of this lane (dims 4 lane ..) turned where they lie in [offset, offset + 64)
__device__ __forceinline__ void turn_k(float (&x)[4], float2 cs, int offset, bool half_layout) {
  const int lane = threadIdx.x & 31;
  const int li = lane - (offset >> 2);  // 0..15 inside the rotary part
  const bool mine = li >= 0 && li < kRot / 4;
  if (half_layout) {
    const bool first = li < 8;
    float other[4], c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      other[j] = __shfl_sync(0xffffffffu, x[j], first ? lane + 8 : lane - 8);
      c[j] = __shfl_sync(0xffffffffu, cs.x, 4 * (li & 7) + j);
      s[j] = __shfl_sync(0xffffffffu, cs.y, 4 * (li & 7) + j);
    }
    if (mine) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = first ? x[j] * c[j] - other[j] * s[j] : other[j] * s[j] + x[j] * c[j];
    }
  } else {
    float c[2], s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = __shfl_sync(0xffffffffu, cs.x, 2 * li + j);
      s[j] = __shfl_sync(0xffffffffu, cs.y, 2 * li + j);
    }
    if (mine) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p = x[2 * j], q = x[2 * j + 1];
        x[2 * j] = p * c[j] - q * s[j];
        x[2 * j + 1] = p * s[j] + q * c[j];
      }
    }
  }
}

// the rope tile's values of this lane (2 lane, 2 lane + 1 of 64), turned
__device__ __forceinline__ void turn_kv(float& x0, float& x1, float2 cs, bool half_layout) {
  const int lane = threadIdx.x & 31;
  if (half_layout) {
    const float o0 = __shfl_xor_sync(0xffffffffu, x0, 16), o1 = __shfl_xor_sync(0xffffffffu, x1, 16);
    const float c0 = __shfl_sync(0xffffffffu, cs.x, 2 * lane), c1 = __shfl_sync(0xffffffffu, cs.x, 2 * lane + 1);
    const float s0 = __shfl_sync(0xffffffffu, cs.y, 2 * lane), s1 = __shfl_sync(0xffffffffu, cs.y, 2 * lane + 1);
    x0 = lane < 16 ? x0 * c0 - o0 * s0 : o0 * s0 + x0 * c0;
    x1 = lane < 16 ? x1 * c1 - o1 * s1 : o1 * s1 + x1 * c1;
  } else {
    const float p = x0, q = x1;
    x0 = p * cs.x - q * cs.y;
    x1 = p * cs.y + q * cs.x;
  }
}

__global__ void __launch_bounds__(kWarpsPerBlock * 32)
rope_quant_kernel(RopeQuantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t turns = a.turns[lane];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + (threadIdx.x >> 5); t < a.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarpsPerBlock) {
    const int64_t slot = a.slots[t];
    if (slot < 0) continue;
    uint2 kraw = make_uint2(0u, 0u), raws[4];
    uint32_t rope = 0;
    if (a.k) kraw = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.k) + t * a.k_stride + 4 * lane);
    if (a.kv) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.kv) + t * a.kv_stride;
#pragma unroll
      for (int tile = 0; tile < 4; ++tile) raws[tile] = *reinterpret_cast<const uint2*>(src + tile * 128 + 4 * lane);
      rope = *reinterpret_cast<const uint32_t*>(src + 512 + 2 * lane);
    }
    const float2 cs = phase_cs(a.pos[t], turns, a.amplitude);
    if (a.k) {
      const float2 p = bf16x2_to_f32(kraw.x), q = bf16x2_to_f32(kraw.y);
      float x[4] = {p.x, p.y, q.x, q.y};
      turn_k(x, cs, a.k_offset, a.k_layout == DSA_ROPE_HALF);
      store_k_values(x, slot, a.k_cache, a.num_slots, a.status);
    }
    if (a.kv) {
      const float2 p = bf16x2_to_f32(rope);
      float x0 = p.x, x1 = p.y;
      turn_kv(x0, x1, cs, a.kv_layout == DSA_ROPE_HALF);
      store_kv_values(raws, x0, x1, slot, a.kv_cache, a.num_slots, a.status);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  if (a.dtype == DSA_DTYPE_BF16) return launch_rope_t<__nv_bfloat16>(a, s);
  if (a.dtype == DSA_DTYPE_FP16) return launch_rope_t<__half>(a, s);
  return launch_rope_t<float>(a, s);
}

cudaError_t launch_rope_quant(const RopeQuantArgs& a, cudaStream_t s) {
  DevInfo di;
  const char* why = nullptr;
  const int cap = device_info(&di, &why) ? di.n_sm * 16 : 2048;
  const int blocks = a.n_tokens / kWarpsPerBlock + (a.n_tokens % kWarpsPerBlock != 0);
  return launch_pdl(rope_quant_kernel, dim3(blocks < cap ? blocks : cap), dim3(kWarpsPerBlock * 32), 0, s, 1, a);
}

}  // namespace dsa
