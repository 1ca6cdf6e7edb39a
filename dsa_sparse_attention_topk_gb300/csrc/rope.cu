// Rotary positions: queries and keys turned by their positions (dsa_rope), and the cache
// writers with the turn on the way (dsa_rope_quant_kv).
//
// A pair (a, b) of a head's rotary part with frequency f (radians per position) at position
// p becomes  amp * (a cos(p f) - b sin(p f),  a sin(p f) + b cos(p f)).
//
// The angle.  p f is taken modulo a whole turn in 64-bit fixed point: the table holds
// f / 2 pi * 2^64, and the integer product with p wraps exactly where the angle does, so a
// far position costs no accuracy (p f in fp32 would be off by 2^-24 p f radians) and no
// double arithmetic, which is slow on this GPU, is needed.
//
// Sine and cosine.  The phase is split into quarter turns and a rest of at most an eighth of
// a turn; the rest becomes radians as an unevaluated sum hi + lo of two floats, and the
// Taylor polynomials of sine and cosine (to degree 11 and 10: the first terms left out are
// below 7e-12 and 1.2e-10) are summed so that each result is again hi + lo, good to about
// 2^-27, and rounded once.  The writers, whose results are cut to four bits and must land on the
// right side of a border, do again what that does not decide, in pairs of floats throughout.
//
// Both kernels are bound by memory: a rotation is 3 multiply-adds per pair.

#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_launch.h"
#include "quant_tok.cuh"

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

struct RopeGeom {
  int slots;         // work items of one head (vectors, or pairs and single elements)
  int slots_block;   // of them in one block; blockIdx.y picks the block's share
  int lo;            // first element an item covers (the rotary part's start in place, else 0)
};

// The sines of a block's tokens, each computed once, by all threads: the heads of a token share
// them, and few lanes of a warp hold rotary dims.  It pays with one row a thread (1842 x 16 heads of
// 192 bf16: 17 -> 8.3 us) and with full vectors in the half layout, as many pairs a thread as rows
// (4096 x 64 x 128 bf16, all rotary: 29 -> 23 us); elsewhere several rows share a thread's sines,
// and waiting for the table costs more (4096 x 128 x 576 interleaved: 174 -> 181 us; 4096 x 63 x 192,
// 8-byte vectors: 76 -> 93).  Blocks whose tokens have more than kTableSize pairs, two a thread (few
// heads), leave them to the threads that turn them (65536 x 1 x 64: 8.4 us, by a table 14.1).
constexpr int kTableSize = 512;
struct Table {
  float2* cs;
  int first, half;   // token of its first row; pairs a token
  bool there;
  __device__ __forceinline__ float2 at(int t, int i) const { return cs[(t - first) * half + i]; }
};
__device__ __forceinline__ float2 pair_cs(const RopeArgs& a, int t, int i) {
  float2 cs = phase_cs(a.pos[t], a.turns[i], a.amplitude);
  if (a.transpose) cs.y = -cs.y;
  return cs;
}
// the table of the block's `rows` rows from row r0 on
__device__ __forceinline__ Table fill_table(const RopeArgs& a, float2* cs, int64_t r0, int rows) {
  const int64_t end = min(r0 + rows, static_cast<int64_t>(a.n) * a.h) - 1;
  Table tab{cs, static_cast<int>(static_cast<uint32_t>(r0) / static_cast<uint32_t>(a.h)), a.rot >> 1, false};
  const int last = static_cast<int>(static_cast<uint32_t>(end) / static_cast<uint32_t>(a.h));
  const int64_t size = static_cast<int64_t>(last - tab.first + 1) * tab.half;
  tab.there = size <= kTableSize;
  if (tab.there)
    for (int i = threadIdx.x; i < size; i += blockDim.x) {
      const int t = i / tab.half;
      cs[i] = pair_cs(a, tab.first + t, i - t * tab.half);
    }
  __syncthreads();
  return tab;
}

// A thread owns one vector position of a head, V elements (with its partner half a rotary part
// further on in the half layout), and takes R consecutive (token, head) rows, so that the
// sines of its pairs are computed once per token and the R loads are in flight together.
// V elements are the widest power of two, up to 16 bytes, that divides every address, stride and
// part of a head.
template <typename T, bool HALF, int V, int R>
__global__ void __launch_bounds__(256)
rope_vec_kernel(RopeArgs a, RopeGeom g) {
  using W = typename Word<V * sizeof(T)>::type;
  constexpr bool TABLE = R == 1 || (HALF && V * sizeof(T) == 16);
  constexpr int P = HALF ? V : V / 2;  // pairs per item
  pdl_launch_dependents();
  pdl_wait();
  const int groups = blockDim.x / g.slots_block, grp = threadIdx.x / g.slots_block;
  const int slot = blockIdx.y * g.slots_block + threadIdx.x % g.slots_block;
  const int64_t rows = static_cast<int64_t>(a.n) * a.h, block0 = static_cast<int64_t>(blockIdx.x) * groups * R;
  // (a thread without an item helps with the table and takes the rows behind the last)
  const int64_t r0 = grp < groups && slot < g.slots ? min(block0 + static_cast<int64_t>(grp) * R, rows) : rows;
  if (!TABLE && r0 == rows) return;
  int e0 = g.lo + slot * V;
  const int half = a.rot >> 1;
  if (HALF && e0 >= a.offset + half) e0 += half;  // the second halves go with the first
  const bool turn = e0 >= a.offset && e0 < a.offset + (HALF ? half : a.rot);
  int t = static_cast<int>(static_cast<uint32_t>(r0) / static_cast<uint32_t>(a.h));
  int hh = static_cast<int>(static_cast<uint32_t>(r0) - static_cast<uint32_t>(t) * static_cast<uint32_t>(a.h));
  const int h0 = hh;
  const T* src = static_cast<const T*>(a.x) + t * a.x_stride_t + hh * a.x_stride_h + e0;
  T* dst = static_cast<T*>(a.out) + t * a.out_stride_t + hh * a.out_stride_h + e0;
  // from a token's last head to the next one's first
  const int64_t src_wrap = a.x_stride_t - (a.h - 1) * a.x_stride_h, dst_wrap = a.out_stride_t - (a.h - 1) * a.out_stride_h;
  Vec<T, V> v[R], w[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k < rows) {
      v[k].u = *reinterpret_cast<const W*>(src);
      if (HALF && turn) w[k].u = *reinterpret_cast<const W*>(src + half);
    }
    const bool last = ++hh == a.h;
    src += last ? src_wrap : a.x_stride_h;
    if (last) hh = 0;
  }
  Table tab{};
  if constexpr (TABLE) {
    __shared__ float2 s_cs[kTableSize];
    tab = fill_table(a, s_cs, block0, groups * R);
  }
  float2 cs[P];
  int have = -1;
  hh = h0;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k >= rows) break;
    if (turn) {
      if (t != have) {
        const int f0 = HALF ? e0 - a.offset : (e0 - a.offset) >> 1;
        if (TABLE && tab.there) {
#pragma unroll
          for (int i = 0; i < P; ++i) cs[i] = tab.at(t, f0 + i);
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) cs[i] = pair_cs(a, t, f0 + i);
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
      if (HALF) *reinterpret_cast<W*>(dst + half) = w[k].u;
    }
    *reinterpret_cast<W*>(dst) = v[k].u;
    const bool last = ++hh == a.h;
    dst += last ? dst_wrap : a.out_stride_h;
    if (last) { hh = 0; ++t; }
  }
}

// Pairs of neighbours that no vector boundary holds (an odd offset, stride or head): a work item
// is one pair or, out of place, one element beside the rotary part; R rows a thread as above.
template <typename T, int R>
__global__ void __launch_bounds__(256)
rope_pair_kernel(RopeArgs a, RopeGeom g) {
  constexpr bool TABLE = R == 1;
  pdl_launch_dependents();
  pdl_wait();
  const int groups = blockDim.x / g.slots_block, grp = threadIdx.x / g.slots_block;
  const int slot = blockIdx.y * g.slots_block + threadIdx.x % g.slots_block;
  const int64_t rows = static_cast<int64_t>(a.n) * a.h, block0 = static_cast<int64_t>(blockIdx.x) * groups * R;
  // (a thread without an item helps with the table and takes the rows behind the last)
  const int64_t r0 = grp < groups && slot < g.slots ? min(block0 + static_cast<int64_t>(grp) * R, rows) : rows;
  if (!TABLE && r0 == rows) return;
  const int half = a.rot >> 1;
  const bool turn = slot < half;
  const int c = slot - half;
  const int e0 = turn ? a.offset + 2 * slot : c < a.offset ? c : c + a.rot;
  int t = static_cast<int>(static_cast<uint32_t>(r0) / static_cast<uint32_t>(a.h));
  int hh = static_cast<int>(static_cast<uint32_t>(r0) - static_cast<uint32_t>(t) * static_cast<uint32_t>(a.h));
  const int h0 = hh;
  const T* src = static_cast<const T*>(a.x) + t * a.x_stride_t + hh * a.x_stride_h + e0;
  T* dst = static_cast<T*>(a.out) + t * a.out_stride_t + hh * a.out_stride_h + e0;
  const int64_t src_wrap = a.x_stride_t - (a.h - 1) * a.x_stride_h, dst_wrap = a.out_stride_t - (a.h - 1) * a.out_stride_h;
  T v[R], w[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k < rows) {
      v[k] = src[0];
      if (turn) w[k] = src[1];
    }
    const bool last = ++hh == a.h;
    src += last ? src_wrap : a.x_stride_h;
    if (last) hh = 0;
  }
  Table tab{};
  if constexpr (TABLE) {
    __shared__ float2 s_cs[kTableSize];
    tab = fill_table(a, s_cs, block0, groups * R);
  }
  float2 cs = make_float2(1.f, 0.f);
  int have = -1;
  hh = h0;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (r0 + k >= rows) break;
    if (turn) {
      if (t != have) {
        cs = TABLE && tab.there ? tab.at(t, slot) : pair_cs(a, t, slot);
        have = t;
      }
      const float p = Elem<T>::get(v[k]), q = Elem<T>::get(w[k]);
      dst[0] = Elem<T>::put(p * cs.x - q * cs.y);
      dst[1] = Elem<T>::put(p * cs.y + q * cs.x);
    } else {
      dst[0] = v[k];
    }
    const bool last = ++hh == a.h;
    dst += last ? dst_wrap : a.out_stride_h;
    if (last) { hh = 0; ++t; }
  }
}

// Rows a thread, where there are many: with vectors of 4 bytes or less eight keep more bytes in flight
// (4096 x 64 heads of 100 bf16, elements: 65 -> 50 us; 60000 rows of 576, 4 bytes: 48 -> 38), with wider
// ones four do (8 bytes, 4096 x 63 heads of 192 dims: 76 us, with eight rows 116).
template <typename T, int V> constexpr int kManyRows = V * sizeof(T) <= 4 ? 8 : 4;

template <typename T, bool HALF, int V>
cudaError_t launch_rope_v(const RopeArgs& a, const RopeGeom& g, dim3 grid, dim3 block, int R, cudaStream_t s) {
  constexpr int kMany = kManyRows<T, V>;
  return R > 1 ? launch_pdl(rope_vec_kernel<T, HALF, V, kMany>, grid, block, 0, s, 1, a, g)
               : launch_pdl(rope_vec_kernel<T, HALF, V, 1>, grid, block, 0, s, 1, a, g);
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  constexpr int kMost = 16 / sizeof(T);
  const bool in_place = a.x == a.out, half = a.layout == DSA_ROPE_HALF;
  // the widest vector that divides everything, in elements
  const uint64_t all = (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) / sizeof(T) |
                       static_cast<uint64_t>(a.x_stride_t | a.x_stride_h | a.out_stride_t | a.out_stride_h | a.offset |
                                             (half ? a.rot / 2 : a.rot) | (in_place ? 0 : a.d)) | kMost;
  const int V = static_cast<int>(all & (~all + 1));
  const bool vec = half || V >= 2;
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
  // Several rows a thread once one row each would fill every SM (1842 x 16 x 192 bf16: 8.6 -> 6.7 us).
  // A single head with full vectors in the half layout has one, so that a block's tokens fit the
  // table (60000 x 1 x 192: 32 us with four, 21 with one).
  const bool single = rows * g.slots < static_cast<int64_t>(multiprocessors()) * 2048 || (half && V == kMost && a.h == 1);
  const int R = single ? 1 : !vec || V * sizeof(T) <= 4 ? 8 : 4;
  const dim3 grid(static_cast<unsigned>((rows + static_cast<int64_t>(groups) * R - 1) / (static_cast<int64_t>(groups) * R)),
                  static_cast<unsigned>((g.slots + g.slots_block - 1) / g.slots_block));
  if (!vec)
    return R > 1 ? launch_pdl(rope_pair_kernel<T, 8>, grid, dim3(threads), 0, s, 1, a, g)
                 : launch_pdl(rope_pair_kernel<T, 1>, grid, dim3(threads), 0, s, 1, a, g);
  if constexpr (kMost == 8) {
    if (V == 8) return half ? launch_rope_v<T, true, 8>(a, g, grid, threads, R, s) : launch_rope_v<T, false, 8>(a, g, grid, threads, R, s);
  }
  if (V == 4) return half ? launch_rope_v<T, true, 4>(a, g, grid, threads, R, s) : launch_rope_v<T, false, 4>(a, g, grid, threads, R, s);
  if (V == 2) return half ? launch_rope_v<T, true, 2>(a, g, grid, threads, R, s) : launch_rope_v<T, false, 2>(a, g, grid, threads, R, s);
  return launch_rope_v<T, true, 1>(a, g, grid, threads, R, s);
}

// ---- the cache writers with the rotation on the way ---------------------------------
// One warp per token, as in the plain writers: lane i computes the sine and cosine of
// frequency i of the token's position, and the lanes that hold a pair's values fetch them
// by shuffle.  The turned values are not rounded to bf16 in between: each code is the nearest of
// the turned value, known to 2^-41 of its pair's size (times the amplitude in fp32).
constexpr int kWarpsPerBlock = 8;
constexpr int kRot = 64;

// Sums and products of such pairs of floats (Dekker, "A floating-point technique for extending the
// available precision", 1971; Knuth's two-sum), good to some 2^-46.
__device__ __forceinline__ Two mul(const Two& a, const Two& b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return two_sum_ordered(p, fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi));
}
__device__ __forceinline__ Two add(const Two& a, const Two& b) {  // |a| >= |b|
  const Two s = two_sum_ordered(a.hi, b.hi);
  return two_sum_ordered(s.hi, s.lo + (a.lo + b.lo));
}
struct CosSin {
  Two c, s;
};
// phase_cs to 2^-41: the terms down to x^7 and x^6 in pairs of floats, those behind them (below 4e-7 and
// 4e-6 together, to x^15 and x^14) in floats.  Out of line, for one token in some 10^4.
__device__ __noinline__ CosSin phase_two(int pos, int64_t turns, float amp) {
  uint32_t quarter;
  const int64_t rest = phase_rest(pos, turns, quarter);
  const float rh = static_cast<float>(rest);
  constexpr double kRad = 6.283185307179586476925 / 18446744073709551616.0;  // 2 pi 2^-64
  constexpr float kHi = static_cast<float>(kRad);
  const Two x = mul({rh, static_cast<float>(rest - static_cast<int64_t>(rh))}, {kHi, static_cast<float>(kRad - static_cast<double>(kHi))});
  const Two z = mul(x, x);
  auto fraction = [](int n) {  // 1 / n
    const float h = static_cast<float>(1.0 / n);
    return Two{h, static_cast<float>(1.0 / n - static_cast<double>(h))};
  };
  float S = -1.0f / 1307674368000.0f, C = -1.0f / 87178291200.0f;
  S = fmaf(S, z.hi, 1.0f / 6227020800.0f);
  S = fmaf(S, z.hi, -1.0f / 39916800.0f);
  S = fmaf(S, z.hi, 1.0f / 362880.0f);
  C = fmaf(C, z.hi, 1.0f / 479001600.0f);
  C = fmaf(C, z.hi, -1.0f / 3628800.0f);
  C = fmaf(C, z.hi, 1.0f / 40320.0f);
  Two sn = add(fraction(-5040), {S * z.hi, 0.f}), cn = add(fraction(-720), {C * z.hi, 0.f});
  sn = add(fraction(120), mul(sn, z));
  sn = add(fraction(-6), mul(sn, z));
  sn = add(x, mul(mul(x, z), sn));
  cn = add(fraction(24), mul(cn, z));
  cn = add({-0.5f, 0.f}, mul(cn, z));
  cn = add({1.0f, 0.f}, mul(cn, z));
  // a quarter turn: (c, s) -> (-s, c)
  const bool swap = quarter & 1u;
  const Two c = swap ? sn : cn, s = swap ? cn : sn;
  return {mul(c, {((quarter + 1u) & 2u) ? -amp : amp, 0.f}), mul(s, {(quarter & 2u) ? -amp : amp, 0.f})};
}

// a c + b s as hi + lo (a, b exact inputs); an infinity or NaN has no low part
__device__ __forceinline__ Two dot2(float a, const Two& c, float b, const Two& s) {
  const float p = __fmul_rn(a, c.hi), q = __fmul_rn(b, s.hi);
  const float e = fmaf(a, c.hi, -p) + fmaf(b, s.hi, -q);   // the products' roundings
  const float h = p + q, t = h - p;
  if (!(fabsf(h) < INFINITY)) return {h, 0.f};
  const float f = (p - (h - t)) + (q - t);                 // the sum's rounding (Knuth's two-sum)
  const float l = f + e + fmaf(a, c.lo, b * s.lo);
  return two_sum_ordered(h, l);
}
__device__ __forceinline__ Two neg(const Two& v) { return {-v.hi, -v.lo}; }
__device__ __forceinline__ Two shfl(const Two& v, int lane) {
  return {__shfl_sync(0xffffffffu, v.hi, lane), __shfl_sync(0xffffffffu, v.lo, lane)};
}

// the k values of this lane (dims 4 lane ..) turned where they lie in [offset, offset + 64),
// rounded to odd (see quotient_round_to_odd): their E4M3 codes and the exponent of the
// largest are then those of the unrounded values
__device__ __forceinline__ float to_odd(const Two& v) {
  uint32_t b = __float_as_uint(v.hi);
  if (v.lo != 0.f && (b & 1u) == 0u) b += ((v.lo > 0.f) == (v.hi > 0.f)) ? 1u : 0xFFFFFFFFu;
  return __uint_as_float(b);
}
__device__ __forceinline__ void turn_k(float (&x)[4], const CosSin& cs, int offset, bool half_layout) {
  const int lane = threadIdx.x & 31;
  const int li = lane - (offset >> 2);  // 0..15 inside the rotary part
  const bool mine = li >= 0 && li < kRot / 4;
  if (half_layout) {
    const bool first = li < 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float other = __shfl_sync(0xffffffffu, x[j], first ? lane + 8 : lane - 8);
      const Two c = shfl(cs.c, 4 * (li & 7) + j), s = shfl(cs.s, 4 * (li & 7) + j);
      const float y = to_odd(dot2(x[j], c, other, first ? neg(s) : s));
      // (the partner's shuffle of this j has read x[j] already)
      if (mine) x[j] = y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Two c = shfl(cs.c, 2 * li + j), s = shfl(cs.s, 2 * li + j);
      const float p = x[2 * j], q = x[2 * j + 1];
      const float y0 = to_odd(dot2(p, c, q, neg(s))), y1 = to_odd(dot2(q, c, p, s));
      if (mine) {
        x[2 * j] = y0;
        x[2 * j + 1] = y1;
      }
    }
  }
}

// the rope tile's values of this lane (2 lane, 2 lane + 1 of 64), turned
__device__ __forceinline__ void turn_kv(float x0, float x1, const CosSin& cs, bool half_layout, Two& y0, Two& y1) {
  const int lane = threadIdx.x & 31;
  if (half_layout) {
    const float o0 = __shfl_xor_sync(0xffffffffu, x0, 16), o1 = __shfl_xor_sync(0xffffffffu, x1, 16);
    const Two c0 = shfl(cs.c, 2 * lane), c1 = shfl(cs.c, 2 * lane + 1);
    const Two s0 = shfl(cs.s, 2 * lane), s1 = shfl(cs.s, 2 * lane + 1);
    y0 = dot2(x0, c0, o0, lane < 16 ? neg(s0) : s0);
    y1 = dot2(x1, c1, o1, lane < 16 ? neg(s1) : s1);
  } else {
    y0 = dot2(x0, cs.c, x1, neg(cs.s));
    y1 = dot2(x1, cs.c, x0, cs.s);
  }
}

// two packed bf16 values -> fp32 (exact)
__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t v) {
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&v);
  return make_float2(__low2float(b), __high2float(b));
}
// |x| / s rounded to odd as quotient_round_to_odd does, for a value known as x + low (low at
// most half an ulp of x): the remainder's sign decides, and low has its share in it.  (low may move
// the quotient by an ulp or more, past the neighbours of x's own: hence the second quotient.)
__device__ __forceinline__ float sum_quotient_round_to_odd(float x, float low, float s) {
  const float a = fabsf(x), b = x < 0.f ? -low : low, q0 = __fdiv_rn(a, s);
  const float q = q0 + __fdiv_rn(__fmaf_rn(-q0, s, a) + b, s);
  const float r = __fmaf_rn(-q, s, a) + b;
  uint32_t qb = __float_as_uint(q);
  if (r != 0.f && (qb & 1u) == 0u) qb += (r > 0.f) ? 1u : 0xFFFFFFFFu;
  return copysignf(__uint_as_float(qb), x);
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

// What the screened forms below allow for: 2^-22 of |a c| + |b s| covers the roundings of
// the fp32 rotation (c, s, the products and the sum, half an ulp each).
constexpr float kTurnErr = 2.384185791015625e-07f;

// One token's key.  The fp32 rotation decides every code and exponent that is the same at
// both ends of its error interval; a token with any other (one in some 10^4) is done again
// from hi + lo.
__device__ __forceinline__ void turn_store_k(uint2 raw, float2 cr, int pos, int64_t turns, const RopeQuantArgs& a,
                                             int64_t slot) {
  const int lane = threadIdx.x & 31;
  const float2 r0 = bf16x2_to_f32(raw.x), r1 = bf16x2_to_f32(raw.y);
  float x[4] = {r0.x, r0.y, r1.x, r1.y};
  const int li = lane - (a.k_offset >> 2);
  const bool mine = li >= 0 && li < kRot / 4;
  float y[4], err[4];
  if (a.k_layout == DSA_ROPE_HALF) {
    const bool first = li < 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float other = __shfl_sync(0xffffffffu, x[j], first ? lane + 8 : lane - 8);
      const float c = __shfl_sync(0xffffffffu, cr.x, 4 * (li & 7) + j);
      const float s = __shfl_sync(0xffffffffu, cr.y, 4 * (li & 7) + j);
      const float p = other * (first ? -s : s);
      y[j] = fmaf(x[j], c, p);
      err[j] = fmaf(fabsf(x[j]), fabsf(c), fabsf(p)) * kTurnErr;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float c = __shfl_sync(0xffffffffu, cr.x, 2 * li + j);
      const float s = __shfl_sync(0xffffffffu, cr.y, 2 * li + j);
      const float p = x[2 * j], q = x[2 * j + 1], u = q * -s, v = p * s;
      y[2 * j] = fmaf(p, c, u);
      y[2 * j + 1] = fmaf(q, c, v);
      err[2 * j] = fmaf(fabsf(p), fabsf(c), fabsf(u)) * kTurnErr;
      err[2 * j + 1] = fmaf(fabsf(q), fabsf(c), fabsf(v)) * kTurnErr;
    }
  }
  if (!mine) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = x[j];
      err[j] = 0.f;
    }
  }
  // (the maxima of a group of 32 dims, eight lanes)
  auto group_max = [](float v) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  };
  auto top4 = [](const float (&v)[4]) { return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))); };
  float amax = group_max(top4(y));
  const float emax = group_max(top4(err));
  int e = mx_shared_exp(amax);
  float inv = exp2i(-e);  // exact power of two: y * inv is exact
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    lo[j] = f32x2_to_e4m3x2((y[2 * j] - err[2 * j]) * inv, (y[2 * j + 1] - err[2 * j + 1]) * inv);
    hi[j] = f32x2_to_e4m3x2((y[2 * j] + err[2 * j]) * inv, (y[2 * j + 1] + err[2 * j + 1]) * inv);
  }
  const bool same = lo[0] == hi[0] && lo[1] == hi[1] && mx_shared_exp(amax - emax) == e &&
                    mx_shared_exp(amax + emax) == e && amax > 0.f;
  if (__any_sync(0xffffffffu, !same && emax > 0.f)) {  // (a group without rotary dims is exact as it is)
    turn_k(x, phase_two(pos, turns, a.amplitude), a.k_offset, a.k_layout == DSA_ROPE_HALF);
    amax = group_max(top4(x));
    e = mx_shared_exp(amax);
    inv = exp2i(-e);
    lo[0] = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv);
    lo[1] = f32x2_to_e4m3x2(x[2] * inv, x[3] * inv);
  }
  uint8_t* page = a.k_cache + (slot / kPage) * kKPageBytes;
  const int row = static_cast<int>(slot % kPage);
  *reinterpret_cast<uint32_t*>(page + row * kIdxDim + 4 * lane) = amax > 0.f ? lo[0] | (lo[1] << 16) : 0u;
  if ((lane & 7) == 0) page[kKScaleOff + row * 4 + (lane >> 3)] = static_cast<uint8_t>(e + 127);
}

// One token's latent row.
//
// The four unturned tiles.  Code = E4M3(x / s), s = fp32(amax / 448), x and amax of 8
// significant bits.  Unless 448 x = B amax for a border B between two codes (of 5 bits or
// fewer), the two sides are integers of at most 13 bits and differ by 2^-13 or more of
// their size, so x times an approximate 1 / s decides.  If they are equal, x / s lies beside
// B by as little as s's own rounding, on the side that the sign of amax - 448 s gives for
// the whole tile: a reciprocal pushed that way by 2^-18 decides both cases with one
// product per value.  Where s is exact (amax a multiple of 7, one tile in seven) the tie is a true
// one, and the corrected quotient (exact where it is representable: Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990) leaves it to the
// conversion.  Division instead of this took 60% of the writer's instructions.
//
// The rope tile goes like the key: the fp32 rotation decides where its error interval, widened
// by the scale's, holds one code; else hi + lo does.
//
// Lane t works out tile t's scale and reciprocal, so that the five cost one division.
__device__ __forceinline__ void turn_store_kv(const uint2 (&raws)[4], uint32_t rope, float2 cr, int pos, int64_t turns,
                                              const RopeQuantArgs& a, int64_t slot) {
  const int lane = threadIdx.x & 31;
  uint8_t* rec = a.kv_cache + slot * kKvTokBytes;
  const bool half_layout = a.kv_layout == DSA_ROPE_HALF;
  const float2 x = bf16x2_to_f32(rope);
  float y0, y1, err0, err1;
  {
    if (half_layout) {
      const float o0 = __shfl_xor_sync(0xffffffffu, x.x, 16), o1 = __shfl_xor_sync(0xffffffffu, x.y, 16);
      const float c0 = __shfl_sync(0xffffffffu, cr.x, 2 * lane), c1 = __shfl_sync(0xffffffffu, cr.x, 2 * lane + 1);
      const float s0 = __shfl_sync(0xffffffffu, cr.y, 2 * lane), s1 = __shfl_sync(0xffffffffu, cr.y, 2 * lane + 1);
      const float p0 = o0 * (lane < 16 ? -s0 : s0), p1 = o1 * (lane < 16 ? -s1 : s1);
      y0 = fmaf(x.x, c0, p0);
      y1 = fmaf(x.y, c1, p1);
      err0 = fmaf(fabsf(x.x), fabsf(c0), fabsf(p0)) * kTurnErr;
      err1 = fmaf(fabsf(x.y), fabsf(c1), fabsf(p1)) * kTurnErr;
    } else {
      const float p0 = -x.y * cr.y, p1 = x.x * cr.y;
      y0 = fmaf(x.x, cr.x, p0);
      y1 = fmaf(x.y, cr.x, p1);
      err0 = fmaf(fabsf(x.x), fabsf(cr.x), fabsf(p0)) * kTurnErr;
      err1 = fmaf(fabsf(x.y), fabsf(cr.x), fabsf(p1)) * kTurnErr;
    }
  }
  float amax = warp_amax(fmaxf(fabsf(y0), fabsf(y1)));  // lane t: tile t's from here on
#pragma unroll
  for (int tile = 0; tile < 4; ++tile) {
    const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&raws[tile].x)),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raws[tile].y)));
    const float v = warp_amax(fmaxf(__low2float(m), __high2float(m)));
    if (lane == tile) amax = v;
  }
  float s = __fdiv_rn(amax, 448.0f);
  const bool usable = s > 1e-30f && s < 1e30f;  // 1 / s and s itself are far from the range's ends
  const float rem = fmaf(-448.0f, s, amax);
  float inv = usable ? __fdividef(1.0f, s) : 0.f;
  if (lane < 4 && rem != 0.f) inv = fmaf(inv, copysignf(3.814697265625e-06f, rem), inv);  // 2^-18
  const uint32_t exact = __ballot_sync(0xffffffffu, rem == 0.f);
  const uint32_t fast = __ballot_sync(0xffffffffu, usable);
#pragma unroll
  for (int tile = 0; tile < 4; ++tile) {
    const float2 p = bf16x2_to_f32(raws[tile].x), q = bf16x2_to_f32(raws[tile].y);
    const float ti = __shfl_sync(0xffffffffu, inv, tile);
    float v[4] = {p.x * ti, p.y * ti, q.x * ti, q.y * ti};
    if (!((fast >> tile) & 1u) || ((exact >> tile) & 1u)) {
      const float ts = __shfl_sync(0xffffffffu, s, tile);
      const float xs[4] = {p.x, p.y, q.x, q.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = (fast >> tile) & 1u ? fmaf(fmaf(-v[i], ts, xs[i]), ti, v[i])
                                   : ts > 0.f ? quotient_round_to_odd(xs[i], ts) : 0.f;
    }
    *reinterpret_cast<uint32_t*>(rec + tile * 128 + 4 * lane) = codes4(v[0], v[1], v[2], v[3]);
  }
  {
    float rs = __shfl_sync(0xffffffffu, s, 4);
    const float ri = __shfl_sync(0xffffffffu, inv, 4);
    // (2^-20 of the value: the scale's and the reciprocal's own errors)
    const float d0 = fmaf(fabsf(y0), 4.0f * kTurnErr, err0), d1 = fmaf(fabsf(y1), 4.0f * kTurnErr, err1);
    uint16_t codes = f32x2_to_e4m3x2((y0 - d0) * ri, (y1 - d1) * ri);
    const bool same = codes == f32x2_to_e4m3x2((y0 + d0) * ri, (y1 + d1) * ri);
    if (!((fast >> 4) & 1u) || __any_sync(0xffffffffu, !same)) {
      Two t0, t1;
      turn_kv(x.x, x.y, phase_two(pos, turns, a.amplitude), half_layout, t0, t1);
      const float top = warp_amax(fmaxf(fabsf(t0.hi), fabsf(t1.hi)));
      // the low part that goes with the largest: the scale is (top + low) / 448 rounded once
      float low = -INFINITY;
      if (fabsf(t0.hi) == top) low = t0.hi < 0.f ? -t0.lo : t0.lo;
      if (fabsf(t1.hi) == top) low = fmaxf(low, t1.hi < 0.f ? -t1.lo : t1.lo);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) low = fmaxf(low, __shfl_xor_sync(0xffffffffu, low, o));
      rs = __fdiv_rn(top, 448.0f);
      const float rest = fmaf(-448.0f, rs, top) + low;
      if (fabsf(rest) < top) rs += rest * (1.0f / 448.0f);  // (not where either is 0, infinite or NaN)
      codes = rs > 0.f ? f32x2_to_e4m3x2(sum_quotient_round_to_odd(t0.hi, t0.lo, rs),
                                         sum_quotient_round_to_odd(t1.hi, t1.lo, rs)) : 0;
      if (lane == 4) s = rs;
    }
    *reinterpret_cast<uint16_t*>(rec + 512 + 2 * lane) = codes;
  }
  if (lane < 8) *reinterpret_cast<float*>(rec + kKvScaleOff + 4 * lane) = lane < 5 ? s : 0.f;
}

__global__ void __launch_bounds__(kWarpsPerBlock * 32, 4)
rope_quant_kernel(RopeQuantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t turns = a.turns[lane];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + (threadIdx.x >> 5); t < a.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarpsPerBlock) {
    const int64_t slot = a.slots[t];
    const int pos = a.pos[t];
    uint2 k, kv[4];
    uint32_t rope;
    if (a.k) k = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.k) + t * a.k_stride + 4 * lane);
    if (a.kv) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.kv) + t * a.kv_stride;
#pragma unroll
      for (int tile = 0; tile < 4; ++tile) kv[tile] = *reinterpret_cast<const uint2*>(src + tile * 128 + 4 * lane);
      rope = *reinterpret_cast<const uint32_t*>(src + 512 + 2 * lane);
    }
    if (slot >= a.num_slots) {
      if (lane == 0) flag(a.status, DSA_STATUS_BAD_PAGE);
    } else if (slot >= 0) {
      const float2 cs = phase_cs(pos, turns, a.amplitude);
      if (a.k) turn_store_k(k, cs, pos, turns, a, slot);
      if (a.kv) turn_store_kv(kv, rope, cs, pos, turns, a, slot);
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
  const int cap = multiprocessors() * 16;
  const int blocks = a.n_tokens / kWarpsPerBlock + (a.n_tokens % kWarpsPerBlock != 0);
  return launch_pdl(rope_quant_kernel, dim3(blocks < cap ? blocks : cap), dim3(kWarpsPerBlock * 32), 0, s, 1, a);
}

}  // namespace dsa
