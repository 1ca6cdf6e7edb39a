// What the per-head norm with rotation (norm_rope.cu) and its gradient (norm_rope_grad.cu) share: how the
// rows of a call are laid over lanes, the tables of a block, and the turn of a row's rotary part.
//
// A row is one head of one token.  A group of G lanes holds a whole row in registers, vector
// first + j part of it in a lane's j-th word, so that it is read once however often it is summed over.  Ordinarily
// first is the lane and part is G; where the layout turns vectors of 16 bytes half a rotary part of 2^k of them
// apart, part is that distance and a lane holds both of a pair (norm_pairs).
// With vectors of 16 bytes eight lanes cover 128 consecutive bytes, as much as a memory request wants,
// and a warp has four rows under way; longer rows take 16 or 32 lanes so that a lane holds at most 32
// elements in fp32.
#pragma once

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "dsa_common.cuh"
#include "dsa_launch.h"
#include "rope_math.cuh"

namespace dsa {
namespace {

constexpr int kNormThreads = 256;
// Shared memory that a block takes at most: of 1024 dims weights and biases 8 KB, and of the rows of one step, 8192
// elements, a sine and a cosine a pair and the exchange 32 KB each; the gradient's sums 64 KB in their place.  What a kernel may
// ask for is always this, whatever a call needs: another thread's call may set it between this one's and its launch.
constexpr int kNormShared = 76 * 1024;

struct NormGeom {
  int lanes;          // G: lanes a row, a power of two of 8..32
  int vectors;        // of one row
  int rows_step;      // rows of a block at a time: kNormThreads / lanes
  int rows_table;     // rows whose tokens' sines are in shared memory together, a multiple of rows_step
  int tokens_table;   // tokens that those can touch
  int step_t, step_h; // rows_step as whole tokens and heads
  int span_pad;       // norm_dim rounded up to 4, floats of the weights' table
  int part;           // vectors between a lane's words
  int pair_word, pair_block;  // the word whose pairs are in the next, and the block of `part` lanes that has them; -1: none
  int turn_word;      // the word of the lanes that is the whole rotary part, -1: there is none
};

// one float of the weight or bias
__device__ __forceinline__ float norm_param(const void* p, int dtype, int i) {
  if (dtype == DSA_DTYPE_FP32) return static_cast<const float*>(p)[i];
  if (dtype == DSA_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// A block's shared memory: weights (ones where there are none) and biases (zeros) in fp32, the sines of the
// tokens at hand, and each row's rotary part for exchange.
struct NormShared {
  float* weight;
  float* bias;
  float2* cs;
  float* ex;
  int first;         // token of cs's first row
  int64_t rows_end;  // rows before it have their sines there
};
__device__ __forceinline__ NormShared norm_shared(const NormArgs& a, const NormGeom& g, unsigned char* raw) {
  NormShared s;
  s.weight = reinterpret_cast<float*>(raw);
  s.bias = s.weight + g.span_pad;
  s.cs = reinterpret_cast<float2*>(s.bias + g.span_pad);
  s.ex = reinterpret_cast<float*>(s.cs + g.tokens_table * ((a.rot / 2 + 1) & ~1));
  s.first = 0;
  s.rows_end = 0;
  return s;
}
// Where the tables have dim e: vectors of eight in two halves, so that eight lanes read 128 bytes next to one another (from
// vectors as they are, every second bank twice, 4096 x 64 rows of 128 took 28.9 us instead of 28.0).
template <int V>
__device__ __forceinline__ int norm_param_at(const NormGeom& g, int e) {
  return V == 8 ? (e & 4 ? g.span_pad >> 1 : 0) + (e >> 3) * 4 + (e & 3) : e;
}
template <int V>
__device__ __forceinline__ void norm_fill_params(const NormArgs& a, const NormGeom& g, const NormShared& s) {
  for (int i = threadIdx.x; i < a.span; i += kNormThreads) {
    const int at = norm_param_at<V>(g, i);
    s.weight[at] = a.weight ? norm_param(a.weight, a.w_dtype, i) : 1.f;
    s.bias[at] = a.bias ? norm_param(a.bias, a.w_dtype, i) : 0.f;
  }
}
// the sines of the tokens of the rows from r0 on, as many as the table holds; every thread of the block calls it, and it
// synchronises them whenever the table changes
__device__ __forceinline__ void norm_fill_cs(const NormArgs& a, const NormGeom& g, NormShared& s, int64_t r0, int64_t end) {
  if (r0 < s.rows_end) return;
  s.rows_end = min(r0 + g.rows_table, end);
  s.first = static_cast<int>(static_cast<uint32_t>(r0) / static_cast<uint32_t>(a.h));
  const int last = static_cast<int>(static_cast<uint32_t>(s.rows_end - 1) / static_cast<uint32_t>(a.h));
  __syncthreads();
  const int half = a.rot >> 1, pitch = (half + 1) & ~1, count = (last - s.first + 1) * half;
  for (int i = threadIdx.x; i < count; i += kNormThreads) {
    const int t = i / half, f = i - t * half;
    const float2 v = phase_cs(a.pos[s.first + t], a.turns[f], a.amplitude);
    if (g.pair_word >= 0) {  // a token's cosines, then its sines
      float* to = reinterpret_cast<float*>(s.cs + t * pitch);
      to[f] = v.x;
      to[half + f] = v.y;
    } else {
      s.cs[t * pitch + f] = v;
    }
  }
  __syncthreads();
}

// A thread's place among the rows: token and head of its row
struct RowAt {
  int t, hh;
  __device__ __forceinline__ RowAt(int64_t row, int h)
      : t(static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(h))),
        hh(static_cast<int>(static_cast<uint32_t>(row) - static_cast<uint32_t>(t) * static_cast<uint32_t>(h))) {}
  // on by a step of rows; whether that is into a later token's first heads
  __device__ __forceinline__ bool step(const NormGeom& g, int h) {
    t += g.step_t;
    hh += g.step_h;
    const bool wrap = hh >= h;
    if (wrap) {
      hh -= h;
      ++t;
    }
    return wrap;
  }
};
// Its address in a tensor: kept by addition
template <typename P>
struct RowPtr {
  P* p;
  int64_t by, by_wrap;
  __device__ __forceinline__ RowPtr(P* base, const RowAt& at, const NormGeom& g, int h, int64_t stride_t, int64_t stride_h)
      : p(base + at.t * stride_t + at.hh * stride_h), by(g.step_t * stride_t + g.step_h * stride_h),
        by_wrap(by + stride_t - h * stride_h) {}
  __device__ __forceinline__ void step(bool wrap) { p += wrap ? by_wrap : by; }
};

// pairs of floats in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// y[i] = y[i] * w[i] (+ b[i]) over V elements, and sums of products
template <int V>
__device__ __forceinline__ void scale_by(float* y, const float* w) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = mul2(make_float2(y[i], y[i + 1]), make_float2(w[i], w[i + 1]));
      y[i] = r.x;
      y[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] *= w[i];
  }
}
template <int V>
__device__ __forceinline__ void scale_all(float* y, float f) {
  const float w[2] = {f, f};
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) scale_by<2>(y + i, w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] *= f;
  }
}
// sum += a[i] b[i], even and odd elements apart
template <int V>
__device__ __forceinline__ void add_products(float2& sum, const float* a, const float* b) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) sum = fma2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), sum);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) sum.x = fmaf(a[i], b[i], sum.x);
  }
}

// V elements of T as floats, and back, pairs of 16 bits in one conversion
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& x, float* y) {
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = Elem<T>::get(x.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> narrow(const float* y) {
  Vec<T, V> o;
  if constexpr (sizeof(T) == 2 && V > 1) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (sizeof(T) == sizeof(__half) && std::is_same<T, __half>::value) {
        const __half2 p = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
    memcpy(&o, w, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = Elem<T>::put(y[i]);
  }
  return o;
}

// The sum over a row's lanes, in every one of them.
__device__ __forceinline__ float row_sum(float v, int lanes) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lanes > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
  if (lanes > 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
  return v;
}

// V floats from or to shared memory, 16 bytes at a time where they are aligned
template <int V>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
  }
}
// the V weights or biases from dim e0 on
template <int V>
__device__ __forceinline__ void load_params(const NormGeom& g, const float* table, int e0, float (&v)[V]) {
  if constexpr (V == 8) {
    float lo[4], hi[4];
    load_floats(table + (e0 >> 1), lo);
    load_floats(table + (g.span_pad >> 1) + (e0 >> 1), hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = lo[i];
      v[4 + i] = hi[i];
    }
  } else {
    load_floats(table + e0, v);
  }
}

// Turn the rotary part of the row in y (fp32, in the lanes' layout); TRANSPOSE turns back.  Pairs of neighbours
// lie in one vector, and a partner half a rotary part away in the same lane where norm_pairs could place it there.
// Elsewhere it comes by shuffle where the whole rotary part is one word of the
// lanes (g.turn_word: as many pairs as one exchange can carry); otherwise, and with vectors of one element, through
// shared memory, ex: the row's own rot floats there.
template <int V, int NV, bool TRANSPOSE>
__device__ __forceinline__ void turn_row(const NormArgs& a, const NormGeom& g, float (&y)[NV * V], const float2* cs,
                                         float* ex, int lane, int first) {
  const bool half_layout = a.layout == DSA_ROPE_HALF;
  const int half = a.rot >> 1;
  if (V >= 4 && NV > 1 && g.pair_word >= 0) {
    const int at = lane & (g.part - 1);
    if ((lane - at) != g.pair_block * g.part) return;
    float c[V], s[V];
    load_floats(reinterpret_cast<const float*>(cs) + at * V, c);
    load_floats(reinterpret_cast<const float*>(cs) + half + at * V, s);
#pragma unroll
    for (int j = 0; j + 1 < NV; ++j) {
      if (j != g.pair_word) continue;  // (the same in all threads)
#pragma unroll
      for (int i = 0; i + 1 < V; i += 2) {
        float *p = y + j * V + i, *q = p + V;
        const float2 x0 = make_float2(p[0], p[1]), x1 = make_float2(q[0], q[1]), co = make_float2(c[i], c[i + 1]);
        const float2 plus = TRANSPOSE ? make_float2(-s[i], -s[i + 1]) : make_float2(s[i], s[i + 1]);
        const float2 z0 = fma2(x1, make_float2(-plus.x, -plus.y), mul2(x0, co)), z1 = fma2(x0, plus, mul2(x1, co));
        p[0] = z0.x;
        p[1] = z0.y;
        q[0] = z1.x;
        q[1] = z1.y;
      }
    }
  } else if (V > 1 && half_layout && g.turn_word >= 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j != g.turn_word) continue;  // (the same in all threads)
      const int rel = (first + j * g.part) * V - a.offset;
      const bool mine = rel >= 0 && rel < a.rot, second = rel >= half;
      const int from = (threadIdx.x & 31) + (second ? -half / V : half / V);
      // the first of a pair becomes a c - b s, the second b c + a s: the one that sends gives the sign
      const float sign = second == TRANSPOSE ? 1.f : -1.f;
      float other[V];
#pragma unroll
      for (int i = 0; i < V; ++i) other[i] = sign * y[j * V + i];
#pragma unroll
      for (int i = 0; i < V; ++i) other[i] = __shfl_sync(0xffffffffu, other[i], from);
      if (mine) {
        float c[2 * V];
        load_floats(reinterpret_cast<const float*>(cs + (second ? rel - half : rel)), c);
#pragma unroll
        for (int i = 0; i < V; i += 2) {  // (a word of several elements has an even number)
          const float2 p = mul2(make_float2(other[i], other[i + 1]), make_float2(c[2 * i + 1], c[2 * i + 3]));
          const float2 z = fma2(make_float2(y[j * V + i], y[j * V + i + 1]), make_float2(c[2 * i], c[2 * i + 2]), p);
          y[j * V + i] = z.x;
          y[j * V + i + 1] = z.y;
        }
      }
    }
  } else if (half_layout || V == 1) {
    __syncwarp();  // (the row before has been read)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int rel = (first + j * g.part) * V - a.offset;
      if (rel >= 0 && rel < a.rot) {
#pragma unroll
        for (int i = 0; i < V; ++i) ex[rel + i] = y[j * V + i];
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int rel = (first + j * g.part) * V - a.offset;
      if (rel >= 0 && rel < a.rot) {
        const bool second = half_layout ? rel >= half : rel & 1;
        const int f = half_layout ? (second ? rel - half : rel) : rel >> 1;
        const int other = half_layout ? (second ? rel - half : rel + half) : rel ^ 1;
        const float sign = second == TRANSPOSE ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 c = cs[f + i];
          y[j * V + i] = fmaf(y[j * V + i], c.x, sign * c.y * ex[other + i]);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int rel = (first + j * g.part) * V - a.offset;
      if (rel >= 0 && rel < a.rot) {
        float c[V];
        load_floats(reinterpret_cast<const float*>(cs + (rel >> 1)), c);
#pragma unroll
        for (int i = 0; i + 1 < V; i += 2) {
          const float p = y[j * V + i], q = y[j * V + i + 1], s = TRANSPOSE ? -c[i + 1] : c[i + 1];
          y[j * V + i] = p * c[i] - q * s;
          y[j * V + i + 1] = p * s + q * c[i];
        }
      }
    }
  }
}

// The widest vector, in elements, that divides every address, stride and part of a row, at most 16 bytes.
inline int norm_vector(uint64_t address_bits, uint64_t stride_bits, const NormArgs& a, int size) {
  const uint64_t all = address_bits / size | stride_bits | static_cast<uint64_t>(a.d | a.span | a.offset) |
                       static_cast<uint64_t>(a.layout == DSA_ROPE_HALF ? a.rot / 2 : a.rot) | static_cast<uint64_t>(16 / size);
  return static_cast<int>(all & (~all + 1));
}
inline NormGeom norm_geom(const NormArgs& a, int v, int size) {
  NormGeom g;
  g.vectors = a.d / v;
  g.lanes = v * size < 16 ? 32 : g.vectors <= 32 ? 8 : g.vectors <= 64 ? 16 : 32;
  g.rows_step = kNormThreads / g.lanes;
  g.step_t = g.rows_step / a.h;
  g.step_h = g.rows_step % a.h;
  g.span_pad = (a.span + 3) & ~3;
  const int first = a.offset / v, last = (a.offset + a.rot) / v - 1;  // (V divides both in the half layout)
  g.part = g.lanes;
  g.pair_word = g.pair_block = -1;
  g.turn_word = v > 1 && first / g.lanes == last / g.lanes ? first / g.lanes : -1;
  return g;
}
// Whether a lane can hold both of a pair: vectors half a rotary part apart then are its words j and j + 1.  (Rows of 128 with
// 64 turned, 4096 x 64 bf16: 28.9 us, by shuffle 29.6.)  Vectors of 16 bytes alone, two next to one another, so that no
// sector of memory is asked for twice.
template <int V, int NV>
void norm_pairs(const NormArgs& a, NormGeom& g, int size) {
  const int apart = a.rot / 2 / V;
  if (V * size != 16 || a.layout != DSA_ROPE_HALF || (a.rot / 2) % V || apart < 2 || apart > g.lanes || (apart & (apart - 1)) ||
      (g.vectors + g.lanes - 1) / g.lanes != NV || a.offset / V % apart)
    return;
  const int word = a.offset / V / apart % NV;
  if (word + 1 >= NV) return;
  g.part = apart;
  g.pair_word = word;
  g.pair_block = a.offset / V / apart / NV;
}
// a lane's first vector
template <int NV>
__device__ __forceinline__ int norm_first(const NormGeom& g, int lane) {
  const int at = lane & (g.part - 1);
  return (lane - at) * NV + at;
}
// The table holds the sines of one step's tokens at least; of a block's whole share where that takes 16 KB at most.
inline void norm_table(const NormArgs& a, NormGeom& g, int64_t rows_block) {
  const int64_t bytes = sizeof(float2) * ((a.rot / 2 + 1) & ~1);
  auto tokens = [&](int64_t rows) { return std::min<int64_t>((rows + a.h - 2) / a.h + 1, a.n); };
  int64_t rows = rows_block;
  while (rows > g.rows_step && tokens(rows) * bytes > 16384) rows = (rows / 2 + g.rows_step - 1) / g.rows_step * g.rows_step;
  g.rows_table = static_cast<int>(std::min<int64_t>(rows, 1 << 30));
  g.tokens_table = static_cast<int>(tokens(rows));
}
template <typename K>
cudaError_t norm_allow_shared(K kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  if (bytes > kNormShared) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormShared);
}
inline size_t norm_shared_bytes(const NormArgs& a, const NormGeom& g) {
  const bool exchange = !(a.layout == DSA_ROPE_HALF ? g.turn_word >= 0 || g.pair_word >= 0 : g.vectors < a.d);  // (see turn_row)
  return 2 * sizeof(float) * g.span_pad + sizeof(float2) * g.tokens_table * ((a.rot / 2 + 1) & ~1) +
         (exchange ? sizeof(float) * g.rows_step * a.rot : 0);
}

}  // namespace
}  // namespace dsa
