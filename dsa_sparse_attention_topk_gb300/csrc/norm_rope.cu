// Queries and keys normed per head and turned by their positions in one pass (dsa_norm_rope), and the cache
// writers with both on the way (dsa_norm_rope_quant_kv).
//
// The first `span` dims of a head become (x - mu) / sqrt(mean (x - mu)^2 + eps) * w + b, mu their mean or
// zero; then pairs of the rotary part are turned as in rope.cu.  Sums, the normed values and the turn are
// fp32, and the result is rounded once: a value is good to a few roundings of fp32 of the row's size.  The
// mean is taken off before anything is squared, so that a row far from zero loses nothing.
//
// Bound: memory, each value read and written once.  A row stays in the registers of 8 to 32 lanes between the
// sums and the turn, 8 to 32 values a lane.  4096 x 64 x 128 bf16 take 26 us, 5.2 TB/s (a plain copy 20, this kernel
// without weights, sums and turn 22.5): the rest is issue and the tables' way through shared memory.

#include "norm_rope.cuh"

namespace dsa {
namespace {

// blocks on an SM together, by the registers that a lane's elements take; up to 16 of them leave room for the
// weights (rows of 128, three blocks: 26.9 us; four and the weights from shared memory 28.0)
template <int E> constexpr int kBlocksSm = E <= 8 ? 4 : E <= 24 ? 3 : 2;
template <int E> constexpr bool kKeepWeights = E <= 16;

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kNormThreads, kBlocksSm<V * NV>)
norm_rope_kernel(NormArgs a, NormGeom g, int64_t rows_block) {
  using W = typename Word<V * sizeof(T)>::type;
  extern __shared__ __align__(16) unsigned char raw[];
  pdl_launch_dependents();
  pdl_wait();
  NormShared sh = norm_shared(a, g, raw);
  const int lane = threadIdx.x & (g.lanes - 1), grp = threadIdx.x / g.lanes;
  const int first = norm_first<NV>(g, lane);
  float* ex = sh.ex + grp * a.rot;
  const int64_t rows = static_cast<int64_t>(a.n) * a.h;
  const int64_t begin = blockIdx.x * rows_block, end = min(begin + rows_block, rows);
  const float inv_span = 1.0f / static_cast<float>(a.span);
  RowAt at(min(begin + grp, rows - 1), a.h), next = at;
  RowPtr<const T> src(static_cast<const T*>(a.x) + first * V, at, g, a.h, a.x_stride_t, a.x_stride_h);
  RowPtr<T> dst(static_cast<T*>(a.out) + first * V, at, g, a.h, a.out_stride_t, a.out_stride_h);
  bool there[NV], normed[NV];  // (a vector is normed as a whole or not at all: V divides span)
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    there[j] = first + j * g.part < g.vectors;
    normed[j] = (first + j * g.part) * V < a.span;
  }
  Vec<T, V> x[NV];  // the row at hand, then the next one
  auto load = [&](bool live) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (live && there[j]) x[j].u = *reinterpret_cast<const W*>(src.p + j * g.part * V);
      else x[j].u = W{};
    src.step(next.step(g, a.h));
  };
  load(begin + grp < end);
  norm_fill_params<V>(a, g, sh);
  float kept[kKeepWeights<NV * V> ? NV * V : 1];
  if constexpr (kKeepWeights<NV * V>) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[V];
      load_params(g, sh.weight, min((first + j * g.part) * V, a.span - V), w);
#pragma unroll
      for (int i = 0; i < V; ++i) kept[j * V + i] = w[i];
    }
  }
  for (int64_t r0 = begin; r0 < end; r0 += g.rows_step) {
    const bool live = r0 + grp < end;
    float y[NV * V];
#pragma unroll
    for (int j = 0; j < NV; ++j) widen<T, V>(x[j], y + j * V);
    load(r0 + g.rows_step + grp < end);
    norm_fill_cs(a, g, sh, r0, end);
    if (a.center) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (normed[j])
#pragma unroll
          for (int i = 0; i < V; ++i) s += y[j * V + i];
      const float mean = row_sum(s, g.lanes) * inv_span;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (normed[j])
#pragma unroll
          for (int i = 0; i < V; ++i) y[j * V + i] -= mean;
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (normed[j]) add_products<V>(s2, y + j * V, y + j * V);
    const float r = rsqrtf(fmaf(row_sum(s2.x + s2.y, g.lanes), inv_span, a.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (normed[j]) {
        const int e0 = (first + j * g.part) * V;
        scale_all<V>(y + j * V, r);
        if (a.weight) {
          if constexpr (kKeepWeights<NV * V>) {
            scale_by<V>(y + j * V, kept + j * V);
          } else {
            float w[V];
            load_params(g, sh.weight, e0, w);
            scale_by<V>(y + j * V, w);
          }
        }
        if (a.bias) {
          float b[V];
          load_params(g, sh.bias, e0, b);
#pragma unroll
          for (int i = 0; i < V; ++i) y[j * V + i] += b[i];
        }
      }
    turn_row<V, NV, false>(a, g, y, sh.cs + (live ? at.t - sh.first : 0) * ((a.rot / 2 + 1) & ~1), ex, lane, first);
    if (live)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (there[j]) *reinterpret_cast<W*>(dst.p + j * g.part * V) = narrow<T, V>(y + j * V).u;
    dst.step(at.step(g, a.h));
  }
}

template <typename T, int V, int NV>
cudaError_t launch_fwd(const NormArgs& a, NormGeom g, cudaStream_t s) {
  norm_pairs<V, NV>(a, g, sizeof(T));
  const int64_t steps = (static_cast<int64_t>(a.n) * a.h + g.rows_step - 1) / g.rows_step;
  // one wave: a block's start, two round trips to memory, is then paid once (4096 x 64 x 128: 38 us with four)
  const int64_t most = static_cast<int64_t>(multiprocessors()) * kBlocksSm<V * NV>;
  const int64_t per = (steps + most - 1) / most;
  norm_table(a, g, per * g.rows_step);
  const size_t smem = norm_shared_bytes(a, g);
  const cudaError_t e = norm_allow_shared(norm_rope_kernel<T, V, NV>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_rope_kernel<T, V, NV>, dim3(static_cast<unsigned>((steps + per - 1) / per)), dim3(kNormThreads),
                    smem, s, 1, a, g, per * g.rows_step);
}

template <typename T>
cudaError_t launch_fwd_t(const NormArgs& a, cudaStream_t s) {
  constexpr int kMost = 16 / sizeof(T);
  const int v = norm_vector(reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out),
                            static_cast<uint64_t>(a.x_stride_t | a.x_stride_h | a.out_stride_t | a.out_stride_h), a, sizeof(T));
  const NormGeom g = norm_geom(a, v, sizeof(T));
  const int nv = (g.vectors + g.lanes - 1) / g.lanes;
  if (v == kMost) {
    if (nv == 1) return launch_fwd<T, kMost, 1>(a, g, s);
    if (nv == 2) return launch_fwd<T, kMost, 2>(a, g, s);
    if (nv == 3) return launch_fwd<T, kMost, 3>(a, g, s);
    if (nv == 4) return launch_fwd<T, kMost, 4>(a, g, s);
    if constexpr (kMost == 4) {
      if (nv == 5) return launch_fwd<T, kMost, 5>(a, g, s);
      return launch_fwd<T, kMost, 8>(a, g, s);
    }
  }
  if constexpr (kMost == 8) {
    if (v >= 4) return nv <= 1 ? launch_fwd<T, 4, 1>(a, g, s) : nv <= 2 ? launch_fwd<T, 4, 2>(a, g, s) : launch_fwd<T, 4, 8>(a, g, s);
  }
  if (v == 2) return nv <= 2 ? launch_fwd<T, 2, 2>(a, g, s) : launch_fwd<T, 2, 16>(a, g, s);
  return nv <= 4 ? launch_fwd<T, 1, 4>(a, g, s) : launch_fwd<T, 1, 32>(a, g, s);
}

// ---- the cache writers with norm and rotation on the way -----------------------------
// One warp per token, lane i the sine and cosine of frequency i, as in the other writers.  The normed and turned
// values are quantised from fp32: a code is the nearest of a value that is good to 2^-19 of the sizes of its parts and
// its pair's (a mean adds 2^-21 of what it takes off), so one that close to the border between two codes may land on either side.  A row whose sum of squares is
// not finite, or 0 without eps, has no norm: it is stored as NaN.
constexpr int kWarpsPerBlock = 8;
constexpr int kRot = 64;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// 1 / sqrt(mean square + eps), NaN where that sum is not finite; infinite where it is 0
__device__ __forceinline__ float norm_factor(float sum, float inv_n, float eps) {
  const float m = fmaf(sum, inv_n, eps);
  return m < INFINITY ? rsqrtf(m) : NAN;
}

// phase_cs without its last correction: a sine and a cosine of two roundings, the second the amplitude's, 8 units of 2^-24
// with all others.  The angle x + xl is as exact as there (of one float, 15% more keys' codes landed on the other side of a
// border, and 65536 tokens took 39.4 us instead of 40.4); the lower part of the phase has a sign, so that
// angles around 0, which may be all that a key's group of 32 holds, keep their relative accuracy on both sides.
__device__ __forceinline__ float2 phase_cs_near(int pos, int64_t turns, float amp) {
  uint32_t quarter;
  // the rest of the phase in 2^-33 turns: hi + lo 2^-31
  const int64_t rest = phase_rest(pos, turns, quarter) + (1ll << 30);
  const int hi = static_cast<int>(rest >> 31), lo = static_cast<int>(static_cast<uint32_t>(rest) & 0x7FFFFFFFu) - (1 << 30);
  const float rh = static_cast<float>(hi);
  const float rl = fmaf(static_cast<float>(lo), 1.0f / 2147483648.0f, static_cast<float>(hi - static_cast<int>(rh)));
  constexpr double kRad = 6.283185307179586476925 / 8589934592.0;  // 2 pi 2^-33
  constexpr float kHi = static_cast<float>(kRad);
  constexpr float kLo = static_cast<float>(kRad - static_cast<double>(kHi));
  const float x = __fmul_rn(rh, kHi);
  const float xl = fmaf(rh, kHi, -x) + fmaf(rl, kHi, rh * kLo);
  const float z = x * x;
  float S = fmaf(1.0f / 362880.0f, z, -1.0f / 5040.0f), C = fmaf(-1.0f / 3628800.0f, z, 1.0f / 40320.0f);
  S = fmaf(S, z, 1.0f / 120.0f);
  S = fmaf(S, z, -1.0f / 6.0f);
  C = fmaf(C, z, -1.0f / 720.0f);
  C = fmaf(C, z, 1.0f / 24.0f);
  // sin = x + (x^3 S(z) + xl cos x),  cos = 1 + (-z/2 + z^2 C(z) - x xl)
  const float sn = x + fmaf(x * z, S, fmaf(-0.5f * z, xl, xl)), cn = 1.0f + fmaf(-x, xl, fmaf(z * z, C, -0.5f * z));
  const bool swap = quarter & 1u;  // a quarter turn: (c, s) -> (-s, c)
  return make_float2((swap ? sn : cn) * (((quarter + 1u) & 2u) ? -amp : amp), (swap ? cn : sn) * ((quarter & 2u) ? -amp : amp));
}

__device__ __forceinline__ void norm_store_k(uint2 raw, float4 w, float4 b, float2 cs, const NormQuantArgs& a, int64_t slot) {
  const int lane = threadIdx.x & 31;
  const float2 r0 = bf16x2_to_f32(raw.x), r1 = bf16x2_to_f32(raw.y);
  float x[4] = {r0.x, r0.y, r1.x, r1.y};
  if (a.k_center) {
    const float mean = warp_sum((x[0] + x[1]) + (x[2] + x[3])) * (1.0f / kIdxDim);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] -= mean;
  }
  float r = norm_factor(warp_sum(fmaf(x[0], x[0], x[1] * x[1]) + fmaf(x[2], x[2], x[3] * x[3])), 1.0f / kIdxDim, a.eps);
  if (!(r < INFINITY)) r = NAN;
  x[0] = fmaf(x[0] * r, w.x, b.x);
  x[1] = fmaf(x[1] * r, w.y, b.y);
  x[2] = fmaf(x[2] * r, w.z, b.z);
  x[3] = fmaf(x[3] * r, w.w, b.w);
  const int li = lane - (a.r.k_offset >> 2);  // 0..15 inside the rotary part
  const bool mine = li >= 0 && li < kRot / 4;
  float y[4];
  if (a.r.k_layout == DSA_ROPE_HALF) {
    const bool first = li < 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float other = __shfl_sync(0xffffffffu, x[j], first ? lane + 8 : lane - 8);
      const float c = __shfl_sync(0xffffffffu, cs.x, 4 * (li & 7) + j), s = __shfl_sync(0xffffffffu, cs.y, 4 * (li & 7) + j);
      y[j] = fmaf(x[j], c, other * (first ? -s : s));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float c = __shfl_sync(0xffffffffu, cs.x, 2 * li + j), s = __shfl_sync(0xffffffffu, cs.y, 2 * li + j);
      y[2 * j] = fmaf(x[2 * j], c, -x[2 * j + 1] * s);
      y[2 * j + 1] = fmaf(x[2 * j + 1], c, x[2 * j] * s);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = mine ? y[j] : x[j];
  float amax = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = amax < INFINITY ? mx_shared_exp(amax) : 0;
  const float inv = exp2i(-e);  // exact power of two
  const uint32_t codes = codes4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
  uint8_t* page = a.r.k_cache + static_cast<int64_t>(static_cast<uint64_t>(slot) / kPage) * kKPageBytes;
  const int row = static_cast<int>(slot & (kPage - 1));
  *reinterpret_cast<uint32_t*>(page + row * kIdxDim + 4 * lane) = amax == 0.f ? 0u : codes;
  if ((lane & 7) == 0) page[kKScaleOff + row * 4 + (lane >> 3)] = static_cast<uint8_t>(e + 127);
}

__device__ __forceinline__ void norm_store_kv(const uint2 (&raws)[4], uint32_t rope, const float4 (*w)[32], float2 cs,
                                              const NormQuantArgs& a, int64_t slot) {
  const int lane = threadIdx.x & 31;
  uint8_t* rec = a.r.kv_cache + slot * kKvTokBytes;
  float y[16];
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int tile = 0; tile < 4; ++tile) {
    const float2 p = bf16x2_to_f32(raws[tile].x), q = bf16x2_to_f32(raws[tile].y);
    y[4 * tile] = p.x;
    y[4 * tile + 1] = p.y;
    y[4 * tile + 2] = q.x;
    y[4 * tile + 3] = q.y;
    sum = fma2(q, q, fma2(p, p, sum));
  }
  const float r = norm_factor(warp_sum(sum.x + sum.y), 1.0f / kVDim, a.eps);
  const float2 x = bf16x2_to_f32(rope);
  float t0, t1;
  if (a.r.kv_layout == DSA_ROPE_HALF) {
    const float o0 = __shfl_xor_sync(0xffffffffu, x.x, 16), o1 = __shfl_xor_sync(0xffffffffu, x.y, 16);
    const float c0 = __shfl_sync(0xffffffffu, cs.x, 2 * lane), c1 = __shfl_sync(0xffffffffu, cs.x, 2 * lane + 1);
    const float s0 = __shfl_sync(0xffffffffu, cs.y, 2 * lane), s1 = __shfl_sync(0xffffffffu, cs.y, 2 * lane + 1);
    t0 = fmaf(x.x, c0, o0 * (lane < 16 ? -s0 : s0));
    t1 = fmaf(x.y, c1, o1 * (lane < 16 ? -s1 : s1));
  } else {
    t0 = fmaf(x.x, cs.x, -x.y * cs.y);
    t1 = fmaf(x.y, cs.x, x.x * cs.y);
  }
  // lane t works out tile t's scale and its reciprocal, so that the five cost one division
  float amax = warp_amax(fmaxf(fabsf(t0), fabsf(t1)));
#pragma unroll
  for (int tile = 0; tile < 4; ++tile) {
    const float4 wt = w[tile][lane];
    const float f[4] = {wt.x, wt.y, wt.z, wt.w};
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 z = mul2(make_float2(y[4 * tile + i], y[4 * tile + i + 1]), mul2(make_float2(r, r), make_float2(f[i], f[i + 1])));
      y[4 * tile + i] = z.x;
      y[4 * tile + i + 1] = z.y;
      m = fmaxf(m, fmaxf(fabsf(z.x), fabsf(z.y)));
    }
    m = warp_amax(r < INFINITY ? m : NAN);
    if (lane == tile) amax = m;
  }
  const float s = __fdiv_rn(amax, 448.0f);
  const bool usable = s > 1e-30f && s < 1e30f;  // 1 / s and s itself are far from the range's ends
  const float inv = usable ? __frcp_rn(s) : 0.f;
  const uint32_t fast = __ballot_sync(0xffffffffu, usable);
  uint32_t codes[4];
  uint16_t tail;
  if ((fast & 0x1Fu) == 0x1Fu) {
#pragma unroll
    for (int tile = 0; tile < 4; ++tile) {
      const float ti = __shfl_sync(0xffffffffu, inv, tile);
      const float2 both = make_float2(ti, ti), p = mul2(make_float2(y[4 * tile], y[4 * tile + 1]), both),
                   q = mul2(make_float2(y[4 * tile + 2], y[4 * tile + 3]), both);
      codes[tile] = codes4(p.x, p.y, q.x, q.y);
    }
    const float ti = __shfl_sync(0xffffffffu, inv, 4);
    tail = f32x2_to_e4m3x2(t0 * ti, t1 * ti);
  } else {  // (a tile of zeros, or at the ends of fp32: the one branch for all five)
    auto quotient = [](float v, float ts) { return ts > 0.f ? __fdiv_rn(v, ts) : 0.f; };
#pragma unroll
    for (int tile = 0; tile < 4; ++tile) {
      const float ts = __shfl_sync(0xffffffffu, s, tile);
      codes[tile] = codes4(quotient(y[4 * tile], ts), quotient(y[4 * tile + 1], ts), quotient(y[4 * tile + 2], ts),
                           quotient(y[4 * tile + 3], ts));
    }
    const float ts = __shfl_sync(0xffffffffu, s, 4);
    tail = f32x2_to_e4m3x2(quotient(t0, ts), quotient(t1, ts));
  }
#pragma unroll
  for (int tile = 0; tile < 4; ++tile) *reinterpret_cast<uint32_t*>(rec + tile * 128 + 4 * lane) = codes[tile];
  *reinterpret_cast<uint16_t*>(rec + 512 + 2 * lane) = tail;
  if (lane < 8) *reinterpret_cast<float*>(rec + kKvScaleOff + 4 * lane) = lane < 5 ? s : 0.f;
}

__global__ void __launch_bounds__(kWarpsPerBlock * 32, 4)
norm_rope_quant_kernel(NormQuantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  // weights and bias of a token's dims, four a lane: the key's, then the latent row's tiles (in registers they left room
  // for 16 warps an SM, and 65536 tokens took 62 us)
  __shared__ float4 s_param[6][32];
  const int lane = threadIdx.x & 31;
  const int64_t turns = a.r.turns[lane];
  if (threadIdx.x < 6 * 32) {
    const int which = threadIdx.x >> 5;
    const float* src = which == 0 ? a.k_weight : which == 1 ? a.k_bias : a.kv_weight ? a.kv_weight + (which - 2) * 128 : nullptr;
    s_param[which][lane] = src ? *reinterpret_cast<const float4*>(src + 4 * lane)
                               : which == 1 ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(1.f, 1.f, 1.f, 1.f);
  }
  __syncthreads();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + (threadIdx.x >> 5); t < a.r.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarpsPerBlock) {
    const int64_t slot = a.r.slots[t];
    const int pos = a.r.pos[t];
    uint2 k, kv[4];
    uint32_t rope;
    if (a.r.k) k = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.r.k) + t * a.r.k_stride + 4 * lane);
    if (a.r.kv) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.r.kv) + t * a.r.kv_stride;
#pragma unroll
      for (int tile = 0; tile < 4; ++tile) kv[tile] = *reinterpret_cast<const uint2*>(src + tile * 128 + 4 * lane);
      rope = *reinterpret_cast<const uint32_t*>(src + 512 + 2 * lane);
    }
    if (slot >= a.r.num_slots) {
      if (lane == 0) flag(a.r.status, DSA_STATUS_BAD_PAGE);
    } else if (slot >= 0) {
      const float2 cs = phase_cs_near(pos, turns, a.r.amplitude);
      if (a.r.k) norm_store_k(k, s_param[0][lane], s_param[1][lane], cs, a, slot);
      if (a.r.kv) norm_store_kv(kv, rope, s_param + 2, cs, a, slot);
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormArgs& a, cudaStream_t s) {
  if (a.dtype == DSA_DTYPE_BF16) return launch_fwd_t<__nv_bfloat16>(a, s);
  if (a.dtype == DSA_DTYPE_FP16) return launch_fwd_t<__half>(a, s);
  return launch_fwd_t<float>(a, s);
}

cudaError_t launch_norm_rope_quant(const NormQuantArgs& a, cudaStream_t s) {
  const int cap = multiprocessors() * 16;
  const int blocks = a.r.n_tokens / kWarpsPerBlock + (a.r.n_tokens % kWarpsPerBlock != 0);
  return launch_pdl(norm_rope_quant_kernel, dim3(blocks < cap ? blocks : cap), dim3(kWarpsPerBlock * 32), 0, s, 1, a);
}

}  // namespace dsa
