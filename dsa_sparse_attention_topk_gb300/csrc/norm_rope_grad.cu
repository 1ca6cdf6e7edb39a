// The gradient of dsa_norm_rope (dsa_norm_rope_grad).
//
// With g the output's gradient turned back, u = (x - mu) r the normed value and du = g w:
//     dx = r (du - u mean(du u) [- mean(du), with a mean]),   dw = sum g u,   db = sum g,
// sums of dw and db over all rows; dims that are not normed have dx = g.  u is formed again from x, which
// costs no memory that the sums would not read anyway; nothing is kept from the forward pass.
//
// Bound: memory, dy and x read and dx written once.  A block takes a run of rows and each lane keeps the sums of its
// own dims in registers; the blocks' sums go to the workspace and a second kernel adds them, always in the same
// order, so that equal inputs give equal bits.  4096 x 64 x 128 bf16 take 41 us, 4.9 TB/s, 2047 x 63 x 192 fp32 52 us, 5.7
// TB/s (at a plain copy's rate 30 and 44.5).  Where a lane has 24 or 32 elements, the two rows' values and the sums do not fit
// its registers (16-bit heads of 256: 3.4 TB/s, with a bias 2.2).

#include "norm_rope.cuh"

namespace dsa {
namespace {

constexpr int kMostBlocks = 1024;  // partial sums in the workspace
constexpr int kBlocksSm = 2;       // blocks an SM gets: one wave

// SHIFT: the bias's sums too
template <typename T, int V, int NV, bool SHIFT>
__global__ void __launch_bounds__(kNormThreads, 2)
norm_rope_grad_kernel(NormArgs a, NormGeom g, int64_t rows_block) {
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
  float dw[NV * V], db[SHIFT ? NV * V : 1];
#pragma unroll
  for (int i = 0; i < NV * V; ++i) {
    dw[i] = 0.f;
    if (SHIFT) db[i] = 0.f;
  }
  RowAt at(min(begin + grp, rows - 1), a.h), next = at;
  RowPtr<const T> xs(static_cast<const T*>(a.x) + first * V, at, g, a.h, a.x_stride_t, a.x_stride_h);
  RowPtr<const T> ys(static_cast<const T*>(a.dy) + first * V, at, g, a.h, a.dy_stride_t, a.dy_stride_h);
  RowPtr<T> dst(static_cast<T*>(a.out) + first * V, at, g, a.h, a.out_stride_t, a.out_stride_h);
  bool there[NV], normed[NV];  // (a vector is normed as a whole or not at all: V divides span)
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    there[j] = first + j * g.part < g.vectors;
    normed[j] = (first + j * g.part) * V < a.span;
  }
  Vec<T, V> p[NV], q[NV];  // x and dy of the row at hand, then of the next one
  auto load = [&](bool live) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (live && there[j]) {
        p[j].u = *reinterpret_cast<const W*>(xs.p + j * g.part * V);
        q[j].u = *reinterpret_cast<const W*>(ys.p + j * g.part * V);
      } else {
        p[j].u = W{};
        q[j].u = W{};
      }
    }
    const bool wrap = next.step(g, a.h);
    xs.step(wrap);
    ys.step(wrap);
  };
  load(begin + grp < end);
  norm_fill_params<V>(a, g, sh);
  for (int64_t r0 = begin; r0 < end; r0 += g.rows_step) {
    const bool live = r0 + grp < end;
    float u[NV * V], d[NV * V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      widen<T, V>(p[j], u + j * V);
      widen<T, V>(q[j], d + j * V);
    }
    load(r0 + g.rows_step + grp < end);
    norm_fill_cs(a, g, sh, r0, end);
    turn_row<V, NV, true>(a, g, d, sh.cs + (live ? at.t - sh.first : 0) * ((a.rot / 2 + 1) & ~1), ex, lane, first);
    if (a.center) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (normed[j])
#pragma unroll
          for (int i = 0; i < V; ++i) s += u[j * V + i];
      const float mean = row_sum(s, g.lanes) * inv_span;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (normed[j])
#pragma unroll
          for (int i = 0; i < V; ++i) u[j * V + i] -= mean;
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (normed[j]) add_products<V>(s2, u + j * V, u + j * V);
    const float r = rsqrtf(fmaf(row_sum(s2.x + s2.y, g.lanes), inv_span, a.eps));
    const float ru = live ? r : 0.f;  // (a row behind the last has x = 0, and with eps = 0 no factor)
    float2 c1 = make_float2(0.f, 0.f);
    float c2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (normed[j]) {
        scale_all<V>(u + j * V, ru);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int k = j * V + i;
          dw[k] = fmaf(d[k], u[k], dw[k]);
          if (SHIFT) db[k] += d[k];
        }
        if (a.weight) {
          float w[V];
          load_params(g, sh.weight, (first + j * g.part) * V, w);
          scale_by<V>(d + j * V, w);
        }
        add_products<V>(c1, d + j * V, u + j * V);
        if (a.center)
#pragma unroll
          for (int i = 0; i < V; ++i) c2 += d[j * V + i];
      }
    const float m1 = row_sum(c1.x + c1.y, g.lanes) * -inv_span;
    const float m2 = a.center ? row_sum(c2, g.lanes) * inv_span : 0.f;
    if (live)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (normed[j]) {
          const float2 f = make_float2(m1, m1), off = make_float2(-m2, -m2);
          if constexpr (V % 2 == 0) {
#pragma unroll
            for (int i = j * V; i < j * V + V; i += 2) {
              float2 z = fma2(make_float2(u[i], u[i + 1]), f, make_float2(d[i], d[i + 1]));
              z = fma2(make_float2(1.f, 1.f), z, off);
              d[i] = z.x;
              d[i + 1] = z.y;
            }
          } else {
#pragma unroll
            for (int i = j * V; i < j * V + V; ++i) d[i] = fmaf(u[i], m1, d[i]) - m2;
          }
          scale_all<V>(d + j * V, r);
        }
        if (there[j]) *reinterpret_cast<W*>(dst.p + j * g.part * V) = narrow<T, V>(d + j * V).u;
      }
    dst.step(at.step(g, a.h));
  }
  if (!a.dweight && !a.dbias) return;
  // the block's sums: first over the groups of a warp, then over the warps through shared memory
  constexpr int kKinds = SHIFT ? 2 : 1, kWarps = kNormThreads / 32;
  float* sums = reinterpret_cast<float*>(raw);  // [kinds][warps][span], over the tables
  __syncthreads();
  const int warp = threadIdx.x >> 5, in_warp = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < NV * V; ++k) {
    for (int o = g.lanes; o < 32; o <<= 1) {
      dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
      if (SHIFT) db[k] += __shfl_xor_sync(0xffffffffu, db[k], o);
    }
    const int e = (first + (k / V) * g.part) * V + k % V;
    if (in_warp < g.lanes && e < a.span) {
      sums[warp * a.span + e] = dw[k];
      if (SHIFT) sums[(kWarps + warp) * a.span + e] = db[k];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kKinds * a.span; i += kNormThreads) {
    const int which = i >= a.span, e = i - which * a.span;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[(which * kWarps + w) * a.span + e];
    a.workspace[static_cast<int64_t>(blockIdx.x) * kKinds * a.span + i] = v;
  }
}

// The sums of `blocks` partial sums: 32 columns a block, 32 rows of threads that each take every 32nd partial.
__global__ void __launch_bounds__(1024)
norm_grad_sum_kernel(const float* part, int blocks, int span, int kinds, float* dweight, float* dbias) {
  __shared__ float s[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int col = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (col < kinds * span)
#pragma unroll 8
    for (int b = threadIdx.y; b < blocks; b += 32) v += part[static_cast<int64_t>(b) * kinds * span + col];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int mine = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && mine < kinds * span) {
    if (mine < span && dweight) dweight[mine] = v;
    if (mine >= span && dbias) dbias[mine - span] = v;
  }
}

template <typename T, int V, int NV, bool SHIFT>
cudaError_t launch_bwd_k(const NormArgs& a, NormGeom g, cudaStream_t s) {
  norm_pairs<V, NV>(a, g, sizeof(T));
  const int64_t steps = (static_cast<int64_t>(a.n) * a.h + g.rows_step - 1) / g.rows_step;
  const int64_t most = std::min<int64_t>(static_cast<int64_t>(multiprocessors()) * kBlocksSm, kMostBlocks);
  const int64_t per = (steps + most - 1) / most;
  const int blocks = static_cast<int>((steps + per - 1) / per), kinds = SHIFT ? 2 : 1;
  norm_table(a, g, per * g.rows_step);
  const size_t smem = std::max(norm_shared_bytes(a, g), sizeof(float) * kinds * (kNormThreads / 32) * a.span);
  cudaError_t e = norm_allow_shared(norm_rope_grad_kernel<T, V, NV, SHIFT>, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(norm_rope_grad_kernel<T, V, NV, SHIFT>, dim3(blocks), dim3(kNormThreads), smem, s, 1, a, g,
                             per * g.rows_step);
  if (e != cudaSuccess || (!a.dweight && !a.dbias)) return e;
  return launch_pdl(norm_grad_sum_kernel, dim3((kinds * a.span + 31) / 32), dim3(32, 32), 0, s, 1,
                    static_cast<const float*>(a.workspace), blocks, a.span, kinds, a.dweight, a.dbias);
}
template <typename T, int V, int NV>
cudaError_t launch_bwd(const NormArgs& a, const NormGeom& g, cudaStream_t s) {
  // (of the narrow vectors one kernel serves both)
  if constexpr (V * sizeof(T) == 16) {
    if (!a.dbias) return launch_bwd_k<T, V, NV, false>(a, g, s);
  }
  return launch_bwd_k<T, V, NV, true>(a, g, s);
}

template <typename T>
cudaError_t launch_bwd_t(const NormArgs& a, cudaStream_t s) {
  constexpr int kMost = 16 / sizeof(T);
  const int v = norm_vector(reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.dy),
                            static_cast<uint64_t>(a.x_stride_t | a.x_stride_h | a.out_stride_t | a.out_stride_h | a.dy_stride_t | a.dy_stride_h),
                            a, sizeof(T));
  const NormGeom g = norm_geom(a, v, sizeof(T));
  const int nv = (g.vectors + g.lanes - 1) / g.lanes;
  if (v == kMost) {
    if (nv == 1) return launch_bwd<T, kMost, 1>(a, g, s);
    if (nv == 2) return launch_bwd<T, kMost, 2>(a, g, s);
    if (nv == 3) return launch_bwd<T, kMost, 3>(a, g, s);
    if (nv == 4) return launch_bwd<T, kMost, 4>(a, g, s);
    if constexpr (kMost == 4) {
      if (nv == 5) return launch_bwd<T, kMost, 5>(a, g, s);
      return launch_bwd<T, kMost, 8>(a, g, s);
    }
  }
  if constexpr (kMost == 8) {
    if (v >= 4) return nv <= 1 ? launch_bwd<T, 4, 1>(a, g, s) : nv <= 2 ? launch_bwd<T, 4, 2>(a, g, s) : launch_bwd<T, 4, 8>(a, g, s);
  }
  if (v == 2) return nv <= 2 ? launch_bwd<T, 2, 2>(a, g, s) : launch_bwd<T, 2, 16>(a, g, s);
  return nv <= 4 ? launch_bwd<T, 1, 4>(a, g, s) : launch_bwd<T, 1, 32>(a, g, s);
}

}  // namespace

size_t norm_grad_workspace_bytes(int span) { return sizeof(float) * 2 * kMostBlocks * static_cast<size_t>(span); }

cudaError_t launch_norm_rope_grad(const NormArgs& a, cudaStream_t s) {
  if (a.dtype == DSA_DTYPE_BF16) return launch_bwd_t<__nv_bfloat16>(a, s);
  if (a.dtype == DSA_DTYPE_FP16) return launch_bwd_t<__half>(a, s);
  return launch_bwd_t<float>(a, s);
}

}  // namespace dsa
