// Dense attention of query rows with few heads over their own positions, straight from the FP8
// latent cache (dsa_prefix_attn with up to 32 heads).
//
// With 16 heads a position is 596 bytes for 35 K flop: memory sets the floor, and the 128-row
// tiles of the tensor-memory path would be seven eighths empty, after an expansion that
// moves three times the bytes.  Here a block takes one query row's heads (one or two tiles of
// 16) and a share of its positions, 32 at a time: it copies their records to shared memory
// (cp.async, one tile ahead), widens the codes to bf16, and feeds mma.sync.m16n8k16.
//
//   logits   S[h, j] = sum over the five scale tiles of scale[j, tile] (q_tile . codes_tile): codes are
//            exact in bf16, as the query is, and each tile's scale multiplies its partial sum in
//            fp32, so nothing is rounded before the softmax.  Warp w takes positions 16 (w & 1) ..
//            and scale tile w / 2 (the last: tiles 3 and 4); its share of the query stays in
//            registers.
//   weights  one warp per two rows of 16: running maximum and sum in fp32; per scale tile the
//            weight times the position's scale, as bf16 (2^-8: the one rounding).
//   output   O[h, d] += weights(tile of d) . codes: warp w takes dims 64 w .., in registers.
//
// Two blocks per SM for one head tile (91 KB of shared memory each), so that one's barriers
// hide behind the other's work.

#include "prefix_common.cuh"

namespace dsa {
namespace {

constexpr int kTok = 32;                          // positions per step
constexpr int kThreads = 256;
constexpr int kRec = kKvTokBytes;                 // 608
constexpr int kPitch = kLatent + 8;               // widened row, elements (rows shift by 16 bytes mod 128)
constexpr int kPPitch = kTok + 8;
constexpr int kSPitch = kTok + 4;

template <int HT> struct FewSmem {
  static constexpr uint32_t raw = 0, tile = raw + 2 * kTok * kRec, p = tile + kTok * kPitch * 2;
  static constexpr uint32_t s = p + 4 * HT * 16 * kPPitch * 2, alpha = s + 4 * HT * 16 * kSPitch * 4;
  static constexpr uint32_t top = alpha + HT * 16 * 4, sum = top + HT * 16 * 4, ref = sum + HT * 16 * 4;
  static constexpr uint32_t words = ref + HT * 16 * 4, bytes = words + 16;
};
static_assert(FewSmem<1>::bytes * 2 <= 232448 - 2048 && FewSmem<2>::bytes <= 232448, "shared memory");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes, in the upper bytes of w's halves, as bf16 (exact): the seven bits below the sign
// are shifted to the bottom of bf16's exponent and the top of its fraction, and 2^120 makes up
// for the exponents' offsets (127 and 7), subnormals included.  A NaN code becomes 480: such
// positions are marked before.
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  const uint32_t v = (w & 0x80008000u) | ((w & 0x7F007F00u) >> 4);
  const __nv_bfloat162 p = *reinterpret_cast<const __nv_bfloat162*>(&v);
  const uint32_t up = 0x7B807B80u;  // 2^120 twice
  const __nv_bfloat162 r = __hmul2(p, *reinterpret_cast<const __nv_bfloat162*>(&up));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int HT>
__global__ void __launch_bounds__(kThreads, HT == 1 ? 2 : 1)
few_kernel(FewArgs f) {
  using Sm = FewSmem<HT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const PrefixArgs& a = f.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x / f.splits, split = blockIdx.x - t * f.splits;
  float* s_s = reinterpret_cast<float*>(smem + Sm::s);
  float* s_alpha = reinterpret_cast<float*>(smem + Sm::alpha);
  unsigned* s_top = reinterpret_cast<unsigned*>(smem + Sm::top);
  float* s_sum = reinterpret_cast<float*>(smem + Sm::sum);
  float* s_ref = reinterpret_cast<float*>(smem + Sm::ref);
  unsigned* s_words = reinterpret_cast<unsigned*>(smem + Sm::words);  // poisonous positions, by step parity
  pdl_launch_dependents();
  pdl_wait();

  const int lim = prefix_row_limit(a, t, tid == 0 && split == 0);
  const int steps_all = lim > f.lo ? (lim - f.lo + kTok - 1) / kTok : 0;
  const int step0 = static_cast<int>(static_cast<int64_t>(split) * steps_all / f.splits);
  const int steps = static_cast<int>(static_cast<int64_t>(split + 1) * steps_all / f.splits) - step0;
  const int64_t row0 = static_cast<int64_t>(t) * a.h_s;
  if (steps == 0) {
    if (f.ns > 1) {
      for (int h = tid; h < a.h_s; h += kThreads) f.ml[(row0 + h) * f.ns + f.slot0 + split] = split_state(0.f, 0.f, 0);
    } else {
      for (int i = tid; i < a.h_s * (kVDim / 8); i += kThreads)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row0 * kVDim + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
      if (a.out_lse)
        for (int h = tid; h < a.h_s; h += kThreads) a.out_lse[row0 + h] = -INFINITY;
    }
    return;
  }
  const int32_t* table = a.page_table + static_cast<int64_t>(a.q_seq[t]) * a.max_pages;

  // ---- copies: eight threads a position, up to five 16-byte chunks each ----
  const int c_tok = tid >> 3, c_sub = tid & 7;
  // physical page of this thread's position of a step (-1: none)
  auto page_of = [&](int step) -> int {
    const int p = f.lo + (step0 + step) * kTok + c_tok;
    if (step >= steps || p >= lim) return -1;
    return p < a.prefix_len ? a.prefix_pages[p / kPage] : table[p / kPage];
  };
  auto copy = [&](int step, int page) {
    const int p = f.lo + (step0 + step) * kTok + c_tok;
    const bool inside = step < steps && p < lim;
    const bool real = inside && page >= 0 && page < a.num_pages;
    if (inside && !real && c_sub == 0) flag(a.status, DSA_STATUS_BAD_PAGE);
    const uint8_t* src = a.kv_cache + (real ? (static_cast<int64_t>(page) * kPage + p % kPage) * kRec : 0);
    const uint32_t dst = smem_u32(smem + Sm::raw) + ((step & 1) * kTok + c_tok) * kRec;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int ch = c_sub + 8 * k;
      if (ch < kRec / 16) cp_async16(dst + 16 * ch, src + 16 * ch, real);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return real;
  };
  bool real_next = copy(0, page_of(0));
  int page_next = page_of(1);

  // ---- this warp's share of the query: K-steps of scale tile w / 2 (the last: tiles 3 and 4) ----
  const int g = lane >> 2, q4 = lane & 3;
  const int tg = warp & 1, ks = warp >> 1, n_k = ks == 3 ? 12 : 8;
  uint32_t qf[HT][12][4];
  {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row0 * kLatent;
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int k = 0; k < 12; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int head = 16 * h + g + 8 * (i & 1), d = 128 * ks + 16 * k + 2 * q4 + 8 * (i >> 1);
          qf[h][k][i] = head < a.h_s && k < n_k ? *reinterpret_cast<const uint32_t*>(q + static_cast<int64_t>(head) * kLatent + d) : 0u;
        }
  }
  float o[HT][8][4] = {};
  // the weights' warp: rows 2 HT warp .. of the 16 HT, lane = position
  float m_ref[2 * HT], l_sum[2 * HT];
#pragma unroll
  for (int i = 0; i < 2 * HT; ++i) {
    m_ref[i] = -INFINITY;
    l_sum[i] = 0.f;
  }
  const float c2 = a.sm_scale * 1.4426950408889634f;  // logits in powers of two
  if (tid < 2) s_words[tid] = 0;
  // (a position's validity goes to the weights' warps by a word per step)
  __shared__ unsigned s_valid[2];

#pragma unroll 1
  for (int j = 0; j < steps; ++j) {
    const int par = j & 1;
    const uint8_t* raw = smem + Sm::raw + par * kTok * kRec;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 0) s_valid[par] = 0, s_words[par] = 0;
    const bool real = real_next;
    __syncthreads();  // this step's records are there; the last step's products are done
    if (c_sub == 0 && real) atomicOr(&s_valid[par], 1u << c_tok);
    real_next = copy(j + 1, page_next);
    page_next = page_of(j + 2);
    // ---- widen: 16 codes a piece, and mark positions with NaN codes or scales that are not finite ----
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int i = k * kThreads + tid;
      if (i < kTok * (kLatent / 16)) {
        const int tok = i / (kLatent / 16), ch = i - tok * (kLatent / 16);
        const uint4 u = *reinterpret_cast<const uint4*>(raw + tok * kRec + 16 * ch);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t v[8];
        bool bad = false;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          v[2 * n] = widen(__byte_perm(w[n], 0u, 0x1404));
          v[2 * n + 1] = widen(__byte_perm(w[n], 0u, 0x3424));
          bad |= has_nan_code(w[n]);
        }
        if ((ch & 7) == 0) bad |= !(fabsf(*reinterpret_cast<const float*>(raw + tok * kRec + kKvScaleOff + 4 * (ch >> 3))) * 448.0f < INFINITY);
        if (bad) atomicOr(&s_words[par], 1u << tok);
        uint4* dst = reinterpret_cast<uint4*>(smem + Sm::tile + (tok * kPitch + 16 * ch) * 2);
        dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
        dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
      }
    }
    __syncthreads();
    // ---- logits ----
    {
      const float* scale0 = reinterpret_cast<const float*>(raw + kKvScaleOff);  // of position 0; the next record + kRec bytes
      auto scale = [&](int tok, int tile) { return *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(scale0) + tok * kRec + 4 * tile); };
      const int i = lane >> 3, r = lane & 7;
      const uint32_t base = smem_u32(smem + Sm::tile) + ((16 * tg + (i >> 1) * 8 + r) * kPitch + 128 * ks + (i & 1) * 8) * 2;
      float acc[HT][2][4] = {}, tot[HT][2][4] = {};
      auto fold = [&](int tile) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int tok = 16 * tg + 8 * n + 2 * q4;
          const float sa = scale(tok, tile), sb = scale(tok + 1, tile);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
            tot[h][n][0] = fmaf(acc[h][n][0], sa, tot[h][n][0]);
            tot[h][n][1] = fmaf(acc[h][n][1], sb, tot[h][n][1]);
            tot[h][n][2] = fmaf(acc[h][n][2], sa, tot[h][n][2]);
            tot[h][n][3] = fmaf(acc[h][n][3], sb, tot[h][n][3]);
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[h][n][z] = 0.f;
          }
        }
      };
#pragma unroll
      for (int k = 0; k < 12; ++k) {
        if (k < 8 || ks == 3) {
          uint32_t b[4];
          ldmatrix4(base + 32 * k, b);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
            mma16816(acc[h][0], qf[h][k], b[0], b[1]);
            mma16816(acc[h][1], qf[h][k], b[2], b[3]);
          }
        }
        if (k == 7) fold(ks);
      }
      if (ks == 3) fold(4);
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float* dst = s_s + (ks * HT * 16 + 16 * h + g) * kSPitch + 16 * tg + 8 * n + 2 * q4;
          *reinterpret_cast<float2*>(dst) = make_float2(tot[h][n][0], tot[h][n][1]);
          *reinterpret_cast<float2*>(dst + 8 * kSPitch) = make_float2(tot[h][n][2], tot[h][n][3]);
        }
    }
    __syncthreads();
    // ---- weights ----
    {
      const bool seen = (s_valid[par] >> lane) & 1u, poison = (s_words[par] >> lane) & 1u;
      float sc[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) sc[n] = *reinterpret_cast<const float*>(raw + lane * kRec + kKvScaleOff + 4 * n);
#pragma unroll
      for (int i = 0; i < 2 * HT; ++i) {
        const int row = 2 * HT * warp + i;
        float x = 0.f;
#pragma unroll
        for (int z = 0; z < 4; ++z) x += s_s[(z * HT * 16 + row) * kSPitch + lane];
        x = !seen ? -INFINITY : poison ? __uint_as_float(0x7FFFFFFFu) : x * c2;
        float mt = x;
#pragma unroll
        for (int z = 16; z; z >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, z));
        const float m_new = fmaxf(m_ref[i], mt);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2_approx(m_ref[i] - ref), p = exp2_approx(x - ref);
        float sum = p;
#pragma unroll
        for (int z = 16; z; z >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
        l_sum[i] = fmaf(l_sum[i], alpha, sum);
        m_ref[i] = m_new;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(smem + Sm::p) + row * kPPitch + lane;
#pragma unroll
        for (int n = 0; n < 4; ++n)  // (no scale of a position that is not seen may come in: 0 times it could be NaN)
          dst[n * HT * 16 * kPPitch] = __float2bfloat16_rn(!seen ? 0.f : poison ? p : p * sc[n]);
        if (lane == 0) s_alpha[row] = alpha;
      }
    }
    __syncthreads();
    // ---- output ----
    {
      const int i = lane >> 3, r = lane & 7;
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const float f0 = s_alpha[16 * h + g], f1 = s_alpha[16 * h + g + 8];
        if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            o[h][n][0] *= f0;
            o[h][n][1] *= f0;
            o[h][n][2] *= f1;
            o[h][n][3] *= f1;
          }
        }
      }
      const uint32_t pb = smem_u32(smem + Sm::p) + (((warp >> 1) * HT * 16 + (i & 1) * 8 + r) * kPPitch + (i >> 1) * 8) * 2;
      const uint32_t vb = smem_u32(smem + Sm::tile) + (((i & 1) * 8 + r) * kPitch + 64 * warp + (i >> 1) * 8) * 2;
#pragma unroll
      for (int k = 0; k < kTok / 16; ++k) {
        uint32_t pa[HT][4];
#pragma unroll
        for (int h = 0; h < HT; ++h) ldmatrix4(pb + (16 * h * kPPitch + 16 * k) * 2, pa[h]);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          uint32_t b[4];
          ldmatrix4_trans(vb + (16 * k * kPitch + 16 * n) * 2, b);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
            mma16816(o[h][2 * n], pa[h], b[0], b[1]);
            mma16816(o[h][2 * n + 1], pa[h], b[2], b[3]);
          }
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // ---- this split's result ----
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 2 * HT; ++i) {
      s_ref[2 * HT * warp + i] = m_ref[i];
      s_sum[2 * HT * warp + i] = l_sum[i];
    }
  }
  if (tid < HT * 16) s_top[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HT; ++h) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int row = 16 * h + g + 8 * z;
      const float l = s_sum[row], inv = l > 0.f || l != l ? 1.f / l : 0.f;
      float top = 0.f;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        o[h][n][2 * z] *= inv;
        o[h][n][2 * z + 1] *= inv;
        top = fmaxf(top, fmaxf(fabsf(o[h][n][2 * z]), fabsf(o[h][n][2 * z + 1])));
      }
      if (f.ns > 1 && top < INFINITY) atomicMax(&s_top[row], __float_as_uint(top));
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HT; ++h) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int row = 16 * h + g + 8 * z;
      if (row >= a.h_s) continue;
      // the row's largest value below 2^15 in what is stored
      const int e = f.ns > 1 ? max(static_cast<int>(s_top[row] >> 23) - 127 - 14, -120) : 0;
      const float down = exp2i(-e);
      const int64_t at = f.ns > 1 ? (row0 + row) * f.ns + f.slot0 + split : row0 + row;
      uint32_t* dst = reinterpret_cast<uint32_t*>(f.ns > 1 ? static_cast<void*>(f.o) : a.out) + (at * kVDim + 64 * warp) / 2 + q4;
#pragma unroll
      for (int n = 0; n < 8; ++n)
        dst[4 * n] = f.ns > 1 ? pack_half2(o[h][n][2 * z] * down, o[h][n][2 * z + 1] * down)
                              : pack_bf162(o[h][n][2 * z], o[h][n][2 * z + 1]);
      if (warp == 0 && q4 == 0) {
        if (f.ns > 1) f.ml[at] = split_state(s_ref[row], s_sum[row], e);
        else if (a.out_lse) a.out_lse[at] = natural_lse(s_ref[row], s_sum[row]);
      }
    }
  }
}

template <int HT>
cudaError_t launch(const FewArgs& f, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(few_kernel<HT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(FewSmem<HT>::bytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(few_kernel<HT>, dim3(static_cast<unsigned>(f.splits) * f.a.n_q), dim3(kThreads), FewSmem<HT>::bytes, s, 1, f);
}

}  // namespace

cudaError_t launch_prefix_few(const FewArgs& f, cudaStream_t s) {
  return f.a.h_s <= 16 ? launch<1>(f, s) : launch<2>(f, s);
}

}  // namespace dsa
