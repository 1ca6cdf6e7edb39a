// Dense attention of query rows with few heads over their own positions, straight from the FP8
// latent cache (dsa_prefix_attn with up to 32 heads).
//
// With 16 heads a position is 596 bytes for 35 K flop: memory sets the floor, and the 128-row
// tiles of the tensor-memory path would be seven eighths empty, after an expansion that
// moves three times the bytes.  Here a block takes one query row's heads (one or two tiles of
// 16) and a run of its positions, 64 at a time: it copies their records to shared memory (bulk
// copies of eight records a warp, one step ahead) and feeds mma.sync.m16n8k16 in fp16 from the
// codes themselves, which each thread widens for its own fragment: tcgen05 would have 16 of its
// 128 rows filled and could not read the codes.  The order of the products' inner index is
// free, so a thread's fragments are eight neighbouring codes of a position (logits) or of
// four positions (output), and no widened tile goes through shared memory.
//
//   logits   S[h, j] = sum over the five scale tiles of scale[j, tile] (q_tile . codes_tile): codes
//            are exact in fp16, the query too after a power of two per head (what falls below
//            2^-39 of the head's largest is lost), and each tile's scale multiplies its partial
//            sum in fp32.  Warp w takes positions 32 (w & 1) .., scale tile w / 2 and a quarter
//            of the fifth; its share of the query stays in registers.
//   weights  one warp per two rows of 16: running maximum and sum in fp32; per scale tile the
//            weight times the position's scale, in fp16 (2^-11: the one rounding) with a power of two per
//            row that follows the largest of them.
//   output   O[h, d] += weights(tile of d) . codes: warp w takes dims 64 w .., in registers.
//
// Two blocks per SM for one head tile (103 KB of shared memory each), so that one's barriers
// hide behind the other's work.
//
// Rows are cut by device-side lengths: all rows' steps are laid end to end and every block takes an
// equal share, which may end one row and begin the next; a row's parts meet in the merge.
//
// Measured (16 heads, two blocks an SM): 3.6 us a step of 64 positions and block, 5 us before and
// behind a block's steps; 128 rows of 1..2048 own positions 42 us, 1.8 TB/s.  A step is bound by
// the latency of its three dependent stages: half of all issue slots are filled, the
// tensor pipe is busy for a quarter of the time; without the logits' products 128 rows of
// 2048..4096 positions take 66 instead of 80 us, without the output's 70, without the weights 73,
// and the copies alone 49.

#include "prefix_common.cuh"
#include "tc_utils.cuh"

namespace dsa {
namespace {

constexpr int kTok = 64;                          // positions per step
constexpr int kThreads = 256;
constexpr int kPitch = kKvTokBytes;               // a position's record: four rows start 96 bytes apart mod 128
constexpr int kKs = 9;                            // K-steps of 16 dims a warp
// A step's positions stand in the products in this order: columns 2 q and 2 q + 1 of eight are the
// positions q and 4 + (q ^ 2), so that four threads' eight positions start in different banks both
// where columns go along them (logits) and where rows do (output).
__device__ __forceinline__ int second(int q) { return 4 + (q ^ 2); }
constexpr int kNoUnit = -112;                     // smallest unit of the output's sums
constexpr int kPPitch = kTok + 8, kSPitch = kTok + 8;

template <int HT> struct FewSmem {
  // two steps' records; weights; partial logits
  static constexpr uint32_t codes = 0, p = codes + 2 * kTok * kPitch, s = p + 4 * HT * 16 * kPPitch * 2;
  static constexpr uint32_t alpha = s + 4 * HT * 16 * kSPitch * 4, inv = alpha + HT * 16 * 4, bytes = inv + HT * 16 * 4;
};
static_assert(FewSmem<1>::bytes * 2 <= 232448 - 2048 && FewSmem<2>::bytes <= 232448, "shared memory");

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero sums
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// two products, or products and sums, in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)),
        "l"(*reinterpret_cast<const unsigned long long*>(&c)));
  return r;
}
// Four E4M3 codes as two pairs of fp16: exact, and NaN stays NaN.
__device__ __forceinline__ void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi) : "r"(codes));
}
__device__ __forceinline__ float warp_max(float x) {  // NaN lanes do not take part
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ int exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }

template <int HT>
__global__ void __launch_bounds__(kThreads, HT == 1 ? 2 : 1)
few_kernel(FewArgs f) {
  using Sm = FewSmem<HT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const PrefixArgs& a = f.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* s_s = reinterpret_cast<float*>(smem + Sm::s);
  float* s_alpha = reinterpret_cast<float*>(smem + Sm::alpha);
  float* s_inv = reinterpret_cast<float*>(smem + Sm::inv);
  __shared__ uint64_t s_full[2];          // a step's records are there
  __shared__ uint8_t s_seen[2][kTok / 8];  // and which of eight positions exist
  __shared__ uint8_t s_bad[kTok / 8];     // of eight positions: which are poisonous
  __shared__ int s_abort;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) tc::mbar_init(&s_full[i], 2 * kThreads / 32);
    s_abort = 0;
    tc::mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  auto steps_of = [&](int lim) { return lim > f.lo ? (lim - f.lo + kTok - 1) / kTok : 0; };
  // ---- this block's share: a row, or `share` steps of all rows' steps end to end ----
  int t = blockIdx.x, step0 = 0, slot = 0;
  int left;
  if (f.splits == 1) {
    left = steps_of(prefix_row_limit(a, t, tid == 0));
    if (left == 0) {
      if (f.ns > 1) {
        if (tid == 0) f.used[t] = 0;
        return;
      }
      const int64_t row0 = static_cast<int64_t>(t) * a.h_s;
      for (int i = tid; i < a.h_s * (kVDim / 8); i += kThreads)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row0 * kVDim + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
      if (a.out_lse)
        for (int h = tid; h < a.h_s; h += kThreads) a.out_lse[row0 + h] = -INFINITY;
      return;
    }
  } else {
    __shared__ int s_total[kThreads / 32], s_most[kThreads / 32], s_first[3];
    // every thread adds up a run of rows, and the block their sums (below 2^31: kFewCutRows)
    const int run = (a.n_q + kThreads - 1) / kThreads, first = min(tid * run, a.n_q), last = min(first + run, a.n_q);
    int sum = 0, most = 0;
#pragma unroll 1
    for (int r = first; r < last; ++r) {
      const int n = steps_of(prefix_row_limit(a, r, blockIdx.x == 0));
      sum += n;
      most = max(most, n);
      if (n == 0 && r % gridDim.x == blockIdx.x) f.used[r] = 0;
    }
    int upto = sum;
#pragma unroll
    for (int z = 1; z < 32; z <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, z);
      if (lane >= z) upto += v;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) {
      s_total[warp] = upto;
      s_most[warp] = most;
    }
    if (tid == 0) s_first[0] = a.n_q;
    __syncthreads();
    int before = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_total[w];
      total += s_total[w];
      most = max(most, s_most[w]);
    }
    // a row of n steps reaches into at most (n - 1) / share + 2 shares
    const int blocks = gridDim.x, block = blockIdx.x;
    const int share = max((total + blocks - 1) / blocks, (most + f.splits - 2) / (f.splits - 1));
    // (total <= blocks * share, but share times the block's number may pass 2^31 in the blocks left over)
    if (share == 0 || block > (total - 1) / share) return;
    const int from = block * share;
    left = min(share, total - from);
    if (before <= from && from < before + sum) {
#pragma unroll 1
      for (int r = first; r < last; ++r) {
        const int n = steps_of(prefix_row_limit(a, r, false));
        if (from < before + n) {
          s_first[0] = r;
          s_first[1] = from - before;
          s_first[2] = block - before / share;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
    t = s_first[0];
    step0 = s_first[1];
    slot = s_first[2];
  }

  const int g = lane >> 2, q4 = lane & 3;
  __syncthreads();
  const int tg = warp & 1, ks = warp >> 1;   // logits: positions 32 tg .., scale tile ks
  uint32_t it = ~0u;                         // steps so far less 1: the records of step i go to buffer i % 2
  const float c2 = a.sm_scale * 1.4426950408889634f;  // logits in powers of two
#pragma unroll 1
  while (t < a.n_q) {
    const int64_t row0 = static_cast<int64_t>(t) * a.h_s;
    // ---- this warp's share of the query (used last of what is read here, so asked for first) ----
    // K-steps 2 j and 2 j + 1: dims 128 ks + 32 j + 8 q4 + 0 .. 3 and 4 .. 7; the ninth: 512 + 16 ks + 4 q4 ..
    uint32_t qf[HT][kKs][4];
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int head = 16 * h + g + 8 * i;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (row0 + head) * kLatent;
#pragma unroll
        for (int k = 0; k < kKs; ++k) {
          const int d = k < 8 ? 128 * ks + 16 * (k & 6) + 8 * q4 + 4 * (k & 1) : kVDim + 16 * ks + 4 * q4;
          uint2 v = make_uint2(0u, 0u);
          if (head < a.h_s) v = *reinterpret_cast<const uint2*>(q + d);
          qf[h][k][i] = v.x;
          qf[h][k][i + 2] = v.y;
        }
      }
    const int lim = prefix_row_limit(a, t, false), rest = steps_of(lim) - step0;
    const int steps = min(rest, left);
    if (f.ns > 1 && steps == rest && tid == 0) f.used[t] = slot + 1;
    const int32_t* table = a.page_table + static_cast<int64_t>(a.q_seq[t]) * a.max_pages;

    // Copies: a warp's eight positions of a step lie in one page, or in two where a page or the prefix
    // ends among them: lane 0 or 1 copies n positions from `first` on.
    static_assert(kTok == 8 * (kThreads / 32), "eight positions a warp");
    const int end = min(lim, f.lo + (step0 + steps) * kTok);
    auto run_of = [&](int step, int& first) {
      const int p = f.lo + (step0 + step) * kTok + 8 * warp, e = min(p + 8, end);
      const int cut = min(e, p < a.prefix_len ? min(a.prefix_len, p / kPage * kPage + kPage) : p / kPage * kPage + kPage);
      first = lane == 0 ? p : cut;
      return lane == 0 ? cut - p : lane == 1 ? e - cut : 0;
    };
    auto page_of = [&](int step) {
      int first, page = -1;
      const int n = run_of(step, first);
      const int32_t* at = (first < a.prefix_len ? a.prefix_pages : table) + first / kPage;
      if (step < steps && n > 0) page = *at;
      return page;
    };
    // what does not exist becomes zero
    auto copy = [&](int step, uint32_t nth, int page) {
      int first;
      const int n = run_of(step, first), place = first - (f.lo + (step0 + step) * kTok);
      const bool found = n > 0 && page >= 0 && page < a.num_pages, real = found && !*static_cast<volatile int*>(&s_abort);
      if (n > 0 && !found) flag(a.status, DSA_STATUS_BAD_PAGE);
      const unsigned seen = __reduce_or_sync(0xffffffffu, real ? (255u >> (8 - n)) << (place & 7) : 0u);
      uint8_t* dst = smem + Sm::codes + (nth & 1) * kTok * kPitch;
      if (seen != 255u) {
#pragma unroll 1
        for (unsigned rest = ~seen & 255u; rest; rest &= rest - 1) {
          uint8_t* row = dst + (8 * warp + __ffs(rest) - 1) * kPitch;
          for (int i = 16 * lane; i < kPitch; i += 512) *reinterpret_cast<uint4*>(row + i) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_async_smem();  // before later copies to the same place
        __syncwarp();
      }
      uint64_t* full = &s_full[nth & 1];
      if (lane == 0) s_seen[nth & 1][warp] = static_cast<uint8_t>(seen);
      if (real) {
        tc::mbar_arrive_expect_tx(full, n * kPitch);
        tc::bulk_load(dst + place * kPitch, a.kv_cache + (static_cast<int64_t>(page) * kPage + first % kPage) * kPitch, n * kPitch, full);
      } else if (lane < 2) {
        tc::mbar_arrive(full);
      }
      __syncwarp();
    };
    int page_next = page_of(0);
    // the query as fp16 times a power of two per head
    float q_back[HT][2];  // the power's inverse, for heads g and g + 8
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kKs; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&qf[h][k][i + 2 * z])));
        float top = fmaxf(__low2float(top2), __high2float(top2));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max(exponent(top) - 14, -126), 112);  // the largest below 2^15 (infinities and NaN stay)
        const float up = exp2i(-e);
        q_back[h][i] = exp2i(e);
#pragma unroll
        for (int k = 0; k < kKs; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t& v = qf[h][k][i + 2 * z];
            const float2 x = mul2(make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)), make_float2(up, up));
            v = pack_half2(x.x, x.y);
          }
      }
    }
    float o[HT][8][4] = {};
    // the weights' warp: rows 2 HT warp .. of the 16 HT, lane = columns 2 lane and 2 lane + 1; the sum is the lane's own
    float m_ref[2 * HT], l_sum[2 * HT], w_sum[2 * HT];  // reference, and the sums of weights and of weights times largest scales
    int unit[2 * HT];  // the output's unit is 2^(unit - 14)
#pragma unroll
    for (int i = 0; i < 2 * HT; ++i) {
      m_ref[i] = -INFINITY;
      l_sum[i] = w_sum[i] = 0.f;
      unit[i] = kNoUnit;
    }

#pragma unroll 1
    for (int j = -1; j < steps; ++j, ++it) {
      // this step's records are there, the last step's products are done, and the next step's records
      // are asked for
      if (j >= 0) {
        tc::mbar_wait(&s_full[it & 1], (it >> 1) & 1, &s_abort, a.status);
        __syncthreads();
      }
      if (j + 1 < steps) {
        copy(j + 1, it + 1, page_next);
        page_next = page_of(j + 2);
      }
      if (j < 0) continue;
      const uint8_t* codes = smem + Sm::codes + (it & 1) * kTok * kPitch;
      auto scale = [&](int tok) { return reinterpret_cast<const float*>(codes + tok * kPitch + kKvScaleOff); };
      // eight positions a warp: a scale that makes a value infinite poisons the position, as a NaN
      // code does through its logit
      {
        const float* sc = scale(8 * warp + (lane & 7));
        float sum = 0.f, top = 0.f;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
          sum += fabsf(sc[k]);
          top = fmaxf(top, fabsf(sc[k]));
        }
        const unsigned bad = __ballot_sync(0xffffffffu, sum != sum || !(top * 448.f < INFINITY));
        if (lane == 0) s_bad[warp] = static_cast<uint8_t>(bad);
      }
      // ---- logits ----
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int tok0 = 32 * tg + 16 * half;
        const uint8_t* src = codes + (tok0 + (g & 1 ? second(g >> 1) : g >> 1)) * kPitch + 8 * q4;
        float acc[HT][2][4];
        float2 tot[HT][2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint2 u = *reinterpret_cast<const uint2*>(src + 8 * n * kPitch + 128 * ks + 32 * i);
            uint32_t b0, b1, b2, b3;
            widen(u.x, b0, b1);
            widen(u.y, b2, b3);
#pragma unroll
            for (int h = 0; h < HT; ++h) {
              if (i == 0) mma16816_first(acc[h][n], qf[h][0], b0, b1);
              else mma16816(acc[h][n], qf[h][2 * i], b0, b1);
              mma16816(acc[h][n], qf[h][2 * i + 1], b2, b3);
            }
          }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int tok_a = tok0 + 8 * n + q4, tok_b = tok0 + 8 * n + second(q4);
          const float2 sc = make_float2(scale(tok_a)[ks], scale(tok_b)[ks]), sc4 = make_float2(scale(tok_a)[4], scale(tok_b)[4]);
          const uint32_t u = *reinterpret_cast<const uint32_t*>(src + 8 * n * kPitch + kVDim + 16 * ks - 4 * q4);
          uint32_t b0, b1;
          widen(u, b0, b1);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
#pragma unroll
            for (int z = 0; z < 2; ++z)
              tot[h][n][z] = mul2(mul2(make_float2(acc[h][n][2 * z], acc[h][n][2 * z + 1]), make_float2(q_back[h][z], q_back[h][z])), sc);
            mma16816_first(acc[h][n], qf[h][8], b0, b1);
#pragma unroll
            for (int z = 0; z < 2; ++z)
              *reinterpret_cast<float2*>(s_s + (ks * HT * 16 + 16 * h + g + 8 * z) * kSPitch + tok0 + 8 * n + 2 * q4) =
                  fma2(mul2(make_float2(acc[h][n][2 * z], acc[h][n][2 * z + 1]), make_float2(q_back[h][z], q_back[h][z])), sc4, tot[h][n][z]);
          }
        }
      }
      __syncthreads();
      // ---- weights ----
      {
        const unsigned some = s_seen[it & 1][lane >> 2], bad = s_bad[lane >> 2];
        bool seen[2], poison[2];
        float4 sc[2];
        float sc_top[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = u ? second(lane & 3) : lane & 3;
          seen[u] = some >> k & 1u;
          poison[u] = bad >> k & 1u;
          sc[u] = *reinterpret_cast<const float4*>(scale(8 * (lane >> 2) + k));
          sc_top[u] = fmaxf(fmaxf(fabsf(sc[u].x), fabsf(sc[u].y)), fmaxf(fabsf(sc[u].z), fabsf(sc[u].w)));
        }
#pragma unroll
        for (int i = 0; i < 2 * HT; ++i) {
          const int row = 2 * HT * warp + i;
          const float* s = s_s + row * kSPitch + 2 * lane;
          float x[2] = {0.f, 0.f};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float2 part = *reinterpret_cast<const float2*>(s + z * HT * 16 * kSPitch);
            x[0] += part.x;
            x[1] += part.y;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) x[u] = !seen[u] ? -INFINITY : poison[u] ? __uint_as_float(0x7FFFFFFFu) : x[u] * c2;
          const float m_new = fmaxf(m_ref[i], warp_max(fmaxf(x[0], x[1])));
          const float ref = m_new == -INFINITY ? 0.f : m_new;
          const float alpha = exp2_approx(m_ref[i] - ref), p0 = exp2_approx(x[0] - ref), p1 = exp2_approx(x[1] - ref);
          l_sum[i] = fmaf(l_sum[i], alpha, p0 + p1);
          m_ref[i] = m_new;
          // the unit: the larger of what was there, shrunk by alpha, and this step's largest weight
          const float b0 = p0 * sc_top[0], b1 = p1 * sc_top[1], big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(b0, b1))));
          w_sum[i] = fmaf(w_sum[i], alpha, b0 + b1);
          const int was = alpha > 0.f ? unit[i] + exponent(alpha) : kNoUnit;
          const int now = max(max(was, kNoUnit), exponent(big));
          const float up = exp2i(14 - now);
          if (lane == 0) s_alpha[row] = alpha * exp2i(min(max(unit[i] - now, -126), 126));
          unit[i] = now;
          const float w0 = p0 * up, w1 = p1 * up;
          uint32_t* dst = reinterpret_cast<uint32_t*>(smem + Sm::p) + (row * kPPitch + 2 * lane) / 2;
          constexpr int kStride = HT * 16 * kPPitch / 2;
          dst[0] = pack_half2(w0 * sc[0].x, w1 * sc[1].x);
          dst[kStride] = pack_half2(w0 * sc[0].y, w1 * sc[1].y);
          dst[2 * kStride] = pack_half2(w0 * sc[0].z, w1 * sc[1].z);
          dst[3 * kStride] = pack_half2(w0 * sc[0].w, w1 * sc[1].w);
        }
      }
      __syncthreads();
      // ---- output: dims 64 warp + 8 (column of the product) + n of the n-th product ----
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const float f0 = s_alpha[16 * h + g], f1 = s_alpha[16 * h + g + 8];
        if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float2 v = mul2(make_float2(o[h][n][2 * z], o[h][n][2 * z + 1]), z ? make_float2(f1, f1) : make_float2(f0, f0));
              o[h][n][2 * z] = v.x;
              o[h][n][2 * z + 1] = v.y;
            }
          }
        }
      }
      const uint32_t pb = smem_u32(smem + Sm::p) + (((warp >> 1) * HT * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * kPPitch + (lane >> 4) * 8) * 2;
      const uint8_t* src_a = codes + q4 * kPitch + 64 * warp + 8 * g;
      const uint8_t* src_b = codes + second(q4) * kPitch + 64 * warp + 8 * g;
#pragma unroll
      for (int k = 0; k < kTok / 16; ++k) {
        uint32_t pa[HT][4];
#pragma unroll
        for (int h = 0; h < HT; ++h) ldmatrix4(pb + (16 * h * kPPitch + 16 * k) * 2, pa[h]);
        uint2 u[4];  // the inner indices 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9
#pragma unroll
        for (int r = 0; r < 4; ++r) u[r] = *reinterpret_cast<const uint2*>((r & 1 ? src_b : src_a) + (16 * k + 8 * (r >> 1)) * kPitch);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          const uint32_t order = n & 2 ? 0x7362 : 0x5140;
          uint32_t b[2][2];
          widen(__byte_perm(n < 4 ? u[0].x : u[0].y, n < 4 ? u[1].x : u[1].y, order), b[0][0], b[1][0]);
          widen(__byte_perm(n < 4 ? u[2].x : u[2].y, n < 4 ? u[3].x : u[3].y, order), b[0][1], b[1][1]);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
            mma16816(o[h][n], pa[h], b[0][0], b[0][1]);
            mma16816(o[h][n + 1], pa[h], b[1][0], b[1][1]);
          }
        }
      }
    }
    // ---- this part's result ----
    const int out_slot = f.slot0 + min(slot, f.splits - 1);
    float l = 0.f, w = 0.f, m = 0.f;  // lane i has row i of this warp's
    int u = 0;
#pragma unroll
    for (int i = 0; i < 2 * HT; ++i) {
#pragma unroll
      for (int z = 16; z; z >>= 1) {
        l_sum[i] += __shfl_xor_sync(0xffffffffu, l_sum[i], z);
        w_sum[i] += __shfl_xor_sync(0xffffffffu, w_sum[i], z);
      }
      if (lane == i) l = l_sum[i], w = w_sum[i], m = m_ref[i], u = unit[i];
    }
    if (lane < 2 * HT) {
      const int row = 2 * HT * warp + lane;
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      // no output is above 448 w / l: a part's goes below 2^15
      const int e = f.ns > 1 ? max(exponent(w * inv) - 5, -120) : 0;
      s_inv[row] = inv * exp2i(u - 14 - e);
      if (row < a.h_s) {
        if (f.ns > 1) f.ml[(row0 + row) * f.ns + out_slot] = split_state(m, l, e);
        else if (a.out_lse) a.out_lse[row0 + row] = natural_lse(m, l);
      }
    }
    __syncthreads();
    // (halves of 16 bits; from here on a part's rows are ns apart)
    uint16_t* out = (f.ns > 1 ? reinterpret_cast<uint16_t*>(f.o) + (row0 * f.ns + out_slot) * kVDim : static_cast<uint16_t*>(a.out) + row0 * kVDim) +
                    64 * warp + 16 * q4;
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int row = 16 * h + g + 8 * z;
        if (row >= a.h_s) continue;
        const float inv = s_inv[row];
        uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * f.ns * kVDim);
        float2 x[8];
#pragma unroll
        for (int n = 0; n < 8; ++n)  // dims 2 n and 2 n + 1 of this thread's 16
          x[n] = mul2(make_float2(o[h][2 * n % 8][2 * z + n / 4], o[h][2 * n % 8 + 1][2 * z + n / 4]), make_float2(inv, inv));
        if (f.ns > 1) {
          dst[0] = make_uint4(pack_half2(x[0].x, x[0].y), pack_half2(x[1].x, x[1].y), pack_half2(x[2].x, x[2].y), pack_half2(x[3].x, x[3].y));
          dst[1] = make_uint4(pack_half2(x[4].x, x[4].y), pack_half2(x[5].x, x[5].y), pack_half2(x[6].x, x[6].y), pack_half2(x[7].x, x[7].y));
        } else {
          dst[0] = make_uint4(pack_bf162(x[0].x, x[0].y), pack_bf162(x[1].x, x[1].y), pack_bf162(x[2].x, x[2].y), pack_bf162(x[3].x, x[3].y));
          dst[1] = make_uint4(pack_bf162(x[4].x, x[4].y), pack_bf162(x[5].x, x[5].y), pack_bf162(x[6].x, x[6].y), pack_bf162(x[7].x, x[7].y));
        }
      }
    }
    // ---- the next row with positions, if the share goes on ----
    --it;
    left -= steps;
    if (left <= 0 || f.splits == 1) break;
    step0 = slot = 0;
#pragma unroll 1
    for (++t; t < a.n_q; t += 32) {
      const int r = t + lane;
      const unsigned some = __ballot_sync(0xffffffffu, r < a.n_q && steps_of(prefix_row_limit(a, r, false)) > 0);
      if (some) {
        t += __ffs(some) - 1;
        break;
      }
    }
  }
  // after a wait that gave up, copies may still be in flight
  if (tid == 0 && *static_cast<volatile int*>(&s_abort))
    for (int i = 0; i < 2; ++i) {
      const uint32_t uses = (it + 2 - i) / 2;
      if (uses) tc::mbar_drain(&s_full[i], (uses - 1) & 1, tc::kWaitLimitNs);
    }
}

template <int HT>
cudaError_t launch(const FewArgs& f, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(few_kernel<HT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(FewSmem<HT>::bytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(few_kernel<HT>, dim3(static_cast<unsigned>(f.blocks)), dim3(kThreads), FewSmem<HT>::bytes, s, 1, f);
}

}  // namespace

cudaError_t launch_prefix_few(const FewArgs& f, cudaStream_t s) {
  return f.a.h_s <= 16 ? launch<1>(f, s) : launch<2>(f, s);
}

}  // namespace dsa
