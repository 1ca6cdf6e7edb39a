// Accumulated attention weights: how much every cached position was attended to, from queries and the
// log-sum-exps their attention returned (dsa_attn_mass, dsa_sparse_attn_mass).
//
//     m[p] += sum over rows t and heads h of exp(scale q[t, h] . kv[p] - lse[t, h])
//
// The probabilities are formed again from the cache; nothing of size rows x positions is written.
//
// Exact products.  kv[p] is five tiles of E4M3 codes with an fp32 scale each.  Codes are exact in fp16, and so is
// a bf16 query times a power of two per (row, head), but for what lies 2^39 below its largest value.  So the tensor
// cores multiply codes, each tile into an accumulator of its own, and the scales are applied to those in fp32:
// a logit is off by fp32 roundings alone, where rounding kv to 16 bits first would put the weights off by a percent.
//
// Sums in fixed point.  A position's rows are worked on by several CTAs, and its weight is added up over calls.
// m holds whole numbers of 2^-36 and takes additions atomically: integers add up the same in any order, so equal
// calls give equal bits.
//
// Layout.  M = 128 positions (a TMEM lane each), N = up to 96 columns, a column being one head of one query
// row; the sum over columns then stays within a thread.  Positions are the A operand in tensor memory, 288
// columns of widened codes; the columns' queries stream through shared memory by TMA in blocks of 64 dims, or stay there
// while a group's columns fit.  A group is a sequence with its rows (dense) or one row with its entries
// (sparse); units (group, tile of 128 positions, chunk of N columns) are shared out evenly over one CTA per SM.
//
// Bound: tensor cores with many columns (128 x 96 x 576 products a chunk); the cache's bytes with few.

#include <cuda.h>

#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_launch.h"
#include "tc_utils.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                        // positions of an MMA
constexpr int kBlocks = kLatent / 64;             // 64-dim blocks of a row
constexpr int kPitch = kKvTokBytes + 16;          // a staged record: lanes 16 bytes apart modulo 128 read without conflicts
constexpr int kStageBytes = kTile * kPitch;
constexpr int kWarpB = 0, kWarpMma = 1, kWarpRec = 2, kWarpCol = 3, kWarpEpi0 = 8;  // 4..7 convert
// tensor memory columns: A (32 a block), two accumulators of up to 96, the scales of two tiles
constexpr int kColD = 32 * kBlocks, kColScale = 480;
constexpr float kMassOne = 68719476736.0f;        // 2^36
constexpr float kMassMost = 67108864.0f;          // 2^26: one addition's limit

// What the columns of a chunk (N) decide.
template <int N> struct Shape {
  static constexpr int width = N == 96 || N == 64 ? 32 : N / 2;  // columns of four warps
  static constexpr int parts = N / width;                        // of them
  static constexpr int threads = 32 * (kWarpEpi0 + 4 * parts);
  static constexpr int stages = N <= 32 ? 2 : 1;                 // tiles of staged records
  static constexpr int slots = N == 96 ? 1 : N == 64 ? 2 : N == 32 ? 1 : 3;  // chunks of queries in shared memory
  static constexpr int block = N * 128;                          // bytes of 64 dims
  static constexpr int off_stage = slots * kBlocks * block;
  static constexpr int off_pos = off_stage + stages * kStageBytes;
  static constexpr int off_col = off_pos + stages * kTile * 4;   // [2][N / 2] pairs of columns, 16 bytes
  static constexpr int off_limit = off_col + 2 * N * 8;          // [2][N] positions seen
  static constexpr int off_ctl = off_limit + 2 * N * 4;
};
constexpr int kMostSlots = 3, kMostParts = 3;

struct MassPlan {
  int n;             // columns of a chunk: 16, 32, 64 or 96
  int groups;
  size_t off_cols, off_groups, off_rank;
};
struct MassWs {
  __half* q;         // [columns][576], times a power of two per column
  float4* cols;      // per column: logit per product (log2 units), -lse, positions it sees (int)
  int4* groups;      // positions or entries, first column, columns, sequence
  int* rank;         // dense: place of a row in the order of sequences, -1: none
};

// ---- queries, columns and groups ---------------------------------------------------------
// positions a row sees
__device__ __forceinline__ int row_limit(const MassArgs& a, int t, bool report) {
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
  if (!a.q_pos) return len;
  const int pos = a.q_pos[t];
  return pos < 0 ? 0 : min(pos, len - 1) + 1;
}

// Dense: rows in the order of their sequences.  A thread per row counts the rows before it, a thread per
// sequence its rows and the furthest position they see.
__global__ void __launch_bounds__(256)
mass_order_kernel(MassArgs a, MassWs ws) {
  __shared__ int s_seq[1024], s_limit[1024];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const bool is_row = i < a.n_q, is_group = !is_row && i < static_cast<int64_t>(a.n_q) + a.n_seq;
  // (a row that sees nothing has no place)
  const bool live = is_row && row_limit(a, static_cast<int>(i), true) > 0;
  const int seq = is_row ? (live ? a.q_seq[i] : -1) : static_cast<int>(i - a.n_q);
  int before = 0, own = 0, furthest = 0;
  for (int t0 = 0; t0 < a.n_q; t0 += 1024) {
    __syncthreads();
    for (int t = t0 + threadIdx.x; t < min(t0 + 1024, a.n_q); t += 256) {
      const int lim = row_limit(a, t, false);
      s_limit[t - t0] = lim;
      s_seq[t - t0] = lim > 0 ? a.q_seq[t] : INT32_MAX;
    }
    __syncthreads();
    const int n = min(1024, a.n_q - t0);
    for (int k = 0; k < n; ++k) {
      const int s = s_seq[k];
      if (s < seq || (s == seq && is_row && t0 + k < i)) ++before;
      if (s == seq) {
        ++own;
        furthest = max(furthest, s_limit[k]);
      }
    }
  }
  if (is_row) ws.rank[i] = live ? before : -1;
  if (is_group) ws.groups[seq] = make_int4(furthest, before * a.h_s, own * a.h_s, seq);
}

// One warp per (row, head): the query as fp16 with its largest value in [2^14, 2^15), and the column's constants.
// A head whose query or lse is NaN (or its query infinite) gets zeros and weight 0.
__global__ void __launch_bounds__(256)
mass_query_kernel(MassArgs a, MassWs ws) {
  __shared__ int s_last[8];
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 8 + warp;
  if (a.idx && blockIdx.y == 0) {  // the row's entries up to the last one, and its weights' empty places
    const int seen = row_limit(a, t, threadIdx.x == 0);
    int last = 0;
    for (int e = threadIdx.x; e < a.topk; e += 256) {
      if (seen > 0 && a.idx[static_cast<int64_t>(t) * a.topk + e] >= 0) last = e + 1;
      if (a.weights) a.weights[static_cast<int64_t>(t) * a.topk + e] = 0.f;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) s_last[warp] = last;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 8; ++w) last = max(last, s_last[w]);
      ws.groups[t] = make_int4(last, t * a.h_s, a.h_s, last > 0 ? a.q_seq[t] : 0);
    }
  }
  if (h >= a.h_s) return;
  const int rank = a.idx ? t : ws.rank[t];
  if (rank < 0) return;
  const int64_t from = static_cast<int64_t>(t) * a.h_s + h, to = static_cast<int64_t>(rank) * a.h_s + h;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + from * kLatent);
  uint32_t raw[kBlocks];
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    raw[i] = src[32 * i + lane];
    top = max(top, max(raw[i] & 0x7FFFu, raw[i] >> 16 & 0x7FFFu));
  }
  top = __reduce_max_sync(0xffffffffu, top);   // bf16 bits order like the values
  const float lse = a.lse[from];
  const bool dead = top >= 0x7F80u || lse != lse;
  // largest in [2^14, 2^15); a subnormal largest counts as the smallest normal one.  The factor in two powers of two
  const int k = 14 + 127 - max(static_cast<int>(top >> 7), 1);
  const float f0 = exp2i(k / 2), f1 = exp2i(k - k / 2);
  uint32_t* dst = reinterpret_cast<uint32_t*>(ws.q + to * kLatent);
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const float x = __uint_as_float(raw[i] << 16) * f0 * f1, y = __uint_as_float(raw[i] & 0xFFFF0000u) * f0 * f1;
    const __half2 v = dead ? __floats2half2_rn(0.f, 0.f) : __floats2half2_rn(x, y);
    dst[32 * i + lane] = *reinterpret_cast<const uint32_t*>(&v);
  }
  if (lane == 0) {
    if (dead) flag(a.status, DSA_STATUS_NAN_SCORE);
    const float c = a.sm_scale * 1.4426950408889634f;
    const bool none = dead || lse == -INFINITY;
    ws.cols[to] = make_float4(dead ? 0.f : c * (1.0f / f0) * (1.0f / f1), none ? -INFINITY : -lse * 1.4426950408889634f,
                              __int_as_float(a.idx ? 0 : row_limit(a, t, false)), 0.f);
  }
}

// ---- the kernel -----------------------------------------------------------------------------
struct MassCtl {
  uint64_t b_full[kMostSlots][5], b_empty[kMostSlots][5];   // a chunk's queries, 128 dims (two blocks) a barrier
  uint64_t rec_full[8], rec_empty[8];                       // [stage][quarter]
  uint64_t a_full[5], a_empty[5];                           // tiles of 128 dims
  uint64_t d_full[2], d_free[2];
  uint64_t part_full[2];
  uint64_t col_full[2], col_empty[2];
  uint64_t drained;
  float part[2][kMostParts - 1][kTile];
  int all_seen[2];                      // every column of the chunk sees the whole tile
  long long scan[20];
  int start_group, start_tile, start_chunk, abort;
  long long units;
  uint32_t tmem;
};
constexpr int kMostSmem = 232448;
static_assert(Shape<96>::off_ctl + sizeof(MassCtl) <= kMostSmem && Shape<64>::off_ctl + sizeof(MassCtl) <= kMostSmem &&
              Shape<32>::off_ctl + sizeof(MassCtl) <= kMostSmem && Shape<16>::off_ctl + sizeof(MassCtl) <= kMostSmem, "shared memory");

// A walk over the CTA's units, tile by tile: chunks [c0, c1) of tile `tile` of group g
struct Walk {
  long long left;
  int g, tile, c0, c1, chunks, tiles;
  int4 grp;
};
template <int N>
__device__ __forceinline__ void open_group(const MassWs& ws, Walk& w) {
  w.grp = ws.groups[w.g];
  w.tiles = (w.grp.x + kTile - 1) / kTile;
  w.chunks = (w.grp.z + N - 1) / N;
}
template <bool SPARSE, int N>
__device__ __forceinline__ bool walk_begin(const MassWs& ws, const MassCtl& ctl, Walk& w) {
  w.left = ctl.units;
  if (w.left <= 0) return false;
  w.g = ctl.start_group;
  w.tile = ctl.start_tile;
  open_group<N>(ws, w);
  w.c0 = SPARSE ? 0 : ctl.start_chunk;
  w.c1 = SPARSE ? w.chunks : static_cast<int>(min(static_cast<long long>(w.chunks), w.c0 + w.left));
  return true;
}
// on to the next tile; false at the end.  (The groups behind have units as long as some are left.)
template <bool SPARSE, int N>
__device__ __forceinline__ bool walk_next(const MassWs& ws, int groups, Walk& w) {
  w.left -= SPARSE ? 1 : w.c1 - w.c0;
  if (w.left <= 0) return false;
  if (++w.tile >= w.tiles) {
    w.tile = 0;
    do {
      if (++w.g >= groups) return false;
      open_group<N>(ws, w);
    } while (!w.tiles || !w.chunks);
  }
  w.c0 = 0;
  w.c1 = SPARSE ? w.chunks : static_cast<int>(min(static_cast<long long>(w.chunks), w.left));
  return true;
}

__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
  return r;
}
// D (+)= A B, fp16 operands, A in tensor memory
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, bool accumulate,
                                           uint32_t leader) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 e, %5, 0;\n setp.ne.b32 p, %4, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      :: "r"(d), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(leader) : "memory");
}
__device__ __forceinline__ void commit_if(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      :: "r"(smem_u32(bar)), "r"(leader) : "memory");
}
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pairs of floats in one instruction
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// W columns of this warp's lanes
template <int W>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&v)[W]) {
  if constexpr (W == 32) tc::tmem_ld32(taddr, v);
  else if constexpr (W == 16) tc::tmem_ld16(taddr, v);
  else tmem_ld8(taddr, v);
}
// a bounded wait (tc::mbar_wait) out of line, behind one attempt in line
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status) {
  return tc::mbar_wait(bar, parity, abort, status);
}

template <bool SPARSE, int N>
__global__ void __launch_bounds__(Shape<N>::threads, 1)
attn_mass_kernel(const __grid_constant__ CUtensorMap q_map, MassArgs a, MassPlan pl, MassWs ws) {
  using S = Shape<N>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* s_stage = smem + S::off_stage;
  int* s_pos = reinterpret_cast<int*>(smem + S::off_pos);
  MassCtl& ctl = *reinterpret_cast<MassCtl*>(smem + S::off_ctl);
  pdl_launch_dependents();
  if (smem_u32(smem) & 1023u) {  // (the swizzled blocks need it; the same in every thread)
    if (tid == 0) flag(a.status, DSA_STATUS_INTERNAL);
    return;
  }
  if (tid == 0) {
    ctl.abort = 0;
    for (int i = 0; i < S::slots; ++i)
      for (int k = 0; k < 5; ++k) {
        tc::mbar_init(&ctl.b_full[i][k], 1);
        tc::mbar_init(&ctl.b_empty[i][k], 1);
      }
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(&ctl.rec_full[i], 1);
      tc::mbar_init(&ctl.rec_empty[i], 1);
    }
    for (int i = 0; i < 5; ++i) {
      tc::mbar_init(&ctl.a_full[i], 4);
      tc::mbar_init(&ctl.a_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&ctl.d_full[i], 1);
      tc::mbar_init(&ctl.d_free[i], 4 * S::parts);
      tc::mbar_init(&ctl.part_full[i], 4 * (S::parts - 1));
      tc::mbar_init(&ctl.col_full[i], 1);
      tc::mbar_init(&ctl.col_empty[i], 4 * S::parts);
    }
    tc::mbar_init(&ctl.drained, 1);
    tc::mbar_fence_init();
    ctl.start_group = ctl.start_tile = ctl.start_chunk = 0;
  }
  if (warp == kWarpMma) tc::tmem_alloc(&ctl.tmem, 512);
  pdl_wait();
  // ---- the CTA's share of the units ----
  {
    const int per = (pl.groups + S::threads - 1) / S::threads;
    const int g0 = min(tid * per, pl.groups), g1 = min(g0 + per, pl.groups);
    long long sum = 0;
    auto units_of = [&](int g) {
      const int4 grp = ws.groups[g];
      const long long tiles = (grp.x + kTile - 1) / kTile;
      return grp.z == 0 ? 0ll : SPARSE ? tiles : tiles * ((grp.z + N - 1) / N);
    };
    for (int g = g0; g < g1; ++g) sum += units_of(g);
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) ctl.scan[warp] = incl;
    __syncthreads();
    long long before = incl - sum, total = 0;
    for (int w = 0; w < S::threads / 32; ++w) {
      if (w < warp) before += ctl.scan[w];
      total += ctl.scan[w];
    }
    const long long start = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
    if (tid == 0) ctl.units = end - start;
    if (start < end && start >= before && start < before + sum) {
      int g = g0;
      long long rest = start - before;
      for (long long u; rest >= (u = units_of(g)); ++g) rest -= u;
      const int chunks = (ws.groups[g].z + N - 1) / N;
      ctl.start_group = g;
      ctl.start_tile = static_cast<int>(SPARSE ? rest : rest / chunks);
      ctl.start_chunk = static_cast<int>(SPARSE ? 0 : rest % chunks);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort = &ctl.abort;
  // (a warp that waits as a whole leaves as a whole: an abort may reach its lanes at different times)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return tc::mbar_try_wait(bar, parity & 1u) || wait_on(bar, parity & 1u, &ctl.abort, a.status);
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  // chunk slots in order; of a group whose chunks all fit, the slots stay while its tiles last
  auto skip = [](int& slot, uint32_t& phase, int by) {  // (by at most all slots)
    slot += by;
    if (slot >= S::slots) {
      slot -= S::slots;
      phase ^= 1u;
    }
  };
  Walk w;

  if (warp == kWarpB) {
    // ---- the columns' queries: 128 dims of a chunk at a time ----
    if (lane == 0 && walk_begin<SPARSE, N>(ws, ctl, w)) {
      int slot = 0, have = -1;
      uint32_t phase = 0;
      bool ok = true;
      do {
        const bool keep = w.chunks <= S::slots;
        if (keep && have == w.g) continue;
        have = w.g;
        const int c0 = keep ? 0 : w.c0, c1 = keep ? w.chunks : w.c1;
        for (int c = c0; ok && c < c1; ++c) {
          for (int k = 0; k < 5; ++k) {
            ok = wait(&ctl.b_empty[slot][k], phase ^ 1u);
            if (!ok) break;
            uint64_t* bar = &ctl.b_full[slot][k];
            uint8_t* to = smem + (slot * kBlocks + 2 * k) * S::block;
            tc::mbar_arrive_expect_tx(bar, (k < 4 ? 2 : 1) * S::block);
            tc::tma_load_3d(to, &q_map, 128 * k, w.grp.y + c * N, 0, bar);
            if (k < 4) tc::tma_load_3d(to + S::block, &q_map, 128 * k + 64, w.grp.y + c * N, 0, bar);
          }
          if (ok) skip(slot, phase, 1);
        }
      } while (ok && walk_next<SPARSE, N>(ws, pl.groups, w));
      // copies in flight must land before the CTA ends (a share may not use all chunks of a group that stays); a
      // slot that was never loaded is past the phase before its first
      for (int i = 0; i < S::slots; ++i)
        for (int k = 0; k < 5; ++k) tc::mbar_drain(&ctl.b_full[i][k], i < slot ? phase : phase ^ 1u, 100000000ull);
      if (*abort) __nanosleep(1000000);  // (and those of a chunk begun)
    }
  } else if (warp == kWarpMma) {
    // ---- products ----
    const uint32_t leader = elect_leader();
    constexpr uint32_t idesc = idesc_f16(N);
    const uint64_t desc0 = tc::desc_kmajor_sw128(smem_u32(smem));
    int slot = 0, base = 0;  // the next chunk's; of a group that stays, its first
    uint32_t phase = 0, base_phase = 0, d = 0, visit = 0;
    if (walk_begin<SPARSE, N>(ws, ctl, w)) {
      bool ok = true, more = true;
      int have = -1;
      while (ok && more) {
        const bool keep = w.chunks <= S::slots;
        if (keep && have != w.g) {
          base = slot;
          base_phase = phase;
          skip(slot, phase, w.chunks);
        }
        have = w.g;
        const int g = w.g, c0 = w.c0, c1 = w.c1, chunks = w.chunks;
        more = walk_next<SPARSE, N>(ws, pl.groups, w);
        const bool leave = !more || w.g != g;
        for (int c = c0; ok && c < c1; ++c) {
          int at = keep ? base : slot;
          uint32_t ph = keep ? base_phase : phase;
          if (keep) skip(at, ph, c);
          else skip(slot, phase, 1);
          const uint64_t desc = desc0 + static_cast<uint32_t>(at * kBlocks * S::block >> 4);
#pragma unroll
          for (int s = 0; s < 5; ++s) {
            if (c == c0) ok = ok && wait_warp(&ctl.a_full[s], visit);
            ok = ok && wait_warp(&ctl.d_free[d & 1], (d >> 1) ^ 1u);
            ok = ok && wait_warp(&ctl.b_full[at][s], ph);
            if (!ok) break;
            tc::fence_after_sync();
            const uint32_t to = tmem + kColD + (d & 1) * N;
#pragma unroll
            for (int k = 0; k < (s < 4 ? 8 : 4); ++k)
              mma_f16_ts(to, tmem + 64 * s + 8 * k, desc + ((2 * s + k / 4) * S::block >> 4) + 2 * (k & 3), idesc, k > 0, leader);
            commit_if(&ctl.d_full[d & 1], leader);
            if (!keep) commit_if(&ctl.b_empty[at][s], leader);
            if (c == c1 - 1) commit_if(&ctl.a_empty[s], leader);
            ++d;
          }
        }
        if (ok && keep && leave) {  // the group's slots go once its last product is done
          int at = base;
          uint32_t ph = base_phase;
          for (int c = 0; c < chunks; ++c) {
            for (int k = 0; k < 5; ++k) commit_if(&ctl.b_empty[at][k], leader);
            skip(at, ph, 1);
          }
        }
        ++visit;
      }
    }
    if (*abort) {  // products in flight must end before the tensor memory is freed
      __syncwarp();
      commit_if(&ctl.drained, leader);
      tc::mbar_drain(&ctl.drained, 0, 100000000ull);
    }
  } else if (warp == kWarpRec) {
    // ---- records of a tile, 32 to a converting warp, a bulk copy a lane ----
    if (walk_begin<SPARSE, N>(ws, ctl, w)) {
      const int64_t table_end = static_cast<int64_t>(a.max_pages) * kPage;
      // the records of a tile, one of each quarter a lane: positions (-1: none) and where they lie.  All loads of
      // a tile are under way together, while the copies of the tile before are.
      auto find = [&](const Walk& at, int (&pos)[4], const uint8_t* (&src)[4]) {
        const int len = SPARSE ? a.seq_lens[at.grp.w] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = at.tile * kTile + k * 32 + lane;
          pos[k] = i < at.grp.x ? (SPARSE ? a.idx[static_cast<int64_t>(at.g) * a.topk + i] : i) : -1;
        }
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (SPARSE && pos[k] >= 0 && (pos[k] >= len || pos[k] >= table_end)) {
            flag(a.status, DSA_STATUS_BAD_INDEX);
            pos[k] = -1;
          }
          page[k] = pos[k] >= 0 ? a.page_table[static_cast<int64_t>(at.grp.w) * a.max_pages + pos[k] / kPage] : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (pos[k] >= 0 && (page[k] < 0 || page[k] >= a.num_pages)) {
            flag(a.status, DSA_STATUS_BAD_PAGE);
            pos[k] = -1;
          }
          pos[k] = max(pos[k], -1);
          src[k] = a.kv_cache + (static_cast<int64_t>(page[k]) * kPage + (pos[k] & (kPage - 1))) * kKvTokBytes;
        }
      };
      uint32_t visit = 0;
      bool ok = true, more = true;
      while (ok && more) {
        const int stage = static_cast<int>(visit % S::stages);
        const uint32_t phase = visit / S::stages;
        int pos[4];
        const uint8_t* src[4];
        find(w, pos, src);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned there = __ballot_sync(0xffffffffu, pos[k] >= 0);
          ok = ok && wait_warp(&ctl.rec_empty[stage * 4 + k], phase ^ 1u);
          if (!ok) break;
          s_pos[stage * kTile + k * 32 + lane] = pos[k];
          __syncwarp();
          uint64_t* bar = &ctl.rec_full[stage * 4 + k];
          if (lane == 0) tc::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(there)) * kKvTokBytes);
          __syncwarp();
          if (pos[k] >= 0) tc::bulk_load(s_stage + stage * kStageBytes + (k * 32 + lane) * kPitch, src[k], kKvTokBytes, bar);
        }
        if (!ok) break;
        more = walk_next<SPARSE, N>(ws, pl.groups, w);
        ++visit;
      }
      if (*abort && lane == 0)  // copies in flight must land before the CTA ends
        for (uint32_t v = visit > static_cast<uint32_t>(S::stages) ? visit - S::stages : 0; v < visit; ++v)
          for (int quarter = 0; quarter < 4; ++quarter)
            tc::mbar_drain(&ctl.rec_full[(v % S::stages) * 4 + quarter], (v / S::stages) & 1u, 100000000ull);
      if (*abort) __nanosleep(1000000);  // (and those of a tile begun)
    }
  } else if (warp == kWarpCol) {
    // ---- the columns' constants, a chunk ahead of the weights; columns behind the group's last have no weight ----
    if (walk_begin<SPARSE, N>(ws, ctl, w)) {
      uint32_t n = 0;
      bool ok = true, more = true;
      while (ok && more) {
        for (int c = w.c0; ok && c < w.c1; ++c, ++n) {
          const int buf = n & 1;
          float4 info[(N + 31) / 32];
          int least = INT32_MAX;
#pragma unroll
          for (int i = 0; i < (N + 31) / 32; ++i) {
            const int col = c * N + 32 * i + lane;
            info[i] = make_float4(0.f, -INFINITY, __int_as_float(INT32_MAX), 0.f);
            if (32 * i + lane < N && col < w.grp.z) info[i] = ws.cols[w.grp.y + col];
            least = min(least, __float_as_int(info[i].z));
          }
          least = __reduce_min_sync(0xffffffffu, least);
          ok = wait_warp(&ctl.col_empty[buf], (n >> 1) ^ 1u);
          if (!ok) break;
          float* pairs = reinterpret_cast<float*>(smem + S::off_col) + buf * 2 * N;
          int* limits = reinterpret_cast<int*>(smem + S::off_limit) + buf * N;
#pragma unroll
          for (int i = 0; i < (N + 31) / 32; ++i) {
            const int at = 32 * i + lane;
            if (at >= N) continue;
            pairs[4 * (at >> 1) + (at & 1)] = info[i].x;
            pairs[4 * (at >> 1) + 2 + (at & 1)] = info[i].y;
            limits[at] = __float_as_int(info[i].z);
          }
          if (lane == 0) ctl.all_seen[buf] = SPARSE || least >= (w.tile + 1) * kTile;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.col_full[buf]);
        }
        more = ok && walk_next<SPARSE, N>(ws, pl.groups, w);
      }
    }
  } else if (warp < kWarpEpi0) {
    // ---- codes widened to fp16 into tensor memory, a position a lane ----
    const int quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t visit = 0;
    if (walk_begin<SPARSE, N>(ws, ctl, w)) {
      bool ok = true, more = true;
      while (ok && more) {
        const int stage = static_cast<int>(visit % S::stages);
        ok = wait_warp(&ctl.rec_full[stage * 4 + quarter], visit / S::stages);
        if (!ok) break;
        const int row = quarter * 32 + lane;
        const uint8_t* rec = s_stage + stage * kStageBytes + row * kPitch;
        uint32_t scales[8];
        bool fine = true;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const float v = *reinterpret_cast<const float*>(rec + kKvScaleOff + 4 * i);
          fine = fine && fabsf(v) * 448.0f < INFINITY;
          scales[i] = __float_as_uint(v);
        }
        if (!fine) scales[0] = 0x7FC00000u;  // NaN: the position has no weight
        scales[5] = static_cast<uint32_t>(s_pos[stage * kTile + row]);
        scales[6] = scales[7] = 0;
#pragma unroll 1
        for (int s = 0; s < 5; ++s) {
          ok = wait_warp(&ctl.a_empty[s], visit ^ 1u);
          if (!ok) break;
          tc::fence_after_sync();
          if (s == 0) tmem_st8(tmem + lanes + kColScale + 8 * (visit & 1), scales);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // 32 codes, 16 columns
            if (s == 4 && j >= 2) break;
            const uint4 lo = *reinterpret_cast<const uint4*>(rec + 128 * s + 32 * j);
            const uint4 hi = *reinterpret_cast<const uint4*>(rec + 128 * s + 32 * j + 16);
            const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const __half2 p = e4m3x2_to_f16x2(static_cast<uint16_t>(u[i] & 0xFFFFu)), q = e4m3x2_to_f16x2(static_cast<uint16_t>(u[i] >> 16));
              o[2 * i] = *reinterpret_cast<const uint32_t*>(&p);
              o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&q);
            }
            tc::tmem_st16(tmem + lanes + 64 * s + 16 * j, o);
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.a_full[s]);
        }
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive(&ctl.rec_empty[stage * 4 + quarter]);
        more = walk_next<SPARSE, N>(ws, pl.groups, w);
        ++visit;
      }
    }
  } else {
    // ---- weights: a position a lane, S::width of a chunk's columns each four warps ----
    constexpr int W = S::width;
    const int quarter = warp & 3, part = (warp - kWarpEpi0) >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t d = 0, n = 0, visit = 0;
    if (walk_begin<SPARSE, N>(ws, ctl, w)) {
      bool ok = true, more = true;
      while (ok && more) {
        uint64_t scale[5];
        float total = 0.f;
        int pos = -1;
        for (int c = w.c0; ok && c < w.c1; ++c) {
          uint64_t acc[W / 2];
#pragma unroll
          for (int s = 0; s < 5; ++s) {
            ok = ok && wait_warp(&ctl.d_full[d & 1], d >> 1);
            if (!ok) break;
            tc::fence_after_sync();
            if (s == 0 && c == w.c0) {
              uint32_t v[8];
              tmem_ld8(tmem + lanes + kColScale + 8 * (visit & 1), v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 5; ++i) scale[i] = pair(__uint_as_float(v[i]), __uint_as_float(v[i]));
              pos = static_cast<int>(v[5]);
            }
            uint32_t v[W];
            tmem_load<W>(tmem + lanes + kColD + (d & 1) * N + part * W, v);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.d_free[d & 1]);
            ++d;
#pragma unroll
            for (int i = 0; i < W / 2; ++i)
              acc[i] = fma_pair(scale[s], pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s ? acc[i] : 0ull);
          }
          const int buf = n & 1;
          ok = ok && wait_warp(&ctl.col_full[buf], n >> 1);
          if (!ok) break;
          ++n;
          const ulonglong2* cols = reinterpret_cast<const ulonglong2*>(smem + S::off_col) + (buf * N + part * W) / 2;
          float sum = 0.f;
          if (ctl.all_seen[buf]) {
            float odd = 0.f;
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
              const ulonglong2 k = cols[i];
              const float2 x = unpair(fma_pair(acc[i], k.x, k.y));
              sum += ex2(x.x);
              odd += ex2(x.y);
            }
            sum += odd;
          } else {
            const int2* limits = reinterpret_cast<const int2*>(smem + S::off_limit) + (buf * N + part * W) / 2;
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
              const ulonglong2 k = cols[i];
              const int2 lim = limits[i];
              const float2 x = unpair(fma_pair(acc[i], k.x, k.y));
              sum += (pos < lim.x ? ex2(x.x) : 0.f) + (pos < lim.y ? ex2(x.y) : 0.f);
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.col_empty[buf]);
          total += sum;
        }
        if (!ok) break;
        // (the other parts' sums of the tile before last have been read: d_free holds all parts within two accumulators)
        if (part > 0) {
          ctl.part[visit & 1][part - 1][row] = total;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.part_full[visit & 1]);
        } else {
          ok = wait_warp(&ctl.part_full[visit & 1], visit >> 1);
          if (!ok) break;
          if (pos >= 0) {
#pragma unroll
            for (int i = 0; i < S::parts - 1; ++i) total += ctl.part[visit & 1][i][row];
            if (SPARSE && a.weights) a.weights[static_cast<int64_t>(w.g) * a.topk + w.tile * kTile + row] = total;
            if (a.mass) {
              if (total != total) flag(a.status, DSA_STATUS_NAN_SCORE);
              else if (total > 0.f)
                atomicAdd(reinterpret_cast<unsigned long long*>(a.mass + static_cast<int64_t>(w.grp.w) * a.mass_stride + pos),
                          static_cast<unsigned long long>(__float2ll_rn(fminf(total, kMassMost) * kMassOne)));
            }
          }
        }
        more = walk_next<SPARSE, N>(ws, pl.groups, w);
        ++visit;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kWarpMma) tc::tmem_dealloc(tmem, 512);
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

MassPlan make_plan(int n_q, int h_s, int n_seq, bool sparse) {
  MassPlan p;
  p.groups = sparse ? n_q : n_seq;
  // a chunk's columns: all of a group of average rows where they fit; of more than 128 as many as there can be
  const int64_t cols = static_cast<int64_t>(h_s) * (sparse ? 1 : std::max(1, (n_q + n_seq - 1) / n_seq));
  p.n = cols <= 16 ? 16 : cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 96 ? 96 : cols <= 128 ? 64 : 96;
  const size_t columns = static_cast<size_t>(n_q) * h_s;
  p.off_cols = round_up(columns * kLatent * 2, 256);
  p.off_groups = p.off_cols + round_up(columns * 16, 256);
  p.off_rank = p.off_groups + round_up(static_cast<size_t>(p.groups) * 16, 256);
  return p;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeFn>(p);
    return static_cast<EncodeFn>(nullptr);
  }();
  return fn;
}

template <bool SPARSE, int N>
cudaError_t launch_main(const CUtensorMap& q_map, const MassArgs& a, const MassPlan& pl, const MassWs& ws, int grid, cudaStream_t s) {
  constexpr size_t smem = Shape<N>::off_ctl + sizeof(MassCtl);
  const cudaError_t e = cudaFuncSetAttribute(attn_mass_kernel<SPARSE, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_mass_kernel<SPARSE, N>, dim3(static_cast<unsigned>(grid)), dim3(Shape<N>::threads), smem, s, 1, q_map, a, pl, ws);
}

}  // namespace

size_t mass_workspace_bytes(int n_q, int h_s, int n_seq) {  // (of either kind: groups are sequences or rows)
  const MassPlan p = make_plan(n_q, h_s, std::max(n_q, n_seq), false);
  return p.off_rank + round_up(static_cast<size_t>(n_q) * 4, 256);
}

cudaError_t launch_attn_mass(const MassArgs& a, cudaStream_t s, const char** err) {
  const bool sparse = a.idx != nullptr;
  const MassPlan pl = make_plan(a.n_q, a.h_s, a.n_seq, sparse);
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  const MassWs ws{reinterpret_cast<__half*>(base), reinterpret_cast<float4*>(base + pl.off_cols),
                  reinterpret_cast<int4*>(base + pl.off_groups), reinterpret_cast<int*>(base + pl.off_rank)};
  const EncodeFn enc = encode_fn();
  if (!enc) {
    *err = "attn_mass: cuTensorMapEncodeTiled is not available";
    return cudaErrorNotSupported;
  }
  // rows of 576 fp16 in boxes of 64 dims x n columns, 128-byte swizzle; rows past the end read as zero
  CUtensorMap q_map;
  const cuuint64_t columns = static_cast<cuuint64_t>(a.n_q) * a.h_s;
  const cuuint64_t dims[3] = {kLatent, columns, 1}, strides[2] = {kLatent * 2, kLatent * 2 * columns};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(pl.n), 1}, one[3] = {1, 1, 1};
  if (enc(&q_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, ws.q, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    *err = "attn_mass: tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaSuccess;
  if (!sparse) {
    const int64_t threads = static_cast<int64_t>(a.n_q) + a.n_seq;
    e = launch_pdl(mass_order_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, 1, a, ws);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(mass_query_kernel, dim3(a.n_q, (a.h_s + 7) / 8), dim3(256), 0, s, 1, a, ws);
  if (e != cudaSuccess) return e;
  // one CTA per SM, fewer where there are fewer units
  const int64_t tiles = ((sparse ? a.topk : a.max_ctx) + kTile - 1) / kTile;
  const int64_t rows = sparse ? 1 : a.n_q;
  const int64_t units = tiles * (sparse ? a.n_q : static_cast<int64_t>(a.n_seq) * ((rows * a.h_s + pl.n - 1) / pl.n));
  const int grid = static_cast<int>(std::min<int64_t>(multiprocessors(), units));
  switch (pl.n) {
    case 16: return sparse ? launch_main<true, 16>(q_map, a, pl, ws, grid, s) : launch_main<false, 16>(q_map, a, pl, ws, grid, s);
    case 32: return sparse ? launch_main<true, 32>(q_map, a, pl, ws, grid, s) : launch_main<false, 32>(q_map, a, pl, ws, grid, s);
    case 64: return sparse ? launch_main<true, 64>(q_map, a, pl, ws, grid, s) : launch_main<false, 64>(q_map, a, pl, ws, grid, s);
    default: return sparse ? launch_main<true, 96>(q_map, a, pl, ws, grid, s) : launch_main<false, 96>(q_map, a, pl, ws, grid, s);
  }
}

}  // namespace dsa
