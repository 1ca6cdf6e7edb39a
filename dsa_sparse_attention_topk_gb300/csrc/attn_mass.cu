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
// A product of codes and queries is below 2^34, so that scales from 2^60 on could take a sum out of fp32 whose logit is
// within it: such a position's are held 2^-64 as large, and the factor is put back behind the column's (kLift).
//
// Sums in fixed point.  A position's rows are worked on by several CTAs, and its weight is added up over calls.
// m holds whole numbers of 2^-36 and takes additions atomically: integers add up the same in any order, so equal
// calls give equal bits.
//
// Layout.  M = 128 positions (a TMEM lane each), N = 16..128 columns, a column being one head of one query row;
// the sum over columns then stays within a thread.  Positions are the A operand, widened codes in tensor memory;
// the columns' queries lie in shared memory, by TMA.  A group is a sequence with its rows (dense) or one row with its
// entries (sparse).  Items (group, chunk of N columns, tile of 128 positions) are shared out evenly over one CTA per
// SM; a chunk's queries stay while its tiles pass, each tile a ring of pieces of 128 dims.
//
// Bound.  32 rows of 128 heads over 16-32K positions each take 131 us (what has to be read 72, products 59), 64 rows of
// 128 heads over 32K 310 (products 157), 512 rows of 128 heads over 2048 entries 199 (products 74).  A tile is 6000 to
// 7000 cycles at 128 columns, 2304 of them products: an accumulator waits for the warps that scale and add it, two of
// them fit beside the widened codes, and those warps also have the tile's exponentials, 500 cycles of which the
// accumulators lie full.  Tried and slower: one read of 32 columns instead of two of 16 (145 us: spills), products of
// floats one by one (134), a single lane that polls for its warp (143), suspended waits with a hint (137).

#include <cuda.h>

#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_launch.h"
#include "tc_utils.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                        // positions of an MMA
constexpr int kBlocks = kLatent / 64;             // 64-dim blocks of a row
// A tile's staged records, in the order in which they are worked on: piece 0 dims 512.. with the scales (96 bytes a
// position), pieces 1..4 dims 128 (s - 1) .. of 128 bytes a position in the 128-byte swizzle, which lanes read without
// conflicts.  dim0(s) is the piece's first.
constexpr int kPiece = kTile * 128, kPiece0 = 96, kStageBytes = 4 * kPiece + kTile * kPiece0;
__host__ __device__ constexpr int dim0(int s) { return s == 0 ? 512 : 128 * (s - 1); }
__host__ __device__ constexpr int piece_at(int s) { return s == 0 ? 4 * kPiece : (s - 1) * kPiece; }
constexpr int kWarpB = 0, kWarpMma0 = 1, kWarpRec = 3, kWarpConv0 = 4, kWarpEpi0 = 8;  // (products: 1 and 2)
constexpr float kMassOne = 68719476736.0f;        // 2^36
constexpr float kMassMost = 67108864.0f;          // 2^26: one addition's limit
constexpr float kLarge = 1152921504606846976.0f;  // 2^60: a position with such a scale
constexpr float kLift = 18446744073709551616.0f;  // has them 2^-64 as large

// What the columns of a chunk decide.
template <int N> struct Shape {
  static constexpr int width = N == 128 ? 32 : 16;          // columns of four warps
  static constexpr int parts = N / width;                   // fours of warps
  static constexpr int threads = 32 * (kWarpEpi0 + 4 * parts);  // (sparse: and four warps)
  static constexpr int pieces = N == 128 ? 5 : N == 64 ? 9 : 10;  // of staged records
  static constexpr int tables = (pieces + 4) / 5 + 1;       // tiles whose slots are at hand
  static constexpr int slots = N == 16 ? 3 : 1;             // chunks of queries in shared memory
  static constexpr int block = N * 128;                     // bytes of 64 dims
  static constexpr int off_stage = slots * kBlocks * block;
  // [2][N / 2] pairs of columns, 16 bytes
  static constexpr int off_col = off_stage + (pieces % 5 ? pieces * kPiece : pieces / 5 * kStageBytes);
  static constexpr int off_limit = off_col + 2 * N * 8;     // [2][N] positions seen
  // [parts][128] sums of a position's weights over a part's columns, -1: no position
  static constexpr int off_sum = off_limit + 2 * N * 4;
  // [tables][128] slots of a tile's records, -1: none
  static constexpr int off_slot = off_sum + parts * kTile * 4;
  static constexpr int off_ctl = off_slot + tables * kTile * 4;
  // where piece d of all, piece s of its tile, is staged
  __device__ static __forceinline__ int staged(uint32_t d, int s) {
    return off_stage + (pieces % 5 ? static_cast<int>(d % pieces) * kPiece
                                   : static_cast<int>(d / 5 % (pieces / 5)) * kStageBytes + piece_at(s));
  }
  // tensor memory columns: accumulators, tiles of 128 dims (64 each), scales and positions of three tiles (with two,
  // those of the tile after next could be written while the last accumulator of this one is scaled)
  static constexpr int accs = N == 128 ? 2 : N == 64 ? 3 : 4;
  static constexpr int ring = N == 128 ? 3 : N == 64 ? 4 : 5;
  static constexpr int col_a = accs * N;
  static constexpr int col_info = col_a + 64 * ring;
  static_assert(col_info + 24 <= 512 && ring >= accs, "tensor memory");
};
constexpr int kMostSlots = 3, kMostAccs = 4, kMostPieces = 10;

struct MassPlan {
  int n;             // columns of a chunk: 16, 32, 64 or 128
  int groups;
  size_t off_cols, off_groups, off_rank;
};
struct MassWs {
  __half* q;         // [columns][576], times a power of two per column
  float4* cols;      // per column: logit per product (log2 units), -lse, positions it sees (int)
  int4* groups;      // positions or entries, first column, columns, sequence
  int* rank;         // dense: place of a row in the order of sequences
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

// Dense: rows in the order of their sequences, those that see nothing behind the last.  A thread per row counts the
// rows before it, a thread per sequence its rows and the furthest position they see.
__global__ void __launch_bounds__(256)
mass_order_kernel(MassArgs a, MassWs ws) {
  __shared__ int s_seq[1024], s_limit[1024];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const bool is_row = i < a.n_q, is_group = !is_row && i < static_cast<int64_t>(a.n_q) + a.n_seq;
  const bool live = is_row && row_limit(a, static_cast<int>(i), true) > 0;
  const int seq = is_row ? (live ? a.q_seq[i] : INT32_MAX) : static_cast<int>(i - a.n_q);
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
  if (is_row) ws.rank[i] = before;
  if (is_group) ws.groups[seq] = make_int4(furthest, before * a.h_s, own * a.h_s, seq);
}

// One warp per (row, head): the query as fp16 with its largest value in [2^14, 2^15), and the column's constants.
// A head whose query or lse is NaN (or its query infinite) gets zeros and weight 0; zeros too the heads of a dense row that
// sees nothing: the last sequence's last chunk reads on into them, and what lies there has to be numbers.
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
  const int limit = a.idx ? 0 : row_limit(a, t, false);
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
  const bool unseen = !a.idx && limit == 0, dead = unseen || top >= 0x7F80u || lse != lse;
  // largest in [2^14, 2^15), or the factor 2^109, which makes the smallest bf16 the smallest fp16: beyond it nothing is
  // gained, and the column's own factor would leave the normal range.  In two powers of two
  const int k = min(14 + 127 - max(static_cast<int>(top >> 7), 1), 109);
  const float f0 = exp2i(k / 2), f1 = exp2i(k - k / 2);
  uint32_t* dst = reinterpret_cast<uint32_t*>(ws.q + to * kLatent);
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const float x = __uint_as_float(raw[i] << 16) * f0 * f1, y = __uint_as_float(raw[i] & 0xFFFF0000u) * f0 * f1;
    const __half2 v = dead ? __floats2half2_rn(0.f, 0.f) : __floats2half2_rn(x, y);
    dst[32 * i + lane] = *reinterpret_cast<const uint32_t*>(&v);
  }
  if (lane == 0) {
    if (dead && !unseen) flag(a.status, DSA_STATUS_NAN_SCORE);
    const float c = a.sm_scale * 1.4426950408889634f;
    const bool none = dead || lse == -INFINITY;
    ws.cols[to] = make_float4(dead ? 0.f : c * (1.0f / f0) * (1.0f / f1), none ? -INFINITY : -lse * 1.4426950408889634f,
                              __int_as_float(limit), 0.f);
  }
}

// ---- the kernel -----------------------------------------------------------------------------
struct MassCtl {
  uint64_t b_full[kMostSlots][5], b_empty[kMostSlots][5];   // a chunk's queries, 128 dims (two blocks) a barrier
  uint64_t a_full[5], a_empty[5];                           // tiles of 128 dims
  uint64_t rec_full[kMostPieces], rec_empty[kMostPieces];   // staged pieces
  uint64_t d_full[kMostAccs], d_free[kMostAccs];
  uint64_t part_full, part_empty;                           // a tile's sums
  uint64_t col_full[2], col_empty[2];
  uint64_t slot_full[3], slot_empty[3];                     // sparse: a tile's slots
  uint64_t drained[2];
  int all_seen[2];                      // every column of the chunk sees the whole tile
  long long scan[28];
  int first_group, first_tile, first_chunk, items, abort;
  uint32_t tmem;
};
constexpr int kMostSmem = 232448;
static_assert(Shape<128>::off_ctl + sizeof(MassCtl) <= kMostSmem &&
              Shape<64>::off_ctl + sizeof(MassCtl) <= kMostSmem &&
              Shape<32>::off_ctl + sizeof(MassCtl) <= kMostSmem &&
              Shape<16>::off_ctl + sizeof(MassCtl) <= kMostSmem, "shared memory");

// A walk over the CTA's items: chunk c of tile `tile` of group g
struct Walk {
  int left, g, tile, c, chunks, tiles;
  int4 grp;
  __device__ __forceinline__ bool same_chunk(const Walk& o) const { return g == o.g && c == o.c; }
};
template <int N>
__device__ __forceinline__ void open_group(const MassWs& ws, Walk& w) {
  w.grp = ws.groups[w.g];
  w.tiles = (w.grp.x + kTile - 1) / kTile;
  w.chunks = (w.grp.z + N - 1) / N;
}
template <int N>
__device__ __forceinline__ bool walk_begin(const MassWs& ws, const MassCtl& ctl, Walk& w) {
  w.left = ctl.items;
  if (w.left <= 0) return false;
  w.g = ctl.first_group;
  w.tile = ctl.first_tile;
  w.c = ctl.first_chunk;
  open_group<N>(ws, w);
  return true;
}
// on to the next item; false at the end.  (The groups behind have items as long as some are left.)
template <int N>
__device__ __forceinline__ bool walk_next(const MassWs& ws, int groups, Walk& w) {
  if (--w.left <= 0) return false;
  if (++w.tile < w.tiles) return true;
  w.tile = 0;
  if (++w.c < w.chunks) return true;
  w.c = 0;
  do {
    if (++w.g >= groups) return false;
    open_group<N>(ws, w);
  } while (!w.tiles || !w.chunks);
  return true;
}

__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
  return r;
}
// D (+)= A B, fp16 operands, A in tensor memory; B by the low word of its descriptor (rows of 128 bytes swizzled, groups of
// eight 1024 bytes apart)
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                           uint32_t leader) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 b;\n setp.ne.b32 e, %5, 0;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %6};\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}"
      :: "r"(d), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(leader), "n"(kDescHi) : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void commit_if(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      :: "r"(smem_u32(bar)), "r"(leader) : "memory");
}
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
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
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" :: "r"(taddr), "r"(__float_as_uint(v)) : "memory");
}
// 16 bytes of global to shared memory, asynchronously, where `on`
__device__ __forceinline__ void copy16_if(bool on, uint32_t to, const void* from) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p cp.async.cg.shared.global [%0], [%1], 16;\n}"
               :: "r"(to), "l"(from), "r"(static_cast<uint32_t>(on)) : "memory");
}
// a bounded wait (tc::mbar_wait) out of line, behind one attempt in line
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status) {
  return tc::mbar_wait(bar, parity, abort, status);
}

// weight `total` to position pos of sequence b
__device__ __forceinline__ void add_mass(const MassArgs& a, int b, int pos, float total) {
  if (!a.mass) return;
  if (total != total) flag(a.status, DSA_STATUS_NAN_SCORE);
  else if (total > 0.f)
    atomicAdd(reinterpret_cast<unsigned long long*>(a.mass + static_cast<int64_t>(b) * a.mass_stride + pos),
              static_cast<unsigned long long>(__float2ll_rn(fminf(total, kMassMost) * kMassOne)));
}

// The sum of a lane's weights where one of the warp's positions has large scales: columns without weight are left out, as their
// products here may be no numbers.  (Out of line and rolled up: in line it took the entries' kernel 4% of its time.)
__device__ __noinline__ float sum_lifted(const float* acc, int columns, const float* cols, const int* limits, int pos, float lift) {
  float total = acc[0] != acc[0] ? NAN : 0.f;  // (the position's values: every column's, or none's)
#pragma unroll 1
  for (int i = 0; i < columns; ++i) {
    const float* k = cols + 4 * (i >> 1) + (i & 1);
    if (pos < limits[i]) total += ex2(fmaf(acc[i] * k[0], lift, k[2]));
  }
  return total;
}

template <bool SPARSE, int N>
__global__ void __launch_bounds__(Shape<N>::threads + (SPARSE ? 128 : 0), 1)
attn_mass_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap piece0_map,
                 const __grid_constant__ CUtensorMap piece_map, MassArgs a, MassPlan pl, MassWs ws) {
  using S = Shape<N>;
  constexpr int kThreads = S::threads + (SPARSE ? 128 : 0);
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    for (int i = 0; i < 5; ++i) {
      tc::mbar_init(&ctl.a_full[i], 4);
      tc::mbar_init(&ctl.a_empty[i], 1);
    }
    for (int i = 0; i < S::pieces; ++i) {
      tc::mbar_init(&ctl.rec_full[i], SPARSE ? 128 : 1);
      tc::mbar_init(&ctl.rec_empty[i], 4);
    }
    for (int i = 0; i < S::tables; ++i) {
      tc::mbar_init(&ctl.slot_full[i], 1);
      tc::mbar_init(&ctl.slot_empty[i], 8);
    }
    for (int i = 0; i < S::accs; ++i) {
      tc::mbar_init(&ctl.d_full[i], 1);
      tc::mbar_init(&ctl.d_free[i], 4 * S::parts);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&ctl.drained[i], 1);
      tc::mbar_init(&ctl.col_full[i], 1);
      tc::mbar_init(&ctl.col_empty[i], 4 * S::parts);
    }
    tc::mbar_init(&ctl.part_full, 4 * S::parts);
    tc::mbar_init(&ctl.part_empty, 1);
    tc::mbar_fence_init();
    ctl.first_group = ctl.first_tile = ctl.first_chunk = 0;
  }
  if (warp == kWarpMma0) tc::tmem_alloc(&ctl.tmem, 512);
  pdl_wait();
  // ---- the CTA's share of the items ----
  {
    const int per = (pl.groups + kThreads - 1) / kThreads;
    const int g0 = min(tid * per, pl.groups), g1 = min(g0 + per, pl.groups);
    long long sum = 0;
    auto items_of = [&](int g) {
      const int4 grp = ws.groups[g];
      return static_cast<long long>((grp.x + kTile - 1) / kTile) * ((grp.z + N - 1) / N);
    };
    for (int g = g0; g < g1; ++g) sum += items_of(g);
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) ctl.scan[warp] = incl;
    __syncthreads();
    long long before = incl - sum, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += ctl.scan[w];
      total += ctl.scan[w];
    }
    const long long start = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
    if (tid == 0) ctl.items = static_cast<int>(end - start);
    if (start < end && start >= before && start < before + sum) {
      int g = g0;
      long long rest = start - before;
      for (long long u; rest >= (u = items_of(g)); ++g) rest -= u;
      const int tiles = (ws.groups[g].x + kTile - 1) / kTile;
      ctl.first_group = g;
      ctl.first_tile = static_cast<int>(rest % tiles);
      ctl.first_chunk = static_cast<int>(rest / tiles);
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
  Walk w;
  // (The roles' loops are rolled up: together they have to stay within the instruction cache.)

  if (warp == kWarpB) {
    // ---- a chunk's queries, 128 dims at a time, and its columns' constants; columns behind the group's last have
    // no weight.  And the tiles' sums on their way out, two items behind (left to the first of the parts they
    // were 2400 of its 6000 cycles a tile of entries, for which everything waits) ----
    Walk done;
    uint32_t n_done = 0;
    auto give = [&] {
      if (!wait_warp(&ctl.part_full, n_done)) return false;
      const float* sums = reinterpret_cast<const float*>(smem + S::off_sum);
      const int64_t row = SPARSE ? static_cast<int64_t>(done.g) * a.topk + done.tile * kTile : 0;
#pragma unroll 1
      for (int i = lane; i < kTile; i += 32) {
        float total = sums[i];
        if (total < 0.f) continue;
        const int pos = SPARSE ? a.idx[row + i] : done.tile * kTile + i;
#pragma unroll
        for (int k = 1; k < S::parts; ++k) total += sums[k * kTile + i];
        if (SPARSE && a.weights) a.weights[row + i] = total;
        add_mass(a, done.grp.w, pos, total);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ctl.part_empty);
      walk_next<N>(ws, pl.groups, done);
      ++n_done;
      return true;
    };
    if (walk_begin<N>(ws, ctl, w)) {
      done = w;
      int slot = 0;
      uint32_t phase = 0, n = 0;
      bool ok = true, more = true, fresh = true;  // fresh: other columns than the item's before
      while (ok && more) {
        const int buf = n & 1;
        float4 info[(N + 31) / 32];
        int least = INT32_MAX;
#pragma unroll
        for (int i = 0; i < (N + 31) / 32; ++i) {
          const int col = w.c * N + 32 * i + lane;
          info[i] = make_float4(0.f, -INFINITY, __int_as_float(INT32_MAX), 0.f);
          if (32 * i + lane < N && col < w.grp.z) info[i] = ws.cols[w.grp.y + col];
          least = min(least, __float_as_int(info[i].z));
        }
        if (fresh) {
#pragma unroll 1
          for (int k = 0; k < 5; ++k) {
            ok = wait_warp(&ctl.b_empty[slot][k], phase ^ 1u);
            if (!ok) break;
            if (lane == 0) {
              uint64_t* bar = &ctl.b_full[slot][k];
              uint8_t* to = smem + (slot * kBlocks + dim0(k) / 64) * S::block;
              tc::mbar_arrive_expect_tx(bar, (k ? 2 : 1) * S::block);
              tc::tma_load_3d(to, &q_map, dim0(k), w.grp.y + w.c * N, 0, bar);
              if (k) tc::tma_load_3d(to + S::block, &q_map, dim0(k) + 64, w.grp.y + w.c * N, 0, bar);
            }
          }
          if (!ok) break;
          if (++slot == S::slots) {
            slot = 0;
            phase ^= 1u;
          }
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
          limits[at] = info[i].y == -INFINITY ? 0 : SPARSE ? INT32_MAX : __float_as_int(info[i].z);
        }
        if (lane == 0) ctl.all_seen[buf] = SPARSE || least >= (w.tile + 1) * kTile;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.col_full[buf]);
        const Walk was = w;
        more = walk_next<N>(ws, pl.groups, w);
        fresh = !w.same_chunk(was);
        ++n;
        while (ok && n_done < n && (n_done + 3 <= n || !more)) ok = give();
      }
      // copies in flight must land before the CTA ends; a slot that was never loaded is past the phase before its first
      if (*abort) {
        for (int i = 0; i < S::slots; ++i)
          for (int k = 0; k < 5; ++k) tc::mbar_drain(&ctl.b_full[i][k], i < slot ? phase : phase ^ 1u, 100000000ull);
        __nanosleep(1000000);  // (and those of a chunk begun)
      }
    }
  } else if (warp == kWarpMma0 || warp == kWarpMma0 + 1) {
    // ---- products: the two warps take turns, so that one's waits and issue pass while the other's products run.
    // (A buffer's phases that were the other warp's turn are over: the accumulators that were read say so, and are waited
    // for first.) ----
    const uint32_t leader = elect_leader(), mine = warp - kWarpMma0;
    constexpr uint32_t idesc = idesc_f16(N);
    const uint32_t b_first = smem_u32(smem) >> 4 | 1u << 16;
    int slot = 0;
    uint32_t phase = 0, d = 0;
    if (walk_begin<N>(ws, ctl, w)) {
      bool ok = true, more = true, fresh_b = true;
      while (ok && more) {
        const Walk was = w;
        more = walk_next<N>(ws, pl.groups, w);
        const bool leave_b = !more || !w.same_chunk(was);
        const uint32_t b_chunk = b_first + static_cast<uint32_t>(slot * kBlocks * S::block >> 4);
#pragma unroll 1
        for (int s = 0; s < 5; ++s, ++d) {
          if ((d & 1) != mine) continue;
          const uint32_t acc = d % S::accs, q = d % S::ring;
          ok = wait_warp(&ctl.d_free[acc], (d / S::accs) ^ 1u);
          ok = ok && wait_warp(&ctl.a_full[q], d / S::ring);
          if (fresh_b) ok = ok && wait_warp(&ctl.b_full[slot][s], phase);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t to = uniform(tmem + acc * N), from = uniform(tmem + S::col_a + 64 * q);
          const uint32_t b_lo = uniform(b_chunk + dim0(s) / 64 * (S::block >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16_ts(to, from + 8 * k, b_lo + 2 * k, idesc, k > 0, leader);
          if (s > 0)
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ts(to, from + 32 + 8 * k, b_lo + (S::block >> 4) + 2 * k, idesc, true, leader);
          commit_if(&ctl.d_full[acc], leader);
          commit_if(&ctl.a_empty[q], leader);
          if (leave_b) commit_if(&ctl.b_empty[slot][s], leader);
        }
        if (leave_b && ++slot == S::slots) {
          slot = 0;
          phase ^= 1u;
        }
        fresh_b = leave_b;
      }
    }
    if (*abort) {  // products in flight must end before the tensor memory is freed
      __syncwarp();
      commit_if(&ctl.drained[mine], leader);
      tc::mbar_drain(&ctl.drained[mine], 0, 100000000ull);
    }
  } else if (warp == kWarpRec) {
    // ---- where a tile's records lie, and those of whole pages by TMA, a piece at a time.  Entry and page of the tile
    // behind are looked up meanwhile. ----
    if (walk_begin<N>(ws, ctl, w)) {
      const int64_t table_end = static_cast<int64_t>(a.max_pages) * kPage;
      int pos[4], page[4];  // of positions 32 k + lane of a tile, -1: none
      auto entry = [&] {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = w.tile * kTile + 32 * k + lane;
          pos[k] = i < w.grp.x ? (SPARSE ? a.idx[static_cast<int64_t>(w.g) * a.topk + i] : i) : -1;
        }
      };
      auto lookup = [&] {
        const int len = SPARSE ? a.seq_lens[w.grp.w] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (SPARSE && pos[k] >= 0 && (pos[k] >= len || pos[k] >= table_end)) {
            flag(a.status, DSA_STATUS_BAD_INDEX);
            pos[k] = -1;
          }
          page[k] = pos[k] >= 0 ? a.page_table[static_cast<int64_t>(w.grp.w) * a.max_pages + pos[k] / kPage] : 0;
        }
      };
      entry();
      lookup();
      bool ok = true, more = true;
      for (uint32_t t = 0; ok && more; ++t) {
        const int buf = t % S::tables;
        int* s_slot = reinterpret_cast<int*>(smem + S::off_slot) + buf * kTile;
        if (SPARSE) {
          ok = wait_warp(&ctl.slot_empty[buf], (t / S::tables) ^ 1u);
          if (!ok) break;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (pos[k] >= 0 && (page[k] < 0 || page[k] >= a.num_pages)) {
            flag(a.status, DSA_STATUS_BAD_PAGE);
            pos[k] = -1;
          }
          // (dense: read by the warps that widen before the tile's first piece is given back)
          s_slot[32 * k + lane] = pos[k] >= 0 ? page[k] * kPage + (pos[k] & (kPage - 1)) : -1;
        }
        __syncwarp();
        more = walk_next<N>(ws, pl.groups, w);
        if constexpr (SPARSE) {
          if (lane == 0) tc::mbar_arrive(&ctl.slot_full[buf]);
          if (more) {
            entry();
            lookup();
          }
        } else {
          const int first_page = s_slot[0], second_page = s_slot[64];  // the tile's two pages, if they are there
          if (more) entry();
#pragma unroll 1
          for (int s = 0; s < 5; ++s) {
            const uint32_t d = 5 * t + s;
            ok = wait_warp(&ctl.rec_empty[d % S::pieces], (d / S::pieces) ^ 1u);
            if (!ok) break;
            if (lane == 0) {
              // (what lies behind the sequence in its last page comes with it and is not looked at)
              uint64_t* bar = &ctl.rec_full[d % S::pieces];
              uint8_t* to = smem + S::staged(d, s);
              const int bytes = (s ? 128 : kPiece0) * kPage;
              tc::mbar_arrive_expect_tx(bar, ((first_page >= 0) + (second_page >= 0)) * bytes);
              const CUtensorMap* map = s ? &piece_map : &piece0_map;
              if (first_page >= 0) tc::tma_load_3d(to, map, dim0(s) / 4, first_page, 0, bar);
              if (second_page >= 0) tc::tma_load_3d(to + bytes, map, dim0(s) / 4, second_page, 0, bar);
            }
            if (s == 0 && more) lookup();
          }
        }
      }
      if (!SPARSE && *abort) __nanosleep(1000000);  // copies in flight must land before the CTA ends
    }
  } else if (warp >= kWarpConv0 && warp < kWarpEpi0) {
    // ---- codes widened to fp16 into tensor memory, a position a lane ----
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if (walk_begin<N>(ws, ctl, w)) {
      bool ok = true, more = true;
      uint32_t q = 0;  // tiles of 128 dims widened
      for (uint32_t visit = 0; ok && more; ++visit) {
#pragma unroll 1
        for (int s = 0; s < 5; ++s, ++q) {
          const uint32_t at = q % S::ring;
          ok = wait_warp(&ctl.rec_full[q % S::pieces], q / S::pieces);
          ok = ok && wait_warp(&ctl.a_empty[at], (q / S::ring) ^ 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint8_t* mine = smem + S::staged(q, s) + row * (s ? 128 : kPiece0);
          if (s == 0) {
            uint32_t info[8];
            bool fine = true;
            const uint4 four = *reinterpret_cast<const uint4*>(mine + 64);
            info[0] = four.x;
            info[1] = four.y;
            info[2] = four.z;
            info[3] = four.w;
            info[4] = *reinterpret_cast<const uint32_t*>(mine + 80);
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const float scale = fabsf(__uint_as_float(info[i]));
              fine = fine && scale * 448.0f < INFINITY;
              most = fmaxf(most, scale);
            }
            if (most >= kLarge)
#pragma unroll
              for (int i = 0; i < 5; ++i) info[i] = __float_as_uint(__uint_as_float(info[i]) * (1.0f / kLift));
            if (!fine) info[0] = 0x7FC00000u;  // NaN: the position has no weight
            const int buf = visit % S::tables;
            if (SPARSE) ok = wait_warp(&ctl.slot_full[buf], visit / S::tables);
            // what the scales have to be multiplied by, -1: no position
            const int slot = reinterpret_cast<const int*>(smem + S::off_slot)[buf * kTile + row];
            info[5] = __float_as_uint(slot < 0 ? -1.f : most >= kLarge ? kLift : 1.f);
            if (SPARSE) {
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&ctl.slot_empty[buf]);
            }
            info[6] = info[7] = 0;
            tmem_st8(tmem + lanes + S::col_info + 8 * (visit % 3), info);
          }
          const int turn = s ? (row & 7) << 4 : 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // 32 codes, 16 columns
            if (s == 0 && j >= 2) break;
            const uint4 lo = *reinterpret_cast<const uint4*>(mine + ((32 * j) ^ turn));
            const uint4 hi = *reinterpret_cast<const uint4*>(mine + ((32 * j + 16) ^ turn));
            const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const __half2 x = e4m3x2_to_f16x2(static_cast<uint16_t>(u[i] & 0xFFFFu)), y = e4m3x2_to_f16x2(static_cast<uint16_t>(u[i] >> 16));
              o[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
              o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
            }
            tc::tmem_st16(tmem + lanes + S::col_a + 64 * at + 16 * j, o);
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.rec_empty[q % S::pieces]);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.a_full[at]);
        }
        more = walk_next<N>(ws, pl.groups, w);
      }
    }
  } else if (SPARSE && warp >= kWarpEpi0 + 4 * S::parts) {
    // ---- records of entries, wherever they lie: eight lanes 128 bytes of one, asynchronously.  A warp's request for 512
    // bytes takes it 40 cycles and more, so four warps do nothing else.  (512 rows of 128 heads over 2048 entries: one
    // warp 311 us, the sixteen that form the weights, which then wait for it, 230; these four 213.  A bulk copy a record
    // takes the thread that asks 80 cycles.) ----
    if (walk_begin<N>(ws, ctl, w)) {
      constexpr int kEach = 8;
      const int chunk = lane & 7, r = (warp - kWarpEpi0 - 4 * S::parts) * 4 + (lane >> 3);
      const uint32_t tiles = static_cast<uint32_t>(w.left);
      const uint8_t* mine = a.kv_cache + 16 * chunk;
      bool ok = true;
      for (uint32_t t = 0; ok && t < tiles; ++t) {
        const uint32_t buf = t % S::tables;
        ok = wait_warp(&ctl.slot_full[buf], t / S::tables);
        if (!ok) break;
        const int* s_slot = reinterpret_cast<const int*>(smem + S::off_slot) + buf * kTile + r;
        const uint8_t* from[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int slot = s_slot[16 * i];
          from[i] = slot < 0 ? nullptr : mine + static_cast<int64_t>(slot) * kKvTokBytes;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.slot_empty[buf]);
#pragma unroll 1
        for (int s = 0; s < 5; ++s) {
          const uint32_t d = 5 * t + s;
          ok = wait_warp(&ctl.rec_empty[d % S::pieces], (d / S::pieces) ^ 1u);
          if (!ok) break;
          const int width = s ? 128 : kPiece0;
          const bool on = s || chunk < kPiece0 / 16;
          const uint32_t to = smem_u32(smem) + S::staged(d, s) + r * width + ((s ? chunk ^ (r & 7) : chunk) << 4);
#pragma unroll
          for (int i = 0; i < kEach; ++i) copy16_if(on && from[i], to + 16 * width * i, from[i] + dim0(s));
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(&ctl.rec_full[d % S::pieces])) : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp >= kWarpEpi0) {
    // ---- weights: a position a lane, S::width of a chunk's columns each four warps ----
    constexpr int W = S::width;
    const int quarter = warp & 3, part = (warp - kWarpEpi0) >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t d = 0;
    if (walk_begin<N>(ws, ctl, w)) {
      bool ok = true, more = true;
      for (uint32_t visit = 0; ok && more; ++visit) {
        const uint32_t tile_info = tmem + lanes + S::col_info + 8 * (visit % 3);
        uint64_t acc[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) acc[i] = 0ull;
        float lift = -1.f;
#pragma unroll 1
        for (int s = 0; s < 5; ++s, ++d) {
          const uint32_t at = d % S::accs;
          ok = wait_warp(&ctl.d_full[at], d / S::accs);
          if (!ok) break;
          tc::fence_after_sync();
          const float scale = tmem_ld1(tile_info + (s ? s - 1 : 4));
          if (s == 0) lift = tmem_ld1(tile_info + 5);
#pragma unroll
          for (int h = 0; h < W / 16; ++h) {  // (16 columns at a time: 768 threads have 80 registers each)
            uint32_t v[16];
            tc::tmem_ld16(tmem + lanes + at * N + part * W + 16 * h, v);
            tc::tmem_wait_ld();
            if (h == W / 16 - 1) {
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&ctl.d_free[at]);
            }
            const uint64_t both = pair(scale, scale);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[8 * h + i] = fma_pair(both, pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), acc[8 * h + i]);
          }
        }
        const int buf = visit & 1;
        ok = ok && wait_warp(&ctl.col_full[buf], visit >> 1);
        if (!ok) break;
        const int pos = w.tile * kTile + row;
        const ulonglong2* cols = reinterpret_cast<const ulonglong2*>(smem + S::off_col) + (buf * N + part * W) / 2;
        const int2* limits = reinterpret_cast<const int2*>(smem + S::off_limit) + (buf * N + part * W) / 2;
        float total = 0.f;
        if (__any_sync(0xffffffffu, lift > 1.f)) {
          float each[W];
#pragma unroll
          for (int i = 0; i < W / 2; ++i) {
            each[2 * i] = unpair(acc[i]).x;
            each[2 * i + 1] = unpair(acc[i]).y;
          }
          total = sum_lifted(each, W, reinterpret_cast<const float*>(cols), reinterpret_cast<const int*>(limits), pos, fmaxf(lift, 1.f));
        } else if (SPARSE || ctl.all_seen[buf]) {
          float odd = 0.f;
#pragma unroll
          for (int i = 0; i < W / 2; ++i) {
            const ulonglong2 k = cols[i];
            const float2 x = unpair(fma_pair(acc[i], k.x, k.y));
            total += ex2(x.x);
            odd += ex2(x.y);
          }
          total += odd;
        } else {
#pragma unroll
          for (int i = 0; i < W / 2; ++i) {
            const ulonglong2 k = cols[i];
            const int2 lim = limits[i];
            const float2 x = unpair(fma_pair(acc[i], k.x, k.y));
            total += (pos < lim.x ? ex2(x.x) : 0.f) + (pos < lim.y ? ex2(x.y) : 0.f);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.col_empty[buf]);
        ok = wait_warp(&ctl.part_empty, visit ^ 1u);
        if (!ok) break;
        reinterpret_cast<float*>(smem + S::off_sum)[part * kTile + row] = lift > 0.f ? total : -1.f;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.part_full);
        more = walk_next<N>(ws, pl.groups, w);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kWarpMma0) tc::tmem_dealloc(tmem, 512);
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

MassPlan make_plan(int n_q, int h_s, int n_seq, bool sparse) {
  MassPlan p;
  p.groups = sparse ? n_q : n_seq;
  // a chunk's columns: all of a group of average rows where they fit
  const int64_t cols = static_cast<int64_t>(h_s) * (sparse ? 1 : std::max(1, (n_q + n_seq - 1) / n_seq));
  p.n = cols <= 16 ? 16 : cols <= 32 ? 32 : cols <= 64 ? 64 : 128;
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

struct MassMaps {
  CUtensorMap q, piece0, piece;
};
template <bool SPARSE, int N>
cudaError_t launch_main(const MassMaps& m, const MassArgs& a, const MassPlan& pl, const MassWs& ws, int grid, cudaStream_t s) {
  constexpr size_t smem = Shape<N>::off_ctl + sizeof(MassCtl);
  const cudaError_t e = cudaFuncSetAttribute(attn_mass_kernel<SPARSE, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_mass_kernel<SPARSE, N>, dim3(static_cast<unsigned>(grid)), dim3(Shape<N>::threads + (SPARSE ? 128 : 0)), smem, s, 1, m.q,
                    m.piece0, m.piece, a, pl, ws);
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
  // a 2-d array of rows, boxes of `box_x` x `box_rows` elements; rows past the end read as zero
  auto map = [&](CUtensorMap* m, CUtensorMapDataType type, const void* at, uint64_t width, uint64_t pitch, uint64_t rows, int box_x,
                 int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[3] = {width, rows, 1}, strides[2] = {pitch, pitch * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
    return enc(m, type, 3, const_cast<void*>(at), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  MassMaps maps{};
  const uint64_t columns = static_cast<uint64_t>(a.n_q) * a.h_s, slots = static_cast<uint64_t>(a.num_pages) * kPage;
  if (!map(&maps.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws.q, kLatent, kLatent * 2, columns, 64, pl.n, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (!sparse && !map(&maps.piece0, CU_TENSOR_MAP_DATA_TYPE_INT32, a.kv_cache, kKvTokBytes / 4, kKvTokBytes, slots, kPiece0 / 4, kPage,
           CU_TENSOR_MAP_SWIZZLE_NONE)) ||
      (!sparse && !map(&maps.piece, CU_TENSOR_MAP_DATA_TYPE_INT32, a.kv_cache, kKvTokBytes / 4, kKvTokBytes, slots, 32, kPage,
           CU_TENSOR_MAP_SWIZZLE_128B))) {
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
    case 16: return sparse ? launch_main<true, 16>(maps, a, pl, ws, grid, s) : launch_main<false, 16>(maps, a, pl, ws, grid, s);
    case 32: return sparse ? launch_main<true, 32>(maps, a, pl, ws, grid, s) : launch_main<false, 32>(maps, a, pl, ws, grid, s);
    case 64: return sparse ? launch_main<true, 64>(maps, a, pl, ws, grid, s) : launch_main<false, 64>(maps, a, pl, ws, grid, s);
    default: return sparse ? launch_main<true, 128>(maps, a, pl, ws, grid, s) : launch_main<false, 128>(maps, a, pl, ws, grid, s);
  }
}

}  // namespace dsa
