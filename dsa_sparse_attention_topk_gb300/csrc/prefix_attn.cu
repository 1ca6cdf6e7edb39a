// Attention of a batch whose sequences share a long prefix, on the 5th-generation tensor
// cores: dense absorbed-MLA attention over the paged FP8 latent cache.
//
// Query row t of sequence b sees the positions p < n_t = min(q_pos[t] + 1, seq_lens[b]):
// those below prefix_len from the shared pages, the rest (its tail) from its own page-table
// row.  With kv[p] the dequantised latent row,
//     l_p = sm_scale * q[t, h] . kv[p],  o[t, h] = sum_p softmax(l)_p kv[p][0:512].
// The work is 2 (576 + 512) flop per (row, head, position) against 596 bytes per position:
// with 128 heads or more per position (rows of several sequences, for the prefix) it is
// bound by the tensor cores.
//
// Three kernels.
//   expand   dequantises the prefix once for all rows, and each tail once, into bf16 rows in
//            the workspace (the same rounding the sparse attention makes), so that the main
//            kernel can feed its MMAs by TMA alone.  A position whose page is out of range
//            becomes a zero row that a bit marks invalid; one with NaN or infinite
//            values a zero row marked poisonous, whose logit is NaN for the rows that see it
//            and nothing to the others.
//   attend   one CTA pair per item: 128 rows of (query row, head) against a run of 64-position
//            tiles of the prefix (a tile of the flattened rows, shared by all sequences) or of
//            one query row's tail.
//   merge    joins a row's splits by their log-sum-exps.
//
// The pair.  The output accumulator of 128 rows x 512 columns would fill tensor memory, so
// each CTA of the pair holds one half of the value columns.  Computing the logits in both
// would cost half as much again; instead CTA c computes logits and weights of the tiles
// j = c (mod 2) and sends the weights (bf16, 16 KB) to its peer by a bulk copy into
// distributed shared memory; both then run P V over every tile, each on its half.
//
// The softmax reference.  Weights are 2^(x - r) with one fixed r per row, the row's
// largest logit (in units of log 2) in the item's first tile.  A weight may then exceed 1:
// fp32 and bf16 hold it up to 2^127 with unchanged relative precision, so nothing has to be
// rescaled inside the loop and the two CTAs need no agreement per tile.  At the end the pair
// compares each row's true maximum M with r, and if they lie further apart than 2^64 anywhere
// it runs the item again with r = M.
//
// Per CTA (9 warps): 0 loads the own tiles' blocks, 8 the peer tiles' value blocks, 1 issues
// Q K^T, 2 issues P V, 3 sends the weights, 4-7 turn logits into weights (one row a thread).
// Tensor memory (512 columns): O in 0..255, the logits in 256..319, the query's dims 0..383
// as bf16 pairs in 320..511.  Shared memory: the query's dims 384..575, both weight buffers,
// and 18 blocks of 64 positions x 64 dims: the value blocks of two own tiles (8), those of one
// peer tile (4), and a ring of 6 for the own tile's other five blocks, which only Q K^T reads.

#include <algorithm>
#include <cuda.h>

#include "dsa_common.cuh"
#include "dsa_launch.h"
#include "tc_utils.cuh"

namespace dsa {
namespace {

constexpr int kTile = 64;                     // positions per tile
constexpr int kRows = 128;                    // (query row, head) rows per item
constexpr int kHalfV = kVDim / 2;
constexpr int kBlock = kTile * 128;           // 64 positions x 64 dims, bf16: 8 KB
constexpr int kQBlock = kRows * 128;          // 128 rows x 64 dims: 16 KB
constexpr int kQTmemSteps = 24;               // K-steps of 16 with the query in tensor memory
constexpr int kQSmemBlocks = 3;
constexpr int kRing = 6, kLoose = 5;          // blocks only Q K^T reads: ring slots, per tile
constexpr int kThreads = 32 * 9;
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;
constexpr uint32_t kPBytes = kRows * 128;     // the weights of a tile
constexpr float kRange = 64.0f;               // |M - r| a row may have, in powers of two

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffPOwn = kOffQ + kQSmemBlocks * kQBlock;
constexpr uint32_t kOffPIn = kOffPOwn + kPBytes;
constexpr uint32_t kOffVOwn = kOffPIn + kPBytes;
constexpr uint32_t kOffVPeer = kOffVOwn + 8 * kBlock;
constexpr uint32_t kOffRing = kOffVPeer + 4 * kBlock;
constexpr uint32_t kOffCtl = kOffRing + kRing * kBlock;

struct PairCtl {
  uint64_t q_full, q_tmem;
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t vown_full[2], vown_empty[2];
  uint64_t vpeer_full, vpeer_empty;
  uint64_t s_full, s_free;   // logits written / read into registers
  uint64_t p_full;           // own weights in shared memory
  uint64_t p_empty;          // own weights read: by the own P V and by the peer's (its copy's)
  uint64_t pin_full;         // the peer's weights have landed
  uint64_t o_done;
  uint64_t r_full;           // CTA 1: the references have landed
  uint64_t fin_full;         // the peer's (max, sums) have landed
  uint32_t tmem_base;
  int abort;
  int redo;
  volatile uint32_t peer_vote[2];  // per attempt: 1: run again, 2: a wait ran out there
  float r[kRows];            // CTA 1: from CTA 0
  float2 fin2[kRows];        // the peer's max and sum of rounded weights
  float fin1[kRows];         // the peer's sum of unrounded weights
};
constexpr uint32_t kSmemBytes = kOffCtl + 3072;
static_assert(sizeof(PairCtl) <= 3072 && kSmemBytes <= 232448, "shared memory");
// the output rows are staged where the tiles' blocks were
constexpr int kStagePitch = kHalfV * 2 + 16;
static_assert(kRows * kStagePitch <= 18 * kBlock, "output staging");

struct PrefixPlan {
  int tiles_p, tiles_t;      // tiles of the prefix, and of the longest possible tail
  int sp, st;                // splits of the prefix and of each tail
  int mt;                    // 128-row tiles of the flattened rows
  int64_t rows_kv;           // rows of the expanded cache
  size_t off_words, off_o, off_ml, bytes;
};

struct PrefixWs {
  __nv_bfloat16* kv;         // [tiles_p * 64 + n_seq * tiles_t * 64][576]
  uint64_t* words;           // [tiles][2]: valid, poisonous
  __nv_bfloat16* o;          // [n_q * h_s][sp + st][512]
  float4* ml;                // [n_q * h_s][sp + st]: reference, sum of rounded weights, of unrounded ones
};

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Splits: the plan of least estimated time.  An item of n tiles takes about 5 + 0.65 n us
// on one of the n_sm / 2 CTA pairs; a further split costs every row its partial output, once
// written and once read.
PrefixPlan make_plan(int n_q, int h_s, int n_seq, int prefix_len, int max_ctx, int n_sm) {
  PrefixPlan p{};
  p.tiles_p = (prefix_len + kTile - 1) / kTile;
  p.tiles_t = (max_ctx - prefix_len + kTile - 1) / kTile;
  p.mt = static_cast<int>((static_cast<int64_t>(n_q) * h_s + kRows - 1) / kRows);
  const int pairs = std::max(1, n_sm / 2);
  const double fix = 5.0, per = 0.65;
  const double join = 2048.0 * n_q * h_s / 5.0e6;  // us a split
  double best = 1e30;
  for (int sp = p.tiles_p ? 1 : 0; sp <= std::min(p.tiles_p, 48); ++sp) {
    for (int st = p.tiles_t ? 1 : 0; st <= std::min(p.tiles_t, 16); st = st ? 2 * st : 1) {
      const double lp = sp ? fix + per * ((p.tiles_p + sp - 1) / sp) : 0.0;
      const double lt = st ? fix + per * ((p.tiles_t + st - 1) / st) : 0.0;
      const double np = static_cast<double>(p.mt) * sp, nt = static_cast<double>(n_q) * st;
      const double waves = static_cast<double>(static_cast<int64_t>((np + pairs - 1) / pairs));
      // the tails are counted half full: their lengths are known to the device alone
      const double total = (np * lp + nt * (fix + 0.5 * (lt - fix))) / pairs;
      const double t = std::max({waves * lp, total + (st ? 0.5 * lt : 0.0), lt}) + (sp + st > 1 ? join * (sp + st) + 3.0 : 0.0);
      if (t < best) {
        best = t;
        p.sp = sp;
        p.st = st;
      }
      if (!st) break;
    }
    if (!p.tiles_p) break;
  }
  p.rows_kv = static_cast<int64_t>(p.tiles_p) * kTile + static_cast<int64_t>(n_seq) * p.tiles_t * kTile;
  const size_t parts = p.sp + p.st > 1 ? static_cast<size_t>(n_q) * h_s * (p.sp + p.st) : 0;
  p.off_words = round_up(static_cast<size_t>(p.rows_kv) * kLatent * 2, 256);
  p.off_o = p.off_words + round_up(static_cast<size_t>(p.rows_kv / kTile) * 16, 256);
  p.off_ml = p.off_o + parts * kVDim * 2;
  p.bytes = p.off_ml + round_up(parts * 16, 256);
  return p;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float exp2_approx(float x) {  // relative error ~2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Positions row t sees: 0 for a row whose sequence or length is out of range (flagged).
__device__ __forceinline__ int row_limit(const PrefixArgs& a, int t, bool report) {
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
  const int pos = a.q_pos[t];
  return pos < 0 ? 0 : min(pos, len - 1) + 1;
}

// ---- expand: one block per 64-position tile ------------------------------------------------
// Bound by memory: 608 bytes read and 1152 written a position.
constexpr int kExpandThreads = 288;
constexpr int kChunks = kLatent / 16;  // 16-code chunks of a record
__global__ void __launch_bounds__(kExpandThreads)
expand_kernel(PrefixArgs a, PrefixPlan pl, PrefixWs ws) {
  __shared__ unsigned s_word[4];  // valid (2 words), poisonous (2 words)
  pdl_launch_dependents();
  pdl_wait();
  const int tile = blockIdx.x;
  const int tid = threadIdx.x;
  int pos0, len;
  const int32_t* pages;
  if (tile < pl.tiles_p) {
    pos0 = tile * kTile;
    len = a.prefix_len;
    pages = a.prefix_pages;
  } else {
    const int b = (tile - pl.tiles_p) / pl.tiles_t;
    pos0 = a.prefix_len + (tile - pl.tiles_p) % pl.tiles_t * kTile;
    len = a.seq_lens[b];
    if (len < 0 || len > a.max_ctx) len = 0;
    if (pos0 >= len) return;
    pages = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  }
  if (tid < 4) s_word[tid] = 0;
  __syncthreads();
  constexpr int kPer = kTile * kChunks / kExpandThreads;  // 8
  static_assert(kTile * kChunks % kExpandThreads == 0, "chunks per thread");
  uint4 code[kPer];
  float scale[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int w = i * kExpandThreads + tid, tok = w / kChunks, c = w - tok * kChunks;
    const int p = pos0 + tok;
    code[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    if (p >= len) continue;
    const int pg = pages[p / kPage];
    if (pg < 0 || pg >= a.num_pages) {
      if (c == 0) flag(a.status, DSA_STATUS_BAD_PAGE);
      continue;
    }
    const uint8_t* rec = a.kv_cache + (static_cast<int64_t>(pg) * kPage + p % kPage) * kKvTokBytes;
    code[i] = *reinterpret_cast<const uint4*>(rec + 16 * c);
    scale[i] = *reinterpret_cast<const float*>(rec + kKvScaleOff + 4 * (c >> 3));
    if (c == 0) atomicOr(&s_word[tok >> 5], 1u << (tok & 31));
  }
  uint4 lo[kPer], hi[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int tok = (i * kExpandThreads + tid) / kChunks;
    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
    uint32_t o[8];
    bool bad = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[4];
      e4m3x4_to_f32(w[q], f);
      o[2 * q] = pack2(f[0] * scale[i], f[1] * scale[i]);
      o[2 * q + 1] = pack2(f[2] * scale[i], f[3] * scale[i]);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)  // an exponent of all ones in either half: infinite or NaN
      bad |= (o[q] & 0x7F80u) == 0x7F80u || (o[q] & 0x7F800000u) == 0x7F800000u;
    if (bad) atomicOr(&s_word[2 + (tok >> 5)], 1u << (tok & 31));
    lo[i] = make_uint4(o[0], o[1], o[2], o[3]);
    hi[i] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  __syncthreads();
  __nv_bfloat16* dst = ws.kv + static_cast<int64_t>(tile) * kTile * kLatent;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int w = i * kExpandThreads + tid, tok = w / kChunks;
    if ((s_word[2 + (tok >> 5)] >> (tok & 31)) & 1u) lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
    uint4* out = reinterpret_cast<uint4*>(dst + static_cast<int64_t>(w) * 16);
    out[0] = lo[i];
    out[1] = hi[i];
  }
  if (tid < 4) reinterpret_cast<unsigned*>(ws.words + 2 * static_cast<int64_t>(tile))[tid] = s_word[tid];
}

// ---- attend ----------------------------------------------------------------------------------
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      :: "r"(d), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      :: "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
// arrive on a barrier once the MMAs this warp's elected lane issued have completed: of this
// CTA, or (multicast) of the CTAs in the mask
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void commit_elected_to(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}"
      :: "r"(smem_u32(bar)), "h"(mask) : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
         "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
         "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// shared memory of this CTA -> the peer's, counted on the peer's barrier
__device__ __forceinline__ void bulk_to_peer(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "r"(smem_u32(src)), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void st_async_f32(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
               :: "r"(addr), "r"(__float_as_uint(v)), "r"(bar) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap, PrefixArgs a,
              PrefixPlan pl, PrefixWs ws) {
  extern __shared__ __align__(1024) uint8_t smem[];
  PairCtl& ctl = *reinterpret_cast<PairCtl*>(smem + kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = static_cast<int>(cluster_ctarank()), peer = c ^ 1;
  pdl_launch_dependents();
  pdl_wait();

  // ---- this pair's item: rows row0 .. of the flattened (query row, head), tiles tile0 .. ----
  const int item = blockIdx.x >> 1;
  const int n_prefix = pl.sp * pl.mt;
  const bool tail = item >= n_prefix;
  const int64_t rows_all = static_cast<int64_t>(a.n_q) * a.h_s;
  const int ns = pl.sp + pl.st;
  int64_t row0;
  int n_rows, part, split, tiles, tile_base, first_pos;
  if (!tail) {
    split = item / pl.mt;
    row0 = static_cast<int64_t>(item - split * pl.mt) * kRows;
    n_rows = static_cast<int>(min(static_cast<int64_t>(kRows), rows_all - row0));
    part = pl.sp;
    tiles = pl.tiles_p;
    tile_base = 0;
    first_pos = 0;
  } else {
    const int k = item - n_prefix;
    split = k / a.n_q;
    const int t = k - split * a.n_q;
    row0 = static_cast<int64_t>(t) * a.h_s;
    n_rows = a.h_s;
    part = pl.st;
    const int lim = row_limit(a, t, tid == 0 && c == 0 && split == 0);
    tiles = lim > a.prefix_len ? (lim - a.prefix_len + kTile - 1) / kTile : 0;
    // (a row that sees anything has a sequence in range)
    tile_base = tiles ? pl.tiles_p + a.q_seq[t] * pl.tiles_t : 0;
    first_pos = a.prefix_len;
  }
  const int tile0 = static_cast<int>(static_cast<int64_t>(split) * tiles / part);
  const int nt = static_cast<int>(static_cast<int64_t>(split + 1) * tiles / part) - tile0;
  const int slot = tail ? pl.sp + split : split;
  if (nt == 0) {  // both CTAs alike: nothing of this row lies in this split
    if (c == 0 && ns > 1) {
      for (int m = tid; m < n_rows; m += kThreads)
        ws.ml[(row0 + m) * ns + slot] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    } else if (ns == 1) {
      for (int i = tid; i < n_rows * (kHalfV / 8); i += kThreads)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (row0 + i / (kHalfV / 8)) * kVDim + kHalfV * c +
                                  8 * (i % (kHalfV / 8))) = make_uint4(0u, 0u, 0u, 0u);
      if (c == 0 && a.out_lse)
        for (int m = tid; m < n_rows; m += kThreads) a.out_lse[row0 + m] = -INFINITY;
    }
    return;
  }
  const int n_own = (nt - c + 1) / 2, n_peer = nt - n_own;  // own tile i: 2 i + c; peer tile i: 2 i + peer

  const bool aligned = (smem_u32(smem) & 1023u) == 0;  // the same in both CTAs
  if (!aligned) {
    if (tid == 0) flag(a.status, DSA_STATUS_INTERNAL);
    return;
  }
  if (tid == 0) {
    ctl.abort = 0;
    ctl.redo = 0;
    tc::mbar_init(&ctl.q_full, 1);
    tc::mbar_init(&ctl.q_tmem, 4);
    for (int k = 0; k < kRing; ++k) {
      tc::mbar_init(&ctl.ring_full[k], 1);
      tc::mbar_init(&ctl.ring_empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(&ctl.vown_full[k], 1);
      tc::mbar_init(&ctl.vown_empty[k], 1);
    }
    tc::mbar_init(&ctl.vpeer_full, 1);
    tc::mbar_init(&ctl.vpeer_empty, 1);
    tc::mbar_init(&ctl.s_full, 1);
    tc::mbar_init(&ctl.s_free, 4);
    tc::mbar_init(&ctl.p_full, 4);
    tc::mbar_init(&ctl.p_empty, 2);
    tc::mbar_init(&ctl.pin_full, 1);
    tc::mbar_init(&ctl.o_done, 1);
    tc::mbar_init(&ctl.r_full, 1);
    tc::mbar_init(&ctl.fin_full, 1);
    tc::mbar_fence_init();
    // what the peer will send
    if (c == 1) tc::mbar_arrive_expect_tx(&ctl.r_full, kRows * 4);
    tc::mbar_arrive_expect_tx(&ctl.fin_full, kRows * 12);
    tc::mbar_arrive_expect_tx(&ctl.pin_full, kPBytes);
  }
  if (warp == 1) tc::tmem_alloc(&ctl.tmem_base, 512);
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers are ready
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort = &ctl.abort;
  // (bounded) wait of one thread, and of a converged warp: there the lanes agree on the outcome
  auto wait = [&](uint64_t* bar, uint32_t parity) { return tc::mbar_wait(bar, parity & 1u, abort, a.status); };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = wait(bar, parity);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  // softmax threads: their row's state, kept from the loop to the output
  float r = 0.f, l = 0.f, lx = 0.f;
  // steps done in earlier attempts, by role (barrier phases run on)
  int g_own = 0, g_peer = 0;
  bool gave_up = false;  // a wait ran out, here or in the peer
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (warp == 0) {
      // ---------------- own tiles: the half of the value blocks this CTA keeps, then the rest ----------------
      if (lane == 0) {
        if (attempt == 0) {
          tc::prefetch_tmap(&qmap);
          tc::prefetch_tmap(&kvmap);
          tc::mbar_arrive_expect_tx(&ctl.q_full, kQSmemBlocks * kQBlock);
          for (int kb = 0; kb < kQSmemBlocks; ++kb)
            tc::tma_load_3d(smem + kOffQ + kb * kQBlock, &qmap, kQTmemSteps * 16 + 64 * kb, static_cast<int>(row0), 0,
                            &ctl.q_full);
        }
        for (int i = 0; i < n_own; ++i) {
          const int g = g_own + i, b = g & 1;
          const int y = (tile_base + tile0 + 2 * i + c) * kTile;
          if (!wait(&ctl.vown_empty[b], (g >> 1) + 1)) break;
          tc::mbar_arrive_expect_tx(&ctl.vown_full[b], 4 * kBlock);
          for (int k = 0; k < 4; ++k)
            tc::tma_load_3d(smem + kOffVOwn + (4 * b + k) * kBlock, &kvmap, 64 * (4 * c + k), y, 0, &ctl.vown_full[b]);
          bool ok = true;
          for (int k = 0; k < kLoose && ok; ++k) {
            const int n = kLoose * g + k, slot_k = n % kRing;
            ok = wait(&ctl.ring_empty[slot_k], n / kRing + 1);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(&ctl.ring_full[slot_k], kBlock);
            tc::tma_load_3d(smem + kOffRing + slot_k * kBlock, &kvmap, 64 * (k < 4 ? 4 * peer + k : 8), y, 0,
                            &ctl.ring_full[slot_k]);
          }
          if (!ok) break;
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      // ---------------- the peer's tiles: this CTA's value blocks ----------------
      if (lane == 0) {
        for (int i = 0; i < n_peer; ++i) {
          const int g = g_peer + i;
          const int y = (tile_base + tile0 + 2 * i + peer) * kTile;
          if (!wait(&ctl.vpeer_empty, g + 1)) break;
          tc::mbar_arrive_expect_tx(&ctl.vpeer_full, 4 * kBlock);
          for (int k = 0; k < 4; ++k)
            tc::tma_load_3d(smem + kOffVPeer + k * kBlock, &kvmap, 64 * (4 * c + k), y, 0, &ctl.vpeer_full);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- Q K^T ----------------
      const uint32_t id = tc::idesc_bf16(kTile, false, false);
      const uint64_t qd = tc::desc_kmajor_sw128(smem_u32(smem + kOffQ));
      const uint32_t d = tmem + kColS;
      bool ok = wait_warp(&ctl.q_full, 0) && wait_warp(&ctl.q_tmem, 0);
      // the four K-steps of 64-dim block kb
      auto block = [&](int kb, uint64_t kd, bool first) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if (kb < kQTmemSteps / 4)
            mma_ts(d, tmem + kColQ + 32 * kb + 8 * s, kd + 2 * s, id, !(first && s == 0));
          else
            mma_ss(d, qd + (kb - kQTmemSteps / 4) * (kQBlock >> 4) + 2 * s, kd + 2 * s, id, !(first && s == 0));
        }
      };
      for (int i = 0; i < n_own && ok; ++i) {
        const int g = g_own + i, b = g & 1;
        ok = wait_warp(&ctl.s_free, g + 1) && wait_warp(&ctl.vown_full[b], g >> 1);
        if (!ok) break;
        __syncwarp();
        tc::fence_after_sync();
        const uint64_t vd = tc::desc_kmajor_sw128(smem_u32(smem + kOffVOwn + 4 * b * kBlock));
#pragma unroll
        for (int k = 0; k < 4; ++k) block(4 * c + k, vd + k * (kBlock >> 4), k == 0);
        for (int k = 0; k < kLoose; ++k) {
          const int n = kLoose * g + k, slot_k = n % kRing;
          ok = wait_warp(&ctl.ring_full[slot_k], n / kRing);
          if (!ok) break;
          __syncwarp();
          tc::fence_after_sync();
          block(k < 4 ? 4 * peer + k : 8, tc::desc_kmajor_sw128(smem_u32(smem + kOffRing + slot_k * kBlock)), false);
          commit_elected(&ctl.ring_empty[slot_k]);
        }
        commit_elected(&ctl.s_full);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- P V: this CTA's value half, over own and peer tiles in turn ----------------
      const uint32_t id = tc::idesc_bf16(kHalfV, false, true);
      bool any = false, ok = true;
      auto pv = [&](uint32_t off_p, uint32_t off_v) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {  // 16 positions a step
          const uint64_t pd = tc::desc_kmajor_sw128(smem_u32(smem + off_p)) + 2 * s;
          const uint64_t vd = tc::smem_desc(smem_u32(smem + off_v) + s * 2048, kBlock, 1024, 2);
          mma_ss(tmem + kColO, pd, vd, id, any || s > 0);
        }
        any = true;
      };
      for (int i = 0; i < n_own || i < n_peer; ++i) {
        if (i < n_own) {
          const int g = g_own + i;
          ok = wait_warp(&ctl.p_full, g);
          if (!ok) break;
          __syncwarp();
          tc::fence_after_sync();
          pv(kOffPOwn, kOffVOwn + 4 * (g & 1) * kBlock);
          commit_elected(&ctl.vown_empty[g & 1]);
          commit_elected(&ctl.p_empty);
        }
        if (i < n_peer) {
          const int g = g_peer + i;
          ok = wait_warp(&ctl.pin_full, g);
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(&ctl.pin_full, kPBytes);  // the next weights
          ok = wait_warp(&ctl.vpeer_full, g);
          if (!ok) break;
          __syncwarp();
          tc::fence_after_sync();
          pv(kOffPIn, kOffVPeer);
          commit_elected(&ctl.vpeer_empty);
          commit_elected_to(&ctl.p_empty, static_cast<uint16_t>(1u << peer));
        }
      }
      commit_elected(&ctl.o_done);
      __syncwarp();
    } else if (warp == 3) {
      // ---------------- own weights to the peer ----------------
      if (lane == 0) {
        const uint32_t dst = dsmem_addr(smem + kOffPIn, peer), bar = dsmem_addr(&ctl.pin_full, peer);
        for (int i = 0; i < n_own; ++i) {
          // (the warps that wrote them waited until the peer had read the last ones)
          if (!wait(&ctl.p_full, g_own + i)) break;
          bulk_to_peer(dst, smem + kOffPOwn, kPBytes, bar);
        }
      }
      __syncwarp();
    } else {
      // ---------------- logits -> weights, one row a thread (warps 4..7) ----------------
      const int quarter = warp & 3, m = quarter * 32 + lane;
      const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
      const bool live = m < n_rows;
      if (attempt == 0) {  // the query's first 384 dims into tensor memory
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (row0 + m) * kLatent);
#pragma unroll
        for (int h = 0; h < 6; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (live) u = __ldg(src + 8 * h + i);
            v[4 * i] = u.x; v[4 * i + 1] = u.y; v[4 * i + 2] = u.z; v[4 * i + 3] = u.w;
          }
          tmem_store32(tmem + lane_base + kColQ + 32 * h, v);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.q_tmem);
      }
      // positions of this part the row sees
      int lim = 0;
      if (live) {
        lim = row_limit(a, static_cast<int>((row0 + m) / a.h_s), !tail && split == 0 && c == 0) - first_pos;
        if (!tail) lim = min(lim, a.prefix_len);
      }
      const float c2 = a.sm_scale * 1.4426950408889634f;  // logits in powers of two
      float top = -INFINITY;
      l = lx = 0.f;
      if (attempt == 0 && c == 1) {
        wait_warp(&ctl.r_full, 0);
        r = ctl.r[m];
      }
      for (int i = 0; i < n_own; ++i) {
        const int g = g_own + i, tile = tile0 + 2 * i + c;
        const ulonglong2 w = __ldcg(reinterpret_cast<const ulonglong2*>(ws.words) + tile_base + tile);
        const int nv = lim - tile * kTile;
        const uint64_t seen = w.x & (nv >= kTile ? ~0ull : nv <= 0 ? 0ull : (1ull << nv) - 1ull);
        if (!wait_warp(&ctl.s_full, g)) break;
        tc::fence_after_sync();
        uint32_t s0[32], s1[32];
        tc::tmem_ld32(tmem + lane_base + kColS, s0);
        tc::tmem_ld32(tmem + lane_base + kColS + 32, s1);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.s_free);
        if (!__all_sync(0xffffffffu, seen == ~0ull && w.y == 0)) {
          const uint32_t inf = 0xFF800000u, nan = 0x7FFFFFFFu;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if ((w.y >> k) & 1u) s0[k] = nan;
            if ((w.y >> (32 + k)) & 1u) s1[k] = nan;
            if (!((seen >> k) & 1u)) s0[k] = inf;
            if (!((seen >> (32 + k)) & 1u)) s1[k] = inf;
          }
        }
        float mt = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; ++k) mt = fmaxf(mt, fmaxf(__uint_as_float(s0[k]), __uint_as_float(s1[k])));
        mt *= c2;
        top = fmaxf(top, mt);
        if (attempt == 0 && c == 0 && i == 0) {
          r = mt == -INFINITY ? 0.f : mt;  // nothing seen in the first tile: any guess
          st_async_f32(dsmem_addr(&ctl.r[m], 1), r, dsmem_addr(&ctl.r_full, 1));
        }
        // weights, rounded to the bf16 that the tensor cores read; l sums the rounded ones (it
        // normalises O), lx the unrounded ones (it gives the log-sum-exp)
        uint32_t p[32];
        float la = 0.f, lb = 0.f, xa = 0.f, xb = 0.f;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float a0 = exp2_approx(fmaf(__uint_as_float(s0[k]), c2, -r));
          const float a1 = exp2_approx(fmaf(__uint_as_float(s0[k + 1]), c2, -r));
          const float b0 = exp2_approx(fmaf(__uint_as_float(s1[k]), c2, -r));
          const float b1 = exp2_approx(fmaf(__uint_as_float(s1[k + 1]), c2, -r));
          p[k >> 1] = pack2(a0, a1);
          p[16 + (k >> 1)] = pack2(b0, b1);
          xa += a0 + a1;
          xb += b0 + b1;
          la += __uint_as_float(p[k >> 1] << 16) + __uint_as_float(p[k >> 1] & 0xFFFF0000u);
          lb += __uint_as_float(p[16 + (k >> 1)] << 16) + __uint_as_float(p[16 + (k >> 1)] & 0xFFFF0000u);
        }
        l += la + lb;
        lx += xa + xb;
        if (!wait_warp(&ctl.p_empty, g + 1)) break;
        uint8_t* row = smem + kOffPOwn + m * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(row + ((k ^ (m & 7)) << 4)) = make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.p_full);
      }
      // the last weights have been read, here and by the peer (whose word of it has then arrived)
      if (n_own > 0) wait_warp(&ctl.p_empty, g_own + n_own - 1);
      // ---- both CTAs' maxima and sums ----
      {
        const uint32_t bar = dsmem_addr(&ctl.fin_full, peer);
        dsmem_st_async_v2(dsmem_addr(&ctl.fin2[m], peer), make_uint2(__float_as_uint(top), __float_as_uint(l)), bar);
        st_async_f32(dsmem_addr(&ctl.fin1[m], peer), lx, bar);
      }
      if (wait_warp(&ctl.fin_full, attempt)) {
        const float2 f2 = ctl.fin2[m];
        const float f1 = ctl.fin1[m];
        top = fmaxf(top, f2.x);
        l = c == 0 ? l + f2.y : f2.y + l;  // the same order in both CTAs
        lx = c == 0 ? lx + f1 : f1 + lx;
      }
      const bool far = live && top != -INFINITY && fabsf(top - r) > kRange;
      if (attempt == 0 && far) atomicOr(&ctl.redo, 1);
      if (attempt == 0) {
        // (a second phase is expected only if there is a second attempt)
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (ctl.redo) {
          if (tid == 4 * 32) tc::mbar_arrive_expect_tx(&ctl.fin_full, kRows * 12);
          r = top == -INFINITY ? 0.f : top;
        }
      }
    }
    // every product of this attempt is complete, and nothing the peer sent is still on its way
    wait(&ctl.o_done, attempt);
    __syncthreads();
    if (tid == 0) dsmem_st_u32(dsmem_addr(const_cast<uint32_t*>(&ctl.peer_vote[attempt]), peer), (*abort ? 2u : 0u) | (ctl.redo ? 1u : 0u));
    __syncwarp();
    cluster_sync();
    gave_up = *abort || (ctl.peer_vote[attempt] & 2u);
    if (attempt == 1 || gave_up || !(ctl.redo && (ctl.peer_vote[0] & 1u))) break;
    g_own += n_own;
    g_peer += n_peer;
  }
  tc::fence_after_sync();

  // ---- output: O / l as bf16, through the tiles' shared memory, in whole rows ----
  uint8_t* stage = smem + kOffVOwn;
  if (warp >= 4 && warp < 8) {
    const int m = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    uint8_t* row = stage + m * kStagePitch;
#pragma unroll
    for (int col = 0; col < kHalfV; col += 32) {
      uint32_t v[32];
      tc::tmem_ld32(tmem + lane_base + kColO + col, v);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        *reinterpret_cast<uint4*>(row + 2 * (col + i)) =
            make_uint4(pack2(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv),
                       pack2(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv),
                       pack2(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv),
                       pack2(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv));
    }
    if (c == 0 && m < n_rows) {
      if (ns == 1) {
        if (a.out_lse)
          a.out_lse[row0 + m] = lx > 0.f || lx != lx ? (r + log2f(lx)) * 0.6931471805599453f : -INFINITY;
      } else {
        // the sum's own exponent joins the reference, so that the merge compares true sizes
        const int e = l > 0.f && l < INFINITY ? static_cast<int>(__float_as_uint(l) >> 23) - 127 : 0;
        const float f = exp2i(-e);
        ws.ml[(row0 + m) * ns + slot] =
            l == 0.f ? make_float4(-INFINITY, 0.f, 0.f, 0.f) : make_float4(r + static_cast<float>(e), l * f, lx * f, 0.f);
      }
    }
  }
  __syncthreads();
  {
    const int piece = tid & 31;
    for (int m = tid >> 5; m < n_rows; m += kThreads / 32) {
      __nv_bfloat16* dst = ns == 1 ? static_cast<__nv_bfloat16*>(a.out) + (row0 + m) * kVDim
                                   : ws.o + ((row0 + m) * ns + slot) * kVDim;
      *reinterpret_cast<uint4*>(dst + kHalfV * c + 8 * piece) =
          *reinterpret_cast<const uint4*>(stage + m * kStagePitch + 16 * piece);
    }
  }
  // after a wait that ran out, copies and products may still be in flight: give them time to
  // land before shared and tensor memory are given back
  if (gave_up) {
    const uint64_t t0 = tc::global_ns();
    while (tc::global_ns() - t0 < 100000ull) {
    }
    cluster_sync();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// ---- merge ---------------------------------------------------------------------------------
// Split s holds O_s / l_s with reference m_s; with M = max m_s and w_s = 2^(m_s - M) l_s the
// output is sum_s w_s (O_s / l_s) / sum_s w_s.  64 threads a row, 8 columns each, four
// rows a block, four splits' loads in flight.
constexpr int kMergeRows = 4, kMergeBatch = 4;
__global__ void __launch_bounds__(64 * kMergeRows)
prefix_merge_kernel(PrefixArgs a, PrefixPlan pl, PrefixWs ws) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 6);
  if (row >= static_cast<int64_t>(a.n_q) * a.h_s) return;
  const int d = 8 * static_cast<int>(threadIdx.x & 63);
  const int ns = pl.sp + pl.st;
  float M = -INFINITY, sum = 0.f, sum_x = 0.f, acc[8] = {};
  for (int s0 = 0; s0 < ns; s0 += kMergeBatch) {
    float4 ml[kMergeBatch];
    uint4 v[kMergeBatch];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      ml[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (s0 + i < ns) {
        ml[i] = __ldcg(ws.ml + row * ns + s0 + i);
        v[i] = __ldcg(reinterpret_cast<const uint4*>(ws.o + (row * ns + s0 + i) * kVDim + d));
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) top = fmaxf(top, ml[i].x);
    if (top != M) {
      const float f = M == -INFINITY ? 0.f : exp2f(M - top);
      sum *= f;
      sum_x *= f;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] *= f;
      M = top;
    }
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      if (ml[i].x == -INFINITY) continue;  // an empty split: its output was never written
      const float w = exp2f(ml[i].x - M), wl = w * ml[i].y;
      sum += wl;
      sum_x += w * ml[i].z;
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[2 * k] += wl * __uint_as_float(u[k] << 16);
        acc[2 * k + 1] += wl * __uint_as_float(u[k] & 0xFFFF0000u);
      }
    }
  }
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * kVDim + d) =
      make_uint4(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv),
                 pack2(acc[4] * inv, acc[5] * inv), pack2(acc[6] * inv, acc[7] * inv));
  if (a.out_lse && d == 0)
    a.out_lse[row] = sum_x > 0.f || sum_x != sum_x ? (M + log2f(sum_x)) * 0.6931471805599453f : -INFINITY;
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
// rows of 576 bf16 in boxes of 64 dims x box_rows, 128-byte swizzle; rows past the end read 0
bool encode_rows(EncodeFn enc, CUtensorMap* map, const void* base, int64_t rows, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kLatent), static_cast<cuuint64_t>(rows), 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kLatent) * 2,
                                 static_cast<cuuint64_t>(kLatent) * 2 * static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  DevInfo di;
  const char* why = nullptr;
  return device_info(&di, &why) ? di.n_sm : 152;
}

}  // namespace

size_t prefix_workspace_bytes(int n_q, int h_s, int n_seq, int prefix_len, int max_ctx) {
  return make_plan(n_q, h_s, n_seq, prefix_len, max_ctx, sm_count()).bytes;
}

cudaError_t launch_prefix_attn(const PrefixArgs& a, cudaStream_t s, const char** err) {
  const PrefixPlan pl = make_plan(a.n_q, a.h_s, a.n_seq, a.prefix_len, a.max_ctx, sm_count());
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  PrefixWs ws{reinterpret_cast<__nv_bfloat16*>(base), reinterpret_cast<uint64_t*>(base + pl.off_words),
              reinterpret_cast<__nv_bfloat16*>(base + pl.off_o), reinterpret_cast<float4*>(base + pl.off_ml)};
  const int64_t rows = static_cast<int64_t>(a.n_q) * a.h_s;
  const int64_t items = static_cast<int64_t>(pl.sp) * pl.mt + static_cast<int64_t>(pl.st) * a.n_q;
  if (pl.rows_kv > INT32_MAX - kTile || rows > INT32_MAX - kRows || items > INT32_MAX / 2) {
    *err = "prefix_attn: more rows than 32 bits count";
    return cudaErrorInvalidValue;
  }
  const EncodeFn enc = encode_fn();
  if (!enc) {
    *err = "prefix_attn: cuTensorMapEncodeTiled is not available";
    return cudaErrorNotSupported;
  }
  CUtensorMap qmap, kvmap;
  if (!encode_rows(enc, &qmap, a.q, rows, kRows) || !encode_rows(enc, &kvmap, ws.kv, pl.rows_kv, kTile)) {
    *err = "prefix_attn: tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  e = launch_pdl(expand_kernel, dim3(static_cast<unsigned>(pl.rows_kv / kTile)), dim3(kExpandThreads), 0, s, 1, a, pl, ws);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attend_kernel, dim3(static_cast<unsigned>(2 * items)), dim3(kThreads), kSmemBytes, s, 2, qmap, kvmap, a,
                 pl, ws);
  if (e != cudaSuccess || pl.sp + pl.st == 1) return e;
  return launch_pdl(prefix_merge_kernel, dim3(static_cast<unsigned>((rows + kMergeRows - 1) / kMergeRows)),
                    dim3(64 * kMergeRows), 0, s, 1, a, pl, ws);
}

}  // namespace dsa
