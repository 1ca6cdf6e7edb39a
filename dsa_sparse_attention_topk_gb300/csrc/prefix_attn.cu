// Attention of a batch whose sequences share a long prefix, on the 5th-generation tensor
// cores: dense absorbed-MLA attention over the paged FP8 latent cache.
//
// Query row t of sequence b sees the positions p < n_t = min(q_pos[t] + 1, seq_lens[b]):
// those below prefix_len from the shared pages, the rest (its tail) from its own page-table
// row.  With kv[p] the dequantised latent row,
//     l_p = sm_scale * q[t, h] . kv[p],  o[t, h] = sum_p softmax(l)_p kv[p][0:512].
// The work is 2 (576 + 512) flop per (row, head, position) against 596 bytes per position:
// with 128 heads or more per position (rows of several sequences, for the prefix) it is
// bound by the tensor cores; with up to 32 heads a path of its own (prefix_few.cu) may take the
// tails, or everything, straight from the cache: make_plan chooses.
//
// Three kernels.
//   expand   dequantises the prefix once for all rows, and each tail once, into fp16 rows in
//            the workspace, so that the main kernel can feed its MMAs by TMA alone.  A tile of 64
//            positions shares one power of two, taken from its largest scale, which keeps fp16's
//            11 bits for everything within 2^-29 of the tile's largest value; bf16 operands
//            would cost three more bits, in the logits above all.  A position whose page
//            is out of range becomes a zero row that a bit marks invalid; one with NaN or
//            infinite values a zero row marked poisonous, whose logit is NaN for the rows
//            that see it and nothing to the others.
//   attend   one CTA pair per item: 128 rows of (query row, head) against a run of 64-position
//            tiles of the prefix (a tile of the flattened rows, shared by all sequences) or of
//            one sequence's tail (as many of its adjacent query rows as fit).
//   merge    joins a row's splits by their log-sum-exps.
//
// The pair.  The output accumulator of 128 rows x 512 columns would fill tensor memory, so
// each CTA of the pair holds one half of the value columns.  Computing the logits in both
// would cost half as much again; instead CTA c computes logits and weights of the tiles
// j = c (mod 2), stores the weights (fp16, 16 KB) in its own shared memory and copies them to its
// peer's (one bulk copy a tile); both then run P V over every tile, each on its half, in the
// order own 0, peer 0, own 1, peer 1 ...
//
// The softmax reference.  With e the exponent of its tile, a position's weight is stored as
// 2^(x + e - rho), x its logit in powers of two and rho the row's reference.  fp16 has room for
// weights up to 2^15 and 11 bits down to 2^-14, so rho goes by the level that the first tile's
// positions share, not by its largest alone: the lowest of four maxima of 16, plus 2, but at least
// 3 and at most 14 below the largest of all.  A position far above the rest (an attention
// sink, often with next to nothing in its value) then keeps 2^14 and leaves the others their bits;
// without one, later tiles may grow by 12 powers of two before rho changes.  CTA 0 sends the first
// rho to CTA 1; the sum of 2^(x - rho) is kept in fp32 from the unrounded weights, in units of
// 2^-e of the item's first tile (in units of 1, values of 2^-106 would take it past 2^127).  A tile of
// zeros may have any exponent and takes that one too, so that it sets no reference far from the
// others' weights.  Where a tile's largest weight would pass 2^15 its owner raises rho, to 5 below
// the largest behind the first tile, for all rows of the warp that this would raise (waiting for
// the products is the cost, and the rows share it), and rescales its accumulator; the references
// travel with the weights, and the receiving CTA raises its own (rescaling its accumulator) or,
// where it has itself gone ahead, scales the received row down.  After each tile in the order
// above both CTAs hold the largest reference used so far, so the results do not depend on timing.
// Measured, 32 rows behind 32K, logits of a spread of 2.5, 4, 6 and 10 powers of two: 202, 204, 216
// and 240 us; raising single rows 238 at a spread of 6; 11 below instead of 5: 259 there, 0: 209;
// rho 10 below the first largest whatever its tile looks like: 288 at 2.5.
//
// MMA pairs.  Where there are rows enough, four CTAs share an item of 256 rows: two per parity,
// whose tensor cores work as one (cta_group::2) on 128 rows each, every B operand split between
// their shared memories.  With one CTA per parity an SM moves some 370 KB through its shared
// memory in a step of two tiles (operand reads, tile loads, weights), more than its 128 bytes a
// cycle allow in the 2270 cycles of the products; with pairs it is 260 KB.
//
// Per CTA (13 warps): 0 loads the tiles for Q K^T, 3 the others, 1 issues Q K^T, 2 issues P V,
// 4-11 turn logits into weights (a row's 64 positions in two threads), 12 copies the weights.
// Descriptors and tensor-memory addresses are constants of the unrolled issue loops.
// Tensor memory (512 columns): O in 0..255, the logits in 256..319, the query's dims 0..383
// as fp16 pairs in 320..511; shared memory as in Layout below.
// The query is scaled to fp16 by a power of two per row (exact: bf16 has 8 bits).
//
// Measured (128 heads): 32 rows behind 32K positions 202 us, of it 8 us expand, some 11 us before an
// item's first and behind its last product, and 2400 cycles a step of two tiles against
// the products' 2270; 512 causal rows behind 16K 1.50 ms, 82% of the cuBLAS bf16 rate.

#include <algorithm>
#include <cuda.h>

#include "prefix_common.cuh"
#include "tc_utils.cuh"

namespace dsa {
namespace {

constexpr int kTile = 64;                     // positions per tile
constexpr int kRows = 128;                    // (query row, head) rows per item
constexpr int kHalfV = kVDim / 2;
constexpr int kBlock = kTile * 128;           // 64 positions x 64 dims, fp16: 8 KB
constexpr int kQBlock = kRows * 128;          // 128 rows x 64 dims: 16 KB
constexpr int kQTmemBlocks = 6;               // 64-dim blocks with the query in tensor memory
constexpr int kQSmemBlocks = 3;
constexpr int kLoose = 5;                     // blocks of a tile that only Q K^T reads
constexpr int kThreads = 32 * 13;
constexpr int kSoftWarps = 8;                 // warps 4..11
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;
constexpr uint32_t kPBytes = kRows * 128;     // the weights of a tile
constexpr uint32_t kPMsg = kPBytes + kRows * 4;  // with the rows' references
constexpr uint32_t kPStride = (kPMsg + 1023) / 1024 * 1024;
// Powers of two: what a weight may reach before its row's reference is raised (2^16 is too large for
// fp16); the first tile's largest weight at most and at least, and its reference's height above the
// lowest of four maxima in between; the largest weight behind a raise.
constexpr float kHeadroom = 15.0f, kMost = 14.0f, kLeast = 3.0f, kAbove = 2.0f, kRaised = 5.0f;

// Shared memory behind the query's part: own weights, the peer's weights, value tiles, tiles for
// Q K^T.  Loads and copies between CTAs take some 2000 cycles, nearly a step of two tiles, so
// what crosses has buffers to spare.  G = 1: the value blocks (64 positions x 64 dims) of two own
// tiles (slots 0, 1; Q K^T reads them too) and one peer tile (slot 2), and the own tile's other
// five blocks.  G = 2: each CTA of an MMA pair holds half of every B operand: 64 positions x 128
// dims of own and peer tiles in turn (a ring of three slots), and 32 positions of tiles for Q K^T
// (a ring of five pieces of 192 dims, three pieces a tile); two buffers each way for the weights.
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffP = kOffQ + kQSmemBlocks * kQBlock;
constexpr int kPiece = 3 * kBlock / 2, kPieces = 5;  // G = 2: 32 positions x 192 dims, ring slots
template <int G> struct Layout {
  static constexpr int kVBytes = 4 * kBlock / G, kVSlots = 3, kBufs = G;
  static constexpr uint32_t p_own = kOffP, p_in = p_own + kBufs * kPStride, v = p_in + kBufs * kPStride;
  static constexpr uint32_t k = v + kVSlots * kVBytes, ctl = k + (G == 1 ? kLoose * kBlock : kPieces * kPiece);
  // the query's 64-dim blocks: dims 0..383 staged where the first tiles for Q K^T do not go, so that
  // these load meanwhile (G = 1: value slot 0; G = 2: pieces 0..2)
  static __host__ __device__ constexpr uint32_t q_block(int kb) {
    return kb >= kQTmemBlocks ? kOffQ + (kb - kQTmemBlocks) * kQBlock
           : G == 1           ? (kb < 4 ? v + kVBytes + kb * kQBlock : kb == 4 ? p_own : k)
                              : (kb < 3 ? v + kb * kQBlock : kb < 5 ? p_own + (kb - 3) * kPStride : k + 3 * kPiece);
  }
  // slot of a tile's values and how often the slot was filled before: own tile i is product 2 i, peer
  // tile i follows it (or, where there is none, the last one)
  static __host__ __device__ constexpr int own_slot(int i) { return G == 1 ? i % 2 : 2 * i % 3; }
  static __host__ __device__ constexpr int own_phase(int i) { return G == 1 ? i / 2 : 2 * i / 3; }
  static __host__ __device__ constexpr int peer_slot(int i, int n_own) {
    return G == 1 ? 2 : (i + (i < n_own ? i + 1 : n_own)) % 3;
  }
  static __host__ __device__ constexpr int peer_phase(int i, int n_own) {
    return G == 1 ? i : (i + (i < n_own ? i + 1 : n_own)) / 3;
  }
};

struct PairCtl {
  uint64_t q_full;                             // the query's rows have landed
  uint64_t q_moved;                            // and their staging space is free for tiles
  uint64_t q_ready;                            // the query is in tensor and shared memory
  uint64_t k_full[kLoose], k_empty[kLoose];    // G = 1: the five loose blocks; G = 2: the five pieces
  uint64_t v_full[3], v_empty[3];              // value tiles: landed; read by their P V
  uint64_t s_full, s_free;                     // logits written / read into registers
  // per weight buffer:
  uint64_t p_mine[2];                          // this CTA's weights are in shared memory
  uint64_t p_full[2];                          // every row's weights are, and O is at their reference
  uint64_t p_empty[2];                         // own weights read: by the own P V and by the peer's (of its copy)
  uint64_t pin_full[2];                        // the peer's weights have landed
  uint64_t pin_go[2];                          // they and O are at one reference
  uint64_t o_done;
  uint64_t r_full;                             // parity 1: the first references have landed
  uint64_t fin_full;                           // the peer's sums have landed
  uint32_t tmem_base;
  int abort;
  float sent[kRows];                           // by the peer: the first references (to parity 1), at the end the sums
  float part[2][2][kRows];                     // tile maxima of a row's two threads, by tile parity
};
template <int G> constexpr uint32_t kSmemBytes = Layout<G>::ctl + 3 * 1024;
static_assert(sizeof(PairCtl) <= 3 * 1024 && kPieces == kLoose && kSmemBytes<1> <= 232448 && kSmemBytes<2> <= 232448, "shared memory");
// the query's dims 0..383 and the output rows are staged where the tiles go
constexpr int kStagePitch = kHalfV * 2 + 16;
static_assert(4 * kQBlock == 2 * Layout<1>::kVBytes && kQBlock <= kLoose * kBlock && 3 * kQBlock == 3 * Layout<2>::kVBytes &&
                  kQBlock <= 2 * kPiece && Layout<2>::q_block(5) % 1024 == 0,
              "query staging");
static_assert(kRows * kStagePitch <= Layout<1>::ctl - Layout<1>::v && kRows * kStagePitch <= Layout<2>::ctl - Layout<2>::v,
              "output staging");

// A split costs every row its partial output, once written and once read, at some 5 TB/s.
constexpr int kShortPrefix = 1024;  // (expanded for every sequence, it should not fill the workspace)
constexpr double kJoinUs = 2048.0 / 5.0e6, kFewUs16 = 1.5, kFewUs16Pair = 3.6, kFewUs32 = 2.2;

// What expand writes per tile.
constexpr int kLowest = -120, kZeros = kLowest - 1;
struct alignas(32) TileInfo {
  uint64_t valid, poison;    // a bit per position
  int32_t e;                 // stored value = value * 2^-e; kZeros where all are 0
  int32_t pad[3];
};

struct PrefixPlan {
  int tiles_p, tiles_t;      // tiles of the prefix, and of the longest possible tail
  int tail_lo, tail_sure;    // the tails' first position (0: a short prefix goes with them), tiles all of them have
  int sp, st;                // splits of the prefix and of each tail on the tensor-memory path
  int few_lo, few;           // the path for few heads: first position and most parts of a row (0: not taken)
  int few_blocks;
  int ns;                    // all splits of a row
  int mt;                    // 128-row tiles of the flattened rows
  int n_seq, h_s;
  int g;                     // of them in one item: MMAs of one CTA or of a pair
  int64_t rows_kv;           // rows of the expanded cache
  size_t off_info, off_o, off_ml, off_used, bytes;
};

struct PrefixWs {
  __half* kv;                // [tiles_p * 64 + n_seq * tiles_t * 64][576]
  TileInfo* info;            // [tiles]
  __half* o;                 // [n_q * h_s][ns][512], times 2^-(its exponent)
  float4* ml;                // [n_q * h_s][ns]: reference, sum, the outputs' exponent
  int* used;                 // [n_q]: parts of the row on the path for few heads
};

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// The tensor-memory path's plan of least estimated time: MMAs of one CTA (128 rows an item, two
// CTAs) or of CTA pairs (256 rows, four CTAs), and the splits: of the prefix up to 64 and of a tail up
// to 16, in powers of two, which bounds the search and the merge (more were not measured).  An item
// of n tiles takes about 9 + 1.33 n us with one CTA per parity and 11 + 0.62 n us with pairs, on one
// of the clusters that fit at once.  A tail's item holds as many adjacent rows of its sequence as fit; the rows are
// counted as if spread evenly over the sequences.  Returns the us.
double plan_tiles(PrefixPlan& p, int n_q, int n_sm) {
  double best = 1e30;
  if (!p.tiles_p && !p.tiles_t) return 0.0;
  for (int g = 1; g <= 2; ++g) {
    const int run = std::max(1, std::min(kRows * g / p.h_s, n_q / p.n_seq));  // query rows in a tail's item
    if (g == 2 && (p.mt < 2 || (!p.tiles_p && run * p.h_s <= kRows))) break;
    // (152 SMs hold 76 clusters of two CTAs of this size, 36 of four)
    const int fit = std::max(1, g == 1 ? n_sm / 2 : n_sm / 4 - n_sm / 76);
    const int mt = (p.mt + g - 1) / g;
    const double fix = g == 1 ? 9.0 : 11.0, per = g == 1 ? 1.33 : 0.62;
    for (int waves = 1; waves <= 6; ++waves) {  // as many splits as fill so many waves
      const int sp = p.tiles_p ? std::min({p.tiles_p, std::max(1, static_cast<int>(static_cast<int64_t>(waves) * fit / mt)), 64}) : 0;
      for (int st = p.tiles_t ? 1 : 0; st <= std::min(p.tiles_t, 16); st = st ? 2 * st : 1) {
        const double lp = sp ? fix + per * ((p.tiles_p + sp - 1) / sp) : 0.0;
        const double lt = st ? fix + per * ((p.tiles_t + st - 1) / st) : 0.0;
        const int64_t np = static_cast<int64_t>(mt) * sp;
        // the tails are counted half full: their lengths are known to the device alone
        const double full = p.tiles_t ? 0.5 + 0.5 * p.tail_sure / p.tiles_t : 0.0;
        const int live = (n_q + run - 1) / run;  // (an empty item takes a cluster for 1 us)
        const double total = (np * lp + static_cast<double>(st) * (live * (fix + full * (lt - fix)) + (n_q - live))) / fit;
        const double t = std::max({static_cast<double>((np + fit - 1) / fit) * lp, total + 0.5 * lt, lt}) + kJoinUs * n_q * p.h_s * (sp + st);
        if (t < best) {
          best = t;
          p.g = g;
          p.sp = sp;
          p.st = st;
        }
        if (!st) break;
      }
      if (!p.tiles_p) break;
    }
  }
  // the expansion, at some 5 TB/s, and one or two more launches
  const double positions = 64.0 * p.tiles_p + 32.0 * (p.tiles_t + p.tail_sure) * p.n_seq;
  return best + positions * (kKvTokBytes + 2 * kLatent) / 5.0e6 + (p.sp + p.st > 1 ? 5.0 : 2.5);
}

// All of it on the tensor-memory path, or (up to 32 heads) the tails or everything on the path for
// few heads.  There 64 positions of a row take 1.5 us alone on an SM and 3.6 us with two blocks on
// it (17 heads and more: 2.2 us, one block), a block's start and end some 5 us and a further row in
// it 4.5 us; it reads nothing twice but a prefix, once for every row.
PrefixPlan make_plan(int n_q, int h_s, int n_seq, int prefix_len, int max_ctx, int n_sm) {
  PrefixPlan p{};
  p.n_seq = n_seq;
  p.h_s = h_s;
  p.tiles_p = (prefix_len + kTile - 1) / kTile;
  p.tiles_t = (max_ctx - prefix_len + kTile - 1) / kTile;
  p.tail_lo = prefix_len;
  p.mt = static_cast<int>((static_cast<int64_t>(n_q) * h_s + kRows - 1) / kRows);
  double best = plan_tiles(p, n_q, n_sm);
  // A short prefix may go with every row's tail instead: expanded once a sequence, but no items and
  // partial results of its own (208 rows of 128 heads, 8 + 486..662 positions: 156 -> 102 us).
  if (prefix_len > 0 && prefix_len <= kShortPrefix && max_ctx > prefix_len) {
    PrefixPlan q = p;
    q.tiles_p = q.sp = q.tail_lo = 0;
    q.tiles_t = (max_ctx + kTile - 1) / kTile;
    q.tail_sure = prefix_len / kTile;
    const double t = plan_tiles(q, n_q, n_sm);
    if (t < best) {
      best = t;
      p = q;
    }
  }
  if (h_s <= kFewHeads) {
    const int fit = h_s <= 16 ? 2 * n_sm : n_sm;
    for (int whole = 0; whole < 2; ++whole) {  // the tails, then everything
      const int lo = whole ? 0 : prefix_len;
      if ((!whole && !prefix_len) || lo == max_ctx) continue;
      PrefixPlan q = p;
      q.sp = q.st = q.tiles_t = q.tail_sure = 0;
      q.tiles_p = whole ? 0 : (prefix_len + kTile - 1) / kTile;
      const double rest = plan_tiles(q, n_q, n_sm);
      const int steps = (max_ctx - lo + 63) / 64, sure = whole ? prefix_len / 64 : 0;
      const double mean = 0.5 * (steps + sure) * n_q;  // of all rows, tails half full
      const int even = static_cast<int>(std::min<int64_t>(fit, static_cast<int64_t>(steps) * n_q));
      for (int few = 1; few <= (n_q > kFewCutRows ? 1 : std::min(2 * steps, 512)); few *= 2) {
        // a row a block, the longest one last; or even shares
        const int blocks = few == 1 ? n_q : even;
        const double step = h_s > 16 ? kFewUs32 : blocks <= n_sm ? kFewUs16 : kFewUs16Pair, parts = std::min<double>(few, 1.0 + even / n_q);
        const double t = rest + 5.0 + kJoinUs * n_q * h_s * (few == 1 ? 1 : parts) + (few > 1 || q.sp ? 3.0 : 0.0) +
                         (few == 1 ? step * std::max<double>(steps, mean / fit + (n_q > fit ? 0.5 * steps : 0.0)) + 4.5 * (n_q / fit)
                                   : step * std::max({mean / even, steps / (few - 1.0), 1.0}) + 4.5 * n_q / even);
        if (t < best) {
          best = t;
          q.few_lo = lo;
          q.few = few;
          q.few_blocks = few == 1 ? n_q : even;
          p = q;
        }
      }
    }
  }
  p.ns = p.sp + p.st + p.few;
  p.rows_kv = static_cast<int64_t>(p.tiles_p) * kTile + static_cast<int64_t>(n_seq) * p.tiles_t * kTile;
  const size_t parts = p.ns > 1 ? static_cast<size_t>(n_q) * h_s * p.ns : 0;
  p.off_info = round_up(static_cast<size_t>(p.rows_kv) * kLatent * 2, 256);
  p.off_o = p.off_info + round_up(static_cast<size_t>(p.rows_kv / kTile) * sizeof(TileInfo), 256);
  p.off_ml = p.off_o + parts * kVDim * 2;
  p.off_used = p.off_ml + round_up(parts * 16, 256);
  p.bytes = std::max<size_t>(256, p.off_used + (p.ns > 1 && p.few ? round_up(static_cast<size_t>(n_q) * 4, 256) : 0));
  return p;
}

// ---- expand: one block per 64-position tile ------------------------------------------------
// Bound by memory: 608 bytes read and 1152 written a position.
constexpr int kExpandThreads = 288;
constexpr int kChunks = kLatent / 16;  // 16-code chunks of a record
__global__ void __launch_bounds__(kExpandThreads)
expand_kernel(PrefixArgs a, PrefixPlan pl, PrefixWs ws) {
  __shared__ unsigned s_word[4];  // valid (2 words), poisonous (2 words)
  __shared__ unsigned s_scale;    // the largest finite scale's bits
  pdl_launch_dependents();
  pdl_wait();
  const int tile = blockIdx.x;
  const int tid = threadIdx.x;
  int pos0, len;
  const int32_t* table = nullptr;
  if (tile < pl.tiles_p) {
    pos0 = tile * kTile;
    len = a.prefix_len;
  } else {
    const int b = (tile - pl.tiles_p) / pl.tiles_t;
    pos0 = pl.tail_lo + (tile - pl.tiles_p) % pl.tiles_t * kTile;
    len = a.seq_lens[b];
    if (len < 0 || len > a.max_ctx) len = 0;
    if (pos0 >= len) return;
    table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  }
  if (tid < 4) s_word[tid] = 0;
  if (tid == 4) s_scale = 0;
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
    const int pg = (p < a.prefix_len ? a.prefix_pages : table)[p / kPage];
    if (pg < 0 || pg >= a.num_pages) {
      if (c == 0) flag(a.status, DSA_STATUS_BAD_PAGE);
      continue;
    }
    const uint8_t* rec = a.kv_cache + (static_cast<int64_t>(pg) * kPage + p % kPage) * kKvTokBytes;
    code[i] = *reinterpret_cast<const uint4*>(rec + 16 * c);
    scale[i] = *reinterpret_cast<const float*>(rec + kKvScaleOff + 4 * (c >> 3));
    if (c == 0) atomicOr(&s_word[tok >> 5], 1u << (tok & 31));
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int tok = (i * kExpandThreads + tid) / kChunks;
    const bool bad = !(fabsf(scale[i]) * 448.0f < INFINITY) || has_nan_code(code[i].x) || has_nan_code(code[i].y) ||
                     has_nan_code(code[i].z) || has_nan_code(code[i].w);
    if (bad) {
      atomicOr(&s_word[2 + (tok >> 5)], 1u << (tok & 31));
      scale[i] = 0.f;
    }
    top = fmaxf(top, fabsf(scale[i]));
  }
  const unsigned warp_top = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if ((tid & 31) == 0) atomicMax(&s_scale, warp_top);
  __syncthreads();
  // 448 * scale < 2^(floor(log2 scale) + 10): below 2^15 once stored
  // (not below -120: powers of two up and down from there stay inside fp32's normal range)
  const int e = s_scale ? max(static_cast<int>(s_scale >> 23) - 127 - 5, kLowest) : kZeros;
  uint4* dst = reinterpret_cast<uint4*>(ws.kv + static_cast<int64_t>(tile) * kTile * kLatent);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int w = i * kExpandThreads + tid, tok = w / kChunks;
    const bool drop = (s_word[2 + (tok >> 5)] >> (tok & 31)) & 1u;
    const float f = drop ? 0.f : scale[i] * exp2i(-e);
    const uint32_t u[4] = {drop ? 0u : code[i].x, drop ? 0u : code[i].y, drop ? 0u : code[i].z, drop ? 0u : code[i].w};
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4];
      e4m3x4_to_f32(u[q], v);
      o[2 * q] = pack_half2(v[0] * f, v[1] * f);
      o[2 * q + 1] = pack_half2(v[2] * f, v[3] * f);
    }
    dst[2 * w] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[2 * w + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  if (tid == 0) {
    TileInfo t;
    t.valid = s_word[0] | static_cast<uint64_t>(s_word[1]) << 32;
    t.poison = s_word[2] | static_cast<uint64_t>(s_word[3]) << 32;
    t.e = e;
    ws.info[tile] = t;
  }
}

// ---- attend ----------------------------------------------------------------------------------
// A bounded wait (as mbar_wait) in two parts: one attempt in line, the rest out of line, so
// that the warps' loops, two dozen waits between them, stay within the instruction cache (with the
// whole wait in line a third of all warp cycles went into fetching instructions).
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status) {
  const uint64_t t0 = tc::global_ns();
  for (uint32_t it = 0;; ++it) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 15u) {
      if (*abort) return false;
      if (tc::global_ns() - t0 > tc::kWaitLimitNs) {
        *abort = 1;
        flag(status, DSA_STATUS_TIMEOUT);
        return false;
      }
    }
  }
}
// Arrive on the same barrier of the cluster's CTA `rank`.  What the arrival announces is read by
// tensor cores alone, behind the writer's proxy fence or tcgen05 fence, so it needs no release at
// cluster scope (which took some 1500 cycles here).
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(dsmem_addr(bar, rank)) : "memory");
}

// tcgen05 for one CTA (G = 1) or for the pair of CTAs 2 i, 2 i + 1 (G = 2).  The pair's even CTA
// issues: an MMA then has 256 rows, 128 in each CTA's tensor memory, and each CTA's shared memory
// holds half of B.
template <int G>
__device__ __forceinline__ void tmem_alloc_all(uint32_t* slot) {
  if constexpr (G == 1) {
    tc::tmem_alloc(slot, 512);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int G>
__device__ __forceinline__ void tmem_dealloc_all(uint32_t base) {
  if constexpr (G == 1) tc::tmem_dealloc(base, 512);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(base) : "memory");
}
// A box of the expanded rows; in a pair it counts on the even CTA's barrier (the same offset
// there: bit 24 of a shared address is the lowest of the CTA's rank).
template <int G>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  if constexpr (G == 1) {
    tc::tma_load_3d(dst, map, x, y, 0, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(0),
           "r"(smem_u32(bar) & 0xFEFFFFFFu)
        : "memory");
  }
}

// fp16 MMAs with operand descriptors given by their low word (address and leading offset); the
// high word is the same for every operand here: 8-row groups 1024 bytes apart, 128-byte swizzle.
// Dynamic shared memory starts behind the block's reserved 1 KB (the kernel checks it), so the
// descriptors are constants of the code.  One elected lane of the converged warp issues
// (`leader`, found once).
#define DSA_DESC_HI "0x40004040"
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
static_assert(kDescHi == 0x40004040u, "descriptor high word");
constexpr uint32_t kSmemBase = 1024;
constexpr uint32_t desc_lo(uint32_t off, uint32_t lead) { return (kSmemBase + off) >> 4 | (lead >> 4) << 16; }
template <int G, bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t leader) {
#define DSA_MMA_TS(group)                                                                             \
  asm volatile(                                                                                       \
      "{\n .reg .pred p, e;\n .reg .b64 b;\n setp.ne.b32 e, %4, 0;\n setp.ne.b32 p, %5, 0;\n"         \
      "mov.b64 b, {%2, " DSA_DESC_HI "};\n"                                                           \
      "@e tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%1], b, %3, p;\n}"                        \
      :: "r"(d), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(leader), "n"(ACC ? 1 : 0) : "memory")
  if constexpr (G == 1) DSA_MMA_TS("1"); else DSA_MMA_TS("2");
#undef DSA_MMA_TS
}
template <int G, bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t leader) {
#define DSA_MMA_SS(group)                                                                             \
  asm volatile(                                                                                       \
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n setp.ne.b32 e, %4, 0;\n setp.ne.b32 p, %5, 0;\n"      \
      "mov.b64 a, {%1, " DSA_DESC_HI "};\n mov.b64 b, {%2, " DSA_DESC_HI "};\n"                       \
      "@e tcgen05.mma.cta_group::" group ".kind::f16 [%0], a, b, %3, p;\n}"                           \
      :: "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(leader), "n"(ACC ? 1 : 0) : "memory")
  if constexpr (G == 1) DSA_MMA_SS("1"); else DSA_MMA_SS("2");
#undef DSA_MMA_SS
}
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
  return r;
}
// arrive on a barrier of the CTAs in the mask once the MMAs the leader issued have completed
template <int G>
__device__ __forceinline__ void commit_to(uint64_t* bar, uint16_t mask, uint32_t leader) {
#define DSA_COMMIT(group)                                                                                            \
  asm volatile(                                                                                                      \
      "{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n"                                                                  \
      "@e tcgen05.commit.cta_group::" group ".mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" \
      :: "r"(smem_u32(bar)), "h"(mask), "r"(leader) : "memory")
  if constexpr (G == 1) DSA_COMMIT("1"); else DSA_COMMIT("2");
#undef DSA_COMMIT
}
// fp16 A and B, fp32 accumulator, M = 128 G
__host__ __device__ constexpr uint32_t idesc_f16(int g, int n, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 * g >> 4) << 24);
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

// S = Q K^T of 64-dim block KB of a tile (four K-steps of 16 dims), its rows at descriptor k_lo.
template <int G, int KB, bool FIRST>
__device__ __forceinline__ void qk_block(uint32_t k_lo, uint32_t leader) {
  constexpr uint32_t id = idesc_f16(G, kTile, false);
  if constexpr (KB < kQTmemBlocks) {
    mma_ts<G, !FIRST>(kColS, kColQ + 32 * KB, k_lo, id, leader);
    mma_ts<G, true>(kColS, kColQ + 32 * KB + 8, k_lo + 2, id, leader);
    mma_ts<G, true>(kColS, kColQ + 32 * KB + 16, k_lo + 4, id, leader);
    mma_ts<G, true>(kColS, kColQ + 32 * KB + 24, k_lo + 6, id, leader);
  } else {
    constexpr uint32_t q = desc_lo(kOffQ + (KB - kQTmemBlocks) * kQBlock, 16);
    mma_ss<G, !FIRST>(kColS, q, k_lo, id, leader);
    mma_ss<G, true>(kColS, q + 2, k_lo + 2, id, leader);
    mma_ss<G, true>(kColS, q + 4, k_lo + 4, id, leader);
    mma_ss<G, true>(kColS, q + 6, k_lo + 6, id, leader);
  }
}
// O (+)= P V of one tile: four K-steps of 16 positions, 256 value columns
template <int G, bool ACC>
__device__ __forceinline__ void pv_tile(uint32_t p_lo, uint32_t v_lo, uint32_t leader) {
  constexpr uint32_t id = idesc_f16(G, kHalfV, true);
  mma_ss<G, ACC>(kColO, p_lo, v_lo, id, leader);
  mma_ss<G, true>(kColO, p_lo + 2, v_lo + (2048 >> 4), id, leader);
  mma_ss<G, true>(kColO, p_lo + 4, v_lo + 2 * (2048 >> 4), id, leader);
  mma_ss<G, true>(kColO, p_lo + 6, v_lo + 3 * (2048 >> 4), id, leader);
}

// The Q K^T warp, G = 1, of CTA C: the own tiles' value blocks (dims 256 C ..) first, the other
// five blocks as they come.
template <int C, typename Wait>
__device__ __forceinline__ void qk_loop_single(PairCtl& ctl, int n_own, Wait wait_warp) {
  const uint32_t leader = elect_leader();
  constexpr uint32_t kStep = kBlock >> 4, v0 = desc_lo(Layout<1>::v, 16), v1 = v0 + 4 * kStep;
  constexpr uint32_t lo = desc_lo(Layout<1>::k, 16);
  constexpr uint16_t me = 1u << C;
#pragma unroll 1
  for (int i = 0; i < n_own; ++i) {
    const int b = i & 1;
    if (!wait_warp(&ctl.s_free, i + 1) || !wait_warp(&ctl.v_full[b], i >> 1)) return;
    tc::fence_after_sync();
    if (b == 0) {
      qk_block<1, 4 * C, true>(v0, leader);
      qk_block<1, 4 * C + 1, false>(v0 + kStep, leader);
      qk_block<1, 4 * C + 2, false>(v0 + 2 * kStep, leader);
      qk_block<1, 4 * C + 3, false>(v0 + 3 * kStep, leader);
    } else {
      qk_block<1, 4 * C, true>(v1, leader);
      qk_block<1, 4 * C + 1, false>(v1 + kStep, leader);
      qk_block<1, 4 * C + 2, false>(v1 + 2 * kStep, leader);
      qk_block<1, 4 * C + 3, false>(v1 + 3 * kStep, leader);
    }
    constexpr int L = 4 * (1 - C);
    if (!wait_warp(&ctl.k_full[0], i)) return;
    qk_block<1, L, false>(lo, leader);
    commit_to<1>(&ctl.k_empty[0], me, leader);
    if (!wait_warp(&ctl.k_full[1], i)) return;
    qk_block<1, L + 1, false>(lo + kStep, leader);
    commit_to<1>(&ctl.k_empty[1], me, leader);
    if (!wait_warp(&ctl.k_full[2], i)) return;
    qk_block<1, L + 2, false>(lo + 2 * kStep, leader);
    commit_to<1>(&ctl.k_empty[2], me, leader);
    if (!wait_warp(&ctl.k_full[3], i)) return;
    qk_block<1, L + 3, false>(lo + 3 * kStep, leader);
    commit_to<1>(&ctl.k_empty[3], me, leader);
    if (!wait_warp(&ctl.k_full[4], i)) return;
    qk_block<1, 8, false>(lo + 4 * kStep, leader);
    commit_to<1>(&ctl.k_empty[4], me, leader);
    commit_to<1>(&ctl.s_full, me, leader);
  }
}
// G = 2: a tile comes in three pieces of 192 dims, half of its positions in each CTA.
template <int PIECE>
__device__ __forceinline__ void qk_piece(uint32_t k_lo, uint32_t leader) {
  constexpr uint32_t kStep = kBlock / 2 >> 4;
  qk_block<2, 3 * PIECE, PIECE == 0>(k_lo, leader);
  qk_block<2, 3 * PIECE + 1, false>(k_lo + kStep, leader);
  qk_block<2, 3 * PIECE + 2, false>(k_lo + 2 * kStep, leader);
}
template <typename Wait>
__device__ __forceinline__ void qk_loop_pair(PairCtl& ctl, int n_own, uint16_t pair, Wait wait_warp) {
  const uint32_t leader = elect_leader();
  constexpr uint32_t k0 = desc_lo(Layout<2>::k, 16);
  int slot = 0, phase = 0;
  auto next = [&] {
    if (++slot == kPieces) {
      slot = 0;
      ++phase;
    }
  };
#pragma unroll 1
  for (int i = 0; i < n_own; ++i) {
    if (!wait_warp(&ctl.k_full[slot], phase) || !wait_warp(&ctl.s_free, i + 1)) return;
    tc::fence_after_sync();
    qk_piece<0>(k0 + slot * (kPiece >> 4), leader);
    commit_to<2>(&ctl.k_empty[slot], pair, leader);
    next();
    if (!wait_warp(&ctl.k_full[slot], phase)) return;
    qk_piece<1>(k0 + slot * (kPiece >> 4), leader);
    commit_to<2>(&ctl.k_empty[slot], pair, leader);
    next();
    if (!wait_warp(&ctl.k_full[slot], phase)) return;
    qk_piece<2>(k0 + slot * (kPiece >> 4), leader);
    commit_to<2>(&ctl.s_full, pair, leader);
    commit_to<2>(&ctl.k_empty[slot], pair, leader);
    next();
  }
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap tile_map,
              const __grid_constant__ CUtensorMap half_map, PrefixArgs a, PrefixPlan pl, PrefixWs ws) {
  using Lay = Layout<G>;
  extern __shared__ __align__(1024) uint8_t smem[];
  PairCtl& ctl = *reinterpret_cast<PairCtl*>(smem + Lay::ctl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // rank = G c + g: c the parity of the own tiles and the half of the value columns, g the CTA's
  // 128 rows of the item's 128 G.  Its peer has the same rows; the pair's even CTA issues MMAs.
  const int rank = static_cast<int>(cluster_ctarank());
  const int c = rank / G, g = rank % G, peer = rank ^ G, other = c ^ 1, chief = G * c;
  const uint16_t mine = static_cast<uint16_t>(((1 << G) - 1) << (G * c));            // the CTAs of this parity
  const uint16_t theirs = static_cast<uint16_t>(((1 << G) - 1) << (G * (c ^ 1)));  // and of the other
  pdl_launch_dependents();
  pdl_wait();

  // ---- the item: rows row0 .. of the flattened (query row, head), tiles tile0 .. ----
  const int item = blockIdx.x / (2 * G);
  const int mt = (pl.mt + G - 1) / G;
  const int n_prefix = pl.sp * mt;
  const bool tail = item >= n_prefix;
  const int64_t rows_all = static_cast<int64_t>(a.n_q) * a.h_s;
  const int ns = pl.ns;
  int64_t row0;
  int n_rows, part, split, tiles, tile_base, first_pos;
  if (!tail) {
    split = item / mt;
    row0 = (static_cast<int64_t>(item - split * mt) * G + g) * kRows;
    n_rows = static_cast<int>(max(min(static_cast<int64_t>(kRows), rows_all - row0), static_cast<int64_t>(0)));
    part = pl.sp;
    tiles = pl.tiles_p;
    tile_base = 0;
    first_pos = 0;
  } else {
    // Query rows in groups of as many as 128 G rows hold: the item of the first row of a run of one
    // sequence's rows takes the run, the other rows' items are empty.
    const int k = item - n_prefix;
    split = k / a.n_q;
    const int t = k - split * a.n_q, fit = kRows * G / a.h_s, group = t / fit * fit, group_end = min(group + fit, a.n_q);
    const int seq = a.q_seq[t];
    int run = 0, lim = 0;
    if (t == group || a.q_seq[t - 1] != seq) {
      for (int base = t;; base += 32) {
        const int r = base + lane;
        const unsigned same = __ballot_sync(0xffffffffu, r < group_end && a.q_seq[r] == seq);
        const int more = same == ~0u ? 32 : __ffs(~same) - 1;
        if (lane < more) lim = max(lim, prefix_row_limit(a, r, warp == 0 && rank == 0 && split == 0));
        run += more;
        if (more < 32) break;
      }
      lim = __reduce_max_sync(0xffffffffu, lim);
    }
    row0 = static_cast<int64_t>(t) * a.h_s + g * kRows;
    n_rows = max(min(kRows, run * a.h_s - g * kRows), 0);
    part = pl.st;
    tiles = lim > pl.tail_lo ? (lim - pl.tail_lo + kTile - 1) / kTile : 0;
    // (a row that sees anything has a sequence in range)
    tile_base = tiles ? pl.tiles_p + seq * pl.tiles_t : 0;
    first_pos = pl.tail_lo;
  }
  const int tile0 = static_cast<int>(static_cast<int64_t>(split) * tiles / part);
  const int nt = static_cast<int>(static_cast<int64_t>(split + 1) * tiles / part) - tile0;
  const int slot = tail ? pl.sp + split : split;
  if (nt == 0) {  // all CTAs alike: nothing of these rows lies in this split
    if (c == 0 && ns > 1) {
      for (int m = tid; m < n_rows; m += kThreads)
        ws.ml[(row0 + m) * ns + slot] = split_state(0.f, 0.f, 0);
    } else if (ns == 1) {
      for (int i = tid; i < n_rows * (kHalfV / 8); i += kThreads)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (row0 + i / (kHalfV / 8)) * kVDim + kHalfV * c +
                                  8 * (i % (kHalfV / 8))) = make_uint4(0u, 0u, 0u, 0u);
      if (c == 0 && a.out_lse)
        for (int m = tid; m < n_rows; m += kThreads) a.out_lse[row0 + m] = -INFINITY;
    }
    return;
  }
  const int n_own = (nt - c + 1) / 2, n_peer = nt - n_own;  // own tile i: 2 i + c; peer tile i: 2 i + other
  // (the CTA's rank in the cluster stands above a shared address's 24 bits)
  if ((smem_u32(smem) & 0xFFFFFFu) != kSmemBase) {  // (the same in all CTAs)
    if (tid == 0) flag(a.status, DSA_STATUS_INTERNAL);
    return;
  }
  if (tid == 0) {
    ctl.abort = 0;
    tc::mbar_init(&ctl.q_full, 1);
    tc::mbar_init(&ctl.q_moved, kSoftWarps);
    tc::mbar_init(&ctl.q_ready, G * 12);
    for (int k = 0; k < kLoose; ++k) {
      tc::mbar_init(&ctl.k_full[k], 1);
      tc::mbar_init(&ctl.k_empty[k], 1);
    }
    for (int k = 0; k < Lay::kVSlots; ++k) {
      tc::mbar_init(&ctl.v_full[k], 1);
      tc::mbar_init(&ctl.v_empty[k], 1);
    }
    for (int k = 0; k < Lay::kBufs; ++k) {
      tc::mbar_init(&ctl.p_mine[k], kSoftWarps);
      tc::mbar_init(&ctl.p_full[k], G * kSoftWarps);
      tc::mbar_init(&ctl.p_empty[k], 2);
      tc::mbar_init(&ctl.pin_full[k], 1);
      tc::mbar_init(&ctl.pin_go[k], G * kSoftWarps);
    }
    tc::mbar_init(&ctl.s_full, 1);
    tc::mbar_init(&ctl.s_free, G * kSoftWarps);
    tc::mbar_init(&ctl.o_done, 1);
    tc::mbar_init(&ctl.r_full, 1);
    tc::mbar_init(&ctl.fin_full, 1);
    tc::mbar_fence_init();
    // what the peer will send
    if (c == 1) tc::mbar_arrive_expect_tx(&ctl.r_full, kRows * 4);
    tc::mbar_arrive_expect_tx(&ctl.fin_full, kRows * 4);
    for (int k = 0; k < Lay::kBufs; ++k) tc::mbar_arrive_expect_tx(&ctl.pin_full[k], kPMsg);
    // the query's rows (those past the last one read as zero)
    tc::fence_async_smem();
    tc::mbar_arrive_expect_tx(&ctl.q_full, 9 * kQBlock);
#pragma unroll 1
    for (int k = 0; k < 9; ++k)
      tc::tma_load_3d(smem + Lay::q_block(k), &q_map, 64 * k, static_cast<int>(row0), 0, &ctl.q_full);
    tc::prefetch_tmap(&tile_map);
    if constexpr (G == 2) tc::prefetch_tmap(&half_map);
  }
  __syncwarp();
  if (warp == 1) tmem_alloc_all<G>(&ctl.tmem_base);
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // every CTA's barriers are ready
  tc::fence_after_sync();
  // all 512 columns are this CTA's, so its addresses start at 0 and are constants below
  if (tid == 0 && ctl.tmem_base != 0) {
    flag(a.status, DSA_STATUS_INTERNAL);
    ctl.abort = 1;
  }
  __syncwarp();
  volatile int* abort = &ctl.abort;
  // (bounded) wait of one thread, and of a converged warp: there the lanes agree on the outcome
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return tc::mbar_try_wait(bar, parity & 1u) || wait_on(bar, parity & 1u, &ctl.abort, a.status);
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity & 1u))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity & 1u, &ctl.abort, a.status)) != 0;
  };
  // an arrival that the issuing CTA waits for
  auto tell_chief = [&](uint64_t* bar) {
    if constexpr (G == 1) tc::mbar_arrive(bar);
    else arrive_at(bar, chief);
  };

  // ---- the query as fp16 by a power of two per row: warps 4..7 take dims 0..191 and warps 8..11
  // 192..383 into tensor memory, warps 0..3 the rest, in place; three threads a row ----
  float k2 = 0.f;  // logit (in powers of two) = S * k2 * 2^(tile's exponent)
  auto turn_query = [&] {
    const int quarter = warp & 3, m = quarter * 32 + lane, third = warp >> 2;
    const int first = third == 0 ? 6 : 3 * (third - 1);  // 64-dim blocks
    auto chunk = [&](int kb, int j) {                    // 8 dims of this row
      return reinterpret_cast<uint4*>(smem + Lay::q_block(kb) + m * 128 + ((j ^ (m & 7)) << 4));
    };
    wait_warp(&ctl.q_full, 0);
    __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 1
    for (int kb = first; kb < first + 3; ++kb) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 u = *chunk(kb, j);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[n])));
      }
    }
    float top = fmaxf(__low2float(top2), __high2float(top2));
    float* part = &ctl.part[0][0][0];  // (three of the four rows of maxima; free again after the second barrier)
    part[third * kRows + m] = top;
    asm volatile("bar.sync %0, 96;" :: "r"(1 + quarter) : "memory");
    top = fmaxf(fmaxf(part[m], part[kRows + m]), part[2 * kRows + m]);
    asm volatile("bar.sync %0, 96;" :: "r"(1 + quarter) : "memory");
    // top * 2^-qe in [2^14, 2^15) (below that for a row of values under 2^-112 alone)
    const int qe = top > 0.f ? min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -126), 113) : 0;
    // (a row past the item's is another item's data: zero)
    const float f = exp2i(-qe);
    k2 = a.sm_scale * 1.4426950408889634f * exp2i(qe);
    const bool live = m < n_rows;
#pragma unroll 1
    for (int kb = first; kb < first + 3; ++kb) {
      uint32_t v[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 u = *chunk(kb, j);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int n = 0; n < 4; ++n)
          v[4 * j + n] = live ? pack_half2(__uint_as_float(w[n] << 16) * f, __uint_as_float(w[n] & 0xFFFF0000u) * f) : 0u;
      }
      if (third > 0) {
        tmem_store32((static_cast<uint32_t>(quarter * 32) << 16) + kColQ + 32 * kb, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) *chunk(kb, j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    tc::fence_async_smem();  // (also orders the reads above before the tiles that follow them)
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      if (third > 0) tc::mbar_arrive(&ctl.q_moved);
      tell_chief(&ctl.q_ready);
    }
  };
  // loads of own tile i: G = 1: its kept value blocks; G = 2: this CTA's positions for Q K^T
  auto load_values = [&](int i) {
    const int b = i & 1;
    if (!wait(&ctl.v_empty[b], (i >> 1) + 1)) return false;
    tc::mbar_arrive_expect_tx(&ctl.v_full[b], Lay::kVBytes);
#pragma unroll 1
    for (int k = 0; k < 4; ++k)
      load_box<G>(smem + Lay::v + (4 * b + k) * kBlock, &tile_map, 64 * (4 * c + k), (tile_base + tile0 + 2 * i + c) * kTile,
                  &ctl.v_full[b]);
    return true;
  };
  auto load_pieces = [&](int i) {
#pragma unroll 1
    for (int k = 0; k < 3; ++k) {
      const int n = 3 * i + k, slot_k = n % kPieces;
      if (!wait(&ctl.k_empty[slot_k], n / kPieces + 1)) return false;
      if (g == 0) tc::mbar_arrive_expect_tx(&ctl.k_full[slot_k], 2 * kPiece);
#pragma unroll 1
      for (int j = 0; j < 3; ++j)
        load_box<G>(smem + Lay::k + slot_k * kPiece + j * (kBlock / 2), &half_map, 64 * (3 * k + j),
                    (tile_base + tile0 + 2 * i + c) * kTile + 32 * g, &ctl.k_full[slot_k]);
    }
    return true;
  };
  if (tid == 0 && n_own > 0) {  // the first tile's, beside the query
    if constexpr (G == 1) load_values(0);
    else load_pieces(0);
  }
  __syncwarp();
  if (warp < 12) turn_query();

  // softmax threads: their row's state, kept from the loop to the output
  float rho = -INFINITY, top = -INFINITY, l = 0.f;
  int e_top = kZeros, e_unit = 0;  // largest exponent of the tiles; l is in units of 2^-e_unit
  if (warp == 0) {
    // ---------------- own tiles ----------------
    if (lane == 0 && wait(&ctl.q_moved, 0)) {
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < n_own && ok; ++i) {
        if constexpr (G == 1) {
          // the half of the value blocks this CTA keeps, then the other blocks
          if (i > 0 && !load_values(i)) break;
          const int y = (tile_base + tile0 + 2 * i + c) * kTile;
#pragma unroll 1
          for (int k = 0; k < kLoose; ++k) {
            ok = wait(&ctl.k_empty[k], i + 1);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(&ctl.k_full[k], kBlock);
            load_box<G>(smem + Lay::k + k * kBlock, &tile_map, 64 * (k < 4 ? 4 * other + k : 8), y, &ctl.k_full[k]);
          }
        } else if (i > 0) {
          ok = load_pieces(i);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- Q K^T ----------------
    if (g == 0 && wait_warp(&ctl.q_ready, 0)) {
      tc::fence_after_sync();
      if constexpr (G == 2) qk_loop_pair(ctl, n_own, mine, wait_warp);
      else if (c == 0) qk_loop_single<0>(ctl, n_own, wait_warp);
      else qk_loop_single<1>(ctl, n_own, wait_warp);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- P V: this parity's value half, over own and peer tiles in turn ----------------
    if (g == 0) {
      const uint32_t leader = elect_leader();
      constexpr uint32_t p_own = desc_lo(Lay::p_own, 16), p_in = desc_lo(Lay::p_in, 16);
      constexpr uint32_t v0 = desc_lo(Lay::v, kBlock), v_step = Lay::kVBytes >> 4, p_step = kPStride >> 4;
#pragma unroll 1
      for (int i = 0; i < n_own || i < n_peer; ++i) {
        const int b = i % Lay::kBufs, ph = i / Lay::kBufs;
        if (i < n_own) {
          const int vs = Lay::own_slot(i);
          if (G == 2 && !wait_warp(&ctl.v_full[vs], Lay::own_phase(i))) break;
          if (!wait_warp(&ctl.p_full[b], ph)) break;
          tc::fence_after_sync();
          if (i == 0) pv_tile<G, false>(p_own, v0, leader);
          else pv_tile<G, true>(p_own + b * p_step, v0 + vs * v_step, leader);
          commit_to<G>(&ctl.p_empty[b], mine, leader);
          commit_to<G>(&ctl.v_empty[vs], mine, leader);
        }
        if (i < n_peer) {
          const int vs = Lay::peer_slot(i, n_own);
          if (!wait_warp(&ctl.v_full[vs], Lay::peer_phase(i, n_own)) || !wait_warp(&ctl.pin_go[b], ph)) break;
          tc::fence_after_sync();
          if (i == 0 && n_own == 0) pv_tile<G, false>(p_in, v0 + vs * v_step, leader);
          else pv_tile<G, true>(p_in + b * p_step, v0 + vs * v_step, leader);
          commit_to<G>(&ctl.p_empty[b], theirs, leader);
          commit_to<G>(&ctl.v_empty[vs], mine, leader);
        }
      }
      commit_to<G>(&ctl.o_done, mine, leader);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------- value blocks of the peer's tiles, and in a pair of the own ones, in the products' order ----
    if (lane == 0 && wait(&ctl.q_moved, 0)) {
#pragma unroll 1
      for (int i = 0; i < n_peer || (G == 2 && i < n_own); ++i) {
        const int y = (tile_base + tile0 + 2 * i) * kTile;
        auto load = [&](int vs, int phase, int y_tile) {
          if (!wait(&ctl.v_empty[vs], phase + 1)) return false;
          if (g == 0) tc::mbar_arrive_expect_tx(&ctl.v_full[vs], G * Lay::kVBytes);
          for (int k = 0; k < 4 / G; ++k)
            load_box<G>(smem + Lay::v + vs * Lay::kVBytes + k * kBlock, &tile_map, 64 * (4 * c + 4 / G * g + k), y_tile,
                        &ctl.v_full[vs]);
          return true;
        };
        if (G == 2 && i < n_own && !load(Lay::own_slot(i), Lay::own_phase(i), y + c * kTile)) break;
        if (i < n_peer && !load(Lay::peer_slot(i, n_own), Lay::peer_phase(i, n_own), y + other * kTile)) break;
      }
    }
    __syncwarp();
  } else if (warp == 12) {
    // ---------------- own weights to the peer ----------------
    if (lane == 0) {
      const uint32_t dst = dsmem_addr(smem + Lay::p_in, peer), bar = dsmem_addr(&ctl.pin_full[0], peer);
#pragma unroll 1
      for (int i = 0; i < n_own; ++i) {
        const int b = i % Lay::kBufs;
        // (the warps that wrote them waited until the peer had read what this buffer held before)
        if (!wait(&ctl.p_mine[b], i / Lay::kBufs)) break;
        bulk_to_peer(dst + b * kPStride, smem + Lay::p_own + b * kPStride, kPMsg, bar + b * 8);
      }
    }
    __syncwarp();
  } else {
    // ---------------- logits -> weights (warps 4..11): row m, positions 32 hv .. of each tile ----------------
    const int quarter = warp & 3, hv = (warp - 4) >> 2, m = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t pair_bar = 1 + quarter;  // named barrier of the row's two warps
    const bool live = m < n_rows;
    // the larger of v over a row's two threads (slot: alternates, so that a value is read before it
    // is written again)
    auto row_max = [&](float v, int slot_k) {
      ctl.part[slot_k][hv][m] = v;
      asm volatile("bar.sync %0, 64;" :: "r"(pair_bar) : "memory");
      return fmaxf(v, ctl.part[slot_k][hv ^ 1][m]);
    };
    // positions of this part the row sees
    int lim = 0;
    if (live) {
      lim = prefix_row_limit(a, static_cast<int>((row0 + m) / a.h_s), !tail && split == 0 && c == 0 && hv == 0) - first_pos;
      if (!tail) lim = min(lim, a.prefix_len);
    }
    // O's row (this thread's 128 columns) and the sum times 2^-by
    auto rescale = [&](float by, bool any_product) {
      const float f = exp2f(-by);
      l *= f;
      if (!any_product) return;
      tc::fence_after_sync();
      for (int col = 128 * hv; col < 128 * hv + 128; col += 16) {
        uint32_t v[16];
        tc::tmem_ld16(lane_base + kColO + col, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
        tc::tmem_st16(lane_base + kColO + col, v);
      }
      tc::tmem_wait_st();
    };
    // the exponent of the item's first tile that is not of zeros alone
#pragma unroll 1
    for (int base = 0; base < nt; base += 32) {
      const int e = base + lane < nt ? __ldcg(&ws.info[tile_base + tile0 + base + lane].e) : kZeros;
      const unsigned some = __ballot_sync(0xffffffffu, e != kZeros);
      if (some) {
        e_unit = __shfl_sync(0xffffffffu, e, __ffs(some) - 1);
        break;
      }
    }
    if (c == 1) {
      wait_warp(&ctl.r_full, 0);
      rho = ctl.sent[m];
    }
    // Bring the peer's tile i (landed, or waited for) and O to one reference.
    auto reconcile = [&](int i) {
      const int b = i % Lay::kBufs;
      uint8_t* p_in = smem + Lay::p_in + b * kPStride;
      const int e_in = __ldcg(&ws.info[tile_base + tile0 + 2 * i + other].e);
      e_top = max(e_top, e_in == kZeros ? e_unit : e_in);
      wait_warp(&ctl.pin_full[b], i / Lay::kBufs);
      if (tid == 4 * 32) tc::mbar_arrive_expect_tx(&ctl.pin_full[b], kPMsg);  // the buffer's next weights
      __syncwarp();
      const float r_in = reinterpret_cast<const float*>(p_in + kPBytes)[m];
      if (__any_sync(0xffffffffu, r_in != rho)) {
        const bool raise = r_in > rho;
        if (__any_sync(0xffffffffu, raise)) {
          // every product so far: the last was the own tile's, or the peer's before it
          if (i < n_own) wait_warp(&ctl.v_empty[Lay::own_slot(i)], Lay::own_phase(i));
          else if (i > 0) wait_warp(&ctl.v_empty[Lay::peer_slot(i - 1, n_own)], Lay::peer_phase(i - 1, n_own));
          rescale(raise ? r_in - rho : 0.f, i < n_own || i > 0);
          if (raise) rho = r_in;
        }
        if (r_in < rho) {  // sent before the peer learned of this reference (2^-inf = 0)
          const float f = exp2f(r_in - rho);
          uint8_t* row = p_in + m * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4* at = reinterpret_cast<uint4*>(row + (((4 * hv + k) ^ (m & 7)) << 4));
            const uint4 u = *at;
            uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 h = unpack_half2(v[j]);
              v[j] = pack_half2(h.x * f, h.y * f);
            }
            *at = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        tc::fence_async_smem();
        tc::fence_before_sync();
        __syncwarp();
      }
      if (lane == 0) tell_chief(&ctl.pin_go[b]);
    };
    // (after a wait that ran out these warps still go through every step, each wait returning at
    // once: the named barriers need both of a row's warps)
#pragma unroll 1
    for (int i = 0; i < n_own; ++i) {
      const int b = i % Lay::kBufs;
      const int tile = tile0 + 2 * i + c;
      const TileInfo* info = ws.info + tile_base + tile;
      const ulonglong2 w = __ldcg(reinterpret_cast<const ulonglong2*>(info));
      const int e_tile = __ldcg(&info->e), e = e_tile == kZeros ? e_unit : e_tile;
      const int nv = lim - tile * kTile;
      const uint64_t seen64 = w.x & (nv >= kTile ? ~0ull : nv <= 0 ? 0ull : (1ull << nv) - 1ull);
      const uint32_t seen = static_cast<uint32_t>(seen64 >> (32 * hv)), poison = static_cast<uint32_t>(w.y >> (32 * hv));
      e_top = max(e_top, e);
      // (held inside fp32's range: a factor of 0 would turn an unseen position's -inf into NaN)
      const float kt = fminf(fmaxf(k2 * exp2i(e), 1.2e-38f), 3.0e38f);
      const float fe = static_cast<float>(e);
      wait_warp(&ctl.s_full, i);
      tc::fence_after_sync();
      uint32_t s[32];
      tc::tmem_ld32(lane_base + kColS + 32 * hv, s);
      tc::tmem_wait_ld();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tell_chief(&ctl.s_free);
      if (!__all_sync(0xffffffffu, seen == ~0u && poison == 0u)) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if ((poison >> k) & 1u) s[k] = 0x7FFFFFFFu;
          if (!((seen >> k) & 1u)) s[k] = 0xFF800000u;
        }
      }
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        t0 = fmaxf(t0, fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 1])));
        t1 = fmaxf(t1, fmaxf(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])));
      }
      const float mt = row_max(fmaf(fmaxf(t0, t1), kt, fe), i & 1);
      if (i == 0 && c == 0) {
        const float low = -row_max(-fmaf(fminf(t0, t1), kt, fe), 1);
        asm volatile("bar.sync %0, 64;" :: "r"(pair_bar) : "memory");  // read before the next tile's maxima
        rho = fmaxf(fminf(low + kAbove, mt - kLeast), mt - kMost);
        if (hv == 0) st_async_f32(dsmem_addr(&ctl.sent[m], peer), rho, dsmem_addr(&ctl.r_full, peer));
      }
      // the reference these weights are made with: the row's, or a new one where a weight of this warp
      // would pass 2^15 or is a row's first (a row that stands behind its first tile's largest stays there)
      if (i > 0 || c > 0) top = fmaxf(top, mt);
      const bool raise = mt > rho + kHeadroom || (rho == -INFINITY && mt > -INFINITY);
      const float rho_p = __any_sync(0xffffffffu, raise) ? fmaxf(rho, top - kRaised) : rho;
      const float off = fe - (rho_p == -INFINITY ? 0.f : rho_p);
      uint32_t p[16];
      float x0 = 0.f, x1 = 0.f;
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        const float a0 = exp2_approx(fmaf(__uint_as_float(s[k]), kt, off));
        const float a1 = exp2_approx(fmaf(__uint_as_float(s[k + 1]), kt, off));
        p[k >> 1] = pack_half2(a0, a1);
        x0 += a0;
        x1 += a1;
      }
      float sum = x0 + x1;
      // the tile before this one in the order of the products: its weights have had this tile's
      // Q K^T and softmax to arrive
      if (i > 0) reconcile(i - 1);
      if (__any_sync(0xffffffffu, rho_p != rho)) {
        const bool up = rho_p > rho;
        if (__any_sync(0xffffffffu, up)) {
          if (i > 0) wait_warp(&ctl.v_empty[Lay::peer_slot(i - 1, n_own)], Lay::peer_phase(i - 1, n_own));  // every product so far
          rescale(up ? rho_p - rho : 0.f, i > 0);
          if (up) rho = rho_p;
        }
        if (rho_p < rho) {  // the peer went ahead meanwhile (2^-inf = 0)
          const float f = exp2f(rho_p - rho);
          sum *= f;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 h = unpack_half2(p[k]);
            p[k] = pack_half2(h.x * f, h.y * f);
          }
        }
      }
      l = fmaf(sum, exp2i(min(max(e_unit - e, -126), 127)), l);
      wait_warp(&ctl.p_empty[b], i / Lay::kBufs + 1);
      uint8_t* p_own = smem + Lay::p_own + b * kPStride;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(p_own + m * 128 + (((4 * hv + k) ^ (m & 7)) << 4)) =
            make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
      if (hv == 0) reinterpret_cast<float*>(p_own + kPBytes)[m] = rho;
      tc::fence_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&ctl.p_mine[b]);
        tell_chief(&ctl.p_full[b]);
      }
    }
    for (int i = max(0, n_own - 1); i < n_peer; ++i) reconcile(i);
    // the last weights have been read, here and by the peer (whose word of it has then arrived)
    for (int i = max(0, n_own - Lay::kBufs); i < n_own; ++i) wait_warp(&ctl.p_empty[i % Lay::kBufs], i / Lay::kBufs);
    // ---- the row's sum over its two threads and both CTAs ----
    ctl.part[0][hv][m] = l;
    asm volatile("bar.sync %0, 64;" :: "r"(pair_bar) : "memory");
    l = ctl.part[0][0][m] + ctl.part[0][1][m];
    if (hv == 0) st_async_f32(dsmem_addr(&ctl.sent[m], peer), l, dsmem_addr(&ctl.fin_full, peer));
    if (wait_warp(&ctl.fin_full, 0)) l = c == 0 ? l + ctl.sent[m] : ctl.sent[m] + l;  // the same in both CTAs
  }
  // every product is complete, and nothing the peer sends is still on its way
  wait(&ctl.o_done, 0);
  __syncthreads();
  tc::fence_after_sync();

  // ---- output: O / l through the tiles' shared memory, in whole rows: bf16, or with several
  // splits fp16 times 2^-(e_out), e_out the largest exponent of the item's tiles: |O / l| is at
  // most the largest value, below 2^15 2^e_out ----
  uint8_t* stage = smem + Lay::v;
  if (warp >= 4 && warp < 12) {
    const int hv = (warp - 4) >> 2, m = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int e_out = e_top;
    // O / l is this times 2^e_out (O is in units of 1, l of 2^-e_unit)
    const float inv = (l > 0.f || l != l ? 1.f / l : 0.f) * exp2i(max(e_unit - e_out, -126));
    const float up = ns == 1 ? exp2i(e_out) : 1.f;
    uint8_t* row = stage + m * kStagePitch;
#pragma unroll 2
    for (int k = 0; k < 4; ++k) {
      const int col = 128 * hv + 32 * k;
      uint32_t v[32];
      tc::tmem_ld32(lane_base + kColO + col, v);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y0 = __uint_as_float(v[i + 2 * j]) * inv, y1 = __uint_as_float(v[i + 2 * j + 1]) * inv;
          o[j] = ns == 1 ? pack_bf162(y0 * up, y1 * up) : pack_half2(y0, y1);
        }
        *reinterpret_cast<uint4*>(row + 2 * (col + i)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (c == 0 && hv == 0 && m < n_rows) {
      if (ns > 1) ws.ml[(row0 + m) * ns + slot] = split_state(rho - static_cast<float>(e_unit), l, e_out);
      else if (a.out_lse) a.out_lse[row0 + m] = natural_lse(rho - static_cast<float>(e_unit), l);
    }
  }
  __syncthreads();
  {
    const int piece = tid & 31;
    uint16_t* const base = ns == 1 ? static_cast<uint16_t*>(a.out) : reinterpret_cast<uint16_t*>(ws.o);
#pragma unroll 5
    for (int m = tid >> 5; m < n_rows; m += kThreads / 32) {
      const int64_t at = ns == 1 ? row0 + m : (row0 + m) * ns + slot;
      *reinterpret_cast<uint4*>(base + at * kVDim + kHalfV * c + 8 * piece) =
          *reinterpret_cast<const uint4*>(stage + m * kStagePitch + 16 * piece);
    }
  }
  // after a wait that ran out, copies and products may still be in flight: give them time to
  // land before either CTA of the pair gives its memory back
  if (*abort) {
    const uint64_t t0 = tc::global_ns();
    while (tc::global_ns() - t0 < 100000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc::fence_after_sync();
  if (warp == 1) tmem_dealloc_all<G>(ctl.tmem_base);
}

// ---- merge ---------------------------------------------------------------------------------
// Split s holds o_s = O_s / l_s (fp16 times a power of two) with reference m_s; with
// M = max m_s and w_s = 2^(m_s - M) l_s the output is sum_s w_s o_s / sum_s w_s.  64 threads a row, 8
// columns each, four splits' loads in flight; for few rows of many splits four such groups a row.
constexpr int kMergeBatch = 4;
struct MergeSum {
  float top = -INFINITY, sum = 0.f, acc[8] = {};
  __device__ __forceinline__ void raise(float to) {
    if (to == top) return;
    const float f = top == -INFINITY ? 0.f : exp2f(top - to);
    sum *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= f;
    top = to;
  }
};
template <int GROUPS>
__global__ void __launch_bounds__(256)
prefix_merge_kernel(PrefixArgs a, PrefixPlan pl, PrefixWs ws) {
  constexpr int kRowsBlock = 4 / GROUPS;
  pdl_launch_dependents();
  pdl_wait();
  const int grp = threadIdx.x >> 6 & (GROUPS - 1), lane64 = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsBlock + (threadIdx.x >> 6) / GROUPS;
  if (row >= static_cast<int64_t>(a.n_q) * a.h_s) return;  // (whole blocks, where groups meet)
  const int d = 8 * lane64;
  const int ns = pl.sp + pl.st + (pl.few ? min(__ldcg(ws.used + row / a.h_s), pl.few) : 0);
  MergeSum m;
  for (int s0 = kMergeBatch * grp; s0 < ns; s0 += kMergeBatch * GROUPS) {
    float4 ml[kMergeBatch];
    uint4 v[kMergeBatch];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      ml[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (s0 + i < ns) {
        ml[i] = __ldcg(ws.ml + row * pl.ns + s0 + i);
        v[i] = __ldcg(reinterpret_cast<const uint4*>(ws.o + (row * pl.ns + s0 + i) * kVDim + d));
      }
    }
    float top = m.top;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) top = fmaxf(top, ml[i].x);
    m.raise(top);
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      if (ml[i].x == -INFINITY) continue;  // an empty split: its output was never written
      const float wl = exp2f(ml[i].x - m.top) * ml[i].y;
      m.sum += wl;
      const float f = wl * exp2f(ml[i].z);
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 h = unpack_half2(u[k]);
        m.acc[2 * k] = fmaf(f, h.x, m.acc[2 * k]);
        m.acc[2 * k + 1] = fmaf(f, h.y, m.acc[2 * k + 1]);
      }
    }
  }
  if constexpr (GROUPS > 1) {
    __shared__ MergeSum s_part[GROUPS - 1][64];
    if (grp > 0) s_part[grp - 1][lane64] = m;
    __syncthreads();
    if (grp > 0) return;
    for (int i = 0; i < GROUPS - 1; ++i) {
      const MergeSum& other = s_part[i][lane64];
      if (other.top == -INFINITY) continue;
      m.raise(fmaxf(m.top, other.top));
      const float f = exp2f(other.top - m.top);
      m.sum = fmaf(f, other.sum, m.sum);
#pragma unroll
      for (int k = 0; k < 8; ++k) m.acc[k] = fmaf(f, other.acc[k], m.acc[k]);
    }
  }
  const float inv = m.sum > 0.f || m.sum != m.sum ? 1.f / m.sum : 0.f;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * kVDim + d) =
      make_uint4(pack_bf162(m.acc[0] * inv, m.acc[1] * inv), pack_bf162(m.acc[2] * inv, m.acc[3] * inv),
                 pack_bf162(m.acc[4] * inv, m.acc[5] * inv), pack_bf162(m.acc[6] * inv, m.acc[7] * inv));
  if (a.out_lse && d == 0)
    a.out_lse[row] = natural_lse(m.top, m.sum);
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
// rows of 576 16-bit values in boxes of 64 dims x box_rows, 128-byte swizzle; rows past the end
// read as zero
bool encode_rows(EncodeFn enc, CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kLatent), static_cast<cuuint64_t>(rows), 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kLatent) * 2,
                                 static_cast<cuuint64_t>(kLatent) * 2 * static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t prefix_workspace_bytes(int n_q, int h_s, int n_seq, int prefix_len, int max_ctx) {
  return make_plan(n_q, h_s, n_seq, prefix_len, max_ctx, multiprocessors()).bytes;
}

void prefix_plan_numbers(int n_q, int h_s, int n_seq, int prefix_len, int max_ctx, int32_t* out) {
  const PrefixPlan p = make_plan(n_q, h_s, n_seq, prefix_len, max_ctx, multiprocessors());
  const int numbers[8] = {p.sp + p.st ? p.g : 0, p.tiles_p, p.sp, p.tail_lo, p.tiles_t, p.st, p.few, p.few_lo};
  std::copy(numbers, numbers + 8, out);
}

cudaError_t launch_prefix_attn(const PrefixArgs& a, cudaStream_t s, const char** err) {
  const PrefixPlan pl = make_plan(a.n_q, a.h_s, a.n_seq, a.prefix_len, a.max_ctx, multiprocessors());
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  PrefixWs ws{reinterpret_cast<__half*>(base), reinterpret_cast<TileInfo*>(base + pl.off_info),
              reinterpret_cast<__half*>(base + pl.off_o), reinterpret_cast<float4*>(base + pl.off_ml),
              reinterpret_cast<int*>(base + pl.off_used)};
  const int64_t rows = static_cast<int64_t>(a.n_q) * a.h_s;
  const int64_t items = static_cast<int64_t>(pl.sp) * ((pl.mt + pl.g - 1) / std::max(1, pl.g)) + static_cast<int64_t>(pl.st) * a.n_q;
  if (pl.rows_kv > INT32_MAX - kTile || rows > INT32_MAX - kRows || items > INT32_MAX / 4 ||
      static_cast<int64_t>(pl.few) * a.n_q > INT32_MAX) {
    *err = "prefix_attn: more rows than 32 bits count";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaSuccess;
  if (pl.few) {
    e = launch_prefix_few({a, pl.few_lo, pl.few, pl.few_blocks, pl.sp + pl.st, pl.ns, ws.o, ws.ml, ws.used}, s);
    if (e != cudaSuccess) return e;
  }
  if (items) {
    const EncodeFn enc = encode_fn();
    if (!enc) {
      *err = "prefix_attn: cuTensorMapEncodeTiled is not available";
      return cudaErrorNotSupported;
    }
    CUtensorMap q_map, tile_map, half_map;
    if (!encode_rows(enc, &q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, rows, kRows) ||
        !encode_rows(enc, &tile_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws.kv, pl.rows_kv, kTile) ||
        !encode_rows(enc, &half_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws.kv, pl.rows_kv, kTile / 2)) {
      *err = "prefix_attn: tensor map encoding failed";
      return cudaErrorInvalidValue;
    }
    const auto attend = pl.g == 2 ? attend_kernel<2> : attend_kernel<1>;
    const uint32_t smem = pl.g == 2 ? kSmemBytes<2> : kSmemBytes<1>;
    e = cudaFuncSetAttribute(attend, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(expand_kernel, dim3(static_cast<unsigned>(pl.rows_kv / kTile)), dim3(kExpandThreads), 0, s, 1, a, pl, ws);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attend, dim3(static_cast<unsigned>(2 * pl.g * items)), dim3(kThreads), smem, s, 2 * pl.g, q_map, tile_map,
                   half_map, a, pl, ws);
    if (e != cudaSuccess) return e;
  }
  if (pl.ns == 1) return cudaSuccess;
  // (one row of 16 heads, 60000 positions: 52 us with 64 parts at most, 32 with 256 and four groups a row)
  if (pl.ns >= 16 && rows <= 2048)
    return launch_pdl(prefix_merge_kernel<4>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, 1, a, pl, ws);
  return launch_pdl(prefix_merge_kernel<1>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, s, 1, a, pl, ws);
}

}  // namespace dsa
