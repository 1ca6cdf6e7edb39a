// Eviction from the paged caches by accumulated attention weight: which positions of a sequence stay
// (dsa_evict_select), and their records moved to the sequence's first positions (dsa_evict_compact).
//
// Selection.  A sequence's first `sinks` and last `recent` positions stay; of those between, the rest of the
// budget goes to the largest weights, equal ones to the lower position.  One cluster a sequence, each CTA a run of
// its positions: a radix select in digits of 9 bits, from the highest bit in which the weights differ
// at all, each digit one pass over the run (shared memory, if it fits) into a histogram that all CTAs
// read over distributed shared memory.  It ends as soon as a bin is kept whole.  Two more passes count and
// write, in position order.  The weights are read from memory once.  Bound: latency, three to five digits of a pass, a
// cluster barrier and remote loads each (32 sequences of 16-32K to 2048: 23 us, one of 128K to 64K: 28, for 6 MB and 1 MB
// of weights).  Digits of 8 bits took 82 and 72.
//
// Moving.  A warp copies four tokens' 608-byte records and 132-byte keys in words of 16 bytes, all read before any is
// written.  Bound: memory (32 x 2048 tokens to other pages: 18.5 us, 5.3 TB/s read and written).  In place a token's
// new place may hold another's record that has not been read, so the records go through the workspace, where
// the second kernel mostly finds them in L2 (65536 tokens: 31 us; written once it would be 15, but a block would
// have to wait for the blocks that read what it overwrites).

#include <mutex>

#include "dsa_common.cuh"
#include "dsa_launch.h"

namespace dsa {
namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;  // a bin a thread
constexpr int kAhead = 4;                             // keys of a thread under way together
static_assert(kBins == kSelThreads, "a bin a thread");
constexpr int kCacheKeys = 24 * 1024;  // keys of a CTA held in shared memory: 192 KB
constexpr int kCluster = 8, kWideCluster = 16;

// order-preserving: a larger weight has a larger key
__device__ __forceinline__ uint64_t mass_key(int64_t m) { return static_cast<uint64_t>(m) ^ (1ull << 63); }

struct SelShared {
  unsigned hist[2][kBins];
  uint64_t lo, hi;             // smallest and largest key of the CTA's candidates
  unsigned totals[2];          // the CTA's positions above the threshold, and on it
  unsigned warp[2][kSelWarps];
  unsigned pick[3];            // the digit, the candidates above its bin and in it
};
// CTA r's copy of a shared variable, and the barrier of all CTAs of a sequence.  A launch of one CTA a sequence has
// no cluster: nothing there goes through distributed shared memory.
__device__ __forceinline__ uint64_t peer_u64(const uint64_t* p, int r, int ranks) {
  if (ranks == 1) return *p;
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(dsmem_addr(p, r)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t peer_u32(const unsigned* p, int r, int ranks) {
  if (ranks == 1) return *p;
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(p, r)) : "memory");
  return v;
}
__device__ __forceinline__ void peer_sync(int ranks) {
  if (ranks == 1) __syncthreads();
  else cluster_sync();
}

// MOST: CTAs of a sequence, at most
template <int MOST>
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(EvictSelectArgs a, int ranks, int cached) {
  extern __shared__ __align__(16) uint64_t s_keys[];
  __shared__ SelShared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x / ranks, rank = blockIdx.x % ranks;  // (a cluster is `ranks` consecutive blocks)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.seq_lens[b];
  if (len < 0 || len > a.max_ctx) {
    if (rank == 0 && tid == 0) flag(a.status, DSA_STATUS_BAD_LEN);
    len = 0;
  }
  const int64_t* mass = a.mass + b * a.mass_stride;
  int32_t* kept = a.kept + static_cast<int64_t>(b) * a.budget;
  int64_t* kept_mass = a.kept_mass ? a.kept_mass + static_cast<int64_t>(b) * a.budget : nullptr;
  const int stay = min(len, a.budget);
  if (rank == 0 && tid == 0) a.new_lens[b] = stay;
  for (int i = stay + rank * kSelThreads + tid; i < a.budget; i += ranks * kSelThreads) {
    kept[i] = -1;
    if (kept_mass) kept_mass[i] = 0;
  }
  // the CTA's run of positions, a sub-run of whole warps' steps per warp
  const int sub = ((len + ranks * kSelWarps - 1) / (ranks * kSelWarps) + 31) / 32 * 32;
  const int64_t begin = static_cast<int64_t>(rank) * sub * kSelWarps;
  const int run0 = static_cast<int>(min(begin, static_cast<int64_t>(len)));
  const int run1 = static_cast<int>(min(begin + static_cast<int64_t>(sub) * kSelWarps, static_cast<int64_t>(len)));
  if (len <= a.budget) {  // (the same in every CTA of the cluster)
    for (int p = run0 + tid; p < run1; p += kSelThreads) {
      kept[p] = p;
      if (kept_mass) kept_mass[p] = mass[p];
    }
    return;
  }
  // candidates: [c0, c1); the others stay
  const int c0 = a.sinks, c1 = max(len - a.recent, c0);
  unsigned need = static_cast<unsigned>(a.budget - (len - (c1 - c0)));
  const int q0 = max(run0, c0), q1 = min(run1, c1);  // the CTA's candidates, if q0 < q1
  uint64_t threshold = ~0ull;   // keys above it stay, and the first need_equal of those on it
  unsigned need_equal = 0;
  if (need > 0) {
    // the bits in which keys differ; the run's keys go to shared memory
    uint64_t lo = ~0ull, hi = 0;
    for (int p0 = run0 + tid; p0 < run1; p0 += kAhead * kSelThreads) {
      uint64_t k[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int p = p0 + j * kSelThreads;
        k[j] = p < run1 ? mass_key(mass[p]) : 0;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int p = p0 + j * kSelThreads;
        if (cached && p < run1) s_keys[p - run0] = k[j];
        if (p >= q0 && p < q1) {
          lo = min(lo, k[j]);
          hi = max(hi, k[j]);
        }
      }
    }
    if (tid == 0) {
      sh.lo = ~0ull;
      sh.hi = 0;
    }
    sh.hist[0][tid] = 0;
    __syncthreads();
    for (int o = 16; o; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) {
      atomicMin(reinterpret_cast<unsigned long long*>(&sh.lo), lo);
      atomicMax(reinterpret_cast<unsigned long long*>(&sh.hi), hi);
    }
    peer_sync(ranks);
    for (int r = 0; r < ranks; ++r) {
      lo = min(lo, peer_u64(&sh.lo, r, ranks));
      hi = max(hi, peer_u64(&sh.hi, r, ranks));
    }
    int bits = lo == hi ? 0 : 64 - __clzll(lo ^ hi);  // still to decide
    uint64_t prefix = bits == 64 ? 0 : hi >> bits << bits;
    bool whole = false;
    for (int pass = 0; bits > 0 && !whole; ++pass) {
      const int shift = max(bits - kDigitBits, 0), wide = bits - shift;
      unsigned* hist = sh.hist[pass & 1];
      for (int p0 = q0; p0 < q1; p0 += kAhead * kSelThreads) {
        bool in[kAhead];
        unsigned digit[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int p = p0 + j * kSelThreads + tid;
          in[j] = p < q1;
          const uint64_t k = !in[j] ? 0 : cached ? s_keys[p - run0] : mass_key(mass[p]);
          in[j] = in[j] && (bits == 64 || (k >> bits) == (prefix >> bits));
          digit[j] = static_cast<unsigned>(k >> shift) & ((1u << wide) - 1u);
        }
        // (the digit of a warp's first lane in one addition: positions of no weight all share theirs)
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const unsigned ins = __ballot_sync(0xffffffffu, in[j]);
          if (!ins) continue;
          const int lead = __ffs(ins) - 1;
          const unsigned common = __shfl_sync(0xffffffffu, digit[j], lead);
          const unsigned same = __ballot_sync(0xffffffffu, in[j] && digit[j] == common);
          if (lane == lead) atomicAdd(&hist[common], static_cast<unsigned>(__popc(same)));
          if (in[j] && digit[j] != common) atomicAdd(&hist[digit[j]], 1u);
        }
      }
      peer_sync(ranks);
      // (every CTA has read the other histogram by now)
      sh.hist[(pass + 1) & 1][tid] = 0;
      // the bins of all CTAs from the highest down, one a thread
      const int bin = kBins - 1 - tid;
      unsigned sum = 0;
#pragma unroll
      for (int r = 0; r < MOST; ++r)
        if (r < ranks) sum += peer_u32(hist + bin, r, ranks);
      unsigned before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      if (lane == 31) sh.warp[0][warp] = before;
      __syncthreads();
      before -= sum;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) before += sh.warp[0][w];
      if (before < need && need <= before + sum) {
        sh.pick[0] = bin;
        sh.pick[1] = before;
        sh.pick[2] = sum;
      }
      __syncthreads();
      prefix |= static_cast<uint64_t>(sh.pick[0]) << shift;
      need -= sh.pick[1];
      whole = need == sh.pick[2];
      bits = shift;
    }
    // a bin that is kept whole: everything from its lowest value on
    threshold = whole ? prefix - 1 : prefix;
    need_equal = whole ? 0 : need;
    if (whole && prefix == 0) {  // (nothing lies below it: the bin of the lowest weights, kept whole)
      threshold = 0;
      need_equal = 0xFFFFFFFFu;
    }
  }
  const bool chosen = a.budget > len - (c1 - c0);  // some of the candidates stay, and the keys have been read
  // how many of each warp's sub-run stay: above the threshold, and on it
  const int w0 = static_cast<int>(min(static_cast<int64_t>(run0) + static_cast<int64_t>(warp) * sub, static_cast<int64_t>(run1)));
  const int w1 = static_cast<int>(min(static_cast<int64_t>(w0) + sub, static_cast<int64_t>(run1)));
  auto key_of = [&](int p) { return p >= w1 ? 0ull : cached && chosen ? s_keys[p - run0] : mass_key(mass[p]); };
  auto classify = [&](int p, uint64_t k, bool& above, bool& equal) {
    const bool in = p < w1, candidate = in && p >= c0 && p < c1;
    above = in && (!candidate || k > threshold);
    equal = candidate && k == threshold && need_equal > 0;
  };
  unsigned n_above = 0, n_equal = 0;
  for (int p0 = w0; p0 < w1; p0 += 32 * kAhead) {
    uint64_t k[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) k[j] = key_of(p0 + 32 * j + lane);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      bool above, equal;
      classify(p0 + 32 * j + lane, k[j], above, equal);
      n_above += __popc(__ballot_sync(0xffffffffu, above));
      n_equal += __popc(__ballot_sync(0xffffffffu, equal));
    }
  }
  __syncthreads();
  if (lane == 0) {
    sh.warp[0][warp] = n_above;
    sh.warp[1][warp] = n_equal;
  }
  __syncthreads();
  if (tid < 2) {
    unsigned t = 0;
    for (int w = 0; w < kSelWarps; ++w) t += sh.warp[tid][w];
    sh.totals[tid] = t;
  }
  peer_sync(ranks);
  unsigned above0 = 0, equal0 = 0;
  for (int r = 0; r < rank; ++r) {
    above0 += peer_u32(&sh.totals[0], r, ranks);
    equal0 += peer_u32(&sh.totals[1], r, ranks);
  }
  for (int w = 0; w < warp; ++w) {
    above0 += sh.warp[0][w];
    equal0 += sh.warp[1][w];
  }
  for (int p0 = w0; p0 < w1; p0 += 32 * kAhead) {
    uint64_t k[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) k[j] = key_of(p0 + 32 * j + lane);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int p = p0 + 32 * j + lane;
      bool above, equal;
      classify(p, k[j], above, equal);
      const unsigned am = __ballot_sync(0xffffffffu, above), em = __ballot_sync(0xffffffffu, equal);
      const unsigned below = (1u << lane) - 1u;
      const unsigned ea = equal0 + __popc(em & below), ra = above0 + __popc(am & below);
      const unsigned at = ra + min(ea, need_equal);
      if ((above || (equal && ea < need_equal)) && at < static_cast<unsigned>(a.budget)) {
        kept[at] = p;
        if (kept_mass) kept_mass[at] = static_cast<int64_t>(k[j] ^ (1ull << 63));
      }
      above0 += __popc(am);
      equal0 += __popc(em);
    }
  }
  peer_sync(ranks);  // (no CTA leaves while another may read its totals)
}

// ---- moving --------------------------------------------------------------------------
constexpr int kMoveWarps = 8, kMoveTokens = 4;  // tokens of a warp under way at a time
constexpr int kScratchToken = kKvTokBytes + kIdxDim + 16;  // a token in the workspace: record, codes, scales
constexpr int kRecWords = kKvTokBytes / 16, kKeyWords = kIdxDim / 16;

// slot of position p of sequence b, -1 where its page is out of range
__device__ __forceinline__ int64_t move_slot(const EvictCompactArgs& a, const int32_t* table, int max_pages, int b, int64_t p) {
  if (p < 0 || p >= static_cast<int64_t>(max_pages) * kPage) {
    flag(a.status, DSA_STATUS_BAD_INDEX);
    return -1;
  }
  const int page = table[static_cast<int64_t>(b) * max_pages + p / kPage];
  if (page < 0 || page >= a.num_pages) {
    flag(a.status, DSA_STATUS_BAD_PAGE);
    return -1;
  }
  return static_cast<int64_t>(page) * kPage + p % kPage;
}

// Word w of a token (records first, then the key's codes, then its scales in a word of their own) in
// the caches or the workspace
__device__ __forceinline__ uint8_t* cache_word(const EvictCompactArgs& a, int64_t slot, int w) {
  if (w < kRecWords) return a.kv_cache ? a.kv_cache + slot * kKvTokBytes + 16 * w : nullptr;
  if (!a.k_cache) return nullptr;
  uint8_t* page = a.k_cache + slot / kPage * kKPageBytes;
  if (w < kRecWords + kKeyWords) return page + slot % kPage * kIdxDim + 16 * (w - kRecWords);
  return page + kKScaleOff + slot % kPage * 4;
}

// MODE 0: from the caches to the caches (other pages); 1: to the workspace; 2: from it
template <int MODE>
__global__ void __launch_bounds__(kMoveWarps * 32)
evict_move_kernel(EvictCompactArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t tokens = static_cast<int64_t>(a.n_seq) * a.budget;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5)) * kMoveTokens;
  // lane k works out token k's slots
  int64_t src = -1, dst = -1;
  if (lane < kMoveTokens && t0 + lane < tokens) {
    const int b = static_cast<int>((t0 + lane) / a.budget), i = static_cast<int>((t0 + lane) % a.budget);
    const int p = a.kept[t0 + lane];
    if (p != -1 && (MODE == 0 || p != i)) {
      src = MODE == 2 ? 0 : move_slot(a, a.page_table, a.max_pages, b, p);
      dst = MODE == 1 ? 0 : move_slot(a, a.dst_table, a.dst_max_pages, b, i);
      if (MODE == 2 && move_slot(a, a.page_table, a.max_pages, b, p) < 0) src = -1;  // (nothing was read)
    }
  }
  uint4 v[kMoveTokens][2];
  int64_t to[kMoveTokens];
#pragma unroll
  for (int k = 0; k < kMoveTokens; ++k) {
    const int64_t from = __shfl_sync(0xffffffffu, src, k);
    to[k] = __shfl_sync(0xffffffffu, dst, k);
    if (from < 0) to[k] = -1;
    if (to[k] < 0) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int w = lane + 32 * j;
      if (w > kRecWords + kKeyWords) continue;
      const uint8_t* at = cache_word(a, from, w);
      if (!at) continue;
      if (MODE == 2) at = a.workspace + (t0 + k) * kScratchToken + 16 * w;
      if (w == kRecWords + kKeyWords) v[k][j].x = *reinterpret_cast<const uint32_t*>(at);
      else v[k][j] = *reinterpret_cast<const uint4*>(at);
    }
  }
#pragma unroll
  for (int k = 0; k < kMoveTokens; ++k) {
    if (to[k] < 0) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int w = lane + 32 * j;
      if (w > kRecWords + kKeyWords) continue;
      uint8_t* at = cache_word(a, to[k], w);
      if (!at) continue;
      if (MODE == 1) at = a.workspace + (t0 + k) * kScratchToken + 16 * w;
      if (w == kRecWords + kKeyWords) *reinterpret_cast<uint32_t*>(at) = v[k][j].x;
      else *reinterpret_cast<uint4*>(at) = v[k][j];
    }
  }
}

// Clusters of sixteen CTAs, each with all the shared memory that one may take, that fit on the current device at once;
// asked once a device.
int wide_clusters() {
  static std::mutex mu;
  static int known[64] = {};  // the answer and one
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] > 0) return known[dev] - 1;
  const int smem = kCacheKeys * static_cast<int>(sizeof(uint64_t));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kWideCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kWideCluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(evict_select_kernel<kWideCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(evict_select_kernel<kWideCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, evict_select_kernel<kWideCluster>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  known[dev] = n + 1;
  return n;
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectArgs& a, cudaStream_t s) {
  // A CTA for each 2048 positions while all sequences' fit two to an SM, at most eight a sequence; sixteen where
  // such clusters fit for all sequences at once (one of 128K: 35 us with eight)
  int ranks = 1;
  while (ranks < kCluster && ranks * 2048 < a.max_ctx &&
         static_cast<int64_t>(a.n_seq) * ranks * 2 <= static_cast<int64_t>(multiprocessors()) * 2)
    ranks *= 2;
  // (a kernel of its own: with one for both, 32 sequences of 32K took 30 us instead of 23)
  const bool wide = ranks == kCluster && kCluster * 2048 < a.max_ctx && a.n_seq <= wide_clusters();
  if (wide) ranks = kWideCluster;
  const int run = ((a.max_ctx + ranks * kSelWarps - 1) / (ranks * kSelWarps) + 31) / 32 * 32 * kSelWarps;
  const int cached = run <= kCacheKeys;
  const size_t smem = cached ? sizeof(uint64_t) * run : 0;
  const auto kernel = wide ? evict_select_kernel<kWideCluster> : evict_select_kernel<kCluster>;
  if (smem > 0 && !wide) {  // (the wide one's is set)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kCacheKeys * static_cast<int>(sizeof(uint64_t)));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(a.n_seq) * ranks), dim3(kSelThreads), smem, s, ranks, a, ranks, cached);
}

size_t evict_workspace_bytes(int n_seq, int budget) {
  return static_cast<size_t>(n_seq) * static_cast<size_t>(budget) * kScratchToken;
}

cudaError_t launch_evict_compact(const EvictCompactArgs& a, cudaStream_t s) {
  const int64_t tokens = static_cast<int64_t>(a.n_seq) * a.budget;
  const dim3 grid(static_cast<unsigned>((tokens + kMoveWarps * kMoveTokens - 1) / (kMoveWarps * kMoveTokens)));
  const dim3 block(kMoveWarps * 32);
  if (a.dst_table != a.page_table) return launch_pdl(evict_move_kernel<0>, grid, block, 0, s, 1, a);
  const cudaError_t e = launch_pdl(evict_move_kernel<1>, grid, block, 0, s, 1, a);
  return e != cudaSuccess ? e : launch_pdl(evict_move_kernel<2>, grid, block, 0, s, 1, a);
}

}  // namespace dsa
