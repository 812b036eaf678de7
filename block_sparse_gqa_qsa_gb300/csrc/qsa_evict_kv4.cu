// qsa_evict_kv4.cu -- eviction from a 4-bit paged cache by accumulated weight
// (qsa_evict_kv4): of a sequence's L tokens every KV head keeps the first
// `sinks`, the last `recent` and, of those between, the ones with the largest
// totals, `budget` in all; their rows move up, in order, in place.
//
// A cluster of CTAs takes one (sequence, head).
// Selection: totals become 32-bit keys of the same order, kept in shared memory
// where a CTA's run of the tokens fits; three passes of digit counts (11, 11, 10
// bits) give the key of the last token kept and how many of the tokens equal to
// it are; a pass in token order writes the list of kept tokens.  A pass's counts
// are summed over the cluster by every CTA for itself, 256 sums of eight digits
// first, then the eight digits of the one that matters: reading all 2048 of 12
// CTAs took 4 to 6 us a pass, adding them up in one CTA 7.
// Moves: kept token i goes to slot i <= its own, so rows move in rounds of the
// cluster: while a round's rows are read into shared memory, nothing that lies
// behind the round's slots is written, and one cluster barrier per round, after
// its reads and before its writes, is all the order that moving in place needs.
// Two more rounds' rows are on their way across it, and the lists and pages of
// two more behind those.  HBM bounds large calls (every moved row is read and
// written once), the chain of passes small ones.
#include <algorithm>
#include <atomic>

#include "qsa_internal.h"
#include "qsa_kv4.cuh"
#include "qsa_paged.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;  // digits of 11 bits
constexpr int kCoarse = 256;  // of 8 digits each
constexpr int kRows = kThreads;  // of a CTA's round, each looked up by a thread: K rows, then as many V rows
constexpr int kChunks = QSA_KV4_ROW_BYTES / 16;
constexpr int kRounds = 3;  // rounds of rows in shared memory
constexpr int kLooked = kRounds + 1;  // rounds whose places are
constexpr int kKeys = 16384;  // tokens of a CTA's run whose keys fit shared memory
constexpr int kMostCluster = 16;

struct EvictArgs {
  uint8_t* pool;
  const int32_t* pageTable;
  const int32_t* ctx;
  const float* total;
  int32_t* kept;
  int32_t* keptLen;
  float* totalOut;  // may be null
  int32_t* status;  // may be null
  int Hkv, rowBytes, numFlatPages, maxPagesPerSeq, totalLen, budget, sinks, recent;
  int cluster;  // CTAs of a cluster
};

struct Shared {
  union {
    struct {
      alignas(16) int counts[3][kBins];  // of each pass's digits in this CTA's run
      int coarse[3][kCoarse];            // and of eight digits each
      uint32_t keys[kKeys];
    };
    alignas(16) uint8_t rows[kRounds][kRows][QSA_KV4_ROW_BYTES];
  };
  int scan[kWarps];
  int found[2];          // a pass's digit, and how many tokens with it are still to be kept
  int above[kWarps], equal[kWarps];  // tokens of each warp's run above and at the last key kept
  int runs[2];           // the CTA's sums of these
  int src[kLooked][kRows];  // pool rows of a round's moves (-1: none)
  int dst[kLooked][kRows];
  float value[kLooked][kRows];  // and their totals
};

// Keys in the order of the totals: whole-number order of the bits of numbers >= 0, reversed below; -0 as 0, NaN lowest.
__device__ __forceinline__ uint32_t key_of_total(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  if (x != x) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int cluster_ld_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(addr));
  return v;
}
__global__ void __launch_bounds__(kThreads, 1) evict_kv4_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, N = a.cluster;
  const int rank = static_cast<int>(blockIdx.x) % N, pair = static_cast<int>(blockIdx.x) / N;
  const int b = pair / a.Hkv, g = pair - b * a.Hkv;
  const int L = min(min(max(a.ctx[b], 0), a.totalLen), a.maxPagesPerSeq * kTokensPerPage), K = min(L, a.budget);
  const float* total = a.total + static_cast<size_t>(pair) * a.totalLen;
  float* totalOut = a.totalOut ? a.totalOut + static_cast<size_t>(pair) * a.totalLen : nullptr;
  int32_t* kept = a.kept + static_cast<size_t>(pair) * a.budget;
  const int step = N * kThreads, own = rank * kThreads + tid;  // places dealt out over the cluster's threads
  if (g == 0 && own == 0) a.keptLen[b] = K;
  for (int i = K + own; i < a.budget; i += step) kept[i] = -1;
  if (L <= a.budget) {  // (the whole cluster) everything stays where it is
    for (int i = own; i < K; i += step) kept[i] = i;
    if (totalOut)
      for (int i = own; i < a.totalLen; i += step) totalOut[i] = i < L ? total[i] : 0.f;
    return;
  }

  // --- selection among the tokens [lo, hi): `need` >= 0 of them, fewer than there are
  const int lo = a.sinks, hi = L - a.recent;
  int need = a.budget - a.sinks - a.recent;
  const int share = ((hi - lo + N - 1) / N + 31) / 32 * 32;  // tokens of a CTA
  const int from = min(hi, lo + rank * share), to = min(hi, from + share);
  uint32_t last = 0;   // key of the last token kept, as far as it is known
  uint32_t known = 0;  // its known bits
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.counts[0][0])[i] = 0;
  const bool held = share <= kKeys;
  if (held)
#pragma unroll 4
    for (int j = from + tid; j < to; j += kThreads) sh.keys[j - from] = key_of_total(total[j]);
  auto key_at = [&](int j) { return held ? sh.keys[j - from] : key_of_total(total[j]); };
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    int* counts = sh.counts[pass];
    const uint32_t mask = pass == 2 ? kBins / 2 - 1 : kBins - 1;
#pragma unroll 4
    for (int j = from + tid; j < to; j += kThreads) {
      const uint32_t k = key_at(j);
      if ((k & known) == last) atomicAdd(counts + (k >> shift & mask), 1);
    }
    __syncthreads();
    if (tid < kCoarse) {
      const int4 x = *reinterpret_cast<const int4*>(counts + 8 * tid), y = *reinterpret_cast<const int4*>(counts + 8 * tid + 4);
      sh.coarse[pass][tid] = (x.x + x.y + x.z + x.w) + (y.x + y.y + y.z + y.w);
    }
    cluster_sync_all();  // all counts of this pass are in
    // the digit, from above, at which the counts reach `need`: thread i < 256 sums the coarse count 255 - i
    int sum = 0;
    if (tid < kCoarse) {
      const uint32_t mine = smem_addr(&sh.coarse[pass][kCoarse - 1 - tid]);
      int n[kMostCluster];
#pragma unroll
      for (int c = 0; c < kMostCluster; ++c) n[c] = c < N ? cluster_ld_int(cluster_addr(mine, c)) : 0;
#pragma unroll
      for (int c = 0; c < kMostCluster; ++c) sum += n[c];
    }
    int all;
    const int before = cta_exclusive_scan<kThreads>(sum, sh.scan, all);
    if (before < need && need <= before + sum) {
      sh.found[0] = kCoarse - 1 - tid;
      sh.found[1] = need - before;
    }
    __syncthreads();
    if (need > 0 && warp == 0) {  // its eight digits: lane l sums digit 7 - l / 4 over every fourth CTA
      const int fine = 8 * sh.found[0] + 7 - (lane >> 2);
      int n = 0;
      for (int c = lane & 3; c < N; c += 4) n += cluster_ld_int(cluster_addr(smem_addr(counts + fine), c));
      n += __shfl_xor_sync(kFull, n, 1);
      n += __shfl_xor_sync(kFull, n, 2);
      int up = 0;  // of the digits above
#pragma unroll
      for (int o = 0; o < 8; ++o) {
        const int x = __shfl_sync(kFull, n, 4 * o);
        up += o < (lane >> 2) ? x : 0;
      }
      const int left = sh.found[1] - up;
      __syncwarp();
      if ((lane & 3) == 0 && left > 0 && left <= n) {
        sh.found[0] = fine;
        sh.found[1] = left;
      }
    }
    __syncthreads();
    if (need > 0) {  // (none to keep: no digit was found)
      last |= static_cast<uint32_t>(sh.found[0]) << shift;
      known |= mask << shift;
      need = sh.found[1];
    }
    __syncthreads();
  }
  const bool none = need <= 0;  // `need` tokens with key `last` are kept, and all above it

  // --- the list of kept tokens, in order: every warp counts its run, then writes it
  const int run = share / kWarps / 32 * 32 + (share / 32 % kWarps ? 32 : 0);  // tokens of a warp, whole rounds of 32
  const int wfrom = min(to, from + warp * run), wto = min(to, wfrom + run);
  int above = 0, equal = 0;
#pragma unroll 4
  for (int j = wfrom + lane; j < wto; j += 32) {
    const uint32_t k = key_at(j);
    above += !none && k > last;
    equal += !none && k == last;
  }
  above = __reduce_add_sync(kFull, above);
  equal = __reduce_add_sync(kFull, equal);
  if (lane == 0) {
    sh.above[warp] = above;
    sh.equal[warp] = equal;
  }
  __syncthreads();
  // lane w < 16: warp w's counts; then lane c: CTA c's
  above = lane < kWarps ? sh.above[lane] : 0;
  equal = lane < kWarps ? sh.equal[lane] : 0;
  if (warp == 0) {
    const int x = __reduce_add_sync(kFull, above), y = __reduce_add_sync(kFull, equal);
    if (lane == 0) {
      sh.runs[0] = x;
      sh.runs[1] = y;
    }
  }
  above = lane < warp ? above : 0;
  equal = lane < warp ? equal : 0;
  cluster_sync_all();  // every CTA's sums are in
  if (lane < rank) {
    const uint32_t runs = cluster_addr(smem_addr(sh.runs), lane);
    above += cluster_ld_int(runs);
    equal += cluster_ld_int(runs + 4);
  }
  above = __reduce_add_sync(kFull, above);  // now: of the tokens before this warp's run
  equal = __reduce_add_sync(kFull, equal);
  for (int j0 = wfrom; j0 < wto; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < wto ? key_at(j) : 0;
    const bool up = !none && j < wto && k > last, eq = !none && j < wto && k == last;
    const unsigned ups = __ballot_sync(kFull, up), eqs = __ballot_sync(kFull, eq), before = (1u << lane) - 1;
    const int eqBefore = equal + __popc(eqs & before);
    if (up || (eq && eqBefore < need)) kept[lo + above + __popc(ups & before) + min(eqBefore, need)] = j;
    above += __popc(ups);
    equal += __popc(eqs);
  }
  for (int i = own; i < a.sinks; i += step) kept[i] = i;
  for (int i = own; i < a.recent; i += step) kept[K - a.recent + i] = hi + i;
  cluster_sync_all();  // the list is written, and no CTA reads another's shared memory any more

  // --- moves
  constexpr int perRound = kRows / 2;  // tokens of a CTA's round
  const int plane = tid / perRound;    // of this thread's row
  const int rounds = (K + N * perRound - 1) / (N * perRound);
  const size_t tokenBytes = static_cast<size_t>(a.Hkv) * a.rowBytes;
  uint8_t* base = a.pool + static_cast<size_t>(g) * a.rowBytes;
  const int32_t* pt = a.pageTable + (static_cast<size_t>(b) * 2 + plane) * a.maxPagesPerSeq;
  bool bad = false;
  auto slot_of = [&](int round) { return (round * N + rank) * perRound + (tid & (perRound - 1)); };
  // The steps of looking a row up, a round apart: the token of a slot; its pages and total; the pool rows, to shared memory.
  struct Looked {
    int token, from, to;
    float value;
  };
  auto token_of = [&](int round) {
    const int i = slot_of(round);
    return i < K ? *static_cast<volatile int32_t*>(kept + i) : -1;
  };
  auto pages_of = [&](int round, int j) {
    Looked x{j, -1, -1, 0.f};
    if (j >= 0) {
      x.from = pt[j >> 7];
      x.to = pt[slot_of(round) >> 7];
      if (plane == 0 && totalOut) x.value = total[j];
    }
    return x;
  };
  auto put = [&](int round, const Looked& x) {
    const int i = slot_of(round), at = round % kLooked;
    const bool moves = x.token >= 0 && x.token != i;
    const bool ok = moves && static_cast<unsigned>(x.from) < static_cast<unsigned>(a.numFlatPages) &&
                    static_cast<unsigned>(x.to) < static_cast<unsigned>(a.numFlatPages);
    bad |= moves && !ok;
    sh.src[at][tid] = ok ? x.from * kTokensPerPage + (x.token & 127) : -1;
    sh.dst[at][tid] = ok ? x.to * kTokensPerPage + (i & 127) : -1;
    sh.value[at][tid] = x.value;
  };
  constexpr int kCopies = kRows * kChunks / kThreads;  // 16-byte pieces of a round per thread
  auto read_rows = [&](int round) {  // one copy group
    const int at = round % kLooked, buf = round % kRounds;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const int e = k * kThreads + tid, r = e / kChunks, c = e - r * kChunks;
      const int src = sh.src[at][r];
      if (src >= 0) cp_async16(smem_addr(&sh.rows[buf][0][0]) + e * 16, base + src * tokenBytes + c * 16, true);
    }
    cp_async_commit();
  };
  auto write_rows = [&](int round) {
    const int at = round % kLooked, buf = round % kRounds;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const int e = k * kThreads + tid, r = e / kChunks, c = e - r * kChunks;
      const int dst = sh.dst[at][r];
      if (dst >= 0)
        *reinterpret_cast<uint4*>(base + dst * tokenBytes + c * 16) = *reinterpret_cast<const uint4*>(&sh.rows[buf][0][0] + e * 16);
    }
    const int i = slot_of(round);
    if (totalOut && plane == 0 && i < K) totalOut[i] = sh.value[at][tid];
  };
  // (a round past the last has no token)
  constexpr int kAhead = kRounds - 1;  // rounds of rows on their way
  int token = token_of(kAhead);
  Looked looked;
#pragma unroll
  for (int round = 0; round < kAhead; ++round) put(round, pages_of(round, token_of(round)));
  looked = pages_of(kAhead, token);
  token = token_of(kAhead + 1);
  __syncthreads();
#pragma unroll
  for (int round = 0; round < kAhead; ++round) read_rows(round);
  for (int round = 0; round < rounds; ++round) {
    put(round + kAhead, looked);
    looked = pages_of(round + kAhead + 1, token);
    token = token_of(round + kAhead + 2);
    __syncthreads();  // the places of round + kAhead are known, round - 1 is written
    read_rows(round + kAhead);
    cp_async_wait<kAhead>();
    cluster_meet();  // every CTA has read this round's rows and totals
    write_rows(round);
  }
  if (totalOut)
    for (int i = K + own; i < a.totalLen; i += step) totalOut[i] = 0.f;  // (every total that is kept has been read)
  if (a.status && __syncthreads_or(bad) && tid == 0) atomicOr(a.status, kErrBadPage);
}

cudaLaunchConfig_t config(long long pairs, int cluster, cudaStream_t st, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = cluster;
  at->val.clusterDim.y = 1;
  at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t allow() {
  cudaError_t e = cudaFuncSetAttribute(evict_kv4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(evict_kv4_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// Clusters of `size` CTAs that the current device holds at once (a cluster's CTAs lie in one GPC), asked for once per device.
int resident_clusters(int size) {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][kMostCluster + 1];  // 0: not asked yet; -1: none
  int dev = 0;
  const bool cached = cudaGetDevice(&dev) == cudaSuccess && dev < kDevices;
  int n = cached ? known[dev][size].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = config(1, size, nullptr, &at);
    if (allow() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, evict_kv4_kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();  // a failed query is not the launch's error: this size is just not used
      n = 0;
    }
    n = n < 1 ? -1 : n;
    if (cached) known[dev][size].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

cudaError_t launch_evict_kv4(const QsaEvictKv4Params& p) {
  EvictArgs a;
  a.pool = static_cast<uint8_t*>(p.kvPool);
  a.pageTable = p.pageTable;
  a.ctx = p.contextLengths;
  a.total = p.total;
  a.kept = p.kept;
  a.keptLen = p.keptLengths;
  a.totalOut = p.totalOut;
  a.status = p.status;
  a.Hkv = p.numKVHeads;
  a.rowBytes = p.poolRowBytes;
  a.numFlatPages = p.numFlatPages;
  a.maxPagesPerSeq = p.maxPagesPerSeq;
  a.totalLen = p.totalLen;
  a.budget = p.budget;
  a.sinks = p.sinks;
  a.recent = p.recent;
  const long long pairs = static_cast<long long>(p.batchSize) * p.numKVHeads;
  // As many CTAs per (sequence, head) as leave all clusters resident at once, with about 512 tokens each at least (1 x 2 heads
  // of 900 tokens 11.7 us, 2 x 4 of 4000 cut to 3500 15.3; with 1024 tokens 14.1 and 18.6, with 256 11.6 and 15.5).
  a.cluster = kMostCluster;
  while (a.cluster > 1 && ((a.cluster - 1) * 512LL >= p.totalLen || pairs > resident_clusters(a.cluster))) --a.cluster;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = config(pairs, a.cluster, static_cast<cudaStream_t>(p.stream), &at);
  // (the attributes are the context's: set with every launch, which costs less than asking whether they are)
  cudaError_t e = allow();
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, evict_kv4_kernel, static_cast<const EvictArgs>(a));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qsa
