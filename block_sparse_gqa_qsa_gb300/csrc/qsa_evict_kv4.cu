// qsa_evict_kv4.cu -- eviction from a 4-bit paged cache by accumulated weight
// (qsa_evict_kv4): of a sequence's L tokens every KV head keeps the first
// `sinks`, the last `recent` and, of those between, the ones with the largest
// totals, `budget` in all; their rows move up, in order, in place.
//
// A cluster of CTAs takes one (sequence, head).
// Selection: totals as 32-bit keys of the same order; three passes of digit
// counts (11, 11, 10 bits), each CTA over its run of the tokens, joined in the
// first CTA's shared memory, give the key of the last token kept and how many
// of the tokens equal to it are; a pass in token order writes the list of kept
// tokens.
// Moves: kept token i goes to slot i <= its own, so rows move in rounds of the
// cluster: while a round's rows are read into shared memory, nothing that lies
// behind the round's slots is written, and one cluster barrier per round, after
// its reads and before its writes, is all the order that moving in place needs;
// the next round's reads are on their way across it.  HBM bounds large calls
// (every moved row is read and written once), the chain of passes small ones.
#include <algorithm>
#include <atomic>

#include "qsa_internal.h"
#include "qsa_kv4.cuh"
#include "qsa_paged.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kRows = 256;  // of a CTA's round: thread i of the lower half looks up K row i, of the upper half V row i
constexpr int kChunks = QSA_KV4_ROW_BYTES / 16;
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
      int joined[3][kBins];  // of the cluster's first CTA: digit counts of each pass over all CTAs
      int counts[kBins];     // this CTA's
    };
    alignas(16) uint8_t rows[2][2][kRows][QSA_KV4_ROW_BYTES];  // of two rounds, K and V
  };
  int scan[kWarps];
  int found[2];          // a pass's digit, and how many tokens with it are still to be kept
  int above[kWarps], equal[kWarps];  // tokens of each warp's run above and at the last key kept
  int runs[2];           // the CTA's sums of these
  int src[3][2][kRows];  // pool rows of a round's moves (-1: none), K and V
  int dst[3][2][kRows];
  float value[3][kRows];  // and their totals
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
__device__ __forceinline__ void cluster_add(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kThreads) evict_kv4_kernel(const EvictArgs a) {
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
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.joined[0][0])[i] = 0;
  cluster_sync_all();  // the first CTA's counts are zero
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? kBins / 2 : kBins;
    for (int i = tid; i < bins; i += kThreads) sh.counts[i] = 0;
    __syncthreads();
    for (int j = from + tid; j < to; j += kThreads) {
      const uint32_t k = key_of_total(total[j]);
      if ((k & known) == last) atomicAdd(&sh.counts[k >> shift & (bins - 1)], 1);
    }
    __syncthreads();
    const uint32_t joined = cluster_addr(smem_addr(sh.joined[pass]), 0);
    for (int i = tid; i < bins; i += kThreads)
      if (sh.counts[i]) cluster_add(joined + 4 * i, sh.counts[i]);
    cluster_sync_all();  // all counts of this pass are in
    // the digit at which the counts from above reach `need`
    const int per = bins / kThreads, top = bins - 1 - tid * per;  // this thread's digits: top, top - 1, ..
    int c[kBins / kThreads], sum = 0;
#pragma unroll
    for (int k = 0; k < kBins / kThreads; ++k) {
      c[k] = k < per ? cluster_ld_int(joined + 4 * max(top - k, 0)) : 0;
      sum += c[k];
    }
    int all;
    int before = cta_exclusive_scan<kThreads>(sum, sh.scan, all);
    if (before < need && need <= before + sum)
#pragma unroll
      for (int k = 0; k < kBins / kThreads; ++k) {
        if (before < need && need <= before + c[k]) {
          sh.found[0] = top - k;
          sh.found[1] = need - before;
        }
        before += c[k];
      }
    __syncthreads();
    if (need > 0) {  // (none to keep: no digit was found)
      last |= static_cast<uint32_t>(sh.found[0]) << shift;
      known |= static_cast<uint32_t>(bins - 1) << shift;
      need = sh.found[1];
    }
    __syncthreads();
  }
  const bool none = need <= 0;  // `need` tokens with key `last` are kept, and all above it

  // --- the list of kept tokens, in order: every warp counts its run, then writes it
  const int run = share / kWarps / 32 * 32 + (share / 32 % kWarps ? 32 : 0);  // tokens of a warp, whole rounds of 32
  const int wfrom = min(to, from + warp * run), wto = min(to, wfrom + run);
  int above = 0, equal = 0;
  for (int j = wfrom + lane; j < wto; j += 32) {
    const uint32_t k = key_of_total(total[j]);
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
  if (tid == 0) {
    int x = 0, y = 0;
    for (int w = 0; w < kWarps; ++w) {
      x += sh.above[w];
      y += sh.equal[w];
    }
    sh.runs[0] = x;
    sh.runs[1] = y;
  }
  cluster_sync_all();  // every CTA's sums are in
  above = equal = 0;   // now: of the tokens before this warp's run
  for (int c = 0; c < rank; ++c) {
    const uint32_t runs = cluster_addr(smem_addr(sh.runs), c);
    above += cluster_ld_int(runs);
    equal += cluster_ld_int(runs + 4);
  }
  for (int w = 0; w < warp; ++w) {
    above += sh.above[w];
    equal += sh.equal[w];
  }
  for (int j0 = wfrom; j0 < wto; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < wto ? key_of_total(total[j]) : 0;
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
  const int rounds = (K + N * kRows - 1) / (N * kRows);
  const size_t tokenBytes = static_cast<size_t>(a.Hkv) * a.rowBytes;
  uint8_t* base = a.pool + static_cast<size_t>(g) * a.rowBytes;
  const int half = tid / kRows, row = tid % kRows;
  const int32_t* pt = a.pageTable + (static_cast<size_t>(b) * 2 + half) * a.maxPagesPerSeq;
  bool bad = false;
  auto look_up = [&](int round) {
    const int i = (round * N + rank) * kRows + row, at = round % 3;
    int src = -1, dst = -1;
    if (i < K) {
      const int j = *static_cast<volatile int32_t*>(kept + i);
      if (half == 0) sh.value[at][row] = total[j];
      if (j != i) {
        const int from = pt[j >> 7], to = pt[i >> 7];
        if (static_cast<unsigned>(from) < static_cast<unsigned>(a.numFlatPages) &&
            static_cast<unsigned>(to) < static_cast<unsigned>(a.numFlatPages)) {
          src = from * kTokensPerPage + (j & 127);
          dst = to * kTokensPerPage + (i & 127);
        } else {
          bad = true;
        }
      }
    }
    sh.src[at][half][row] = src;
    sh.dst[at][half][row] = dst;
  };
  auto read_rows = [&](int round) {  // one copy group
    const int at = round % 3, buf = round & 1;
#pragma unroll
    for (int k = 0; k < 2 * kRows * kChunks / kThreads; ++k) {
      const int e = k * kThreads + tid, r = e / kChunks, c = e - r * kChunks;  // r: K rows, then V rows
      const int src = (&sh.src[at][0][0])[r];
      if (src >= 0) cp_async16(smem_addr(&sh.rows[buf][0][0][0]) + e * 16, base + src * tokenBytes + c * 16, true);
    }
    cp_async_commit();
  };
  auto write_rows = [&](int round) {
    const int at = round % 3, buf = round & 1;
#pragma unroll
    for (int k = 0; k < 2 * kRows * kChunks / kThreads; ++k) {
      const int e = k * kThreads + tid, r = e / kChunks, c = e - r * kChunks;
      const int dst = (&sh.dst[at][0][0])[r];
      if (dst >= 0)
        *reinterpret_cast<uint4*>(base + dst * tokenBytes + c * 16) = *reinterpret_cast<const uint4*>(&sh.rows[buf][0][0][0] + e * 16);
    }
    const int i = (round * N + rank) * kRows + row;
    if (totalOut && half == 0 && i < K) totalOut[i] = sh.value[at][row];
  };
  look_up(0);
  __syncthreads();
  read_rows(0);
  for (int round = 0; round < rounds; ++round) {
    if (round + 1 < rounds) look_up(round + 1);
    __syncthreads();  // the next round's rows are known, and the one before this is written
    if (round + 1 < rounds)
      read_rows(round + 1);
    else
      cp_async_commit();
    cp_async_wait<1>();
    cluster_sync_all();  // every CTA has read this round's rows and totals
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

// The largest cluster, up to 16, that the current device takes; asked for once per device.
int most_cluster() {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices];  // 0: not asked yet
  int dev = 0;
  const bool cached = cudaGetDevice(&dev) == cudaSuccess && dev < kDevices;
  int n = cached ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    n = 8;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = config(1, kMostCluster, nullptr, &at);
    int fit = 0;
    if (allow() == cudaSuccess && cudaOccupancyMaxActiveClusters(&fit, evict_kv4_kernel, &cfg) == cudaSuccess && fit > 0)
      n = kMostCluster;
    (void)cudaGetLastError();  // a failed query is not the launch's error: this size is just not used
    if (cached) known[dev].store(n, std::memory_order_relaxed);
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
  // As many CTAs per (sequence, head) as about fill the GPU, with at least 1024 tokens each.
  a.cluster = most_cluster();
  while (a.cluster > 1 && (pairs * a.cluster > 2LL * sm_count() || (a.cluster - 1) * 1024LL >= p.totalLen)) a.cluster /= 2;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = config(pairs, a.cluster, static_cast<cudaStream_t>(p.stream), &at);
  // (the attributes are the context's: set with every launch, which costs less than asking whether they are)
  cudaError_t e = allow();
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, evict_kv4_kernel, static_cast<const EvictArgs>(a));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qsa
