// qsa_weights_kv4.cu -- the attention weights of list entries over a 4-bit
// paged pool, and what every cached token has gathered of them
// (qsa_sparse_weights_kv4): for row t, KV head g and entry e naming token j
//
//   w[e] = sum_h exp(scale q_h . k_j - lse_h),   total[j] += sum of w over rows and entries.
//
// With the attention's log-sum-exp every weight stands alone: a warp takes 32
// entries, gathers their K rows, forms S^T = K Q^T as the attention does, and
// sums 2^(x - lse) over the heads of its rows with two shuffles.  K rows and
// lists are read once, weights written once: latency bounds a decode step
// (list -> pages -> rows), so the list is cut into as many warps as fill the
// GPU, two tiles each.
//
// Totals.  With one row per sequence a token is added to once per entry that
// names it (equal addends if twice), so the order of the atomic adds does not
// show.  With several rows the sums go through a second kernel, in which a CTA
// owns a range of a (sequence, head)'s tokens and walks the rows in order, a
// barrier between them: a token's atomic adds come in the order of the rows,
// whatever runs first, and give what a call per row would.
#include <algorithm>

#include "qsa_paged_kv4.cuh"

namespace qsa {
namespace {

constexpr int kThreads = kPagedThreads;
constexpr int kWarps = kPagedWarps;
constexpr int kTileBytes = kKv4CodeBytes + kKv4ScaleBytes;
constexpr int kWarpBytes = 2 * kTileBytes + 2 * kStep * 4;  // two tiles, two steps' row ids

struct WeightArgs {
  PagedArgs a;
  const float* lse;
  float* weights;
  float* total;  // may be null; only with one row per sequence
  int totalLen;
  int steps;  // of a warp
};

template <int NT, bool kBf16>
__global__ void __launch_bounds__(kThreads) sparse_weights_kv4_kernel(const WeightArgs w) {
  const PagedArgs& a = w.a;
  // Groups of up to 8 heads: every warp has the queries to itself and waits for no other (decode of 32 sequences 9.1 us, 10.2
  // with shared ones); larger ones share them (window of 37 rows 26.1 us, 27.4 with its own).
  constexpr bool kShared = NT > 1;
  __shared__ __align__(128) uint8_t smem[kWarps * kWarpBytes + (kShared ? 1 : kWarps) * kKv4QueryBytes<NT>];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Row r = row_of(a, static_cast<int>(blockIdx.x), 1);
  List list(a, r);
  // this warp's run of the list
  const int first = (static_cast<int>(blockIdx.y) * kWarps + warp) * w.steps * kStep;
  const int count = max(0, min(w.steps, (a.topK - first + kStep - 1) / kStep));
  if (!kShared && count == 0) return;
  int j0 = list.at(first + lane), j1 = count > 1 ? list.at(first + kStep + lane) : -1;
  row_lengths(a, r);
  list.L = r.L;
  float* out = w.weights + (r.bt * a.Hkv + r.kvh) * a.topK;
  if (r.t >= r.n) {
    for (int e = first + lane; e < min(first + count * kStep, a.topK); e += 32) out[e] = 0.f;
    return;
  }
  const uint32_t tiles = smem_addr(smem + warp * kWarpBytes);
  int* ids = reinterpret_cast<int*>(smem + warp * kWarpBytes + 2 * kTileBytes);
  const uint32_t rowBytes = static_cast<uint32_t>(a.Hkv) * a.poolHeadDim;
  const uint8_t* base = a.pool + static_cast<size_t>(r.kvh) * a.poolHeadDim;
  auto gather = [&](const Pages& p, int par) {
    const PoolRows rows = list.rows_of(p);
    int* at = ids + par * kStep;
    at[kv4_row_place(lane)] = rows.ok ? rows.k : -1;
    const unsigned mask = __ballot_sync(kFull, rows.ok);
    __syncwarp();
    if (mask) {
      const uint32_t tile = tiles + par * kTileBytes;
      kv4_copy_codes<true>(at, mask, tile + lane * 16, base + (lane & 3) * 16, rowBytes);
      kv4_copy_scales(rows.ok ? rows.k : -1, tile + kKv4CodeBytes + kv4_k_scale(lane) * kKv4Chunk, base, rowBytes);
    }
    cp_async_commit();
    return mask;
  };
  unsigned cur = gather(list.pages_of(j0), 0);
  Pages p1 = list.pages_of(j1);
  int j2 = count > 2 ? list.at(first + 2 * kStep + lane) : -1;
  const uint32_t queries = smem_addr(smem + kWarps * kWarpBytes + (kShared ? 0 : warp * kKv4QueryBytes<NT>));
  float qs[NT][2], l2[NT][2];
  kv4_load_q<NT, kBf16, kShared>(static_cast<const uint4*>(a.q) + r.head0 * (kD / 8), a.G, queries, qs);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // heads past the group, and heads without tokens, weigh 0
      const int h = 8 * nt + 2 * (lane & 3) + j;
      const float l = h < a.G ? __ldg(w.lse + r.head0 + h) : INFINITY;
      l2[nt][j] = l == -INFINITY ? INFINITY : l * kLog2e;
    }
  if constexpr (kShared)
    __syncthreads();  // the queries are in place
  else
    __syncwarp();
  const int q = lane & 3, key = kv4_first_key(lane), mine = key + q;  // the entry whose sum this lane keeps
  for (int i = 0; i < count; ++i) {
    const int par = i & 1;
    const unsigned next = gather(p1, par ^ 1);
    const int jn = j1;
    j1 = j2;
    p1 = list.pages_of(j2);
    j2 = i + 3 < count ? list.at(first + (i + 3) * kStep + lane) : -1;
    float v = 0.f;
    if (cur) {
      const uint32_t tile = tiles + par * kTileBytes;
      float s[2][NT][4];
      cp_async_wait<1>();
      __syncwarp();
      kv4_scores<NT>(s, tile, tile + kKv4CodeBytes, queries);
      float sum[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float tk;
        asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(tk) : "r"(tile + kKv4CodeBytes + kv4_k_scale(key + k) * kKv4Chunk + 8));
        const float ks = read_scale(tk) * a.sl2;
        sum[k] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = s[k >> 1][nt][2 * (k & 1) + j];
            sum[k] += ex2_ftz(kBf16 ? fmaf(x * ks, qs[nt][j], -l2[nt][j]) : fmaf(x, ks, -l2[nt][j]));
          }
        sum[k] += __shfl_xor_sync(kFull, sum[k], 1);
        sum[k] += __shfl_xor_sync(kFull, sum[k], 2);
      }
      v = cur >> mine & 1 ? (q == 0 ? sum[0] : q == 1 ? sum[1] : q == 2 ? sum[2] : sum[3]) : 0.f;
      __syncwarp();  // every lane is done with the tile
    }
    const int e = first + i * kStep + mine, j = __shfl_sync(kFull, j0, mine);
    if (e < a.topK) out[e] = v;
    if (w.total && (cur >> mine & 1) && j < w.totalLen)
      atomicAdd(w.total + (static_cast<size_t>(r.b) * a.Hkv + r.kvh) * w.totalLen + j, v);
    j0 = jn;
    cur = next;
  }
  cp_async_wait<0>();
  list.report();
}

// total += the weights of a sequence's rows, one row after the other, for the tokens [lo, lo + range) of a (sequence, head).
// Every CTA reads the rows' lists; weights only where they count.  What bounds it is a row's chain of instructions from one
// barrier to the next, 0.3 us (37 rows of 3 sequences of up to 24001 tokens: the call 24.7 us, this kernel 13 of it, issue
// slots 38 % busy; more rows on their way, in registers or through shared memory, change nothing).  A tile of rows x tokens,
// filled by asynchronous copies and added column by column, took 24.4 us for that call and 25 instead of 31 for 64 rows of a
// sequence of 8000 tokens, but 84 instead of 37 for 4 rows of each of 32 sequences of 65536.
constexpr int kSumThreads = 512;
constexpr int kPer = 5;    // entries of a thread that are loaded ahead:
constexpr int kLists = 4;  // rows ahead their tokens,
constexpr int kSums = 2;   // rows ahead the weights of those in the range

struct SumArgs {
  const int32_t* indices;
  const int32_t* ctx;
  const int32_t* newLen;
  const float* weights;
  float* total;
  int S, Hkv, topK, totalLen, range;
};

__global__ void __launch_bounds__(kSumThreads) sum_weights_kernel(const SumArgs a) {
  const int b = blockIdx.x / a.Hkv, g = blockIdx.x - b * a.Hkv, lo = blockIdx.y * a.range;
  const int L = max(0, a.ctx[b]), n = max(0, min(a.newLen ? a.newLen[b] : a.S, min(a.S, L)));
  const int range = min(a.range, min(L, a.totalLen) - lo);
  if (range <= 0) return;
  const int32_t* list = a.indices + static_cast<size_t>(b) * a.S * a.topK;
  const float* weight = a.weights + (static_cast<size_t>(b) * a.S * a.Hkv + g) * a.topK;
  const size_t hop = static_cast<size_t>(a.Hkv) * a.topK;
  float* total = a.total + (static_cast<size_t>(b) * a.Hkv + g) * a.totalLen + lo;
  auto mine = [&](int j) { return static_cast<unsigned>(j) - static_cast<unsigned>(lo) < static_cast<unsigned>(range); };
  int j[kLists][kPer];
  float w[kSums][kPer];
  auto load_tokens = [&](int t, int (&jt)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = threadIdx.x + k * kSumThreads;
      jt[k] = t < n && e < a.topK ? __ldg(list + static_cast<size_t>(t) * a.topK + e) : -1;
    }
  };
  auto load_weights = [&](int t, const int (&jt)[kPer], float (&wt)[kPer]) {  // (those of entries that name nothing are 0)
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (mine(jt[k])) wt[k] = __ldg(weight + t * hop + threadIdx.x + k * kSumThreads);
  };
#pragma unroll
  for (int i = 0; i < kLists; ++i) load_tokens(i, j[i]);
#pragma unroll
  for (int i = 0; i < kSums; ++i) load_weights(i, j[i], w[i]);
  for (int t0 = 0; t0 < n; t0 += kLists)
#pragma unroll
    for (int i = 0; i < kLists; ++i) {
      const int t = t0 + i;
      __syncthreads();  // the adds of the rows before this one come first
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (mine(j[i][k])) atomicAdd(total + (j[i][k] - lo), w[i % kSums][k]);
      load_tokens(t + kLists, j[i]);
      load_weights(t + kSums, j[(i + kSums) % kLists], w[i % kSums]);
      if (t < n)
        for (int e = threadIdx.x + kPer * kSumThreads; e < a.topK; e += kSumThreads) {
          const int more = __ldg(list + static_cast<size_t>(t) * a.topK + e);
          if (mine(more)) atomicAdd(total + (more - lo), __ldg(weight + t * hop + e));
        }
    }
}

template <int NT, bool kBf16>
cudaError_t weights_go(WeightArgs w, unsigned pairs, cudaStream_t st) {
  // Two steps a warp (one on its way while the other is computed) where that gives every SM the warps it holds (7 CTAs;
  // larger groups 5, and a few more for rows that end early); more where there are more pairs, so that one wave does (64
  // sequences of 4 heads 14.1 us with 4 steps, 15.6 with 5; 200 42.8 with 13, 44.6 with 16), up to 16 (2000 rows 916 us, with
  // 32 935).
  const long long steps = (w.a.topK + kStep - 1) / kStep, warps = (NT == 1 ? 28LL : 24LL) * sm_count();
  long long per = std::max(2LL, std::min(16LL, (pairs * steps + warps - 1) / warps));
  per = std::max(per, (steps + 32767) / 32768);
  w.steps = static_cast<int>(std::min(per, steps));
  const unsigned parts = static_cast<unsigned>((steps + w.steps * kWarps - 1) / (w.steps * kWarps));
  sparse_weights_kv4_kernel<NT, kBf16><<<dim3(pairs, parts), kThreads, 0, st>>>(w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sparse_weights_kv4(const QsaSparseWeightsKv4Params& p, bool bf16) {
  WeightArgs w;
  PagedArgs& a = w.a;
  a.q = p.qPtr;
  a.pool = static_cast<const uint8_t*>(p.kvPool);
  a.scale = nullptr;
  a.pageTable = p.pageTable;
  a.indices = p.indices;
  a.ctx = p.contextLengths;
  a.newLen = p.newLengths;
  a.o = nullptr;
  a.status = p.status;
  a.S = p.seqLen;
  a.Hq = p.numQHeads;
  a.Hkv = p.numKVHeads;
  a.G = p.numQHeads / p.numKVHeads;
  a.poolHeadDim = p.poolRowBytes;
  a.numFlatPages = p.numFlatPages;
  a.maxPagesPerSeq = p.maxPagesPerSeq;
  a.topK = p.topK;
  a.blockShift = 0;
  a.split = 1;
  a.sl2 = p.attentionScale * kLog2e;
  a.lse = nullptr;
  w.lse = p.lse;
  w.weights = p.weights;
  w.total = p.seqLen == 1 ? p.total : nullptr;
  w.totalLen = p.totalLen;
  const unsigned pairs = static_cast<unsigned>(static_cast<long long>(p.batchSize) * p.seqLen * p.numKVHeads);
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  cudaError_t e;
  if (bf16)
    e = a.G <= 8 ? weights_go<1, true>(w, pairs, st) : weights_go<2, true>(w, pairs, st);
  else
    e = a.G <= 8 ? weights_go<1, false>(w, pairs, st) : weights_go<2, false>(w, pairs, st);
  if (e != cudaSuccess || p.seqLen == 1 || !p.total) return e;
  // Ranges of 1024 to 8192 tokens, as many as give every SM two CTAs.
  const long long both = static_cast<long long>(p.batchSize) * p.numKVHeads;
  long long range = (p.totalLen * both / (2LL * sm_count()) + 255) / 256 * 256;
  range = std::max(1024LL, std::min(8192LL, range));
  SumArgs s{p.indices, p.contextLengths, p.newLengths, p.weights, p.total, p.seqLen, p.numKVHeads, p.topK, p.totalLen,
            static_cast<int>(range)};
  const unsigned ranges = static_cast<unsigned>((p.totalLen + range - 1) / range);
  sum_weights_kernel<<<dim3(static_cast<unsigned>(both), ranges), kSumThreads, 0, st>>>(s);
  return cudaGetLastError();
}

}  // namespace qsa
