// qsa_attention_kv4.cu -- sparse GQA attention over a 4-bit paged cache
// (qsa_sparse_paged_kv4): for every live row and query head
//
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = tk_j s^K_j c^K_j,  v_j = tv_j s^V_j c^V_j
//
// over the row's list, with e2m1 codes c, an e4m3 scale s per 16 dims and an
// fp32 scale t per row.  The softmax is that of the 8-bit pool with the row
// scales in the place of its block scales (qsa_paged.cuh): tv_j rides in the
// exponent, and one pass keeps a maximum, a sum and O.
//
// Two kernels share the arithmetic.  With few (row, KV head) pairs, a CTA of 4
// warps takes one, or a cluster of up to 8 CTAs shares it, the list dealt out
// to the warps in steps of 32 entries; with many, a CTA takes four KV heads of a
// row, a warp each, and resolves a list once for its heads.
// A warp runs its steps by itself: the 32 K and V rows of 80 bytes are gathered
// with cp.async into its own tiles, the K rows' codes together with both rows'
// scale chunks, the V rows' codes after them.
//
// S^T = K Q^T and O^T += V^T P^T are m16n8k16 MMAs in fp16 with the head group
// as N.  For the second, ldmatrix transposes 16 x 16 bytes, so a register holds
// four keys of one byte column, i.e. of two dims: its low codes are row g of an
// MMA tile, its high codes row g + 8, and a tile's 16 dims are one scale group.
// Two registers, 16 keys apart, are paired key by key with two shifts and two
// selections for 16 codes; S^T has its rows in the order that makes P's pairs the
// same ones.  The V scales are transposed the same way once per step and read
// back as f16 pairs of keys.
#include <algorithm>
#include <atomic>

#include "qsa_paged_kv4.cuh"

namespace qsa {
namespace {

constexpr int kThreads = kPagedThreads;
constexpr int kWarps = kPagedWarps;
// A warp's tile set: K codes, V codes, K scale chunks, V scale chunks of a step's rows.
constexpr int kVAt = kKv4CodeBytes;
constexpr int kKScaleAt = 2 * kKv4CodeBytes;
constexpr int kVScaleAt = kKScaleAt + kKv4ScaleBytes;
constexpr int kSetBytes = kVScaleAt + kKv4ScaleBytes;
// A warp's shared memory in the split form: two tile sets, the V scales of the current step by group, the values of its
// entries, the pool rows of two steps' entries (K then V).
constexpr int kGroupsAt = 2 * kSetBytes;
constexpr int kEntriesAt = kGroupsAt + kKv4ScaleBytes;
constexpr int kRowsAt = kEntriesAt + kStep * 8;
constexpr int kWarpBytes = kRowsAt + 2 * 2 * kStep * 4;
// (behind the warps' tiles: the pair's queries)

// What the softmax needs of an entry (see softmax32), from the scale chunks' row scales.
__device__ __forceinline__ float2 entry_of(const PagedArgs& a, bool ok, uint32_t kscale, uint32_t vscale) {
  const int lane = threadIdx.x & 31;
  float tk, tv;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(tk) : "r"(kscale + kv4_k_scale(lane) * kKv4Chunk + 8));
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(tv) : "r"(vscale + lane * kKv4Chunk + 8));
  tv = read_scale(tv);
  return ok ? make_float2(read_scale(tk) * a.sl2, lg2_ftz(tv)) : make_float2(0.f, -INFINITY);
}

// A step's V scales by group: piece 4 j + q of `groups` gets group j's scales of keys 4 q + i and 4 q + i + 16, i = 0..3, as
// f16 pairs.
// (Columns 8 and on of the scale chunks, the row scales, are dropped.)
__device__ __forceinline__ void transpose_scales(uint32_t vscale, uint32_t groups) {
  const int lane = threadIdx.x & 31;
  uint32_t r[4], p[4];
  ldsm_bytes_t(vscale + lane * kKv4Chunk, r);
  e4m3_to_f16(__byte_perm(r[0], r[2], 0x5140), p[0], p[1]);
  e4m3_to_f16(__byte_perm(r[0], r[2], 0x7362), p[2], p[3]);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(groups + lane * 16), "r"(p[0]), "r"(p[1]), "r"(p[2]),
               "r"(p[3])
               : "memory");
}

// O^T += V^T P^T.  Tile j holds dims 16 j + 2 g (rows g) and 16 j + 2 g + 1 (rows g + 8).
template <int NT>
__device__ __forceinline__ void values32(Acc<NT>& A, uint32_t codes, uint32_t groups, const uint32_t (&pb)[2][NT][2]) {
  const int lane = threadIdx.x & 31;
  const uint32_t row = codes + lane * kKv4Codes + ((lane >> 1 & 3) << 4);
  uint32_t next[4];
  ldsm_bytes_t(row, next);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint32_t r[4] = {next[0], next[1], next[2], next[3]};
    if (m < 3) ldsm_bytes_t(row ^ ((m + 1) << 4), next);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 sc = lds16(groups + (4 * (2 * m + c) + (lane & 3)) * 16);
      constexpr uint32_t kLow = 0x0f0f0f0f;
      uint32_t lo[4], hi[4];  // of keys 4 q + i and 4 q + i + 16
      e2m1_to_f16((r[c] & kLow) | (r[2 + c] << 4 & ~kLow), lo[0], lo[1], lo[2], lo[3]);
      e2m1_to_f16((r[c] >> 4 & kLow) | (r[2 + c] & ~kLow), hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
      for (int gk = 0; gk < 2; ++gk) {
        const uint32_t s0 = gk ? sc.z : sc.x, s1 = gk ? sc.w : sc.y;
        const uint32_t a[4] = {hmul2(lo[2 * gk], s0), hmul2(hi[2 * gk], s0), hmul2(lo[2 * gk + 1], s1), hmul2(hi[2 * gk + 1], s1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(A.o[2 * m + c][nt], a, pb[gk][nt][0], pb[gk][nt][1]);
      }
    }
  }
}

// Resident CTAs per SM that the registers allow.  Many rows: 5 and 6 (96 and 80 registers, little of a lane in local memory)
// took 1654 and 1774 us for an 8192-row prompt where 4 took 1650.  Split: decode of 16, 32, 64, 200 sequences with 4 KV heads
// 11.9, 17.7, 26.6, 64.1 us with 3, 12.9, 19.0, 27.7, 68.9 with 4.
template <int NT>
constexpr int kSplitCtasPerSm = NT == 1 ? 3 : 2;
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 4 : 2;
// The tiles, and later the merge buffers: the warps' O, m, l and lse sums, then the CTA's.
template <int NT>
constexpr int kTilesBytes = kWarps * kWarpBytes + kKv4QueryBytes<NT>;
template <int NT>
constexpr int kSmem = kTilesBytes<NT> > (kWarps + 1) * 8 * NT * (kPad + 3) * 4 ? kTilesBytes<NT>
                                                                           : (kWarps + 1) * 8 * NT * (kPad + 3) * 4;

// Where a lane's copies go in a tile set at `set`.
struct SetDst {
  uint32_t k, v, ks, vs;
  __device__ __forceinline__ explicit SetDst(uint32_t set) {
    const int lane = threadIdx.x & 31;
    k = set + lane * 16;
    v = set + kVAt + (lane >> 2) * kKv4Codes + (((lane & 3) ^ (lane >> 3)) << 4);  // chunk c of row r at c ^ (r / 2 % 4)
    ks = set + kKScaleAt + kv4_k_scale(lane) * kKv4Chunk;
    vs = set + kVScaleAt + lane * kKv4Chunk;
  }
};
// Gathers of a step whose row ids lie at `ids` (K, then V): one copy group each, empty if mask names none.
__device__ __forceinline__ void gather_k(const int* ids, unsigned mask, const SetDst& dst, uint32_t off, const uint8_t* base,
                                         uint32_t rowBytes) {
  if (mask) {
    const int lane = threadIdx.x & 31, at = kv4_row_place(lane);
    kv4_copy_codes<true>(ids, mask, dst.k + off, base + (lane & 3) * 16, rowBytes);
    kv4_copy_scales(ids[at], dst.ks + off, base, rowBytes);
    kv4_copy_scales(ids[kStep + at], dst.vs + off, base, rowBytes);
  }
  cp_async_commit();
}
__device__ __forceinline__ void gather_v(const int* ids, unsigned mask, const SetDst& dst, uint32_t off, const uint8_t* base,
                                         uint32_t rowBytes) {
  if (mask) kv4_copy_codes<false>(ids + kStep, mask, dst.v + off, base + (threadIdx.x & 3) * 16, rowBytes);
  cp_async_commit();
}

// Sum over the lanes that share a head.
__device__ __forceinline__ float head_sum(float x) {
  x += __shfl_xor_sync(kFull, x, 4);
  x += __shfl_xor_sync(kFull, x, 8);
  return x + __shfl_xor_sync(kFull, x, 16);
}
// A warp's result to shared memory: o [8 NT heads][kPad] fp32, m, l and the lse sums [8 NT].
template <int NT, bool kLse>
__device__ __forceinline__ void stash(const Acc<NT>& A, const float (&ls)[NT][2], float* o, float* m, float* l, float* s) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = 8 * nt + 2 * q + j;
      const float sum = head_sum(A.l[nt][j]);
      float exact = 0.f;
      if constexpr (kLse) exact = head_sum(ls[nt][j]);
      if (g == 0) {
        m[h] = A.m[nt][j];
        l[h] = sum;
        if constexpr (kLse) s[h] = exact;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        *reinterpret_cast<float2*>(o + h * kPad + 16 * mt + 2 * g) = make_float2(A.o[mt][nt][j], A.o[mt][nt][2 + j]);
    }
}
// log sum_j exp of a head with maximum M (in log2 units) and sum of 2^(x_j - M).
__device__ __forceinline__ float lse_of(float M, float sum) {
  return sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}
// Zeros in the o rows of `heads` heads, -inf in their lse, by `threads` threads.
__device__ __forceinline__ void no_tokens(const PagedArgs& a, size_t head0, int heads, int tid, int threads) {
  uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + head0 * kD);
  for (int e = tid; e < heads * kD / 8; e += threads) out[e] = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (int h = tid; h < heads; h += threads) a.lse[head0 + h] = -INFINITY;
}

// Few (row, KV head) pairs: the warps of a CTA, and the CTAs of a cluster, share one pair's list.
template <int NT, bool kBf16, bool kLse>
__global__ void __launch_bounds__(kThreads, kSplitCtasPerSm<NT>) sparse_paged_kv4_split_kernel(const PagedArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x % a.split);
  Row r = row_of(a, static_cast<int>(blockIdx.x / a.split), 1);
  List list(a, r);
  // the warp's first three steps of the list, on their way while the lengths are read
  const int hop = kStep * kWarps * a.split;  // entries between a warp's steps
  const int first = kStep * (rank * kWarps + warp) + lane;
  const int j0 = list.at(first), j1 = list.at(first + hop);
  int slot = first + 2 * hop, j2 = list.at(slot);
  row_lengths(a, r);
  list.L = r.L;
  uint2* out = static_cast<uint2*>(a.o) + r.head0 * (kD / 4);  // 4 values each
  if (r.t >= r.n) {  // the whole cluster leaves
    if (rank == 0) no_tokens(a, r.head0, a.G, tid, kThreads);
    return;
  }
  uint8_t* mine = smem + warp * kWarpBytes;
  const uint32_t set = smem_addr(mine), groups = set + kGroupsAt;
  float2* entries = reinterpret_cast<float2*>(mine + kEntriesAt);
  int* ids = reinterpret_cast<int*>(mine + kRowsAt);  // [step & 1][K, V][kv4_row_place]
  const uint32_t rowBytes = static_cast<uint32_t>(a.Hkv) * a.poolHeadDim;
  const uint8_t* base = a.pool + static_cast<size_t>(r.kvh) * a.poolHeadDim;
  const SetDst dst(set);

  auto resolve = [&](const Pages& p, int parity) {  // which lanes' entries name a row
    const PoolRows rows = list.rows_of(p);
    int* at = ids + parity * 2 * kStep + kv4_row_place(lane);
    at[0] = rows.ok ? rows.k : -1;
    at[kStep] = rows.ok ? rows.v : -1;
    return __ballot_sync(kFull, rows.ok);
  };
  auto gather_keys = [&](int par, unsigned mask) {
    gather_k(ids + par * 2 * kStep, mask, dst, par * kSetBytes, base, rowBytes);
  };
  auto gather_values = [&](int par, unsigned mask) {
    gather_v(ids + par * 2 * kStep, mask, dst, par * kSetBytes, base, rowBytes);
  };

  Acc<NT> A;
  acc_init(A);
  float ls[NT][2] = {};
  const int steps = max(0, (a.topK - (first - lane) + hop - 1) / hop);
  unsigned cur = resolve(list.pages_of(j0), 0);
  Pages p1 = list.pages_of(j1);
  __syncwarp();
  gather_keys(0, cur);
  gather_values(0, cur);
  slot += hop;
  int j3 = list.at(slot);
  const uint32_t queries = smem_addr(smem + kWarps * kWarpBytes);
  float qs[NT][2];
  kv4_load_q<NT, kBf16, true>(static_cast<const uint4*>(a.q) + r.head0 * (kD / 8), a.G, queries, qs);
  unsigned next = resolve(p1, 1);
  p1 = list.pages_of(j2);
  __syncwarp();
  gather_keys(1, next);
  gather_values(1, next);
  __syncthreads();  // the queries are in place
  for (int i = 0; i < steps; ++i) {
    const int par = i & 1;
    const uint32_t at = set + par * kSetBytes;
    const unsigned then = resolve(p1, par);  // step i + 2: its rows go where step i's are
    p1 = list.pages_of(j3);
    slot += hop;
    j3 = list.at(slot);
    if (cur) {
      float s[2][NT][4];
      uint32_t pb[2][NT][2];
      cp_async_wait<3>();  // this lane's share of the K rows; the V codes and the next step's may be in flight
      __syncwarp();
      entries[lane] = entry_of(a, cur >> lane & 1, at + kKScaleAt, at + kVScaleAt);
      transpose_scales(at + kVScaleAt, groups);
      kv4_scores<NT>(s, at, at + kKScaleAt, queries);
      __syncwarp();  // every lane is done with the K rows and both scales
      gather_keys(par, then);
      softmax32<NT, kBf16, kLse>(A, s, qs, entries + kv4_first_key(lane), pb, ls);
      cp_async_wait<3>();  // the V codes
      __syncwarp();
      values32<NT>(A, at + kVAt, groups, pb);
      __syncwarp();  // every lane is done with the V codes
      gather_values(par, then);
    } else {  // nothing was copied for this step
      __syncwarp();
      gather_keys(par, then);
      gather_values(par, then);
    }
    cur = next;
    next = then;
  }
  cp_async_wait<0>();
  list.report();
  __syncthreads();  // the tiles become the merge buffers

  constexpr int H = 8 * NT;
  float* ow = reinterpret_cast<float*>(smem);   // [kWarps][H][kPad]
  float* oc = ow + kWarps * H * kPad;           // the CTA's merged [H][kPad]
  float* mw = oc + H * kPad;                    // [kWarps][H]
  float* lw = mw + kWarps * H;
  float* sw = lw + kWarps * H;
  float* mc = sw + kWarps * H;                  // [H], then the sums, then the lse sums
  stash<NT, kLse>(A, ls, ow + warp * H * kPad, mw + warp * H, lw + warp * H, sw + warp * H);
  __syncthreads();
  for (int h = warp; h < a.G; h += kWarps) {
    float M, sum, exact = 0.f;
    const float4 o = join<H>(ow, mw, lw, h, M, sum);
    if constexpr (kLse)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) exact = fmaf(exp2f(mw[w * H + h] - M), sw[w * H + h], exact);
    if (a.split > 1) {
      *reinterpret_cast<float4*>(oc + h * kPad + 4 * lane) = o;
      if (lane == 0) {
        mc[h] = M;
        mc[H + h] = sum;
        mc[2 * H + h] = exact;
      }
    } else {
      out[h * 32 + lane] = normalised<kBf16>(o, sum);
      if (kLse && lane == 0) a.lse[r.head0 + h] = lse_of(M, exact);
    }
  }
  if (a.split == 1) return;
  // Join over the cluster: head h by one warp of it.
  cluster_sync_all();
  const uint32_t ocAddr = smem_addr(oc), mcAddr = smem_addr(mc);
  for (int h = rank * kWarps + warp; h < a.G; h += a.split * kWarps) {
    // all CTAs' parts on their way at once (with a meeting below that waits for the writes of o, 0.3 us more)
    float4 x[kMaxCluster];
    float ms[kMaxCluster], part[kMaxCluster], whole[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      ms[c] = -FLT_MAX;
      if (c < a.split) {
        ms[c] = cluster_ld(cluster_addr(mcAddr + h * 4, c));
        part[c] = cluster_ld(cluster_addr(mcAddr + (H + h) * 4, c));
        if constexpr (kLse) whole[c] = cluster_ld(cluster_addr(mcAddr + (2 * H + h) * 4, c));
        x[c] = cluster_ld4(cluster_addr(ocAddr + (h * kPad + 4 * lane) * 4, c));
      }
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -FLT_MAX, sum = 0.f, exact = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) M = fmaxf(M, ms[c]);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < a.split) {
        const float f = exp2f(ms[c] - M);
        sum += f * part[c];
        if constexpr (kLse) exact += f * whole[c];
        o.x += f * x[c].x;
        o.y += f * x[c].y;
        o.z += f * x[c].z;
        o.w += f * x[c].w;
      }
    out[h * 32 + lane] = normalised<kBf16>(o, sum);
    if (kLse && lane == 0) a.lse[r.head0 + h] = lse_of(M, exact);
  }
  cluster_meet();  // no CTA leaves while another reads its shared memory
}

// Many rows: a CTA takes four KV heads of a row, each warp one of them and the whole list.  The heads share the list, so the
// warps resolve its entries once for all of them, a chunk of 128 at a time, 32 per warp: row ids go to shared memory for
// every warp.  Chunk c + 1's are written before the barrier that opens chunk c (its first rows are gathered in chunk c's
// last step).
constexpr int kRowsGroupsAt = kSetBytes;
constexpr int kRowsEntriesAt = kRowsGroupsAt + kKv4ScaleBytes;
constexpr int kRowsQueriesAt = kRowsEntriesAt + kStep * 8;
template <int NT>
constexpr int kRowsWarp = kRowsQueriesAt + kKv4QueryBytes<NT>;
template <int NT>
constexpr int kWarpTiles = kRowsWarp<NT> > 8 * NT * (kPad + 3) * 4 ? kRowsWarp<NT> : 8 * NT * (kPad + 3) * 4;  // later: O, m, l, lse
template <int NT>
constexpr int kIdsAt = kWarps * kWarpTiles<NT>;                    // [chunk % 3][warp's step][K, V][kStep] row ids
template <int NT>
constexpr int kMasksAt = kIdsAt<NT> + 3 * kWarps * kStep * 2 * 4;  // [chunk % 3][warp's step] entries that name a row
template <int NT>
constexpr int kRowsSmem = kMasksAt<NT> + 64;

template <int NT, bool kBf16, bool kLse>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<NT>) sparse_paged_kv4_rows_kernel(const PagedArgs a, int items) {
  constexpr int kChunk = kWarps * kStep;  // entries
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = static_cast<int>(blockIdx.x);
  if (item >= items) return;  // (none is; without the test the compiler puts 48 bytes of a lane in local memory: 1627 us
                              // for an 8192-row prompt instead of 1520)
  Row r = row_of(a, item, kWarps);
  List list(a, r);
  const int j0 = list.at(tid), j1 = list.at(tid + kChunk);
  int slot = tid + 2 * kChunk, j2 = list.at(slot);
  row_lengths(a, r);
  list.L = r.L;
  if (r.t >= r.n) {
    no_tokens(a, r.head0, kWarps * a.G, tid, kThreads);
    return;
  }
  uint8_t* mine = smem + warp * kWarpTiles<NT>;
  const uint32_t set = smem_addr(mine), groups = set + kRowsGroupsAt;
  float2* entries = reinterpret_cast<float2*>(mine + kRowsEntriesAt);
  int* ids = reinterpret_cast<int*>(smem + kIdsAt<NT>);
  unsigned* masks = reinterpret_cast<unsigned*>(smem + kMasksAt<NT>);
  const uint32_t rowBytes = static_cast<uint32_t>(a.Hkv) * a.poolHeadDim;
  const uint8_t* base = a.pool + static_cast<size_t>(r.kvh + warp) * a.poolHeadDim;
  const SetDst dst(set);

  auto put_rows = [&](const Pages& p, int buf) {  // row ids of the thread's entry of a chunk
    const PoolRows rows = list.rows_of(p);
    int* at = ids + (buf * kWarps + warp) * 2 * kStep + kv4_row_place(lane);
    at[0] = rows.ok ? rows.k : -1;
    at[kStep] = rows.ok ? rows.v : -1;
    const unsigned mask = __ballot_sync(kFull, rows.ok);
    if (lane == 0) masks[buf * kWarps + warp] = mask;
  };
  auto ids_of = [&](int buf, int step) { return ids + (buf * kWarps + step) * 2 * kStep; };
  Acc<NT> A;
  acc_init(A);
  float ls[NT][2] = {};
  put_rows(list.pages_of(j0), 0);
  Pages p1 = list.pages_of(j1);
  const uint32_t queries = set + kRowsQueriesAt;
  float qs[NT][2];
  kv4_load_q<NT, kBf16, false>(static_cast<const uint4*>(a.q) + (r.head0 + warp * a.G) * (kD / 8), a.G, queries, qs);
  __syncthreads();
  unsigned mask = masks[0];  // of the current step, whose rows are gathered
  gather_k(ids_of(0, 0), mask, dst, 0, base, rowBytes);
  gather_v(ids_of(0, 0), mask, dst, 0, base, rowBytes);
  const int chunks = (a.topK + kChunk - 1) / kChunk;
  int buf = 0;
  for (int c = 0; c < chunks; ++c) {
    const int nbuf = buf == 2 ? 0 : buf + 1;
    put_rows(p1, nbuf);
    p1 = list.pages_of(j2);
    slot += kChunk;
    j2 = list.at(slot);
    __syncthreads();
#pragma unroll 1
    for (int e = 0; e < kWarps; ++e) {
      const bool last = e == kWarps - 1;
      const int gbuf = last ? nbuf : buf, ge = last ? 0 : e + 1;  // the next step
      const unsigned next = masks[gbuf * kWarps + ge];
      const int* nids = ids_of(gbuf, ge);
      if (mask) {
        float s[2][NT][4];
        uint32_t pb[2][NT][2];
        cp_async_wait<1>();  // this lane's share of the K rows; the V codes may be in flight
        __syncwarp();
        entries[lane] = entry_of(a, mask >> lane & 1, set + kKScaleAt, set + kVScaleAt);
        transpose_scales(set + kVScaleAt, groups);
        kv4_scores<NT>(s, set, set + kKScaleAt, queries);
        __syncwarp();  // every lane is done with the K rows and both scales
        gather_k(nids, next, dst, 0, base, rowBytes);
        softmax32<NT, kBf16, kLse>(A, s, qs, entries + kv4_first_key(lane), pb, ls);
        cp_async_wait<1>();  // the V codes; the next K rows may be in flight
        __syncwarp();
        values32<NT>(A, set + kVAt, groups, pb);
        __syncwarp();  // every lane is done with the V codes
        gather_v(nids, next, dst, 0, base, rowBytes);
      } else {
        gather_k(nids, next, dst, 0, base, rowBytes);
        gather_v(nids, next, dst, 0, base, rowBytes);
      }
      mask = next;
    }
    buf = nbuf;
  }
  cp_async_wait<0>();
  list.report();
  __syncwarp();  // the warp's tiles become its output buffer
  constexpr int H = 8 * NT;
  float* ow = reinterpret_cast<float*>(mine);  // [H][kPad]
  float* mw = ow + H * kPad;                   // [m, l, lse sums][H]
  stash<NT, kLse>(A, ls, ow, mw, mw + H, mw + 2 * H);
  __syncwarp();
  const size_t head0 = r.head0 + warp * a.G;
  uint2* out = static_cast<uint2*>(a.o) + head0 * (kD / 4);
  for (int h = 0; h < a.G; ++h)
    out[h * 32 + lane] = normalised<kBf16>(*reinterpret_cast<const float4*>(ow + h * kPad + 4 * lane), mw[H + h]);
  if (kLse && a.lse && lane < a.G) a.lse[head0 + lane] = lse_of(mw[lane], mw[2 * H + lane]);
}

template <int NT, bool kBf16, bool kLse>
cudaError_t rows_go(const PagedArgs& a, long long pairs, cudaStream_t st) {
  auto kernel = sparse_paged_kv4_rows_kernel<NT, kBf16, kLse>;
  constexpr int kSmemBytes = kRowsSmem<NT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(pairs / kWarps), kThreads, kSmemBytes, st>>>(
      a, static_cast<int>(pairs / kWarps));
  return cudaGetLastError();
}

template <int NT>
cudaLaunchConfig_t split_config(long long pairs, int split, cudaStream_t st, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<NT>;
  cfg.stream = st;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = split;
  at->val.clusterDim.y = 1;
  at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cfg;
}

// Clusters of `split` CTAs that the current device holds at once (a cluster's CTAs lie in one GPC, so this is less than
// the CTAs allow), asked for once per device, when the kernel's shared memory is allowed too.
template <int NT, bool kBf16, bool kLse>
long long resident_clusters(int split) {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];  // 0: not asked yet; -1: none
  int dev = 0;
  const bool cached = cudaGetDevice(&dev) == cudaSuccess && dev < kDevices;
  int n = cached ? known[dev][split].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = split_config<NT>(1, split, nullptr, &at);
    auto kernel = sparse_paged_kv4_split_kernel<NT, kBf16, kLse>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<NT>) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();  // a failed query is not the launch's error: this size is just not used
      n = 0;
    }
    n = n < 1 ? -1 : n;
    if (cached) known[dev][split].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int NT, bool kBf16, bool kLse>
cudaError_t paged_go(PagedArgs a, long long pairs, cudaStream_t st) {
  const long long slots = static_cast<long long>(kCtasPerSm<NT>) * sm_count();  // CTAs resident at once
  // A warp per pair for just under one wave of such CTAs, and from 1.6 waves on: 600 rows of 4 heads of 8 queries (1 wave) 139
  // us, 155 in the other form, 700 (1.15) 181 and 180, 1000 (1.6) 238 and 252, 2048 460 and 508; of 14 queries 280 rows (0.9
  // waves) 97 and 106, 320 156 and 122.  (Two heads of two rows to a CTA, for 2 KV heads: 1200 pairs 96 us instead of 82,
  // 4400 292 instead of 276, 8192 as long.)
  // (bf16 groups up to 8 sum for lse whether it is asked for or not: the compiler then keeps a lane in registers, 918 us for
  // 4096 rows instead of 942.)
  const long long rowCtas = pairs / kWarps;
  if (a.Hkv % kWarps == 0 && ((10 * rowCtas >= 9 * slots && rowCtas <= slots) || 10 * rowCtas >= 16 * slots))
    return rows_go<NT, kBf16, kLse || (kBf16 && NT == 1)>(a, pairs, st);
  // Otherwise 1 to 8 CTAs per pair, all clusters resident at once, at most one CTA per 128 entries of the list: those that cost
  // least, in units of 0.28 us: 1 + 2 CTAs of an SM for each of a warp's steps, 4 for the join, 4 for a third CTA on an SM.
  // (us by CTAs per pair: 128 pairs with lists of 2051 17.7, 16.3, 17.3 with 1, 2, 3, of 1027 11.2, 11.4, 11.9, of 259 5.6, 6.8,
  // 7.6; 64 pairs, 2051, 18.4, 13.0, 13.2, 12.2, 14.1, 11.9 with 1 to 6; 32 pairs, 1027, 11.9, 9.4, 7.5, 7.7, 8.1, 8.2; 192
  // pairs, 2051, 27.7, 22.6, 259 8.4, 8.8.  A count that leaves clusters waiting costs a fifth more at least.)
  const int sms = sm_count(), most = std::min(kMaxCluster, (a.topK + kStep * kWarps - 1) / (kStep * kWarps));
  long long least = 0;
  for (int split = 1; split <= most; ++split) {
    const long long resident = resident_clusters<NT, kBf16, kLse>(split);
    if (split > 1 && pairs > resident) continue;
    const long long steps = (a.topK + kStep * kWarps * split - 1) / (kStep * kWarps * split);
    const long long ctas = (pairs * split + sms - 1) / sms;  // of an SM
    const long long cost = steps * (1 + 2 * ctas) + (split > 1 ? 4 : 0) + (ctas > 2 ? 4 : 0);
    if (split == 1 || cost <= least) {  // (equal ones: with more CTAs fewer warps have the most steps)
      least = cost;
      a.split = split;
    }
  }
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = split_config<NT>(pairs, a.split, st, &at);
  auto kernel = sparse_paged_kv4_split_kernel<NT, kBf16, kLse>;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PagedArgs>(a));
  if (e == cudaErrorInvalidValue) {  // the attribute is the context's: a new one has not got it
    (void)cudaGetLastError();
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<NT>);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PagedArgs>(a));
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT, bool kBf16>
cudaError_t paged_lse(const PagedArgs& a, long long pairs, cudaStream_t st) {
  return a.lse ? paged_go<NT, kBf16, true>(a, pairs, st) : paged_go<NT, kBf16, false>(a, pairs, st);
}

}  // namespace

cudaError_t launch_sparse_paged_kv4(const QsaSparsePagedKv4Params& p, bool bf16) {
  PagedArgs a;
  a.q = p.qPtr;
  a.pool = static_cast<const uint8_t*>(p.kvPool);
  a.scale = nullptr;
  a.pageTable = p.pageTable;
  a.indices = p.indices;
  a.ctx = p.contextLengths;
  a.newLen = p.newLengths;
  a.o = p.oPtr;
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
  a.lse = p.lse;
  const long long pairs = static_cast<long long>(p.batchSize) * p.seqLen * p.numKVHeads;
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  if (bf16) return a.G <= 8 ? paged_lse<1, true>(a, pairs, st) : paged_lse<2, true>(a, pairs, st);
  return a.G <= 8 ? paged_lse<1, false>(a, pairs, st) : paged_lse<2, false>(a, pairs, st);
}

}  // namespace qsa
