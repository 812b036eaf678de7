// qsa_attention_kv8.cu -- sparse GQA attention over an 8-bit paged cache
// (qsa_sparse_paged_kv8): for every live row and query head
//
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = ks_j c^K_j,  v_j = vs_j c^V_j
//
// over the row's list, with e4m3 codes c and one fp32 scale per block of
// tokens and head.  In log2 units, with x_j = ks_j scale log2(e) (q . c^K_j) and
// e_j = x_j + log2(vs_j), one pass keeps a maximum M of e_j, l = sum 2^(e_j - M) / vs_j
// and O = sum 2^(e_j - M) c^V_j: the V scale rides in the exponent, so the
// weights that the second product rounds to fp16 are relative to the largest
// weight times scale, whatever the scales are, and o = O / l.  (log2(vs_j) is
// the hardware's approximation; its error enters O and l alike.)
//
// Two kernels share the arithmetic.  With few (row, KV head) pairs, a CTA of 4
// warps takes one, or a cluster of up to 8 CTAs shares it, the list dealt out
// to the warps in steps of 32 entries; with many, a CTA takes four KV heads of a
// row (or two of two rows), a warp each, and resolves a list once for its heads.
//
// A warp runs its steps by itself.  Every dependent load of a step (list entry,
// page ids, scales) has a step or more to arrive; the 32 K and V rows of 128
// bytes are gathered with cp.async into the warp's own K tile and V tile.  A
// step's K tile is free after its first product, its V tile after the second,
// and the rows of the next step (many rows: one tile of each, half a step of
// copies in flight per warp, which 16 warps cover) or of the one after it (few
// pairs: two of each, more in flight where latency decides) start then.
//
// S^T = C^K Q^T and O^T += (C^V)^T P^T are m16n8k16 MMAs in fp16 with the head
// group as N; codes are converted to fp16 pairs in registers (exact).  The
// summed dims of the first are permuted so that a lane reads its K codes as
// whole 16-byte chunks; for the second, ldmatrix transposes 16 x 16 bytes, so
// a register holds four keys of one dim.  The rows of S^T are the keys in the
// order that makes its columns the second product's fragments of P^T.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <utility>

#include "qsa_internal.h"
#include "qsa_kv8.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kD = 128;
constexpr int kStep = 32;                      // list entries of a warp's step
constexpr int kTileBytes = kStep * kD;         // K (or V) rows of a step
// A warp's shared memory in the split form: two K tiles, two V tiles, the pool rows of two steps' entries (K then V), the
// values of a step's entries.
constexpr int kRowsAt = 4 * kTileBytes;
constexpr int kEntriesAt = kRowsAt + 2 * 2 * kStep * 4;
constexpr int kWarpBytes = kEntriesAt + kStep * 16;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct PagedArgs {
  const void* q;
  const uint8_t* pool;
  const float* scale;
  const int32_t* pageTable;
  const int32_t* indices;
  const int32_t* ctx;
  const int32_t* newLen;  // may be null
  void* o;
  int32_t* status;  // may be null
  int S, Hq, Hkv, G, poolHeadDim, numFlatPages, maxPagesPerSeq, topK;
  int blockShift;  // log2(scaleBlock)
  int split;       // CTAs per pair: the cluster size
  float sl2;       // attentionScale * log2(e)
};

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr));
  return v;
}

template <bool kBf16>
__device__ __forceinline__ uint2 pack4(float4 v) {
  return kBf16 ? make_uint2(pack_bf162(v.x, v.y), pack_bf162(v.z, v.w))
               : make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
}

// Byte offset of 16-byte chunk c of key row r in a step's K tile (a lane group reads chunks 0..3 or 4..7 of two rows of
// different parity) and V tile (ldmatrix reads one chunk of 8 successive rows): each access covers all banks once.
__device__ __forceinline__ uint32_t k_off(int r, int c) { return r * kD + ((c ^ ((r & 1) << 2)) << 4); }
__device__ __forceinline__ uint32_t v_off(int r, int c) { return r * kD + ((c ^ (r & 7)) << 4); }
// Key of row g of an S^T fragment (row g + 8: two keys on), within its 16 keys.
__device__ __forceinline__ int key_of(int g) { return 4 * (g >> 1) + (g & 1); }

// 16-byte copy to dst + kOff.
template <int kOff>
__device__ __forceinline__ void cp_async16_to(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;\n" ::"r"(dst), "l"(src), "n"(kOff) : "memory");
}
template <int kOff>
__device__ __forceinline__ void cp_async16_to(uint32_t dst, const void* src, bool pred) {
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(pred ? 16 : 0), "n"(kOff)
               : "memory");
}
__device__ __forceinline__ float lg2_ftz(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// One lane's eight 16-byte copies of a gather: rows 4 i + (lane >> 3), i = 0..7, each at dst[i & 1] + 512 i.
// base: the lane's chunk of pool row 0.  kAll: every row is named (row >= 0); otherwise the others are zeros.
template <bool kAll, size_t... I>
__device__ __forceinline__ void copy_rows(const int (&row)[8], const uint32_t (&dst)[2], const uint8_t* base,
                                          uint32_t rowBytes, std::index_sequence<I...>) {
  if constexpr (kAll) {
    (cp_async16_to<4 * kD * I>(dst[I & 1], base + static_cast<uint64_t>(static_cast<uint32_t>(row[I])) * rowBytes), ...);
  } else {
    (cp_async16_to<4 * kD * I>(dst[I & 1], base + static_cast<uint64_t>(static_cast<uint32_t>(max(row[I], 0))) * rowBytes,
                               row[I] >= 0),
     ...);
  }
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Two transposed 16 x 16 byte matrices (rows at the addresses of lanes 0..15 and 16..31): of each, the lane gets rows
// 4 q .. 4 q + 3 of column g, then of column g + 8.
__device__ __forceinline__ void ldsm_bytes_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// A warp's running state: O^T fragments, max and sum of its heads 8 nt + 2 q, 8 nt + 2 q + 1 (q = lane & 3).
// Tile mt holds dims 16 mt + g and 16 mt + g + 8, g = lane >> 2.
template <int NT>
struct Acc {
  float o[8][NT][4];
  float m[NT][2];
  float l[NT][2];
};

// S^T = C^K Q^T of a step's 32 keys: s[gk][nt] holds keys 16 gk + key_of(g) and 2 on, heads 8 nt + 2 q and + 1.
template <int NT>
__device__ __forceinline__ void scores32(float (&s)[2][NT][4], uint32_t tile, const uint32_t (&qf)[NT][8][2]) {
  const int lane = threadIdx.x & 31, key = key_of(lane >> 2), q = lane & 3;
#pragma unroll
  for (int gk = 0; gk < 2; ++gk) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[gk][nt][0] = s[gk][nt][1] = s[gk][nt][2] = s[gk][nt][3] = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 r0 = lds16(tile + k_off(16 * gk + key, q + 4 * half));
      const uint4 r1 = lds16(tile + k_off(16 * gk + key + 2, q + 4 * half));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a[4];
        e4m3_to_f16(word(r0, w), a[0], a[2]);
        e4m3_to_f16(word(r1, w), a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(s[gk][nt], a, qf[nt][4 * half + w][0], qf[nt][4 * half + w][1]);
      }
    }
  }
}

// Online softmax of a step: s becomes the weights relative to the running maximum, returned in fp16 as the B
// fragments of the second product.  The maximum moves only when a weight would pass 2^kHeadroom (the weights
// are relative numbers: nothing is lost by their being up to 256 instead of 1), so that O is hardly ever
// rescaled after a warp's first step.  The sums use the weights as the second product does, rounded to 11 bits: where
// few keys decide, a rounding that only one of the two had would show in an fp16 output (up to 2^-11 of it, as much as
// its half step).  The maximum starts at the lowest finite number, so that an entry that names nothing
// (-inf) weighs 0 even before the first that does.  entries[i], of key i: x = K scale * attentionScale * log2(e),
// y = log2(V scale), z = 1 / V scale; (0, -inf, 0) for an entry that names nothing.
template <int NT, bool kBf16>
__device__ __forceinline__ void softmax32(Acc<NT>& A, float (&s)[2][NT][4], const float (&qs)[NT][2],
                                          const float4* entries, uint32_t (&pb)[2][NT][2]) {
  constexpr float kHeadroom = 8.f;
  const int key = key_of((threadIdx.x & 31) >> 2);
  float ks[4], lv[4], iv[4];  // of the lane's keys
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 e = entries[key + 16 * (i >> 1) + 2 * (i & 1)];
    ks[i] = e.x;
    lv[i] = e.y;
    iv[i] = e.z;
  }
  float mx[NT][2];
  bool move = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float& x = s[i >> 1][nt][2 * (i & 1) + h];
        // bf16: the K scale first (the product is below 2^31, so with scales below 2^96 only a logit itself overflows)
        x = kBf16 ? fmaf(x * ks[i], qs[nt][h], lv[i]) : fmaf(x, ks[i], lv[i]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[nt][h] = fmaxf(fmaxf(s[0][nt][h], s[0][nt][2 + h]), fmaxf(s[1][nt][h], s[1][nt][2 + h]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx[nt][h] = fmaxf(mx[nt][h], __shfl_xor_sync(kFull, mx[nt][h], o));
      move |= mx[nt][h] > A.m[nt][h] + kHeadroom;
    }
  }
  if (__any_sync(kFull, move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float al[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mn = fmaxf(A.m[nt][h], mx[nt][h]);
        al[h] = ex2_ftz(A.m[nt][h] - mn);
        A.m[nt][h] = mn;
        A.l[nt][h] *= al[h];
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        A.o[mt][nt][0] *= al[0];
        A.o[mt][nt][1] *= al[1];
        A.o[mt][nt][2] *= al[0];
        A.o[mt][nt][3] *= al[1];
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* x = &s[i >> 1][nt][2 * (i & 1)];
      const uint64_t w = pack_f2(ex2_ftz(x[0] - A.m[nt][0]), ex2_ftz(x[1] - A.m[nt][1]));
      // 8193 w - 8192 w, the first rounded to 24 bits: w to 11
      const uint64_t r = ffma2(pack_f2(-8192.f, -8192.f), w, ffma2(pack_f2(8192.f, 8192.f), w, w));
      x[0] = lo_f2(r);
      x[1] = hi_f2(r);
      A.l[nt][0] = fmaf(x[0], iv[i], A.l[nt][0]);
      A.l[nt][1] = fmaf(x[1], iv[i], A.l[nt][1]);
    }
    // the weights in fp16: as they are from 2^-14 on, to 2^-25 below
#pragma unroll
    for (int gk = 0; gk < 2; ++gk) {
      pb[gk][nt][0] = movmatrix_t(pack_half2(s[gk][nt][0], s[gk][nt][1]));
      pb[gk][nt][1] = movmatrix_t(pack_half2(s[gk][nt][2], s[gk][nt][3]));
    }
  }
}

// O^T += (C^V)^T P^T.
template <int NT>
__device__ __forceinline__ void values32(Acc<NT>& A, uint32_t tile, const uint32_t (&pb)[2][NT][2]) {
  const uint32_t row = tile + v_off(threadIdx.x & 31, 0);
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    uint32_t r[4];
    ldsm_bytes_t(row ^ (mt << 4), r);
#pragma unroll
    for (int gk = 0; gk < 2; ++gk) {
      uint32_t a[4];
      e4m3_to_f16(r[2 * gk], a[0], a[2]);
      e4m3_to_f16(r[2 * gk + 1], a[1], a[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816(A.o[mt][nt], a, pb[gk][nt][0], pb[gk][nt][1]);
    }
  }
}

// The group's Q^T fragments: k-step 4 half + w of a lane covers dims 16 (q + 4 half) + 4 w .. + 3, as the K
// chunks do.  bf16 values are scaled by a power of two per head to fp16's upper range; qs gets its inverse for
// the lane's heads 2 q, 2 q + 1.
template <int NT, bool kBf16>
__device__ __forceinline__ void load_q(const uint4* q, int G, uint32_t (&qf)[NT][8][2], float (&qs)[NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = 8 * nt + g;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      raw[i] = h < G ? __ldg(q + h * (kD / 8) + 2 * (c + 4 * (i >> 1)) + (i & 1)) : make_uint4(0, 0, 0, 0);
    float up = 1.f, down = 1.f;
    if constexpr (kBf16) {
      uint32_t m = 0;  // largest magnitude, as bf16 bits
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) m = max(m, max(word(raw[i], w) & 0x7fff, (word(raw[i], w) >> 16) & 0x7fff));
      m = max(m, __shfl_xor_sync(kFull, m, 1));
      m = max(m, __shfl_xor_sync(kFull, m, 2));
      // exponent e of the largest: scaled by 2^(14 - e), or 2^114 where that is less, so that the inverse is a normal
      // number; not for 0, inf and NaN
      const int e = static_cast<int>(m >> 7) - 127;
      if (m != 0 && e < 128) {
        const int k = 14 - max(e, -100);
        up = __int_as_float((127 + k) << 23);
        down = __int_as_float((127 - k) << 23);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t v = word(raw[i], w);
        if constexpr (kBf16) v = pack_half2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
        // 16-byte piece i holds dims 16 (c + 4 (i / 2)) + 8 (i & 1) + 2 w: k-step 4 (i / 2) + 2 (i & 1) + w / 2
        qf[nt][4 * (i >> 1) + 2 * (i & 1) + (w >> 1)][w & 1] = v;
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) qs[nt][j] = __shfl_sync(kFull, down, 4 * (2 * c + j));
  }
}

constexpr int kPad = kD + 4;  // floats of a head in the merge buffers

// Resident CTAs per SM.  Many rows: the register budget decides.  With 4, groups up to 8 keep a little of a lane in local
// memory (four fp16 heads 28 bytes, four or two bf16 heads 8 and 16); 5 at 96 registers spill far more and took 1333 us
// for an 8192-row prompt against 1275 with 4; 16-head groups at 168 registers 2008 against 1928 with 2.  Split: two tiles of
// each kind per warp (69 KB a CTA) rather than a fourth CTA with one: decode of 8, 16, 38, 64, 200 sequences with 4 KV heads
// took 7.0, 9.7, 18.3, 26.4, 70.6 us instead of 7.5, 10.5, 19.8, 29.1, 78.1, of 32 sequences 17.1 either way.
template <int NT>
constexpr int kSplitCtasPerSm = NT == 1 ? 3 : 2;
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 4 : 2;
// The tiles, and later the merge buffers: the warps' O, m and l, then the CTA's.
template <int NT>
constexpr int kSmem = kWarps * kWarpBytes > (kWarps + 1) * 8 * NT * (kPad + 2) * 4 ? kWarps * kWarpBytes
                                                                               : (kWarps + 1) * 8 * NT * (kPad + 2) * 4;

// What a CTA (or cluster) works on: a row of the call and successive KV heads.
struct Row {
  int kvh, b, t, L, n;  // first KV head, sequence, row, the tokens that its page table holds, its live rows
  size_t bt, head0;     // list row; first query head
};
// The place of work item `id` with `heads` KV heads each; its lengths are read by row_lengths.
__device__ __forceinline__ Row row_of(const PagedArgs& a, int id, int heads) {
  Row r;
  const int per = a.Hkv / heads, rowid = id / per;
  r.kvh = (id - rowid * per) * heads;
  r.b = rowid / a.S;
  r.t = a.S - 1 - (rowid - r.b * a.S);  // a sequence's rows from the last position down: the longest lists start first
  r.bt = static_cast<size_t>(r.b) * a.S + r.t;
  r.head0 = r.bt * a.Hq + static_cast<size_t>(r.kvh) * a.G;
  return r;
}
__device__ __forceinline__ void row_lengths(const PagedArgs& a, Row& r) {
  const int L = max(0, a.ctx[r.b]);
  r.L = min(L, a.maxPagesPerSeq * kTokensPerPage);
  r.n = max(0, min(a.newLen ? a.newLen[r.b] : a.S, min(a.S, L)));
}

// From list entries to pool rows, free of branches: what an entry cannot name is looked up at 0 and dropped.
struct Pages {
  int j, k, v;  // entry (-1: none), its page ids
};
struct PoolRows {
  bool ok;   // the entry names a row
  int k, v;  // its rows of the pool (0 for none)
};
struct List {
  const PagedArgs& a;
  const int32_t *entries, *ptK, *ptV;
  int L, bad;
  __device__ __forceinline__ List(const PagedArgs& args, const Row& r)
      : a(args),
        entries(args.indices + r.bt * args.topK),
        ptK(args.pageTable + static_cast<size_t>(r.b) * 2 * args.maxPagesPerSeq),
        ptV(ptK + args.maxPagesPerSeq),
        L(0),
        bad(0) {}
  __device__ __forceinline__ int at(int slot) const { return slot < a.topK ? __ldg(entries + slot) : -1; }
  __device__ __forceinline__ Pages pages_of(int j) {
    const bool in = static_cast<unsigned>(j) < static_cast<unsigned>(L);
    bad |= !in && j != -1 ? kErrBadIndex : 0;
    const int page = in ? j >> 7 : 0;
    return Pages{in ? j : -1, __ldg(ptK + page), __ldg(ptV + page)};
  }
  __device__ __forceinline__ PoolRows rows_of(const Pages& p) {
    const bool pages = static_cast<unsigned>(p.k) < static_cast<unsigned>(a.numFlatPages) &&
                       static_cast<unsigned>(p.v) < static_cast<unsigned>(a.numFlatPages);
    const bool ok = p.j >= 0 && pages;
    bad |= p.j >= 0 && !pages ? kErrBadPage : 0;
    return PoolRows{ok, ok ? p.k * kTokensPerPage + (p.j & 127) : 0, ok ? p.v * kTokensPerPage + (p.j & 127) : 0};
  }
  __device__ __forceinline__ void report() {
    bad = __reduce_or_sync(kFull, static_cast<unsigned>(bad));
    if (bad && (threadIdx.x & 31) == 0 && a.status) atomicOr(a.status, bad);
  }
};
// The scales of a pool row, from KV head kvh on.
__device__ __forceinline__ const float* scales_of(const PagedArgs& a, int row, int kvh) {
  return a.scale + static_cast<size_t>(row >> a.blockShift) * a.Hkv + kvh;
}
// What the softmax needs of an entry: see softmax32.
__device__ __forceinline__ float4 entry_of(const PagedArgs& a, bool ok, float ks, float vs) {
  vs = read_scale(vs);
  return ok ? make_float4(read_scale(ks) * a.sl2, lg2_ftz(vs), rcp_ftz(vs), 0.f) : make_float4(0.f, -INFINITY, 0.f, 0.f);
}
// Place of a step's entry i among its 32 row ids: a lane gathers rows 4 i + (lane >> 3), which lie together.
__device__ __forceinline__ int row_place(int i) { return (i & 3) * (kStep / 4) + (i >> 2); }

// Where a lane's copies of a step's K and V rows go in a warp's tiles.
struct TileDst {
  uint32_t k[2], v[2];
  __device__ __forceinline__ TileDst(uint32_t ktile, uint32_t vtile) {
    const int r = (threadIdx.x & 31) >> 3, c = threadIdx.x & 7;
    k[0] = k[1] = ktile + k_off(r, c);
    v[0] = vtile + v_off(r, c);
    v[1] = v[0] ^ 64;  // rows 4 i + r: bit 2 of the row flips with i
  }
};
// Gathers the rows whose ids lie at `ids` (by row_place, -1 for none): one copy group, empty if mask names none.
__device__ __forceinline__ void gather_rows(const int* ids, unsigned mask, const uint32_t (&dst)[2], const uint8_t* base,
                                            uint32_t rowBytes) {
  if (mask) {
    const int4* at = reinterpret_cast<const int4*>(ids + ((threadIdx.x & 31) >> 3) * (kStep / 4));
    const int4 x = at[0], y = at[1];
    const int row[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (mask == kFull)
      copy_rows<true>(row, dst, base, rowBytes, std::make_index_sequence<8>{});
    else
      copy_rows<false>(row, dst, base, rowBytes, std::make_index_sequence<8>{});
  }
  cp_async_commit();
}

template <int NT>
__device__ __forceinline__ void acc_init(Acc<NT>& A) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) A.o[mt][nt][0] = A.o[mt][nt][1] = A.o[mt][nt][2] = A.o[mt][nt][3] = 0.f;
    A.m[nt][0] = A.m[nt][1] = -FLT_MAX;
    A.l[nt][0] = A.l[nt][1] = 0.f;
  }
}

// A warp's result to shared memory: o [8 NT heads][kPad] fp32 (kPad puts a fragment's writes in different banks), m, l [8 NT].
template <int NT>
__device__ __forceinline__ void stash(const Acc<NT>& A, float* o, float* m, float* l) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = 8 * nt + 2 * q + j;
      float sum = A.l[nt][j];
      sum += __shfl_xor_sync(kFull, sum, 4);
      sum += __shfl_xor_sync(kFull, sum, 8);
      sum += __shfl_xor_sync(kFull, sum, 16);
      if (g == 0) {
        m[h] = A.m[nt][j];
        l[h] = sum;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        o[h * kPad + 16 * mt + g] = A.o[mt][nt][j];
        o[h * kPad + 16 * mt + g + 8] = A.o[mt][nt][2 + j];
      }
    }
}
// Joins the warps' stashed results of head h: the lane's four dims relative to the largest maximum, which is returned
// with the sum.
template <int H>
__device__ __forceinline__ float4 join(const float* o, const float* m, const float* l, int h, float& M, float& sum) {
  M = -FLT_MAX;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m[w * H + h]);
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int k = w * H + h;
    const float f = exp2f(m[k] - M);
    const float4 x = *reinterpret_cast<const float4*>(o + k * kPad + 4 * (threadIdx.x & 31));
    sum += f * l[k];
    r.x += f * x.x;
    r.y += f * x.y;
    r.z += f * x.z;
    r.w += f * x.w;
  }
  return r;
}
template <bool kBf16>
__device__ __forceinline__ uint2 normalised(const float4& o, float sum) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  return pack4<kBf16>(make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

// Few (row, KV head) pairs: the warps of a CTA, and the CTAs of a cluster, share one pair's list.
template <int NT, bool kBf16>
__global__ void __launch_bounds__(kThreads, kSplitCtasPerSm<NT>) sparse_paged_kv8_split_kernel(const PagedArgs a) {
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
    if (rank == 0)
      for (int e = tid; e < a.G * kD / 8; e += kThreads) reinterpret_cast<uint4*>(out)[e] = make_uint4(0, 0, 0, 0);
    return;
  }
  uint8_t* mine = smem + warp * kWarpBytes;
  const uint32_t ktile = smem_addr(mine), vtile = ktile + 2 * kTileBytes;
  int* ids = reinterpret_cast<int*>(mine + kRowsAt);  // [step & 1][K, V][row_place]
  float4* entries = reinterpret_cast<float4*>(mine + kEntriesAt);
  const uint32_t rowBytes = static_cast<uint32_t>(a.Hkv) * a.poolHeadDim;
  const uint8_t* base = a.pool + static_cast<size_t>(r.kvh) * a.poolHeadDim + (lane & 7) * 16;
  const TileDst dst(ktile, vtile);

  struct Named {
    bool ok;        // the lane's entry names a row
    float ks, vs;   // its scales as stored
    unsigned mask;  // lanes whose entry does
  };
  auto resolve = [&](const Pages& p, int parity) {
    const PoolRows rows = list.rows_of(p);
    const Named n{rows.ok, __ldg(scales_of(a, rows.k, r.kvh)), __ldg(scales_of(a, rows.v, r.kvh)), __ballot_sync(kFull, rows.ok)};
    int* at = ids + parity * 2 * kStep + row_place(lane);
    at[0] = rows.ok ? rows.k : -1;
    at[kStep] = rows.ok ? rows.v : -1;
    return n;
  };
  auto gather = [&](int parity, int plane, unsigned mask) {
    const uint32_t o = parity * kTileBytes;
    const uint32_t d[2] = {(plane ? dst.v[0] : dst.k[0]) + o, (plane ? dst.v[1] : dst.k[1]) + o};
    gather_rows(ids + (parity * 2 + plane) * kStep, mask, d, base, rowBytes);
  };

  Acc<NT> A;
  acc_init(A);
  const int steps = max(0, (a.topK - (first - lane) + hop - 1) / hop);
  Named cur = resolve(list.pages_of(j0), 0);
  Pages p1 = list.pages_of(j1);
  __syncwarp();
  gather(0, 0, cur.mask);
  gather(0, 1, cur.mask);
  slot += hop;
  int j3 = list.at(slot);
  uint32_t qf[NT][8][2];
  float qs[NT][2];
  load_q<NT, kBf16>(static_cast<const uint4*>(a.q) + r.head0 * (kD / 8), a.G, qf, qs);
  Named next = resolve(p1, 1);
  p1 = list.pages_of(j2);
  __syncwarp();
  gather(1, 0, next.mask);
  gather(1, 1, next.mask);
  for (int i = 0; i < steps; ++i) {
    const int par = i & 1;
    const Named then = resolve(p1, par);  // step i + 2: its rows go where step i's are
    p1 = list.pages_of(j3);
    slot += hop;
    j3 = list.at(slot);
    if (cur.mask) {
      entries[lane] = entry_of(a, cur.ok, cur.ks, cur.vs);
      float s[2][NT][4];
      uint32_t pb[2][NT][2];
      cp_async_wait<3>();  // this lane's share of the K tile; its V tile and the next step's two may be in flight
      __syncwarp();
      scores32<NT>(s, ktile + par * kTileBytes, qf);
      __syncwarp();  // every lane is done with the K tile
      gather(par, 0, then.mask);
      softmax32<NT, kBf16>(A, s, qs, entries, pb);
      cp_async_wait<3>();  // the V tile
      __syncwarp();
      values32<NT>(A, vtile + par * kTileBytes, pb);
      __syncwarp();  // every lane is done with the V tile
      gather(par, 1, then.mask);
    } else {  // nothing was copied for this step
      __syncwarp();
      gather(par, 0, then.mask);
      gather(par, 1, then.mask);
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
  float* mc = lw + kWarps * H;                  // [H], then the sums
  stash<NT>(A, ow + warp * H * kPad, mw + warp * H, lw + warp * H);
  __syncthreads();
  for (int h = warp; h < a.G; h += kWarps) {
    float M, sum;
    const float4 o = join<H>(ow, mw, lw, h, M, sum);
    if (a.split > 1) {
      *reinterpret_cast<float4*>(oc + h * kPad + 4 * lane) = o;
      if (lane == 0) {
        mc[h] = M;
        mc[H + h] = sum;
      }
    } else {
      out[h * 32 + lane] = normalised<kBf16>(o, sum);
    }
  }
  if (a.split == 1) return;
  // Join over the cluster: head h by one warp of it.
  cluster_sync_all();
  const uint32_t ocAddr = smem_addr(oc), mcAddr = smem_addr(mc);
  for (int h = rank * kWarps + warp; h < a.G; h += a.split * kWarps) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float ms[kMaxCluster], M = -FLT_MAX, sum = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      ms[c] = c < a.split ? cluster_ld(cluster_addr(mcAddr + h * 4, c)) : -FLT_MAX;
      M = fmaxf(M, ms[c]);
    }
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < a.split) {
        const float f = exp2f(ms[c] - M);
        const float4 x = cluster_ld4(cluster_addr(ocAddr + (h * kPad + 4 * lane) * 4, c));
        sum += f * cluster_ld(cluster_addr(mcAddr + (H + h) * 4, c));
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
    out[h * 32 + lane] = normalised<kBf16>(o, sum);
  }
  cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

// Many rows: a warp takes one KV head of a row and the whole list, a group of kH warps (4 or 2) kH heads of the row, a CTA
// 4 / kH groups.  The heads share the list, so a group's warps resolve its entries once for all of them, a chunk of 32 kH
// at a time, 32 per warp: row ids, and per head what the softmax needs, go to shared memory for every warp of the group.  Chunk c + 1's row ids are written before the barrier that opens chunk c (its first rows are
// gathered in chunk c's last step), its scales, which are loaded meanwhile, behind chunk c's steps.  Groups share
// nothing: each has a barrier of its own and leaves when it is done.
template <int NT>
constexpr int kWarpTiles = 2 * kTileBytes > 8 * NT * (kPad + 2) * 4 ? 2 * kTileBytes : 8 * NT * (kPad + 2) * 4;  // later: O, m, l
template <int NT>
constexpr int kIdsAt = kWarps * kWarpTiles<NT>;                    // [chunk % 3][warp's step][K, V][kStep] row ids
template <int NT>
constexpr int kMasksAt = kIdsAt<NT> + 3 * kWarps * kStep * 2 * 4;  // [chunk % 3][warp's step] entries that name a row
template <int NT>
constexpr int kChunkEntriesAt = kMasksAt<NT> + 64;                 // [chunk & 1][warp][kH kStep]
template <int NT, int kH>
constexpr int kRowsSmem = kChunkEntriesAt<NT> + 2 * kWarps * kH * kStep * 16;

template <int NT, bool kBf16, int kH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<NT>) sparse_paged_kv8_rows_kernel(const PagedArgs a, int items) {
  constexpr int kChunk = kH * kStep;  // entries
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / kH, w0 = group * kH;          // this group and its first warp
  const int tid = static_cast<int>(threadIdx.x) - w0 * 32;  // within the group
  const int item = static_cast<int>(blockIdx.x) * (kWarps / kH) + group;
  if (item >= items) return;
  auto group_sync = [&] {
    if (group == 0)
      asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kH) : "memory");
    else
      asm volatile("bar.sync 2, %0;\n" ::"n"(32 * kH) : "memory");
  };
  Row r = row_of(a, item, kH);
  List list(a, r);
  const int j0 = list.at(tid), j1 = list.at(tid + kChunk);
  int slot = tid + 2 * kChunk, j2 = list.at(slot);
  row_lengths(a, r);
  list.L = r.L;
  uint2* out = static_cast<uint2*>(a.o) + r.head0 * (kD / 4);  // kH G heads of 4 values each
  if (r.t >= r.n) {
    for (int e = tid; e < kH * a.G * kD / 8; e += 32 * kH) reinterpret_cast<uint4*>(out)[e] = make_uint4(0, 0, 0, 0);
    return;
  }
  uint8_t* mine = smem + warp * kWarpTiles<NT>;
  const uint32_t ktile = smem_addr(mine), vtile = ktile + kTileBytes;
  int* ids = reinterpret_cast<int*>(smem + kIdsAt<NT>) + w0 * 2 * kStep;
  unsigned* masks = reinterpret_cast<unsigned*>(smem + kMasksAt<NT>) + w0;
  float4* entries = reinterpret_cast<float4*>(smem + kChunkEntriesAt<NT>) + w0 * kChunk;
  const uint32_t rowBytes = static_cast<uint32_t>(a.Hkv) * a.poolHeadDim;
  const uint8_t* base = a.pool + static_cast<size_t>(r.kvh + warp - w0) * a.poolHeadDim + (lane & 7) * 16;
  const TileDst dst(ktile, vtile);

  struct Scales {
    bool ok;
    float k[kH], v[kH];
  };
  auto put_rows = [&](const Pages& p, int buf) {  // row ids of the thread's entry of a chunk, and its scales' loads
    const PoolRows rows = list.rows_of(p);
    int* at = ids + (buf * kWarps + warp - w0) * 2 * kStep + row_place(lane);
    at[0] = rows.ok ? rows.k : -1;
    at[kStep] = rows.ok ? rows.v : -1;
    const unsigned mask = __ballot_sync(kFull, rows.ok);
    if (lane == 0) masks[buf * kWarps + warp - w0] = mask;
    Scales s;
    s.ok = rows.ok;
    const float *ks = scales_of(a, rows.k, r.kvh), *vs = scales_of(a, rows.v, r.kvh);
#pragma unroll
    for (int c = 0; c < kH; ++c) {
      s.k[c] = __ldg(ks + c);
      s.v[c] = __ldg(vs + c);
    }
    return s;
  };
  auto put_entries = [&](const Scales& s, int buf) {
#pragma unroll
    for (int c = 0; c < kH; ++c) entries[(buf * kWarps + c) * kChunk + tid] = entry_of(a, s.ok, s.k[c], s.v[c]);
  };
  auto gather = [&](int buf, int step, int plane, unsigned mask) {
    gather_rows(ids + ((buf * kWarps + step) * 2 + plane) * kStep, mask, plane ? dst.v : dst.k, base, rowBytes);
  };
  Acc<NT> A;
  acc_init(A);
  Scales sc = put_rows(list.pages_of(j0), 0);
  Pages p1 = list.pages_of(j1);
  uint32_t qf[NT][8][2];
  float qs[NT][2];
  load_q<NT, kBf16>(static_cast<const uint4*>(a.q) + (r.head0 + (warp - w0) * a.G) * (kD / 8), a.G, qf, qs);
  put_entries(sc, 0);
  group_sync();
  unsigned mask = masks[0];  // of the current step, whose rows are gathered
  gather(0, 0, 0, mask);
  gather(0, 0, 1, mask);
  const int chunks = (a.topK + kChunk - 1) / kChunk;
  int buf = 0;
  for (int c = 0; c < chunks; ++c) {
    const int nbuf = buf == 2 ? 0 : buf + 1;
    sc = put_rows(p1, nbuf);
    p1 = list.pages_of(j2);
    slot += kChunk;
    j2 = list.at(slot);
    group_sync();
#pragma unroll 1
    for (int e = 0; e < kH; ++e) {
      const bool last = e == kH - 1;
      const int gbuf = last ? nbuf : buf, ge = last ? 0 : e + 1;  // the next step
      const unsigned next = masks[gbuf * kWarps + ge];
      if (mask) {
        float s[2][NT][4];
        uint32_t pb[2][NT][2];
        cp_async_wait<1>();  // this lane's share of the K tile; the V tile may be in flight
        __syncwarp();
        scores32<NT>(s, ktile, qf);
        __syncwarp();  // every lane is done with the K tile
        gather(gbuf, ge, 0, next);
        softmax32<NT, kBf16>(A, s, qs, entries + ((c & 1) * kWarps + warp - w0) * kChunk + e * kStep, pb);
        cp_async_wait<1>();  // the V tile; the next K tile may be in flight
        __syncwarp();
        values32<NT>(A, vtile, pb);
        __syncwarp();  // every lane is done with the V tile
        gather(gbuf, ge, 1, next);
      } else {
        gather(gbuf, ge, 0, next);
        gather(gbuf, ge, 1, next);
      }
      mask = next;
    }
    put_entries(sc, (c + 1) & 1);
    buf = nbuf;
  }
  cp_async_wait<0>();
  list.report();
  __syncwarp();  // the warp's tiles become its output buffer
  constexpr int H = 8 * NT;
  float* ow = reinterpret_cast<float*>(mine);  // [H][kPad]
  float* mw = ow + H * kPad;                   // [m, l][H]
  stash<NT>(A, ow, mw, mw + H);
  __syncwarp();
  for (int h = 0; h < a.G; ++h)
    out[((warp - w0) * a.G + h) * 32 + lane] =
        normalised<kBf16>(*reinterpret_cast<const float4*>(ow + h * kPad + 4 * lane), mw[H + h]);
}

template <int NT, bool kBf16, int kH>
cudaError_t rows_go(const PagedArgs& a, long long pairs, cudaStream_t st) {
  auto kernel = sparse_paged_kv8_rows_kernel<NT, kBf16, kH>;
  constexpr int kSmemBytes = kRowsSmem<NT, kH>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>((pairs + kWarps - 1) / kWarps), kThreads, kSmemBytes, st>>>(
      a, static_cast<int>(pairs / kH));
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
template <int NT, bool kBf16>
long long resident_clusters(int split) {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];  // 0: not asked yet; -1: none
  int dev = 0;
  const bool cached = cudaGetDevice(&dev) == cudaSuccess && dev < kDevices;
  int n = cached ? known[dev][split].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = split_config<NT>(1, split, nullptr, &at);
    auto kernel = sparse_paged_kv8_split_kernel<NT, kBf16>;
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

template <int NT, bool kBf16>
cudaError_t paged_go(PagedArgs a, long long pairs, cudaStream_t st) {
  const long long slots = static_cast<long long>(kCtasPerSm<NT>) * sm_count();  // CTAs resident at once
  // A warp per pair from two waves of such CTAs on: 2 x 700 rows of 4 heads (2.3 waves) took 202 us instead of 224, 2 x 350
  // (1.2 waves) 146 instead of 127.  With 2 heads 4096 rows (3.4 waves) 294 instead of 301, 8192 618 instead of 657, 12
  // query heads each 887 instead of 987, but 1100 + 1100 rows (1.8 waves) 213 instead of 198.  (All taken
  // before the sums' weights were rounded too, which adds 1 to 3 % to either form: 202 is 205 now, 618 626, 887 911.  Two
  // warps per pair, four heads: 223 us where one took 223.  Lists of their own per warp, for odd numbers of heads: 406 us
  // where the split form took 332, 8192 rows of one head.)
  if (a.Hkv % 2 == 0 && pairs / kWarps >= 2 * slots)
    return a.Hkv % 4 == 0 ? rows_go<NT, kBf16, 4>(a, pairs, st) : rows_go<NT, kBf16, 2>(a, pairs, st);
  // Otherwise as many CTAs per pair as leave all clusters resident at once, at most one per 128 entries of the list.
  a.split = std::min(kMaxCluster, (a.topK + kStep * kWarps - 1) / (kStep * kWarps));
  while (pairs > resident_clusters<NT, kBf16>(a.split) && a.split > 1) --a.split;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = split_config<NT>(pairs, a.split, st, &at);
  auto kernel = sparse_paged_kv8_split_kernel<NT, kBf16>;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PagedArgs>(a));
  if (e == cudaErrorInvalidValue) {  // the attribute is the context's: a new one has not got it
    (void)cudaGetLastError();
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<NT>);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PagedArgs>(a));
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sparse_paged_kv8(const QsaSparsePagedKv8Params& p, bool bf16) {
  PagedArgs a;
  a.q = p.qPtr;
  a.pool = static_cast<const uint8_t*>(p.kvPool);
  a.scale = p.kvScale;
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
  a.poolHeadDim = p.poolHeadDim;
  a.numFlatPages = p.numFlatPages;
  a.maxPagesPerSeq = p.maxPagesPerSeq;
  a.topK = p.topK;
  a.blockShift = 0;
  while ((1 << a.blockShift) < p.scaleBlock) ++a.blockShift;
  a.split = 1;
  a.sl2 = p.attentionScale * kLog2e;
  const long long pairs = static_cast<long long>(p.batchSize) * p.seqLen * p.numKVHeads;
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  if (bf16) return a.G <= 8 ? paged_go<1, true>(a, pairs, st) : paged_go<2, true>(a, pairs, st);
  return a.G <= 8 ? paged_go<1, false>(a, pairs, st) : paged_go<2, false>(a, pairs, st);
}

}  // namespace qsa
