// qsa_attention_kv8.cu -- sparse GQA attention over an 8-bit paged cache
// (qsa_sparse_paged_kv8): for every live row and query head
//
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = ks_j c^K_j,  v_j = vs_j c^V_j
//
// over the row's list, with e4m3 codes c and one fp32 scale per block of
// tokens and head.  In log2 units, with x_j = ks_j scale log2(e) (q . c^K_j) and
// e_j = x_j + log2(vs_j), one pass keeps M = max e_j, l = sum 2^(e_j - M) / vs_j
// and O = sum 2^(e_j - M) c^V_j: the V scale rides in the exponent, so the
// probabilities that the second product rounds to fp16 are at most 1 whatever
// the scales are, and o = O / l.  (log2(vs_j) is the hardware's approximation;
// its error enters O and l alike.)
//
// One CTA of 4 warps takes a (row, KV head) pair; when there are few pairs a
// cluster of up to 8 CTAs shares one.  The list is dealt out to the warps of
// the pair in steps of 32 entries, and each warp runs by itself, with no CTA
// barrier inside the loop: lane i resolves entry i of a step (list entry three
// steps ahead, page ids two, scales one, so that each dependent load has a
// step to arrive), and the warp gathers the 32 K and V rows of 128 bytes with
// cp.async into its own K tile and V tile.  A step's K tile is free after its
// first product, its V tile after the second, and the next step's rows start
// then: one tile of each keeps half a step of copies in flight per warp.
//
// S^T = C^K Q^T and O^T += (C^V)^T P^T are m16n8k16 MMAs in fp16 with the head
// group as N; codes are converted to fp16 pairs in registers (exact).  The
// summed dims of the first are permuted so that a lane reads its K codes as
// whole 16-byte chunks; for the second, ldmatrix transposes 16 x 16 bytes, so
// a register holds four keys of one dim.  The rows of S^T are the keys in the
// order that makes its columns the second product's fragments of P^T.
#include <algorithm>
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
// A warp's shared memory: a K tile, a V tile, the pool rows of two steps' entries (K then V), a step's Entry values.
constexpr int kRowsAt = 2 * kTileBytes;
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
// rescaled after a warp's first step.  It starts at the lowest finite number, so that an entry that names nothing
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
        if constexpr (kBf16) x *= qs[nt][h];
        x = fmaf(x, ks[i], lv[i]);
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
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& x = s[i >> 1][nt][2 * (i & 1) + h];
        x = ex2_ftz(x - A.m[nt][h]);
        A.l[nt][h] = fmaf(x, iv[i], A.l[nt][h]);
      }
    }
    // the weights in fp16: off by 2^-11 of themselves, which the output's own rounding hides
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
      // exponent e of the largest: scaled by 2^(14 - e), in two steps that stay normal; none for 0, inf and NaN
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

// Resident CTAs per SM: the register budget decides (5 at 96 registers spill and took 1333 us for an 8192-row prompt
// against 1275; 16-head groups at 168 registers 2008 against 1928).
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 4 : 2;
// The tiles, and later the merge buffers: the warps' O, m and l, then the CTA's.
template <int NT>
constexpr int kSmem = kWarps * kWarpBytes > (kWarps + 1) * 8 * NT * (kPad + 2) * 4 ? kWarps * kWarpBytes
                                                                               : (kWarps + 1) * 8 * NT * (kPad + 2) * 4;

template <int NT, bool kBf16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<NT>) sparse_paged_kv8_kernel(const PagedArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x % a.split);
  const int pair = static_cast<int>(blockIdx.x / a.split);
  // a sequence's rows from the last position down: the longest lists start first
  const int kvh = pair % a.Hkv, rowid = pair / a.Hkv;
  const int b = rowid / a.S, t = a.S - 1 - rowid % a.S;
  // the warp's first three steps of the list, on their way while the lengths are read
  const size_t bt = static_cast<size_t>(b) * a.S + t;
  const int32_t* lst = a.indices + bt * a.topK;
  const int hop = kStep * kWarps * a.split;  // entries between a warp's steps
  const int first = kStep * (rank * kWarps + warp) + lane;
  auto list_at = [&](int slot) { return slot < a.topK ? __ldg(lst + slot) : -1; };
  const int j0 = list_at(first), j1 = list_at(first + hop);
  int slot = first + 2 * hop, j2 = list_at(slot);
  const int L = max(0, min(a.ctx[b], a.maxPagesPerSeq * kTokensPerPage));
  const int n = max(0, min(a.newLen ? a.newLen[b] : a.S, min(a.S, L)));
  const size_t head0 = bt * a.Hq + static_cast<size_t>(kvh) * a.G;
  uint2* out = static_cast<uint2*>(a.o) + head0 * (kD / 4);  // 4 values each
  if (t >= n) {  // the whole cluster leaves
    if (rank == 0)
      for (int e = tid; e < a.G * kD / 8; e += kThreads) reinterpret_cast<uint4*>(out)[e] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int32_t* ptK = a.pageTable + static_cast<size_t>(b) * 2 * a.maxPagesPerSeq;
  const int32_t* ptV = ptK + a.maxPagesPerSeq;
  uint8_t* mine = smem + warp * kWarpBytes;
  const uint32_t ktile = smem_addr(mine), vtile = ktile + kTileBytes;
  int* rows = reinterpret_cast<int*>(mine + kRowsAt);  // [step & 1][K, V][row & 3][row >> 2]
  float4* entries = reinterpret_cast<float4*>(mine + kEntriesAt);
  const uint32_t rowBytes = static_cast<uint32_t>(a.Hkv) * a.poolHeadDim;
  const uint8_t* base = a.pool + static_cast<size_t>(kvh) * a.poolHeadDim + (lane & 7) * 16;

  // Resolving an entry is free of branches: what an entry cannot name is looked up at 0 and dropped.
  int bad = 0;
  struct Pages {
    int j, k, v;  // entry (-1: none), its page ids
  };
  auto pages_of = [&](int j) {
    const bool in = static_cast<unsigned>(j) < static_cast<unsigned>(L);
    bad |= !in && j != -1 ? kErrBadIndex : 0;
    const int at = in ? j >> 7 : 0;
    return Pages{in ? j : -1, __ldg(ptK + at), __ldg(ptV + at)};
  };
  struct Rows {
    bool ok;        // the lane's entry names a row
    float ks, vs;   // its scales as stored
    unsigned mask;  // lanes whose entry does
  };
  auto resolve = [&](const Pages& p, int parity) {
    Rows r;
    const bool pages = static_cast<unsigned>(p.k) < static_cast<unsigned>(a.numFlatPages) &&
                       static_cast<unsigned>(p.v) < static_cast<unsigned>(a.numFlatPages);
    r.ok = p.j >= 0 && pages;
    bad |= p.j >= 0 && !pages ? kErrBadPage : 0;
    const int krow = r.ok ? p.k * kTokensPerPage + (p.j & 127) : 0;
    const int vrow = r.ok ? p.v * kTokensPerPage + (p.j & 127) : 0;
    r.ks = __ldg(a.scale + static_cast<size_t>(krow >> a.blockShift) * a.Hkv + kvh);
    r.vs = __ldg(a.scale + static_cast<size_t>(vrow >> a.blockShift) * a.Hkv + kvh);
    r.mask = __ballot_sync(kFull, r.ok);
    int* at = rows + parity * 2 * kStep + (lane & 3) * (kStep / 4) + (lane >> 2);
    at[0] = r.ok ? krow : -1;
    at[kStep] = r.ok ? vrow : -1;
    return r;
  };
  // Gathers a step's K (plane 0) or V (1) rows into the tile, 8 lanes to a row of 128 bytes: one copy group.
  const uint32_t kdst[2] = {ktile + k_off(lane >> 3, lane & 7), ktile + k_off(lane >> 3, lane & 7)};
  const uint32_t v0 = vtile + v_off(lane >> 3, lane & 7), vdst[2] = {v0, v0 ^ 64};  // rows 4 i: bit 2 flips with i
  auto gather = [&](int parity, int plane, unsigned mask, const uint32_t (&dst)[2]) {
    const int4* at = reinterpret_cast<const int4*>(rows + (parity * 2 + plane) * kStep + (lane >> 3) * (kStep / 4));
    if (mask) {
      const int4 x = at[0], y = at[1];
      const int row[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      if (mask == kFull)
        copy_rows<true>(row, dst, base, rowBytes, std::make_index_sequence<8>{});
      else
        copy_rows<false>(row, dst, base, rowBytes, std::make_index_sequence<8>{});
    }
    cp_async_commit();
  };

  Acc<NT> A;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) A.o[mt][nt][0] = A.o[mt][nt][1] = A.o[mt][nt][2] = A.o[mt][nt][3] = 0.f;
    A.m[nt][0] = A.m[nt][1] = -FLT_MAX;
    A.l[nt][0] = A.l[nt][1] = 0.f;
  }
  const int steps = max(0, (a.topK - (first - lane) + hop - 1) / hop);
  Rows cur = resolve(pages_of(j0), 0);
  __syncwarp();
  gather(0, 0, cur.mask, kdst);
  gather(0, 1, cur.mask, vdst);
  Pages p1 = pages_of(j1);
  uint32_t qf[NT][8][2];
  float qs[NT][2];
  load_q<NT, kBf16>(static_cast<const uint4*>(a.q) + head0 * (kD / 8), a.G, qf, qs);
  for (int i = 0; i < steps; ++i) {
    const int par = (i + 1) & 1;
    const Rows next = resolve(p1, par);
    p1 = pages_of(j2);
    slot += hop;
    j2 = list_at(slot);
    if (cur.mask) {
      const float vs = read_scale(cur.vs);
      entries[lane] = cur.ok ? make_float4(read_scale(cur.ks) * a.sl2, lg2_ftz(vs), rcp_ftz(vs), 0.f)
                             : make_float4(0.f, -INFINITY, 0.f, 0.f);
      float s[2][NT][4];
      uint32_t pb[2][NT][2];
      cp_async_wait<1>();  // this lane's share of the K tile; the V tile may be in flight
      __syncwarp();
      scores32<NT>(s, ktile, qf);
      __syncwarp();  // every lane is done with the K tile
      gather(par, 0, next.mask, kdst);
      softmax32<NT, kBf16>(A, s, qs, entries, pb);
      cp_async_wait<1>();  // the V tile; the next K tile may be in flight
      __syncwarp();
      values32<NT>(A, vtile, pb);
      __syncwarp();  // every lane is done with the V tile
      gather(par, 1, next.mask, vdst);
    } else {  // nothing was copied for this step
      __syncwarp();
      gather(par, 0, next.mask, kdst);
      gather(par, 1, next.mask, vdst);
    }
    cur = next;
  }
  cp_async_wait<0>();
  bad = __reduce_or_sync(kFull, static_cast<unsigned>(bad));
  if (bad && lane == 0 && a.status) atomicOr(a.status, bad);
  __syncthreads();  // the rings become the merge buffers

  // Per warp [8 NT heads][128 dims, padded] fp32 and (m, l).  kPad puts a fragment's writes in different banks.
  constexpr int H = 8 * NT;
  float* ow = reinterpret_cast<float*>(smem);   // [kWarps][H][kPad]
  float* oc = ow + kWarps * H * kPad;           // the CTA's merged [H][kPad]
  float* mw = oc + H * kPad;                    // [kWarps][H]
  float* lw = mw + kWarps * H;
  float* mc = lw + kWarps * H;                  // [H], then the sums
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = 8 * nt + 2 * q + j;
      float l = A.l[nt][j];
      l += __shfl_xor_sync(kFull, l, 4);
      l += __shfl_xor_sync(kFull, l, 8);
      l += __shfl_xor_sync(kFull, l, 16);
      if (g == 0) {
        mw[warp * H + h] = A.m[nt][j];
        lw[warp * H + h] = l;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        ow[(warp * H + h) * kPad + 16 * mt + g] = A.o[mt][nt][j];
        ow[(warp * H + h) * kPad + 16 * mt + g + 8] = A.o[mt][nt][2 + j];
      }
    }
  __syncthreads();
  for (int h = warp; h < a.G; h += kWarps) {
    float M = -FLT_MAX, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mw[w * H + h]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(mw[w * H + h] - M);
      const float4 x = *reinterpret_cast<const float4*>(ow + (w * H + h) * kPad + 4 * lane);
      l += f * lw[w * H + h];
      o.x += f * x.x;
      o.y += f * x.y;
      o.z += f * x.z;
      o.w += f * x.w;
    }
    if (a.split > 1) {
      *reinterpret_cast<float4*>(oc + h * kPad + 4 * lane) = o;
      if (lane == 0) {
        mc[h] = M;
        mc[H + h] = l;
      }
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      out[h * 32 + lane] = pack4<kBf16>(make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
  }
  if (a.split == 1) return;
  // Join over the cluster: head h by one warp of it.
  cluster_sync_all();
  const uint32_t ocAddr = smem_addr(oc), mcAddr = smem_addr(mc);
  for (int h = rank * kWarps + warp; h < a.G; h += a.split * kWarps) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float ms[kMaxCluster], M = -FLT_MAX, l = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      ms[r] = r < a.split ? cluster_ld(cluster_addr(mcAddr + h * 4, r)) : -FLT_MAX;
      M = fmaxf(M, ms[r]);
    }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.split) {
        const float f = exp2f(ms[r] - M);
        const float4 x = cluster_ld4(cluster_addr(ocAddr + (h * kPad + 4 * lane) * 4, r));
        l += f * cluster_ld(cluster_addr(mcAddr + (H + h) * 4, r));
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    out[h * 32 + lane] = pack4<kBf16>(make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  }
  cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

template <int NT, bool kBf16>
cudaError_t paged_go(PagedArgs a, long long pairs, cudaStream_t st) {
  auto kernel = sparse_paged_kv8_kernel<NT, kBf16>;
  static_assert(kSmem<NT> <= 48 * 1024, "no attribute is set");
  // As many CTAs per pair as stay resident at once, at most one per 128 entries of the list.
  const long long slots = static_cast<long long>(kCtasPerSm<NT>) * sm_count();
  const int most = std::min(kMaxCluster, (a.topK + kStep * kWarps - 1) / (kStep * kWarps));
  a.split = static_cast<int>(std::max<long long>(1, std::min<long long>(most, slots / pairs)));
  if (pairs * a.split > 0x7fffffffLL) a.split = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<NT>;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PagedArgs>(a));
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
