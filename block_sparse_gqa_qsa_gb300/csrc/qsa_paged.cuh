// qsa_paged.cuh -- what the attention kernels over quantised paged pools
// (8 bits and 4 bits) share: their arguments, from list entries to pool rows, the
// online softmax of a step of 32 keys, and the join of several warps' results.
#pragma once

#include <cfloat>

#include "qsa_internal.h"
#include "qsa_kv8.cuh"

namespace qsa {

constexpr int kPagedThreads = 128;
constexpr int kPagedWarps = kPagedThreads / 32;
constexpr int kD = 128;
constexpr int kStep = 32;  // list entries of a warp's step
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct PagedArgs {
  const void* q;
  const uint8_t* pool;
  const float* scale;  // 8-bit pool only
  const int32_t* pageTable;
  const int32_t* indices;
  const int32_t* ctx;
  const int32_t* newLen;  // may be null
  void* o;
  int32_t* status;  // may be null
  int S, Hq, Hkv, G, poolHeadDim /* bytes of a pool row */, numFlatPages, maxPagesPerSeq, topK;
  int blockShift;  // log2(scaleBlock), 8-bit pool only
  int split;       // CTAs per pair: the cluster size
  float sl2;       // attentionScale * log2(e)
  float* lse;      // 4-bit pool only; may be null
};

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// A meeting of the cluster's threads that waits for no write: what a thread has read stays read, and nothing that one of them
// writes before it is read behind it.  (A releasing arrival waits for the thread's global writes.)
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.aligned;\n" ::: "memory");
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

// Online softmax of a step: s becomes the weights relative to the running maximum, returned in fp16 as the B
// fragments of the second product.  The maximum moves only when a weight would pass 2^kHeadroom (the weights
// are relative numbers: nothing is lost by their being up to 256 instead of 1), so that O is hardly ever
// rescaled after a warp's first step, and a step's maximum over the lanes is formed only then.  The sums use the weights as the second product does, rounded to 11 bits: where
// few keys decide, a rounding that only one of the two had would show in an fp16 output (up to 2^-11 of it, as much as
// its half step).  The maximum starts at the lowest finite number, so that an entry that names nothing
// (-inf) weighs 0 even before the first that does.  entries[i], of key i: x = K scale * attentionScale * log2(e),
// y = log2(V scale), z = 1 / V scale; (0, -inf, 0) for an entry that names nothing.  (Entries of two values, 4-bit pool:
// those of the lane's four keys lie together at `entries`; z = 2^-y, kept finite where it meets a weight of 0.)
// kLse: ls gathers the sums of the weights as they are before the rounding.
template <int NT, bool kBf16, bool kLse = false, typename Entry>
__device__ __forceinline__ void softmax32(Acc<NT>& A, float (&s)[2][NT][4], const float (&qs)[NT][2],
                                          const Entry* entries, uint32_t (&pb)[2][NT][2],
                                          float (*ls)[2] = nullptr) {
  constexpr float kHeadroom = 8.f;
  float ks[4], lv[4], iv[4];  // of the lane's keys
  if constexpr (sizeof(Entry) == sizeof(float4)) {
    const int key = key_of((threadIdx.x & 31) >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Entry e = entries[key + 16 * (i >> 1) + 2 * (i & 1)];
      ks[i] = e.x;
      lv[i] = e.y;
      iv[i] = e.z;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 e = reinterpret_cast<const float4*>(entries)[i];
      ks[2 * i] = e.x;
      lv[2 * i] = e.y;
      ks[2 * i + 1] = e.z;
      lv[2 * i + 1] = e.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) iv[i] = fminf(ex2_ftz(-lv[i]), 0x1p126f);
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
        // bf16: the K scale first (the product is below 2^31, 4-bit pool 2^34, so with scales below 2^96, 2^93, only a logit
        // itself overflows)
        x = kBf16 ? fmaf(x * ks[i], qs[nt][h], lv[i]) : fmaf(x, ks[i], lv[i]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[nt][h] = fmaxf(fmaxf(s[0][nt][h], s[0][nt][2 + h]), fmaxf(s[1][nt][h], s[1][nt][2 + h]));
      move |= mx[nt][h] > A.m[nt][h] + kHeadroom;
    }
  }
  if (__any_sync(kFull, move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float al[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        for (int o = 4; o < 32; o <<= 1) mx[nt][h] = fmaxf(mx[nt][h], __shfl_xor_sync(kFull, mx[nt][h], o));
        const float mn = fmaxf(A.m[nt][h], mx[nt][h]);
        al[h] = ex2_ftz(A.m[nt][h] - mn);
        A.m[nt][h] = mn;
        A.l[nt][h] *= al[h];
        if constexpr (kLse) ls[nt][h] *= al[h];
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
      if constexpr (kLse) {
        ls[nt][0] = fmaf(lo_f2(w), iv[i], ls[nt][0]);
        ls[nt][1] = fmaf(hi_f2(w), iv[i], ls[nt][1]);
      }
    }
    // the weights in fp16: as they are from 2^-14 on, to 2^-25 below
#pragma unroll
    for (int gk = 0; gk < 2; ++gk) {
      pb[gk][nt][0] = movmatrix_t(pack_half2(s[gk][nt][0], s[gk][nt][1]));
      pb[gk][nt][1] = movmatrix_t(pack_half2(s[gk][nt][2], s[gk][nt][3]));
    }
  }
}

constexpr int kPad = kD + 4;  // floats of a head in the merge buffers

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

// Joins the warps' stashed results of head h: the lane's four dims relative to the largest maximum, which is returned
// with the sum.
template <int H>
__device__ __forceinline__ float4 join(const float* o, const float* m, const float* l, int h, float& M, float& sum) {
  M = -FLT_MAX;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, m[w * H + h]);
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kPagedWarps; ++w) {
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

}  // namespace qsa
