// qsa_store_kv4.cu -- new tokens' keys and values into a 4-bit paged pool
// (qsa_store_kv4): a row of 128 values x becomes codes c, group scales s_j and
// a row scale t,
//   t = min { 2^k : max |x| <= 2688 2^k },  s_j = e4m3(max_j |x| / (6 t)),  c = e2m1(x / (s_j t)).
//
// A stream: 256 bytes in and 80 out a row (and 256 more where the dense values
// are asked for), so HBM bounds a large call and latency a small one.  Eight
// lanes take a row, one 16-value group each; the row's maximum and its eight
// scale bytes are joined with shuffles, so a row is written as 64 bytes of
// codes and one 16-byte scale chunk.
//
// Quotients that meet a border between two codes (or scales) exactly have to be
// seen as such.  t is a power of two, s_j has 4 significant bits and x at most 11,
// so a quotient lies on a border or 2^-11 of itself away from it; a product with
// a reciprocal, off by 2^-22, is rounded to 2^-16 (codes: an addend of 192) or to
// 16 bits (scales), which puts it back on the border and no other one there.
// (Two divisions and a corrected quotient instead: 50 us for 4 x 16384 ragged
// rows of 4 heads, issue slots 77 % busy.)
#include <algorithm>

#include "qsa_internal.h"
#include "qsa_kv4.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;  // of a row
constexpr int kRowsPerCta = kThreads / kLanes;

struct StoreArgs {
  const void *k, *v;
  void *kOut, *vOut;  // may be null
  const int32_t* ctx;
  const int32_t* newLen;  // may be null
  uint8_t* pool;
  const int32_t* pageTable;
  int32_t* status;  // may be null
  long long kStride, vStride;  // elements between tokens
  int S, Hkv, rowBytes, numFlatPages, maxPagesPerSeq;
  unsigned rows;  // 2 B S Hkv
};

// Words i = 0..7 of a group: values 2 i and 2 i + 1.
__device__ __forceinline__ uint32_t word_of(const uint4 (&r)[2], int i) {
  const uint4& q = r[i >> 2];
  return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Two values times u, rounded to the type, saturating (a scale may round up, so that fp16's largest values are held as up to
// 1/16 more); NaN stays NaN.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_saturated(float lo, float hi) {
  uint32_t d;
  if constexpr (kBf16)  // bf16's end lies far above 2688 2^48
    d = pack_bf162(lo, hi);
  else
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) store_kv4_kernel(const StoreArgs a) {
  const unsigned row = blockIdx.x * kRowsPerCta + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  // rows in the order token, plane, head: a token's rows are neighbours in the pool
  const unsigned rest = row / a.Hkv, h = row - rest * a.Hkv;
  const int plane = rest & 1;
  const unsigned bt = rest >> 1, b = bt / a.S;
  const int t = static_cast<int>(bt - b * a.S);
  const bool in = row < a.rows;
  int L = 0, n = 0;
  if (in) {
    L = max(__ldg(a.ctx + b), 0);
    n = max(0, min(a.newLen ? __ldg(a.newLen + b) : a.S, min(a.S, L)));
  }
  void* out = plane ? a.vOut : a.kOut;
  uint4* dense = in && out ? static_cast<uint4*>(out) + ((static_cast<size_t>(bt) * a.Hkv + h) * kLanes + l) * 2 : nullptr;
  const bool live = t < n;
  if (in && !live && dense) dense[0] = dense[1] = make_uint4(0, 0, 0, 0);
  // a warp's four rows go on together (the shuffles below); those that are not live store nothing
  if (__all_sync(kFull, !live)) return;
  uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  int page = -1;
  const int p = L - n + t;
  if (live) {
    const uint16_t* x = static_cast<const uint16_t*>(plane ? a.v : a.k) + bt * (plane ? a.vStride : a.kStride);
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(h) * 128) + 2 * l;
    raw[0] = __ldg(src);
    raw[1] = __ldg(src + 1);
    if ((p >> 7) < a.maxPagesPerSeq)
      page = __ldg(a.pageTable + (static_cast<size_t>(b) * 2 + plane) * a.maxPagesPerSeq + (p >> 7));
  }
  // the group's largest magnitude, as bits (their order is that of the magnitudes)
  constexpr uint32_t kInf = kBf16 ? 0x7f80 : 0x7c00;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, word_of(raw, i) & 0x7fff7fff);
  m = max(m & 0xffff, m >> 16);
  const bool finite = m < kInf;
  if (!finite) {  // of the finite ones
    m = 0;
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = word_of(raw, i >> 1) >> (16 * (i & 1)) & 0x7fff;
      m = max(m, x < kInf ? x : 0u);
    }
  }
  const float amax = unpack2<kBf16>(m).x;
  uint32_t top = m;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
  // t = 2^k, k the smallest with top <= 2688 2^k: the bits of a float count up with it, 2^23 to a power of two
  const int above = __float_as_int(unpack2<kBf16>(top).x) - __float_as_int(2688.0f);
  const int k = min(48, max(-48, (above + 0x7fffff) >> 23));
  const float ts = __int_as_float((127 + k) << 23), tinv = __int_as_float((127 - k) << 23);
  const float want = amax * tinv * (1.0f / kE2m1Max);
  uint32_t s8 = f32_to_e4m3(fmaf(-256.f, want, fmaf(256.f, want, want)), 0.f, 0.f, 0.f);  // saturates at 448
  uint32_t lo, hi;
  e4m3_to_f16(s8, lo, hi);
  const float s = __low2float(*reinterpret_cast<const __half2*>(&lo));
  const float unit = s * ts;  // exact
  const float inv = s == 0.f ? 0.f : rcp_approx(unit);
  uint32_t code[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<kBf16>(word_of(raw, 4 * w + i));
      const uint64_t r = ffma2(pack_f2(x.x, x.y), pack_f2(inv, inv), pack_f2(192.f, 192.f));
      q[2 * i] = copysignf(lo_f2(r) - 192.f, x.x);
      q[2 * i + 1] = copysignf(hi_f2(r) - 192.f, x.y);
    }
    code[w] = finite ? f32_to_e2m1(q) : 0;
  }
  if (!finite) s8 = 0x7f;
  // the row's scale bytes: lanes 0..3 of it join theirs in word 0, 4..7 in word 1
  uint32_t word = (s8 & 0xff) << (8 * (l & 3));
  word |= __shfl_xor_sync(kFull, word, 1);
  word |= __shfl_xor_sync(kFull, word, 2);
  const uint32_t other = __shfl_xor_sync(kFull, word, 4);
  if (!live) return;
  if (static_cast<unsigned>(page) < static_cast<unsigned>(a.numFlatPages)) {
    uint8_t* dst = a.pool + ((static_cast<size_t>(page) * kTokensPerPage + (p & 127)) * a.Hkv + h) * a.rowBytes;
    *reinterpret_cast<uint2*>(dst + 8 * l) = make_uint2(code[0], code[1]);
    if (l == 0) *reinterpret_cast<uint4*>(dst + kKv4Codes) = make_uint4(word, other, __float_as_uint(ts), 0);
  } else if (a.status) {
    atomicOr(a.status, kErrBadPage);
  }
  if (dense) {
    uint32_t v[8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t c[4];
      e2m1_to_f16(code[w], c[0], c[1], c[2], c[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
        const float u = finite ? unit : NAN;
        v[4 * w + i] = pack_saturated<kBf16>(f.x * u, f.y * u);
      }
    }
    dense[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dense[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace

cudaError_t launch_store_kv4(const QsaStoreKv4Params& p, bool bf16) {
  StoreArgs a;
  a.k = p.k;
  a.v = p.v;
  a.kOut = p.kOut;
  a.vOut = p.vOut;
  a.ctx = p.contextLengths;
  a.newLen = p.newLengths;
  a.pool = static_cast<uint8_t*>(p.kvPool);
  a.pageTable = p.pageTable;
  a.status = p.status;
  a.kStride = p.kTokenStride;
  a.vStride = p.vTokenStride;
  a.S = p.seqLen;
  a.Hkv = p.numKVHeads;
  a.rowBytes = p.poolRowBytes;
  a.numFlatPages = p.numFlatPages;
  a.maxPagesPerSeq = p.maxPagesPerSeq;
  a.rows = static_cast<unsigned>(2LL * p.batchSize * p.seqLen * p.numKVHeads);
  const unsigned blocks = (a.rows + kRowsPerCta - 1) / kRowsPerCta;
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  if (bf16)
    store_kv4_kernel<true><<<blocks, kThreads, 0, st>>>(a);
  else
    store_kv4_kernel<false><<<blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace qsa
