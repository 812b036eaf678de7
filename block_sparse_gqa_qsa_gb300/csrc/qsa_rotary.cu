// qsa_rotary.cu -- rotary positions (qsa_rotary): pairs (a, b) of a head turn
// by p f_i,
//   y_a = m (x_a cos - x_b sin),  y_b = m (x_b cos + x_a sin),
// at positions that the caller names, for pairs of either layout.
//
// A stream: every rotated element is read and written once, so HBM bounds a
// large call and latency a small one.  A thread owns one vector of a token's
// pairs (of up to 16 bytes; half layout: a vector and its partner) for several
// heads: it forms their cosines and sines once, in registers, and the heads'
// loads are independent of each other and all on their way before the first is
// used.  Neighbouring threads hold neighbouring vectors of a head, so that a
// warp reads and writes whole rows.  Out of place, further threads copy the
// vectors behind rotDim.
#include <algorithm>

#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads of a thread in flight

struct RotaryArgs {
  const void* x;
  void* y;
  const int32_t* positions;
  long long xToken, xHead, yToken, yHead;  // elements
  int heads, rot;
  int rotVectors, vectors;  // per head: vectors (or pairs of vectors) that turn, and with those that are copied
  int copyBytes;            // of a vector that is copied: 16, or V elements
  int headGroups;           // threads that share a (token, vector): thread g takes heads g, g + headGroups, ..
  unsigned units;           // tokens * headGroups * vectors
  float magnitude;
  bool inverse;
  unsigned long long turn[kRotaryMaxPairs];
};

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, float& x) { x = v; }

template <typename T, int V>
struct __align__(sizeof(T) * V) Vec {
  T v[V];
};

// Vector `at` of the heads g, g + groups, .. from x to y.
template <typename W, typename T>
__device__ __forceinline__ void copy_heads(const T* x, T* y, int at, long long xHop, long long yHop, int g, int heads, int groups) {
  for (int h = g; h < heads; h += kBatch * groups, x += kBatch * xHop, y += kBatch * yHop) {
    W v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k * groups < heads) v[k] = reinterpret_cast<const W*>(x + k * xHop)[at];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k * groups < heads) reinterpret_cast<W*>(y + k * yHop)[at] = v[k];
  }
}

// kInter: pairs (2i, 2i + 1), else (i, i + rot / 2).  V elements a vector; interleaved with V = 1 a vector is one pair's
// two elements, read one by one.
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  constexpr bool kSingle = kInter && V == 1;
  constexpr bool kTwo = !kInter || kSingle;            // a unit is two vectors
  constexpr int kPairs = kInter ? (V == 1 ? 1 : V / 2) : V;
  using Vector = Vec<T, V>;
  const unsigned unit = blockIdx.x * kThreads + threadIdx.x;
  if (unit >= a.units) return;
  const unsigned rest = unit / a.vectors, c = unit - rest * a.vectors;
  const unsigned token = rest / a.headGroups, g = rest - token * a.headGroups;
  const int p = __ldg(a.positions + token);
  if (p < 0) return;
  const T* x = static_cast<const T*>(a.x) + token * a.xToken + g * a.xHead;
  T* y = static_cast<T*>(a.y) + token * a.yToken + g * a.yHead;
  const long long xHop = a.xHead * a.headGroups, yHop = a.yHead * a.headGroups;
  if (c >= static_cast<unsigned>(a.rotVectors)) {  // behind rotDim: copied (out of place only)
    x += a.rot;
    y += a.rot;
    const int at = static_cast<int>(c) - a.rotVectors;
    if (V * sizeof(T) < 16 && a.copyBytes == 16)
      copy_heads<uint4>(x, y, at, xHop, yHop, g, a.heads, a.headGroups);
    else
      copy_heads<Vector>(x, y, at, xHop, yHop, g, a.heads, a.headGroups);
    return;
  }
  const int at = kSingle ? 2 * c : c * V, partner = at + (kSingle ? 1 : a.rot / 2);
  float cs[kPairs], sn[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    // p * turn mod 2^64 is the angle as an exact fraction of a turn; its top 32 bits, signed, are half turns * 2^31
    const unsigned long long t = a.turn[c * kPairs + i] * static_cast<unsigned>(p);
    sincospif(static_cast<float>(static_cast<int>(static_cast<unsigned>(t >> 32))) * 0x1p-31f, &sn[i], &cs[i]);
    cs[i] *= a.magnitude;
    sn[i] *= a.inverse ? -a.magnitude : a.magnitude;
  }
  for (int h = g; h < a.heads; h += kBatch * a.headGroups, x += kBatch * xHop, y += kBatch * yHop) {
    Vector u[kBatch], w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k * a.headGroups < a.heads) {
        u[k] = *reinterpret_cast<const Vector*>(x + k * xHop + at);
        if constexpr (kTwo) w[k] = *reinterpret_cast<const Vector*>(x + k * xHop + partner);
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k * a.headGroups < a.heads) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          T& ra = kTwo ? u[k].v[i] : u[k].v[(2 * i) % V];
          T& rb = kTwo ? w[k].v[i] : u[k].v[(2 * i + 1) % V];
          const float xa = to_f32(ra), xb = to_f32(rb);
          from_f32(fmaf(xa, cs[i], -(xb * sn[i])), ra);
          from_f32(fmaf(xb, cs[i], xa * sn[i]), rb);
        }
        *reinterpret_cast<Vector*>(y + k * yHop + at) = u[k];
        if constexpr (kTwo) *reinterpret_cast<Vector*>(y + k * yHop + partner) = w[k];
      }
  }
}

// Whether addresses and strides of x and y are multiples of v elements.
bool lies_on(const QsaRotaryParams& p, int v, size_t size) {
  const auto ok = [&](const void* q, int64_t token, int64_t head) {
    return reinterpret_cast<uintptr_t>(q) % (v * size) == 0 && (p.numTokens == 1 || token % v == 0) &&
           (p.numHeads == 1 || head % v == 0);
  };
  return ok(p.x, p.xTokenStride, p.xHeadStride) && ok(p.y, p.yTokenStride, p.yHeadStride);
}

template <typename T, int V>
cudaError_t rotary_go(const QsaRotaryParams& p, const RotaryTurns& rt) {
  RotaryArgs a;
  a.x = p.x;
  a.y = p.y;
  a.positions = p.positions;
  a.xToken = p.xTokenStride;
  a.xHead = p.xHeadStride;
  a.yToken = p.yTokenStride;
  a.yHead = p.yHeadStride;
  a.heads = p.numHeads;
  a.rot = p.rotDim;
  a.rotVectors = p.interleaved && V > 1 ? p.rotDim / V : p.rotDim / 2 / V;
  constexpr int kWide = 16 / sizeof(T);
  const int rest = p.x == p.y ? 0 : p.headDim - p.rotDim;
  const bool wide = rest % kWide == 0 && p.rotDim % kWide == 0 && lies_on(p, kWide, sizeof(T));
  a.copyBytes = wide ? 16 : V * sizeof(T);
  a.vectors = a.rotVectors + rest * static_cast<int>(sizeof(T)) / a.copyBytes;
  a.magnitude = p.magnitude;
  a.inverse = p.inverse != 0;
  std::copy(rt.turn, rt.turn + kRotaryMaxPairs, a.turn);
  // Up to 16 heads a thread (16384 tokens of 36 heads: 50.2 us, with 8 54.6), as few as leave every SM its threads.
  const long long each = static_cast<long long>(p.numTokens) * a.vectors, want = 2048LL * sm_count();
  const int perThread = static_cast<int>(std::max(1LL, std::min(16LL, each * p.numHeads / want)));
  a.headGroups = (p.numHeads + perThread - 1) / perThread;
  a.units = static_cast<unsigned>(each * a.headGroups);
  const unsigned blocks = (a.units + kThreads - 1) / kThreads;
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  if (p.interleaved)
    rotary_kernel<T, V, true><<<blocks, kThreads, 0, st>>>(a);
  else
    rotary_kernel<T, V, false><<<blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// Whether vectors of v elements cut every rotated half (pair row) and every row's rest, at aligned addresses.
bool fits(const QsaRotaryParams& p, int v, size_t size) {
  const int piece = p.interleaved ? p.rotDim : p.rotDim / 2;
  return piece % v == 0 && (p.x == p.y || (p.headDim - p.rotDim) % v == 0) && lies_on(p, v, size);
}

template <typename T>
cudaError_t rotary_t(const QsaRotaryParams& p, const RotaryTurns& rt) {
  constexpr int kMost = 16 / sizeof(T);
  if (fits(p, kMost, sizeof(T))) return rotary_go<T, kMost>(p, rt);
  if (fits(p, kMost / 2, sizeof(T))) return rotary_go<T, kMost / 2>(p, rt);
  if constexpr (kMost == 8)
    if (fits(p, 2, sizeof(T))) return rotary_go<T, 2>(p, rt);
  return rotary_go<T, 1>(p, rt);
}

}  // namespace

cudaError_t launch_rotary(const QsaRotaryParams& p, const RotaryTurns& rt, int elem) {
  return elem == 0 ? rotary_t<__half>(p, rt) : elem == 1 ? rotary_t<__nv_bfloat16>(p, rt) : rotary_t<float>(p, rt);
}

}  // namespace qsa
