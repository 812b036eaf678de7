// qsa_rotary.cu -- rotary positions (qsa_rotary): pairs (a, b) of a head turn
// by p f_i,
//   y_a = m (x_a cos - x_b sin),  y_b = m (x_b cos + x_a sin),
// at positions that the caller names, for pairs of either layout.
//
// A stream: every rotated element is read and written once, so HBM bounds a
// large call and latency a small one.  A CTA takes the heads (or a part) of a
// few tokens: it forms the tokens' cosines and sines once, in shared memory; a
// thread then owns one vector of a token's pairs (of up to 16 bytes; half
// layout: a vector and its partner) for up to 8 heads, keeps its cosines and
// sines in registers, and has four vectors on their way before the first is used.
// Neighbouring threads hold neighbouring vectors of a head.  Out of place, the
// threads then copy the vectors behind rotDim.
// 16384 tokens of 36 16-bit heads of 128, all dims turning: halves 49.6 us, pairs
// 45.4 (0.91 and 0.99 of the copy rate).  What that took: cosines and sines formed by
// every thread for itself 100 us in halves, 145 with rotDim 64 (the copying
// threads being in the same warps); formed by the CTA 76; few registers, so that
// four CTAs lie on an SM (five for pairs, whose 48 registers leave 44 bytes of a
// thread in local memory with 16-bit elements, 8 with fp32), and the first loads in
// front of the table 54; two elements to a conversion 50.
#include <algorithm>
#include <type_traits>

#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kThreads = 256;
// Of a thread: vectors of 16 bytes in flight (with 2 halves 57.8 us and pairs 51.2), heads (with 4 48.6 and 55.6, with 16
// 50.9 and 46.6).
constexpr int kVectors = 4;
constexpr int kMostHeads = 8;

struct RotaryArgs {
  const void* x;
  void* y;
  const int32_t* positions;
  long long xToken, xHead, yToken, yHead;  // elements
  int tokens, heads, rot;
  int rotVectors, copyVectors;  // per head: vectors (or pairs of vectors) that turn; vectors that are copied
  int copyBytes;                // of the latter
  int headGroups;               // threads that share a (token, vector): thread g takes heads g, g + headGroups, ..
  int ctaTokens, ctaGroups;     // of a CTA
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

// Two 16-bit values of a word.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return std::is_same_v<T, __nv_bfloat16> ? pack_bf162(lo, hi) : pack_half2(lo, hi);
}
// (a, b) turned by (c, s).
__device__ __forceinline__ float2 turned(float a, float b, const float2& cs) {
  return make_float2(fmaf(a, cs.x, -(b * cs.y)), fmaf(b, cs.x, a * cs.y));
}

template <typename T, int V>
struct __align__(sizeof(T) * V) Vec {
  T v[V];
};

// Vector `at` of the heads g, g + groups, .. from x to y.
template <typename W, typename T>
__device__ __forceinline__ void copy_heads(const T* x, T* y, int at, long long xHop, long long yHop, int g, int heads, int groups) {
  constexpr int kBatch = kVectors;
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
__global__ void __launch_bounds__(kThreads, kInter && V * sizeof(T) == 16 ? 5 : 4) rotary_kernel(const RotaryArgs a) {
  constexpr bool kSingle = kInter && V == 1;
  constexpr bool kTwo = !kInter || kSingle;            // a unit is two vectors
  constexpr int kPairs = kInter ? (V == 1 ? 1 : V / 2) : V;
  constexpr int kFlight = V * sizeof(T) == 16 ? kVectors : 2 * kVectors;  // (8-byte vectors: 20.2 us with 4, 19.2 with 8)
  constexpr int kBatch = kTwo ? kFlight / 2 : kFlight;  // heads in flight
  using Vector = Vec<T, V>;
  extern __shared__ float2 table[];  // [ctaTokens][rot / 2] cosine, sine, times the magnitude
  const int token0 = blockIdx.x * a.ctaTokens, g0 = blockIdx.y * a.ctaGroups, pairs = a.rot >> 1;
  const long long xHop = a.xHead * a.headGroups, yHop = a.yHead * a.headGroups;
  auto row = [&](auto* base, long long token, long long head, int t, int g) { return base + (token0 + t) * token + g * head; };

  // this thread's vector (a CTA has at most one for each), and its first heads' values on their way
  const int rest = threadIdx.x / a.rotVectors, c = threadIdx.x - rest * a.rotVectors;
  const int t = rest / a.ctaGroups, g = g0 + rest - t * a.ctaGroups;
  const bool mine = t < a.ctaTokens && token0 + t < a.tokens && g < a.headGroups;
  const int at = kSingle ? 2 * c : c * V, partner = at + (kSingle ? 1 : pairs);
  const T* x = row(static_cast<const T*>(a.x), a.xToken, a.xHead, t, g);
  Vector u[kBatch], w[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k * a.headGroups < a.heads) {
        u[k] = *reinterpret_cast<const Vector*>(x + k * xHop + at);
        if constexpr (kTwo) w[k] = *reinterpret_cast<const Vector*>(x + k * xHop + partner);
      }
  };
  if (mine) load(g);

  for (int i = threadIdx.x; i < a.ctaTokens * pairs; i += kThreads) {
    const int token = token0 + i / pairs, k = i % pairs;
    const int p = token < a.tokens ? __ldg(a.positions + token) : -1;
    if (p < 0) continue;
    // p * turn mod 2^64 is the angle as an exact fraction of a turn; its top 32 bits, signed, are half turns * 2^31
    const unsigned long long angle = a.turn[k] * static_cast<unsigned>(p);
    float cv, sv;
    sincospif(static_cast<float>(static_cast<int>(static_cast<unsigned>(angle >> 32))) * 0x1p-31f, &sv, &cv);
    table[i] = make_float2(cv * a.magnitude, sv * (a.inverse ? -a.magnitude : a.magnitude));
  }
  __syncthreads();

  if (mine && __ldg(a.positions + token0 + t) >= 0) {
    T* y = row(static_cast<T*>(a.y), a.yToken, a.yHead, t, g);
    float2 cs[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) cs[i] = table[t * pairs + c * kPairs + i];
    for (int h = g;;) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (h + k * a.headGroups < a.heads) {
          if constexpr (sizeof(T) == 2 && V > 1) {  // whole words
            uint32_t *p = reinterpret_cast<uint32_t*>(&u[k]), *q = reinterpret_cast<uint32_t*>(&w[k]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float2 a0 = unpack2<T>(p[i]);
              if constexpr (kInter) {
                const float2 r = turned(a0.x, a0.y, cs[i]);
                p[i] = pack2<T>(r.x, r.y);
              } else {
                const float2 b0 = unpack2<T>(q[i]), r0 = turned(a0.x, b0.x, cs[2 * i]), r1 = turned(a0.y, b0.y, cs[2 * i + 1]);
                p[i] = pack2<T>(r0.x, r1.x);
                q[i] = pack2<T>(r0.y, r1.y);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
              T& ra = kTwo ? u[k].v[i] : u[k].v[(2 * i) % V];
              T& rb = kTwo ? w[k].v[i] : u[k].v[(2 * i + 1) % V];
              const float2 r = turned(to_f32(ra), to_f32(rb), cs[i]);
              from_f32(r.x, ra);
              from_f32(r.y, rb);
            }
          }
          *reinterpret_cast<Vector*>(y + k * yHop + at) = u[k];
          if constexpr (kTwo) *reinterpret_cast<Vector*>(y + k * yHop + partner) = w[k];
        }
      h += kBatch * a.headGroups;
      if (h >= a.heads) break;
      x += kBatch * xHop;
      y += kBatch * yHop;
      load(h);
    }
  }
  if (!a.copyVectors) return;
  for (int i = threadIdx.x; i < a.ctaTokens * a.ctaGroups * a.copyVectors; i += kThreads) {
    const int r = i / a.copyVectors, v = i - r * a.copyVectors, tt = r / a.ctaGroups, gg = g0 + r - tt * a.ctaGroups;
    if (token0 + tt >= a.tokens || gg >= a.headGroups || __ldg(a.positions + token0 + tt) < 0) continue;
    const T* from = row(static_cast<const T*>(a.x), a.xToken, a.xHead, tt, gg) + a.rot;
    T* to = row(static_cast<T*>(a.y), a.yToken, a.yHead, tt, gg) + a.rot;
    if (a.copyBytes == 16)
      copy_heads<uint4>(from, to, v, xHop, yHop, gg, a.heads, a.headGroups);
    else if (a.copyBytes == 8)
      copy_heads<uint2>(from, to, v, xHop, yHop, gg, a.heads, a.headGroups);
    else if (sizeof(T) == 4 || a.copyBytes == 4)
      copy_heads<uint32_t>(from, to, v, xHop, yHop, gg, a.heads, a.headGroups);
    else
      copy_heads<uint16_t>(from, to, v, xHop, yHop, gg, a.heads, a.headGroups);
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
  a.tokens = p.numTokens;
  a.heads = p.numHeads;
  a.rot = p.rotDim;
  a.rotVectors = p.interleaved && V > 1 ? p.rotDim / V : p.rotDim / 2 / V;
  const int rest = p.x == p.y ? 0 : p.headDim - p.rotDim;
  int wide = 16 / sizeof(T);  // elements of a copied vector
  while (wide > 1 && (rest % wide || p.rotDim % wide || !lies_on(p, wide, sizeof(T)))) wide /= 2;
  a.copyBytes = wide * sizeof(T);
  a.copyVectors = rest / wide;
  a.magnitude = p.magnitude;
  a.inverse = p.inverse != 0;
  std::copy(rt.turn, rt.turn + kRotaryMaxPairs, a.turn);
  // As few heads a thread as leave every SM its threads.
  const long long each = static_cast<long long>(p.numTokens) * a.rotVectors, want = 2048LL * sm_count();
  const int perThread = static_cast<int>(std::max(1LL, std::min<long long>(kMostHeads, each * p.numHeads / want)));
  a.headGroups = (p.numHeads + perThread - 1) / perThread;
  // A CTA takes as many tokens, or as many of a token's groups, as give each of its threads a vector.
  a.ctaGroups = std::max(1, std::min(a.headGroups, kThreads / a.rotVectors));
  a.ctaTokens = std::max(1, std::min(p.numTokens, kThreads / (a.ctaGroups * a.rotVectors)));
  const dim3 grid((p.numTokens + a.ctaTokens - 1) / a.ctaTokens, (a.headGroups + a.ctaGroups - 1) / a.ctaGroups);
  const size_t smem = static_cast<size_t>(a.ctaTokens) * (p.rotDim / 2) * sizeof(float2);  // at most 16 KB
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  if (p.interleaved)
    rotary_kernel<T, V, true><<<grid, kThreads, smem, st>>>(a);
  else
    rotary_kernel<T, V, false><<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

// Whether vectors of v elements cut every rotated half (pair row), at aligned addresses.
bool fits(const QsaRotaryParams& p, int v, size_t size) {
  return (p.interleaved ? p.rotDim : p.rotDim / 2) % v == 0 && lies_on(p, v, size);
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
