// qsa_append.cu -- new tokens' keys and values into a paged cache, with the
// per-head norm and the rotation on the way (qsa_append_kv: a pool of the
// inputs' 16-bit type; qsa_append_kv8: e4m3 codes with block scales).
//
//   y = x / sqrt(mean(x^2) + eps) * (1 + w),  (y_i, y_{i+h}) rotated by p theta^(-2i/rot), h = rot / 2
//
// A stream of the packed heads: every input is read once and every output
// written once, so HBM bounds a large call and latency a small one.  A CTA
// takes the rows of one tile of kTile (or scaleBlock, where that is more)
// consecutive cache positions, aligned in the page: the tile lies in one page,
// its cos/sin table is formed once and shared by all heads, and every block of
// scales lies in one tile, so one warp owns a block and no atomics are needed.
// A warp takes one head of up to 16 of the tile's rows at a time, copied by
// cp.async into its own two-slot ring in shared memory: the next head's rows
// travel while this one is computed.  rotDim is a multiple of 16, so a row's
// 16-byte chunks of 8 values are whole rotation halves; a lane takes a chunk
// of a first half and its partner chunk (or two chunks past rotDim), so the
// rotation needs no exchange, and the D/16 lanes of a row reduce its sum of
// squares with shuffles.  For an 8-bit pool a K or V head is passed over twice
// in shared memory: its blocks' largest values first, then the codes.  Blocks
// of more than 16 tokens are copied twice (the second time from L2).
#include <algorithm>

#include "qsa_internal.h"
#include "qsa_kv8.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;  // most rows of a ring slot
constexpr int kCtasPerSm = 2;

struct AppendArgs {
  const void* qkv;
  const float* qw;
  const float* kw;
  const int32_t* ctx;
  const int32_t* newLen;  // may be null
  void* qout;
  void* kout;  // may be null
  void* vout;  // may be null
  uint8_t* pool;
  float* scale;  // 8-bit only
  const int32_t* pageTable;
  int32_t* status;  // may be null
  int S, Hq, Hkv, rot, poolHeadDim, numFlatPages, maxPagesPerSeq;
  int blockShift;        // log2(scaleBlock)
  int tile;              // positions per CTA: max(kTile, scaleBlock)
  int tiles;             // tiles per sequence
  int slotRows;          // rows of a ring slot: min(kTile, S)
  float eps;
  unsigned long long turn[64];  // inv_freq of pair i as a 64-bit fixed-point fraction of a turn
};

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4 r, uint64_t (&v)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) {
      v[i] = static_cast<uint64_t>(w[i] << 16) | (static_cast<uint64_t>(w[i] & 0xffff0000u) << 32);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[i] = pack_f2(f.x, f.y);
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = kBf16 ? pack_bf162(lo_f2(v[i]), hi_f2(v[i])) : pack_half2(lo_f2(v[i]), hi_f2(v[i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two chunks of a row, as pairs of values.
struct Chunks {
  uint64_t a[4], b[4];
};

// Mean square of a row whose D values the D/16 lanes of a group hold.
template <int D>
__device__ __forceinline__ float mean_square(const Chunks& x) {
  uint64_t p = fmul2(x.a[0], x.a[0]), q = fmul2(x.b[0], x.b[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    p = ffma2(x.a[k], x.a[k], p);
    q = ffma2(x.b[k], x.b[k], q);
  }
  float ss = (lo_f2(p) + hi_f2(p)) + (lo_f2(q) + hi_f2(q));
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  return ss * (1.0f / D);
}

// x (1 + w) / sqrt(mean(x^2) + eps), and for lanes that hold rotated chunks (`rotated`) the rotation of (a, b) by the
// row's table at this lane's chunk: (cos, cos), (sin, sin) of elements 2k, 2k + 1, hl apart.
template <int D, bool kBf16>
__device__ __forceinline__ void norm_rotate(Chunks& x, const Chunks& w, float eps, bool rotated, const ulonglong2* cs,
                                            int hl) {
  float m = mean_square<D>(x) + eps, back = 1.0f;
  if (kBf16 && __any_sync(kFull, m == INFINITY)) {  // squares past fp32: the same on values scaled by 2^-64
    Chunks z;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      z.a[k] = fmul2(x.a[k], pack_f2(0x1p-64f, 0x1p-64f));
      z.b[k] = fmul2(x.b[k], pack_f2(0x1p-64f, 0x1p-64f));
    }
    const float ms = mean_square<D>(z);  // eps is nothing beside squares of 2^128
    back = m == INFINITY ? 0x1p-64f : 1.0f;
    m = m == INFINITY ? ms : m;
  }
  const float r = rsqrtf(m);
  const float inv = back * r * fmaf(-0.5f * m * r, r, 1.5f);  // one Newton step: a few units of 2^-24
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.a[k] = fmul2(x.a[k], w.a[k]);
    x.b[k] = fmul2(x.b[k], w.b[k]);
  }
  if (rotated) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const ulonglong2 t = cs[k * hl];
      const uint64_t u = fmul2(x.a[k], t.x);
      const uint64_t v = ffma2(x.a[k], t.y, fmul2(x.b[k], t.x));
      x.a[k] = pack_f2(fmaf(-lo_f2(x.b[k]), lo_f2(t.y), lo_f2(u)), fmaf(-hi_f2(x.b[k]), hi_f2(t.y), hi_f2(u)));
      x.b[k] = v;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.a[k] = fmul2(x.a[k], pack_f2(inv, inv));
    x.b[k] = fmul2(x.b[k], pack_f2(inv, inv));
  }
}

// Largest finite magnitude of 8 values (0 for none).
__device__ __forceinline__ float finite_max(const uint64_t (&y)[4]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = fabsf(lo_f2(y[k])), b = fabsf(hi_f2(y[k]));
    m = fmaxf(m, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
  }
  return m;
}

// 8 codes of y * inv; infinities become NaN.
__device__ __forceinline__ uint2 quantise8(const uint64_t (&y)[4], float inv) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = lo_f2(y[k]), b = hi_f2(y[k]);
    v[2 * k] = fabsf(a) < INFINITY ? a * inv : NAN;
    v[2 * k + 1] = fabsf(b) < INFINITY ? b * inv : NAN;
  }
  return make_uint2(f32_to_e4m3(v[0], v[1], v[2], v[3]), f32_to_e4m3(v[4], v[5], v[6], v[7]));
}

// 8 stored codes multiplied by f and rounded to codes again (exact for a power of two, above 2^-6).
__device__ __forceinline__ uint2 rescale8(const uint2 c, float f) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3_to_f16(i ? c.y : c.x, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    r[i] = f32_to_e4m3(a.x * f, a.y * f, b.x * f, b.y * f);
  }
  return make_uint2(r[0], r[1]);
}

// Place of chunk c of ring row r: the lanes of a row read chunks 0 .. hl - 1 and 2 hl .. , or the others, at once, and
// for the usual hl those lie in different banks.
template <int D>
__device__ __forceinline__ int place(int r, int c) {
  return r * (D / 8) + (D == 128 ? c ^ ((c >> 3) << 2) : c ^ ((r & 1) << 2));
}

template <int D, bool kBf16, bool kKv8>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) append_kv_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8;    // chunks per row, lanes that copy one
  constexpr int RPW = 32 / LPR; // rows of a warp-wide copy
  constexpr int CPR = D / 16;   // lanes that compute a row, two chunks each
  constexpr int RPI = 32 / CPR; // rows a warp computes at once
  extern __shared__ __align__(16) uint4 smem[];  // [kWarps][2][slotRows][LPR] rows, then the cos/sin table
  __shared__ __align__(16) float w1[2][D];       // 1 + w of q and k heads
  const int slotChunks = a.slotRows * LPR;
  ulonglong2* table = reinterpret_cast<ulonglong2*>(smem + kWarps * 2 * slotChunks);  // [live row][4][rot / 16]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.tiles, tileIdx = blockIdx.x - b * a.tiles;
  const int L = max(a.ctx[b], 0);
  const int n = max(0, min(a.newLen ? a.newLen[b] : a.S, min(a.S, L)));
  const int c = L - n;                            // position of row 0
  const int t0 = tileIdx * a.tile - c % a.tile;   // row at the tile's first position
  if (t0 >= a.S) return;
  const int tlo = max(t0, 0);                     // first row of this CTA
  const int thi = min(min(a.S, n), t0 + a.tile);  // past its last live row; the tile's later rows are padding
  const int NH = a.Hq + 2 * a.Hkv;
  const int step = gridDim.y * kWarps;

  // A warp's work: its heads in turn; for a K or V head of an 8-bit pool with blocks above kTile, all of the
  // tile's chunks of kTile rows for the largest values and once more for the codes; else each chunk once.
  struct Item {
    int h, base;  // head, row at the chunk's first position
    bool second;
  };
  const int c0 = t0 < tlo ? t0 + (tlo - t0) / kTile * kTile : t0;  // first chunk with a row of the CTA
  const bool twice = kKv8 && a.tile > kTile;
  auto next_item = [&](Item it) {
    it.base += kTile;
    if (it.base >= thi) {
      it.base = c0;
      const bool again = twice && it.h >= a.Hq && !it.second;
      it.second = again;
      it.h += again ? 0 : step;
    }
    return it;
  };
  uint4* ring = smem + warp * 2 * slotChunks;
  const uint4* src = static_cast<const uint4*>(a.qkv) + static_cast<size_t>(b) * a.S * NH * LPR + lane % LPR;
  auto copy = [&](const Item& it, int slot) {  // one copy group per item, empty past the last
    if (it.h < NH) {
      const int first = max(it.base, tlo), rows = min(thi, it.base + kTile) - first;
      const uint4* g = src + (static_cast<size_t>(first + lane / LPR) * NH + it.h) * LPR;
      const size_t hop = static_cast<size_t>(RPW) * NH * LPR;
      uint4* d = ring + slot * slotChunks;
      if (rows == kTile) {
#pragma unroll
        for (int i = 0; i < kTile / RPW; ++i)
          cp_async16(smem_addr(d + place<D>(i * RPW + lane / LPR, lane % LPR)), g + i * hop, true);
      } else {
        for (int r = lane / LPR; r < rows; r += RPW, g += hop) cp_async16(smem_addr(d + place<D>(r, lane % LPR)), g, true);
      }
    }
    cp_async_commit();
  };
  Item cur{static_cast<int>(blockIdx.y) * kWarps + warp, c0, false};
  if (thi > tlo) copy(cur, 0);

  const int hl = a.rot >> 4;  // chunks of half a rotation
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) w1[i / D][i % D] = 1.0f + __ldg((i < D ? a.qw : a.kw) + i % D);
  for (int i = threadIdx.x; i < (thi - tlo) * 8 * hl; i += kThreads) {  // pairs of the live rows
    const int r = i / (8 * hl), pair = i - r * 8 * hl;
    float cv, sv;
    rope_cos_sin_turns(static_cast<unsigned>(c + tlo + r), a.turn[pair], cv, sv);
    const int e = pair & 7;
    float* dst = reinterpret_cast<float*>(table + (r * 4 + (e >> 1)) * hl + (pair >> 3)) + (e & 1);
    dst[0] = cv;
    dst[2] = sv;
  }
  // padding rows: zeros in the dense outputs, where the tile's lie together
  const int tpad = min(a.S, t0 + a.tile), tfirst = max(thi, tlo);
  if (tfirst < tpad) {
    auto zero = [&](void* out, int heads) {
      if (!out) return;
      uint4* d = static_cast<uint4*>(out) + (static_cast<size_t>(b) * a.S + tfirst) * heads * LPR;
      const int chunks = (tpad - tfirst) * heads * LPR;
      for (int i = blockIdx.y * kThreads + threadIdx.x; i < chunks; i += gridDim.y * kThreads) d[i] = make_uint4(0, 0, 0, 0);
    };
    zero(a.qout, a.Hq);
    zero(a.kout, a.Hkv);
    zero(a.vout, a.Hkv);
  }
  if (thi <= tlo) return;

  // the tile's pages: it lies in one page of K and one of V
  const int page = (c + tlo) >> 7;
  int pg[2] = {-1, -1};
  if (page < a.maxPagesPerSeq) {
    const int32_t* pt = a.pageTable + static_cast<size_t>(b) * 2 * a.maxPagesPerSeq + page;
    pg[0] = __ldg(pt);
    pg[1] = __ldg(pt + a.maxPagesPerSeq);
  }
  bool badPage = false;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (static_cast<unsigned>(pg[i]) >= static_cast<unsigned>(a.numFlatPages)) {
      pg[i] = -1;
      badPage = true;
    }
  if (badPage && threadIdx.x == 0 && a.status) atomicOr(a.status, kErrBadPage);
  __syncthreads();

  const int l = lane & (CPR - 1), sub = lane / CPR;
  const bool rotated = l < hl;
  const int ca = rotated ? l : hl + l, cb = rotated ? l + hl : l + CPR;  // this lane's chunks
  Chunks w;
  int have = -1;        // whose weights w holds: 0 q heads, 1 k heads
  float bm = 0.f;       // lanes 0..15, 8-bit: largest value of chunk position `lane` (of the whole block, above 16)
  float rowInv = 0.f;   // lanes 0..15, 8-bit: 1 / scale at chunk position `lane`
  for (int slot = 0; cur.h < NH; slot ^= 1) {
    const Item nxt = next_item(cur);
    copy(nxt, slot ^ 1);
    cp_async_wait<1>();
    __syncwarp();
    const int h = cur.h, base = cur.base;
    const int first = max(base, tlo), rows = min(thi, base + kTile) - first, off = first - base;
    const bool isq = h < a.Hq, isv = h >= a.Hq + a.Hkv;
    const int hk = isq ? h : (isv ? h - a.Hq - a.Hkv : h - a.Hq);  // among the q, k or v heads
    const int pageId = isq ? -1 : (isv ? pg[1] : pg[0]);
    const uint4* buf = ring + slot * slotChunks;
    if (!isv && have != (isq ? 0 : 1)) {
      have = isq ? 0 : 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w.a[k] = *reinterpret_cast<const uint64_t*>(&w1[have][8 * ca + 2 * k]);
        w.b[k] = *reinterpret_cast<const uint64_t*>(&w1[have][8 * cb + 2 * k]);
      }
    }
    // The lane's values of the chunk's r-th live row (r past the last: no row, anything).
    auto value = [&](int r, uint4& rawa, uint4& rawb, Chunks& y) {
      const int rc = min(r, rows - 1);
      rawa = buf[place<D>(rc, ca)];
      rawb = buf[place<D>(rc, cb)];
      unpack8<kBf16>(rawa, y.a);
      unpack8<kBf16>(rawb, y.b);
      if (!isv) norm_rotate<D, kBf16>(y, w, a.eps, rotated, table + (first - tlo + rc) * 4 * hl + l, hl);
    };

    if (kKv8 && !isq && !cur.second) {  // the largest value of each row, then of each block
      float rm = 0.f;
      for (int i = 0; i * RPI < rows; ++i) {
        uint4 ra, rb;
        Chunks y;
        value(i * RPI + sub, ra, rb, y);
        float m = fmaxf(finite_max(y.a), finite_max(y.b));
#pragma unroll
        for (int o = CPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        const int r = lane - off - i * RPI;  // lane's row among these
        m = __shfl_sync(kFull, m, (r & (RPI - 1)) * CPR);
        if (r >= 0 && r < RPI && lane - off < rows) rm = m;
      }
      const int sb = 1 << a.blockShift;
      for (int o = 1; o < min(sb, kTile); o <<= 1) rm = fmaxf(rm, __shfl_xor_sync(kFull, rm, o));
      bm = base == c0 ? rm : fmaxf(bm, rm);
      if (base + kTile >= thi) {  // every row is in: the scale of this lane's block
        const int rr = lane & (kTile - 1);
        const int tb = t0 + (twice ? 0 : rr & ~(sb - 1));  // row at the block's first position
        const bool fill = max(tb, tlo) < min(tb + sb, thi) && pageId >= 0;
        float* sp = a.scale +
                    ((static_cast<size_t>(fill ? pageId : 0) << (7 - a.blockShift)) +
                     (fill ? ((c + tb) & 127) >> a.blockShift : 0)) * a.Hkv + hk;
        float now = 1.f, shrink = 1.f;
        if (fill) {
          if (tb < 0) {  // older tokens: keep their scale, or grow it by the smallest power of two that fits
            const float kept = read_scale(*sp);
            const float over = __fdiv_rn(bm, kE4m3Max * kept);
            now = kept;
            if (over > 1.f) {
              const int bits = __float_as_int(over);
              const int k = (bits >> 23) - 127 + ((bits & 0x7fffff) ? 1 : 0);
              now = fminf(ldexpf(kept, k), kScaleHi);
              shrink = kept / now;
            }
          } else {
            now = fminf(fmaxf(__fdiv_rn(bm, kE4m3Max), kScaleLo), kScaleHi);
          }
        }
        __syncwarp();  // every lane of a block has read its scale
        if (fill && (twice ? lane == 0 : lane < kTile && (rr & (sb - 1)) == 0)) *sp = now;
        rowInv = 1.0f / now;
        // older rows of the grown block (at most one block of the tile holds older tokens)
        const float f = __shfl_sync(kFull, shrink, twice || t0 >= 0 ? 0 : (-t0) & ~(sb - 1));
        if (t0 < 0 && f != 1.f && pageId >= 0)
          for (int p = (c & ~(sb - 1)) + lane / LPR; p < c; p += RPW) {
            uint2* row = reinterpret_cast<uint2*>(
                             a.pool + ((static_cast<size_t>(pageId) * kTokensPerPage + (p & 127)) * a.Hkv + hk) *
                                          a.poolHeadDim) + lane % LPR;
            *row = rescale8(*row, f);
          }
      }
    }

    if (!kKv8 || isq || !twice || cur.second) {
      uint4* dense = static_cast<uint4*>(isq ? a.qout : (isv ? a.vout : a.kout));
      const int heads = isq ? a.Hq : a.Hkv;
      if (dense) dense += ((static_cast<size_t>(b) * a.S + first + sub) * heads + hk) * LPR;
      constexpr int kElem = kKv8 ? 1 : 2;
      const size_t rowBytes = static_cast<size_t>(a.Hkv) * a.poolHeadDim * kElem;
      uint8_t* prow = pageId < 0 ? nullptr
                                 : a.pool + (static_cast<size_t>(pageId) * kTokensPerPage + ((c + first) & 127) + sub) * rowBytes +
                                       static_cast<size_t>(hk) * a.poolHeadDim * kElem;
#pragma unroll 2
      for (int i = 0; i * RPI < rows; ++i) {
        const int r = i * RPI + sub;
        uint4 ra, rb;
        Chunks y;
        value(r, ra, rb, y);
        const float qs = kKv8 && !isq ? __shfl_sync(kFull, rowInv, (off + r) & (kTile - 1)) : 0.f;
        if (r < rows) {
          if (!isv && (dense || !kKv8)) {
            ra = pack8<kBf16>(y.a);
            rb = pack8<kBf16>(y.b);
          }
          if (dense) {
            dense[ca] = ra;
            dense[cb] = rb;
          }
          if (prow) {
            if constexpr (kKv8) {
              reinterpret_cast<uint2*>(prow)[ca] = quantise8(y.a, qs);
              reinterpret_cast<uint2*>(prow)[cb] = quantise8(y.b, qs);
            } else {
              reinterpret_cast<uint4*>(prow)[ca] = ra;
              reinterpret_cast<uint4*>(prow)[cb] = rb;
            }
          }
        }
        if (dense) dense += static_cast<size_t>(RPI) * heads * LPR;
        if (prow) prow += RPI * rowBytes;
      }
    }
    __syncwarp();  // every lane is done with the slot
    cur = nxt;
  }
  cp_async_wait<0>();  // the last groups are empty; nothing is in flight at exit
}

template <int D, bool kBf16, bool kKv8>
cudaError_t append_go(const AppendArgs& a, int B, cudaStream_t st) {
  auto kernel = append_kv_kernel<D, kBf16, kKv8>;
  // the warps' rings, and the table of 8 bytes per row and rotated pair: at most 64 KB each
  const size_t smem = kWarps * 2 * static_cast<size_t>(a.slotRows) * (D * 2) +
                      static_cast<size_t>(std::min(a.tile, a.S)) * (a.rot / 2) * 8;
  if (smem > 40 * 1024) {  // past what a kernel may have without asking (48 KB, w1 among it)
    const cudaError_t attr =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (attr != cudaSuccess) return attr;
  }
  // One CTA per tile when the tiles fill the GPU a few times over; otherwise the heads of a tile are dealt
  // out to several CTAs, down to one head per warp.
  const long long tiles = static_cast<long long>(B) * a.tiles;
  const int most = (a.Hq + 2 * a.Hkv + kWarps - 1) / kWarps;
  const long long want = 4LL * sm_count();
  const int parts = static_cast<int>(std::min<long long>(most, std::max<long long>(1, (want + tiles - 1) / tiles)));
  kernel<<<dim3(static_cast<unsigned>(tiles), parts), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const AppendArgs& a, int B, bool bf16, bool kv8, cudaStream_t st) {
  if (kv8) return bf16 ? append_go<D, true, true>(a, B, st) : append_go<D, false, true>(a, B, st);
  return bf16 ? append_go<D, true, false>(a, B, st) : append_go<D, false, false>(a, B, st);
}

}  // namespace

cudaError_t launch_append_kv(const QsaAppendKvParams& p, const RopeFreqs& rf, bool bf16, bool kv8) {
  AppendArgs a;
  a.qkv = p.qkv;
  a.qw = p.qNormW;
  a.kw = p.kNormW;
  a.ctx = p.contextLengths;
  a.newLen = p.newLengths;
  a.qout = p.qOut;
  a.kout = p.kOut;
  a.vout = p.vOut;
  a.pool = static_cast<uint8_t*>(p.kvPool);
  a.scale = p.kvScale;
  a.pageTable = p.pageTable;
  a.status = p.status;
  a.S = p.seqLen;
  a.Hq = p.numQHeads;
  a.Hkv = p.numKVHeads;
  a.rot = p.rotDim;
  a.poolHeadDim = p.poolHeadDim;
  a.numFlatPages = p.numFlatPages;
  a.maxPagesPerSeq = p.maxPagesPerSeq;
  a.blockShift = 0;
  while (kv8 && (1 << a.blockShift) < p.scaleBlock) ++a.blockShift;
  a.tile = std::max(kTile, p.scaleBlock);
  // the most aligned tiles that seqLen consecutive positions touch
  a.tiles = static_cast<int>((static_cast<long long>(p.seqLen) + a.tile - 2) / a.tile + 1);
  a.slotRows = std::min(kTile, p.seqLen);
  a.eps = p.rmsNormEps;
  for (int i = 0; i < 64; ++i) a.turn[i] = rf.turn[i];
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  return p.headDim == 64 ? append_d<64>(a, p.batchSize, bf16, kv8, st) : append_d<128>(a, p.batchSize, bf16, kv8, st);
}

}  // namespace qsa
