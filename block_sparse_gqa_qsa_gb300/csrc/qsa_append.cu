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
// scales lies in one tile, so one CTA (of small blocks one warp) owns a block.
// A warp takes one head of up to 16 of the tile's rows at a time, copied by
// cp.async into its own two-slot ring in shared memory: the next head's rows
// travel while this one is computed.  rotDim is a multiple of 16, so a row's
// 16-byte chunks of 8 values are whole rotation halves; a lane takes a chunk
// of a first half and its partner chunk (or two chunks past rotDim), so the
// rotation needs no exchange, and the D/16 lanes of a row reduce its sum of
// squares with shuffles.  For an 8-bit pool a K or V head is passed over twice
// in shared memory: its blocks' largest values first, then the codes.  A block
// of more than 16 tokens is spread over 2 to 8 successive warps, 16 rows each,
// which join their maxima in shared memory between the two.
#include <algorithm>
#include <type_traits>

#include "qsa_internal.h"
#include "qsa_kv8.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;  // most rows of a ring slot
// CTAs per SM that the registers allow and the dealing counts on.  (The fp16 forms for wide blocks keep 8 or 12 bytes of a
// lane in local memory.)  Shared memory allows them for heads of 64, and for heads of 128 with blocks up to 16 tokens and
// rotations up to 64 wide; blocks of 32 and more or a rotation of 128 leave room for two, both with blocks of 128 for one:
// ragged 4 x 16384 prompts with blocks of 16 take 163 us, of 32 172, of 64 179, of 128 222, a rotation of 128 182.
constexpr int kCtasPerSm = 3;
constexpr int kMaxWideHeads = 512;  // K and V heads of a CTA whose tile is one block of more than kTile tokens

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
  int slotRows;          // rows of a ring slot
  int group;             // rows of a q head's item (any head's, for a 16-bit pool)
  int kvCost, unitsPerCta;  // a K or V head's share of a tile's work, a q head's being 1; a CTA's share
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

// x (1 + w) / sqrt(mean(x^2) + eps), then the rotation of (a, b) by the table entries cs, `hop` apart: (cos, cos),
// (sin, sin) of elements 2k, 2k + 1 (lanes past rotDim get (1, 1), (0, 0)).
template <int D, bool kBf16>
__device__ __forceinline__ void norm_rotate(Chunks& x, const Chunks& w, float eps, const ulonglong2* cs, int hop) {
  float m = mean_square<D>(x) + eps;
  if constexpr (kBf16) {  // squares past fp32's range, or below it beside a small eps: the same on scaled values
    if (__any_sync(kFull, m == INFINITY || m < 0x1p-90f)) {
      // 2^-70: 128 squares of the largest bf16 stay below 2^123, and the largest value that gets here stays above 2^-10
      const float f = m == INFINITY ? 0x1p-70f : m < 0x1p-90f ? 0x1p100f : 1.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x.a[k] = fmul2(x.a[k], pack_f2(f, f));
        x.b[k] = fmul2(x.b[k], pack_f2(f, f));
      }
      m = mean_square<D>(x) + eps * f * f;
    }
  }
  const float r = rsqrtf(m);
  const float inv = r * fmaf(-0.5f * m * r, r, 1.5f);  // one Newton step: a few units of 2^-24
  const uint64_t inv2 = pack_f2(inv, inv);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const ulonglong2 t = cs[k * hop];
    const uint64_t p = fmul2(x.a[k], w.a[k]), q = fmul2(x.b[k], w.b[k]), u = fmul2(p, t.x);
    const uint64_t v = pack_f2(fmaf(-lo_f2(q), lo_f2(t.y), lo_f2(u)), fmaf(-hi_f2(q), hi_f2(t.y), hi_f2(u)));
    x.a[k] = fmul2(v, inv2);
    x.b[k] = fmul2(ffma2(p, t.y, fmul2(q, t.x)), inv2);
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

// 8 codes of y / s; inv is 1 / s in fp32.  y * inv alone is off by up to two roundings, which sends a quotient halfway
// between two codes to either; with its remainder put back, a quotient that fp32 holds is exact.  The remainder of an
// infinity is NaN.
__device__ __forceinline__ uint2 quantise8(const uint64_t (&y)[4], float s, float inv) {
  const uint64_t ms2 = pack_f2(-s, -s), inv2 = pack_f2(inv, inv);
  uint64_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t q = fmul2(y[k], inv2);
    v[k] = ffma2(ffma2(q, ms2, y[k]), inv2, q);
  }
  return make_uint2(f32_to_e4m3(lo_f2(v[0]), hi_f2(v[0]), lo_f2(v[1]), hi_f2(v[1])),
                    f32_to_e4m3(lo_f2(v[2]), hi_f2(v[2]), lo_f2(v[3]), hi_f2(v[3])));
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

// kWide: the tile is one block of more than kTile tokens of an 8-bit pool.
template <int D, bool kBf16, bool kKv8, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) append_kv_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8;    // chunks per row, lanes that copy one
  constexpr int RPW = 32 / LPR; // rows of a warp-wide copy
  constexpr int CPR = D / 16;   // lanes that compute a row, two chunks each
  constexpr int RPI = 32 / CPR; // rows a warp computes at once
  extern __shared__ __align__(16) uint4 smem[];  // [kWarps][2][slotRows][LPR] rows, then the cos/sin table
  __shared__ __align__(16) float w1[2][D];       // 1 + w of q and k heads
  __shared__ ulonglong2 identity;                // the table entry of lanes past rotDim
  __shared__ int blockMax[kWide ? kMaxWideHeads : 1];  // largest value of each K/V head's block, as float bits
  const int slotChunks = a.slotRows * LPR;
  ulonglong2* table = reinterpret_cast<ulonglong2*>(smem + kWarps * 2 * slotChunks);  // [live row][4][rot / 16]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.tiles, tileIdx = blockIdx.x - b * a.tiles;
  const int L = max(a.ctx[b], 0);
  const int n = max(0, min(a.newLen ? a.newLen[b] : a.S, min(a.S, L)));
  const int c = L - n;                            // position of row 0
  const int t0 = tileIdx * a.tile - (c & (a.tile - 1));   // row at the tile's first position
  if (t0 >= a.S) return;
  const int tlo = max(t0, 0);                     // first row of this CTA
  const int thi = min(min(a.S, n), t0 + a.tile);  // past its last live row; the tile's later rows are padding
  const int NH = a.Hq + 2 * a.Hkv;
  auto head_at = [&](int unit) { return unit <= a.Hq ? unit : a.Hq + (unit - a.Hq) / a.kvCost; };
  // The dearer K and V heads of small blocks first, where there is more than a wave (4000 rows of 48 heads: 26.0 us, 28.1
  // with them last).
  const int part = kKv8 && !kWide ? gridDim.y - 1 - blockIdx.y : blockIdx.y;
  const int h0 = head_at(part * a.unitsPerCta), h1 = min(NH, head_at((part + 1) * a.unitsPerCta));

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

  // The work of a CTA, dealt to its warps one item at a time: a head and a group of its rows, kTile for a K or V head of an
  // 8-bit pool, `group` rows for a q head (any head of a 16-bit pool).  Groups start at the tile's first position.  Wide:
  // the K and V heads come first, each with a power of two of groups (the last ones may have no live row), so that a head's
  // groups go to successive warps in the same round.  Otherwise the K and V heads, which take longer, come first where a
  // CTA has all heads (4 x 16384 rows: 165 us instead of 171), last where it has a few (they wait for the table).
  struct Item {
    int h, first, rows;  // head, first live row, live rows (none: <= 0)
  };
  const int hs = kKv8 ? max(h0, min(a.Hq, h1)) : h1;  // heads [h0, hs) take groups of `group` rows, [hs, h1) of kTile
  const int gq0 = (tlo - t0) / a.group, gq = (thi - t0 + a.group - 1) / a.group - gq0;
  const int gk0 = kWide ? (tlo - t0) / kTile : 0, ng = kWide ? (thi - t0 + kTile - 1) / kTile - gk0 : 1;
  const int gk = ng > 4 ? 8 : ng > 2 ? 4 : ng, nkv = (h1 - hs) * gk, nq = (hs - h0) * gq, items = nq + nkv;
  const bool kvFirst = kWide || (kKv8 && gridDim.y == 1);
  const int early = kvFirst ? nkv : nq;  // items of the kind that comes first
  auto item_at = [&](int i) {
    const bool late = i >= early, q = late == kvFirst;
    const int per = q ? gq : gk, size = q ? a.group : kTile, k = late ? i - early : i, h = k / per;
    const int base = t0 + (k - h * per + (q ? gq0 : gk0)) * size, first = max(base, tlo);
    return Item{(q ? h0 : hs) + h, first, min(thi, base + size) - first};
  };
  uint4* ring = smem + warp * 2 * slotChunks;
  const uint4* src = static_cast<const uint4*>(a.qkv) +
                     (static_cast<size_t>(b) * a.S + lane / LPR) * NH * LPR + lane % LPR;
  auto copy = [&](const Item& it, int slot) {  // one copy group
    const uint4* g = src + (static_cast<size_t>(it.first) * NH + it.h) * LPR;
    const size_t hop = static_cast<size_t>(RPW) * NH * LPR;
    uint4* d = ring + slot * slotChunks;
    if (it.rows == kTile) {
#pragma unroll
      for (int i = 0; i < kTile / RPW; ++i)
        cp_async16(smem_addr(d + place<D>(i * RPW + lane / LPR, lane % LPR)), g + i * hop, true);
    } else {
#pragma unroll 2
      for (int r = lane / LPR; r < it.rows; r += RPW, g += hop)
        cp_async16(smem_addr(d + place<D>(r, lane % LPR)), g, true);
    }
  };
  Item next{0, 0, 0};  // the item whose rows are in, or on their way to, ring slot `slot`
  int slot = 0;
  if (warp < items) copy(next = item_at(warp), 0);
  cp_async_commit();

  const int hl = a.rot >> 4;  // chunks of half a rotation
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) w1[i / D][i % D] = 1.0f + __ldg((i < D ? a.qw : a.kw) + i % D);
  if (threadIdx.x == 0) identity = make_ulonglong2(pack_f2(1.f, 1.f), 0);
  if constexpr (kWide)
    for (int i = threadIdx.x; i < h1 - hs; i += kThreads) blockMax[i] = 0;
  if (h0 < a.Hq + a.Hkv)  // V heads need no table
    for (int r = warp; r < thi - tlo; r += kWarps)
      for (int pair = lane; pair < 8 * hl; pair += 32) {
        // pos * turn mod 2^64 is the angle as an exact fraction of a turn; its top 32 bits, signed, are half turns * 2^31
        const unsigned long long t = a.turn[pair] * static_cast<unsigned>(c + tlo + r);
        float cv, sv;
        sincospif(static_cast<float>(static_cast<int>(static_cast<unsigned>(t >> 32))) * 0x1p-31f, &sv, &cv);
        const int e = pair & 7;
        float* dst = reinterpret_cast<float*>(table + (r * 4 + (e >> 1)) * hl + (pair >> 3)) + (e & 1);
        dst[0] = cv;
        dst[2] = sv;
      }

  bool badPage = false;  // an id outside the pool: -1
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
  const int csHop = rotated ? hl : 0;
  Chunks w;
  int have = -1;  // whose weights w holds: 0 q heads, 1 k heads
  // Calls f(r, raw chunks, values) for the lane's rows r of an item in a ring slot, all lanes alike (r past the last: no
  // row, any values).
  auto each_row = [&](const Item& it, int slot, auto norm, auto&& f) {
    const uint4* pa = ring + slot * slotChunks + place<D>(sub, ca);  // RPI is even: the place moves evenly
    const uint4* pb = ring + slot * slotChunks + place<D>(sub, cb);
    const ulonglong2* cs = rotated ? table + (it.first - tlo + sub) * 4 * hl + l : &identity;
    for (int r = sub; r - sub < it.rows; r += RPI, pa += RPI * LPR, pb += RPI * LPR, cs += RPI * 4 * csHop) {
      const uint4 ra = *pa, rb = *pb;
      Chunks y;
      unpack8<kBf16>(ra, y.a);
      unpack8<kBf16>(rb, y.b);
      if constexpr (norm.value) norm_rotate<D, kBf16>(y, w, a.eps, cs, csHop);
      f(r, ra, rb, y);
    }
  };
  using Norm = std::integral_constant<bool, true>;
  using Copy = std::integral_constant<bool, false>;
  // Largest value of row position `lane` of a K or V item's group (0 for none), over all of a block's rows in it.
  auto row_maxima = [&](const Item& it, int slot, bool isv) {
    const int off = (it.first - t0) & (kTile - 1);
    float rm = 0.f;
    auto take = [&](int r, const uint4&, const uint4&, const Chunks& y) {
      float m = fmaxf(finite_max(y.a), finite_max(y.b));
#pragma unroll
      for (int o = CPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const int mine = lane - off - (r - sub);  // lane's row among these
      m = __shfl_sync(kFull, m, (mine & (RPI - 1)) * CPR);
      if (mine >= 0 && mine < RPI && lane - off < it.rows) rm = m;
    };
    if (isv)
      each_row(it, slot, Copy{}, take);
    else
      each_row(it, slot, Norm{}, take);
    for (int o = 1; o < min(1 << a.blockShift, kTile); o <<= 1) rm = fmaxf(rm, __shfl_xor_sync(kFull, rm, o));
    return rm;
  };
  // The scale of a block whose first position is row tb, for a head's largest new value bm: `kept` is its stored scale,
  // used only if it holds older tokens.  Those keep their scale, or grow it by the smallest power of two that fits.
  auto new_scale = [&](int tb, float bm, float kept, float& shrink) {
    shrink = 1.f;
    if (tb >= 0) return fminf(fmaxf(__fdiv_rn(bm, kE4m3Max), kScaleLo), kScaleHi);
    const float was = read_scale(kept);
    const float over = __fdiv_rn(bm, kE4m3Max * was);
    if (!(over > 1.f)) return was;
    const int bits = __float_as_int(over);
    const float now = fminf(ldexpf(was, (bits >> 23) - 127 + ((bits & 0x7fffff) ? 1 : 0)), kScaleHi);
    shrink = was / now;
    return now;
  };
  auto scale_at = [&](int pageId, int tb, int hk) {
    return a.scale +
           ((static_cast<size_t>(pageId) << (7 - a.blockShift)) + (((c + tb) & 127) >> a.blockShift)) * a.Hkv + hk;
  };
  // Older rows of the block that starts in front of row 0, divided by 2^k (a warp's work).
  auto shrink_older = [&](int pageId, int hk, float f) {
    for (int p = (c & ~((1 << a.blockShift) - 1)) + lane / LPR; p < c; p += RPW) {
      uint2* row = reinterpret_cast<uint2*>(
                       a.pool + ((static_cast<size_t>(pageId) * kTokensPerPage + (p & 127)) * a.Hkv + hk) * a.poolHeadDim) +
                   lane % LPR;
      *row = rescale8(*row, f);
    }
  };
  // Meeting of the gk warps that share a block of more than kTile tokens.
  auto block_sync = [&] {
    if (gk == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + warp / gk), "r"(32 * gk) : "memory");
  };
  auto weights = [&](int which) {
    if (have == which) return;
    have = which;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w.a[k] = *reinterpret_cast<const uint64_t*>(&w1[which][8 * ca + 2 * k]);
      w.b[k] = *reinterpret_cast<const uint64_t*>(&w1[which][8 * cb + 2 * k]);
    }
  };

  // this warp's items, each with the next one's rows on their way
  for (int i = warp; i < items; i += kWarps, slot ^= 1) {
    const Item it = next;
    if (i + kWarps < items) copy(next = item_at(i + kWarps), slot ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncwarp();
    const bool isq = it.h < a.Hq, isv = it.h >= a.Hq + a.Hkv;
    const int hk = isq ? it.h : (isv ? it.h - a.Hq - a.Hkv : it.h - a.Hq);  // among the q, k or v heads
    const int heads = isq ? a.Hq : a.Hkv, pageId = isq ? -1 : (isv ? pg[1] : pg[0]);
    constexpr int kElem = kKv8 ? 1 : 2;
    const size_t rowBytes = static_cast<size_t>(a.Hkv) * a.poolHeadDim * kElem, denseRow = static_cast<size_t>(heads) * LPR;
    uint4* dense = static_cast<uint4*>(isq ? a.qout : (isv ? a.vout : a.kout));
    if (dense) dense += (static_cast<size_t>(b) * a.S + it.first) * denseRow + hk * LPR;
    uint8_t* prow = pageId < 0 ? nullptr
                               : a.pool + (static_cast<size_t>(pageId) * kTokensPerPage + ((c + it.first) & 127)) * rowBytes +
                                     static_cast<size_t>(hk) * a.poolHeadDim * kElem;
    if (!isv) weights(isq ? 0 : 1);
    if (!kKv8 || isq) {
      auto put = [&](int r, const uint4& ra, const uint4& rb) {
        if (r >= it.rows) return;
        if (dense) {
          uint4* d = dense + r * denseRow;
          d[ca] = ra;
          d[cb] = rb;
        }
        if (!kKv8 && prow) {
          uint4* d = reinterpret_cast<uint4*>(prow + r * rowBytes);
          d[ca] = ra;
          d[cb] = rb;
        }
      };
      if (!kKv8 && isv)
        each_row(it, slot, Copy{}, [&](int r, const uint4& ra, const uint4& rb, const Chunks&) { put(r, ra, rb); });
      else
        each_row(it, slot, Norm{}, [&](int r, const uint4&, const uint4&, const Chunks& y) {
          put(r, pack8<kBf16>(y.a), pack8<kBf16>(y.b));
        });
    } else if constexpr (kKv8) {
      const int off = (it.first - t0) & (kTile - 1);
      const float bm = row_maxima(it, slot, isv);
      float rowScale, f = 1.f;  // scale at row position `lane` of the group; what older codes are multiplied by
      if constexpr (kWide) {
        float* sp = scale_at(max(pageId, 0), t0, hk);
        const float kept = t0 < 0 ? *sp : 1.f;
        if (lane == 0) atomicMax(&blockMax[it.h - hs], __float_as_int(bm));  // numbers >= 0: whole-number order is theirs
        block_sync();  // the block's warps: all maxima are in, all have read the stored scale
        const float now = new_scale(t0, __int_as_float(*static_cast<volatile int*>(&blockMax[it.h - hs])), kept, f);
        rowScale = now;
        if (pageId >= 0 && warp % gk == 0) {
          if (lane == 0) *sp = now;
          if (f != 1.f) shrink_older(pageId, hk, f);
        }
      } else {
        const int sb = 1 << a.blockShift, rr = lane & (kTile - 1);
        const int tb = t0 + (rr & ~(sb - 1));  // row at the first position of this lane's block
        const bool fill = lane < kTile && max(tb, tlo) < min(tb + sb, thi) && pageId >= 0;
        float* sp = scale_at(fill ? pageId : 0, fill ? tb : 0, hk);
        float now = 1.f;
        if (fill) now = new_scale(tb, bm, tb < 0 ? *sp : 1.f, f);
        __syncwarp();  // every lane of a block has read its scale
        if (fill && (rr & (sb - 1)) == 0) *sp = now;
        rowScale = now;
        f = __shfl_sync(kFull, f, t0 < 0 ? (-t0) & ~(sb - 1) : 0);  // of the block that holds row 0
        if (t0 < 0 && f != 1.f && pageId >= 0) shrink_older(pageId, hk, f);
      }
      const float rowInv = 1.0f / rowScale;
      auto put = [&](int r, const uint4& ra, const uint4& rb, const Chunks& y) {
        const int from = (off + r) & (kTile - 1);
        const float qs = __shfl_sync(kFull, rowScale, from), inv = __shfl_sync(kFull, rowInv, from);
        if (r >= it.rows) return;
        if (dense) {
          uint4* d = dense + r * denseRow;
          d[ca] = isv ? ra : pack8<kBf16>(y.a);
          d[cb] = isv ? rb : pack8<kBf16>(y.b);
        }
        if (prow) {
          uint2* d = reinterpret_cast<uint2*>(prow + r * rowBytes);
          d[ca] = quantise8(y.a, qs, inv);
          d[cb] = quantise8(y.b, qs, inv);
        }
      };
      if (isv)
        each_row(it, slot, Copy{}, put);
      else
        each_row(it, slot, Norm{}, put);
    }
    __syncwarp();  // every lane is done with the slot
  }
  cp_async_wait<0>();  // the last groups are empty; nothing is in flight at exit
}

template <int D, bool kBf16, bool kKv8, bool kWide = false>
cudaError_t append_go(AppendArgs a, int B, cudaStream_t st) {
  auto kernel = append_kv_kernel<D, kBf16, kKv8, kWide>;
  constexpr int RPI = 512 / D;  // rows a warp computes at once
  const int NH = a.Hq + 2 * a.Hkv, sms = sm_count();
  const long long tiles = static_cast<long long>(B) * a.tiles;
  const int rows = std::min(a.tile, a.S);  // most live rows of a tile
  // Groups of kTile rows when that gives every resident warp one; else the fewest rows that fill a warp, so that a small
  // call's rows run side by side.
  const long long warps = static_cast<long long>(kCtasPerSm) * kWarps * sms;
  a.group = tiles * NH * ((rows + kTile - 1) / kTile) >= warps ? kTile : RPI;
  // One CTA per tile when the tiles fill the GPU; otherwise a tile's heads are dealt out to about as many CTAs as are
  // resident at once (to the nearest number, padding rows leave early: 4 x 333..1000 rows of 20 heads took 11.0 us with 512
  // CTAs, 13.6 with 256), down to one item per warp.  K and V heads of wide blocks count twice (with blocks of 32 12.5 us
  // instead of 14.0, one 8192-row prompt with blocks of 64 44.7 instead of 51.7).
  const int perHead = (rows + a.group - 1) / a.group;
  const int most = std::max(1, (NH * perHead + kWarps - 1) / kWarps);
  int parts = static_cast<int>(std::min<long long>({most, NH, std::max<long long>(1, (kCtasPerSm * sms + tiles / 2) / tiles)}));
  a.kvCost = kWide ? 2 : 1;
  const int units = a.Hq + 2 * a.Hkv * a.kvCost;
  if (kWide) parts = std::max(parts, (NH + kMaxWideHeads - 2) / (kMaxWideHeads - 1));
  a.unitsPerCta = (units + parts - 1) / parts;
  parts = (units + a.unitsPerCta - 1) / a.unitsPerCta;
  // the warps' rings, and the table of 8 bytes per row and rotated pair (one access of RPI rows past its end)
  a.slotRows = (std::min(kTile, a.S) + RPI - 1) / RPI * RPI;
  const size_t smem = kWarps * 2 * static_cast<size_t>(a.slotRows) * (D * 2) +
                      static_cast<size_t>(rows + RPI) * (a.rot / 2) * 8;
  if (smem > 40 * 1024) {  // past what a kernel may have without asking (48 KB, the static arrays among it)
    // always the most that any call needs: another thread may launch the same kernel between this and the launch
    constexpr int kMost = kWarps * 2 * kTile * D * 2 + (kTokensPerPage + RPI) * (D / 2) * 8;
    const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (attr != cudaSuccess) return attr;
  }
  kernel<<<dim3(static_cast<unsigned>(tiles), parts), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const AppendArgs& a, int B, bool bf16, bool kv8, cudaStream_t st) {
  if (kv8 && a.tile > kTile) return bf16 ? append_go<D, true, true, true>(a, B, st) : append_go<D, false, true, true>(a, B, st);
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
  a.eps = p.rmsNormEps;
  for (int i = 0; i < 64; ++i) a.turn[i] = rf.turn[i];
  cudaStream_t st = static_cast<cudaStream_t>(p.stream);
  return p.headDim == 64 ? append_d<64>(a, p.batchSize, bf16, kv8, st) : append_d<128>(a, p.batchSize, bf16, kv8, st);
}

}  // namespace qsa
