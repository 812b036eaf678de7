// qsa_paged_kv4.cuh -- tiles of a 4-bit paged pool as the kernels that read it
// by lists hold them: 32 gathered rows of K (and V), their scale chunks, and
// the first product S^T = C^K Q^T.
//
// A row's value is c s_j t.  c s_j has at most 6 significant bits and lies in
// fp16's range, so codes become f16 pairs by a conversion and an exact product
// with their group's scale; t multiplies what comes out in fp32.
#pragma once

#include "qsa_kv4.cuh"
#include "qsa_paged.cuh"

namespace qsa {

constexpr int kKv4CodeBytes = kStep * kKv4Codes;   // codes of a step's K (or V) rows
constexpr int kKv4ScaleBytes = kStep * kKv4Chunk;  // their scale chunks

// First of the four keys of a step (i = 0..3 behind it) that are rows of a lane's S^T fragments: key i is row g of tile i
// (g = lane >> 2; tile 2 gk is rows 0..7, tile 2 gk + 1 rows 8..15 of MMA gk).  Rows 2 q and 2 q + 1 of a tile, which the
// transposed fragment of P holds as a pair, are keys 16 apart: what the V codes of two registers pair at once.
__device__ __forceinline__ int kv4_first_key(int lane) { return 4 * (lane >> 3) + 16 * (lane >> 2 & 1); }
// Place of row r of a step's K codes (rows 16 apart lie in different banks) and of its K scale chunk (so do rows 4 apart).
__device__ __forceinline__ int kv4_k_row(int r) { return r ^ (r >> 4); }
__device__ __forceinline__ int kv4_k_scale(int r) { return (r & 3) * 8 + (r >> 2); }

// Place of a step's entry i among its 32 row ids: a lane gathers rows 8 i + (lane >> 2), which lie together.
__device__ __forceinline__ int kv4_row_place(int i) { return (i & 7) * 4 + (i >> 3); }

// A lane's shares of a gather: 16 bytes of the codes of rows 8 i + (lane >> 2), i = 0..3, to dst + 512 i (K codes: dst ^ 64
// from row 16 on, see kv4_k_row), and its own row's scale chunk.  Rows that no entry names (id -1) become zeros.  (The path of steps that name fewer than 32 rows is a
// loop, so that the compiler branches: as predicated instructions it took a twentieth of the attention's issue slots.)
template <bool kKeys>
__device__ __forceinline__ void kv4_copy_codes(const int* ids, unsigned mask, uint32_t dst, const uint8_t* base,
                                               uint32_t rowBytes) {
  ids += ((threadIdx.x & 31) >> 2) * 4;
  if (mask == kFull) {
    const int4 r = *reinterpret_cast<const int4*>(ids);
    auto src = [&](int row) { return base + static_cast<uint64_t>(static_cast<uint32_t>(row)) * rowBytes; };
    cp_async16_to<0>(dst, src(r.x));
    cp_async16_to<512>(dst, src(r.y));
    const uint32_t upper = kKeys ? dst ^ 64 : dst;
    cp_async16_to<1024>(upper, src(r.z));
    cp_async16_to<1536>(upper, src(r.w));
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int row = ids[i];
      cp_async16((kKeys && i > 1 ? dst ^ 64 : dst) + 512 * i, base + static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * rowBytes, row >= 0);
    }
  }
}
__device__ __forceinline__ void kv4_copy_scales(int row, uint32_t dst, const uint8_t* base, uint32_t rowBytes) {
  cp_async16(dst, base + static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * rowBytes + kKv4Codes, row >= 0);
}

// The group's queries in shared memory as the scores read them: piece (4 nt + w) * 32 + lane holds the lane's B fragments
// of k-steps 2 w and 2 w + 1.
template <int NT>
constexpr int kKv4QueryBytes = NT * 4 * 32 * 16;

// S^T = C^K Q^T of a step's 32 keys: s[gk][nt] holds keys kv4_first_key + 2 gk and + 2 gk + 1, heads 8 nt + 2 q and + 1.
// A lane reads a key's 16 bytes q of codes, 32 dims with two scales: k-step w covers dims 32 q + 4 w .. + 3 of every q.
template <int NT>
__device__ __forceinline__ void kv4_scores(float (&s)[2][NT][4], uint32_t codes, uint32_t scales, uint32_t queries) {
  const int lane = threadIdx.x & 31, key = kv4_first_key(lane), q = lane & 3;
  uint4 r[4];
  uint32_t sc[4][2];  // (s, s) of a row's two groups
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = lds16(codes + kv4_k_row(key + i) * kKv4Codes + q * 16);
    uint32_t b, pair, none;
    asm volatile("{\n .reg .b16 t;\n ld.shared.b16 t, [%1];\n cvt.u32.u16 %0, t;\n}\n"
                 : "=r"(b)
                 : "r"(scales + kv4_k_scale(key + i) * kKv4Chunk + 2 * q));
    e4m3_to_f16(b, pair, none);
    sc[i][0] = __byte_perm(pair, 0, 0x1010);
    sc[i][1] = __byte_perm(pair, 0, 0x3232);
  }
#pragma unroll
  for (int gk = 0; gk < 2; ++gk)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[gk][nt][0] = s[gk][nt][1] = s[gk][nt][2] = s[gk][nt][3] = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint4 b[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) b[nt] = lds16(queries + ((4 * nt + w) * 32 + lane) * 16);
#pragma unroll
    for (int gk = 0; gk < 2; ++gk) {
      uint32_t a[2][4];  // of k-steps 2 w, 2 w + 1
      e2m1_to_f16(word(r[2 * gk], w), a[0][0], a[0][2], a[1][0], a[1][2]);
      e2m1_to_f16(word(r[2 * gk + 1], w), a[0][1], a[0][3], a[1][1], a[1][3]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[k][i] = hmul2(a[k][i], sc[2 * gk + (i & 1)][w >> 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(s[gk][nt], a[k], k ? b[nt].z : b[nt].x, k ? b[nt].w : b[nt].y);
      }
    }
  }
}

// Puts the group's queries at `queries`: k-step w of a lane covers dims 32 q + 4 w .. + 3, as the K codes do.  bf16 values are
// scaled by a power of two per head to fp16's upper range; qs gets its inverse for the lane's heads 2 q, 2 q + 1.
// kShared: the CTA's four warps put a quarter each, all of them before a __syncthreads; otherwise a warp puts its own, before
// a __syncwarp.
template <int NT, bool kBf16, bool kShared>
__device__ __forceinline__ void kv4_load_q(const uint4* q, int G, uint32_t queries, float (&qs)[NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, mine = kShared ? threadIdx.x >> 5 : 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = 8 * nt + g;
    const uint4* src = q + h * (kD / 8) + 4 * c;
    // 16 bytes i hold dims 32 c + 8 i .. + 7: k-steps 2 i and 2 i + 1, two words each
    auto piece = [&](int i) { return h < G ? __ldg(src + i) : make_uint4(0, 0, 0, 0); };
    uint4 raw[4];
    if constexpr (kBf16 || !kShared) {
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = piece(i);
    }
    float up = 1.f, down = 1.f;
    if constexpr (kBf16) {
      uint32_t m = 0;  // largest magnitude, as bf16 bits
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) m = __vmaxu2(m, word(raw[i], w) & 0x7fff7fff);
      m = max(m & 0xffff, m >> 16);
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
    auto put = [&](int i, const uint4& r) {
      uint32_t v[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[w] = word(r, w);
        if constexpr (kBf16) v[w] = pack_half2(__uint_as_float(v[w] << 16) * up, __uint_as_float(v[w] & 0xffff0000u) * up);
      }
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(queries + ((4 * nt + i) * 32 + lane) * 16), "r"(v[0]),
                   "r"(v[1]), "r"(v[2]), "r"(v[3])
                   : "memory");
    };
    if constexpr (!kShared) {
#pragma unroll
      for (int i = 0; i < 4; ++i) put(i, raw[i]);
    } else if constexpr (kBf16) {
      put(mine, mine == 0 ? raw[0] : mine == 1 ? raw[1] : mine == 2 ? raw[2] : raw[3]);
    } else {
      put(mine, piece(mine));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) qs[nt][j] = __shfl_sync(kFull, down, 4 * (2 * c + j));
  }
}

}  // namespace qsa
