// qsa_api.cu -- the C ABI of libqsa.so (declared in include/qsa.h): host-side
// validation, workspace arithmetic, RoPE frequency tables, the TMA tensor map
// of the decode indexer, and the kernel launches.  Nothing here allocates or
// synchronises; a failed check returns before anything is enqueued.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>

#include "qsa_internal.h"

namespace {

thread_local std::string g_last_error;

qsa_status_t fail(qsa_status_t s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

qsa_status_t ok() {
  g_last_error.clear();
  return QSA_OK;
}

qsa_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(QSA_ERR_CUDA, "%s: CUDA error %d (%s)", what, static_cast<int>(e), cudaGetErrorString(e));
}

}  // namespace

qsa_status_t qsa::record_error(qsa_status_t s, const char* msg) { return fail(s, "%s", msg); }

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

qsa::RopeFreqs rope_freqs(float theta, int rot) {
  qsa::RopeFreqs r;
  std::memset(&r, 0, sizeof(r));
  for (int i = 0; i < rot / 2; ++i) {
    r.inv_freq[i] = std::pow(static_cast<double>(theta), -2.0 * i / rot);
    double x = r.inv_freq[i] / 6.283185307179586;
    x -= std::floor(x);
    r.turn[i] = static_cast<unsigned long long>(std::ldexp(x, 64));  // x < 1, so this stays below 2^64
  }
  const double pi = 3.14159265358979323846;
  for (int j = 0; j <= 32; ++j) {  // cos(pi j / 64); past pi / 4 as sin of the complement, so j = 32 is exactly 0
    const double c = j <= 16 ? std::cos(pi * j / 64.0) : std::sin(pi * (32 - j) / 64.0);
    r.qcos_hi[j] = static_cast<float>(c);
    r.qcos_lo[j] = static_cast<float>(c - static_cast<double>(r.qcos_hi[j]));
  }
  return r;
}

// rope_freqs of the calling thread's last (theta, rot): the table is a function of the two alone, and a decode step
// asks for the same one in every layer.
const qsa::RopeFreqs& last_rope_freqs(float theta, int rot) {
  thread_local qsa::RopeFreqs r;
  thread_local float of_theta = 0.f;  // no valid theta
  thread_local int of_rot = 0;
  if (of_theta != theta || of_rot != rot) {
    r = rope_freqs(theta, rot);
    of_theta = theta;
    of_rot = rot;
  }
  return r;
}

constexpr int kMaxAttnListWidth = 16384;  // attention stages one list (or slice) in shared memory

// Indexer arguments shared by both indexers ("Qsa Attention Plugin" constructor
// attributes: indexerNumHeads, indexerHeadDim, indexerBudget, indexerCompressRatio).
qsa_status_t check_indexer_shape(int Hi, int di, int rot, int ratio, int budget, int topK, float theta,
                                 float eps) {
  if (Hi < 1 || di < 1 || rot < 0 || rot > di || (rot & 1) || ratio < 1 || budget < 1 || !(theta > 0.f) ||
      !(eps >= 0.f))
    return fail(QSA_ERR_INVALID_ARG, "indexer: invalid numHeads/headDim/rotDim/compressRatio/budget/theta/eps");
  if (static_cast<long long>(topK) < static_cast<long long>(budget) * ratio + ratio - 1)
    return fail(QSA_ERR_INVALID_ARG, "indexer: topK %d < budget*ratio + ratio - 1 = %lld", topK,
                static_cast<long long>(budget) * ratio + ratio - 1);
  if (Hi > 8) return fail(QSA_ERR_UNSUPPORTED, "indexer: numHeads %d > 8", Hi);
  if (di != 64 && di != 128) return fail(QSA_ERR_UNSUPPORTED, "indexer: headDim %d not 64 or 128", di);
  if (rot > 128) return fail(QSA_ERR_UNSUPPORTED, "indexer: rotDim %d > 128", rot);
  return QSA_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

}  // namespace

namespace {

// The attention entry points share their checks; fn names the caller in messages.
qsa_status_t sparse_prefill_entry(const QsaSparsePrefillParams* p, const char* fn, bool bf16, bool tcgen05 = false) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->qPtr || !p->kPtr || !p->vPtr || !p->oPtr || !p->indices || !p->contextLengths)
    return fail(QSA_ERR_INVALID_ARG, "%s: a tensor pointer is NULL", fn);
  if (p->batchSize < 1 || p->seqLen < 1 || p->numQHeads < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->topK < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->numQHeads % p->numKVHeads)
    return fail(QSA_ERR_INVALID_ARG, "%s: numQHeads %% numKVHeads != 0", fn);
  if (!qsa_sparse_prefill_can_implement(p->numQHeads, p->numKVHeads, p->headDim))
    return fail(QSA_ERR_UNSUPPORTED, "%s: needs headDim 128 and a GQA group of at most 16", fn);
  if (p->topK > kMaxAttnListWidth)
    return fail(QSA_ERR_UNSUPPORTED, "%s: topK > %d", fn, kMaxAttnListWidth);
  if (static_cast<long long>(p->batchSize) * p->seqLen * p->numKVHeads > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize*seqLen*numKVHeads exceeds the grid", fn);
  if (!aligned(p->qPtr, 16) || !aligned(p->kPtr, 16) || !aligned(p->vPtr, 16) || !aligned(p->oPtr, 16))
    return fail(QSA_ERR_INVALID_ARG, "%s: Q/K/V/O must be 16-byte aligned", fn);
  const cudaError_t e = tcgen05 ? qsa::launch_sparse_prefill_tc(*p, bf16) : qsa::launch_sparse_prefill(*p, bf16);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}


qsa_status_t sparse_decode_entry(const QsaSparseDecodeParams* p, const char* fn, bool bf16) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->qPtr || !p->kvPoolPtr || !p->pageTable || !p->indices || !p->contextLengths || !p->oPtr)
    return fail(QSA_ERR_INVALID_ARG, "%s: a tensor pointer is NULL", fn);
  if (!p->partialO || !p->partialStats || !p->splitCounters)
    return fail(QSA_ERR_WORKSPACE, "%s: partialO/partialStats/splitCounters is NULL", fn);
  if (p->batchSize < 1 || p->numQHeads < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->topK < 1 ||
      p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->numQHeads % p->numKVHeads)
    return fail(QSA_ERR_INVALID_ARG, "%s: numQHeads %% numKVHeads != 0", fn);
  if (p->poolHeadDim < p->headDim) return fail(QSA_ERR_INVALID_ARG, "%s: poolHeadDim < headDim", fn);
  if (!qsa_sparse_decode_can_implement(p->numQHeads, p->numKVHeads, p->headDim, p->poolHeadDim))
    return fail(QSA_ERR_UNSUPPORTED,
                "%s: needs headDim 128, a GQA group of at most 16, poolHeadDim a multiple of 8", fn);
  if (p->topK > kMaxAttnListWidth) return fail(QSA_ERR_UNSUPPORTED, "%s: topK > %d", fn, kMaxAttnListWidth);
  if (p->batchSize > 65535 || p->numKVHeads > 65535)
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize/numKVHeads > 65535", fn);
  if (static_cast<long long>(p->maxPagesPerSeq) * 128 > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: maxPagesPerSeq too large", fn);
  if (!aligned(p->qPtr, 16) || !aligned(p->kvPoolPtr, 16) || !aligned(p->oPtr, 16) || !aligned(p->partialO, 16) ||
      !aligned(p->partialStats, 4) || !aligned(p->splitCounters, 4))
    return fail(QSA_ERR_INVALID_ARG, "%s: q/pool/o/partialO must be 16-byte aligned", fn);
  const cudaError_t e = qsa::launch_sparse_decode(*p, bf16);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

bool power_of_two(int x) { return x >= 1 && (x & (x - 1)) == 0; }

// The append entry points share their checks; fn names the caller in messages.
qsa_status_t append_kv_entry(const QsaAppendKvParams* p, const char* fn, bool bf16, bool kv8) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->qkv || !p->qNormW || !p->kNormW || !p->contextLengths || !p->qOut || !p->kvPool || !p->pageTable)
    return fail(QSA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
  if (p->batchSize < 1 || p->seqLen < 1 || p->numQHeads < 1 || p->numKVHeads < 1 || p->headDim < 1 ||
      p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->rotDim < 0 || p->rotDim > p->headDim || (p->rotDim & 1) || !(p->ropeTheta > 0.f) || !(p->rmsNormEps >= 0.f) ||
      std::isinf(p->rmsNormEps))
    return fail(QSA_ERR_INVALID_ARG, "%s: rotDim must be even and <= headDim; theta > 0, eps >= 0 and finite", fn);
  if (p->poolHeadDim < p->headDim) return fail(QSA_ERR_INVALID_ARG, "%s: poolHeadDim < headDim", fn);
  if (kv8) {
    if (!p->kvScale) return fail(QSA_ERR_INVALID_ARG, "%s: kvScale is NULL", fn);
    if (!power_of_two(p->scaleBlock) || p->scaleBlock > qsa::kTokensPerPageHost)
      return fail(QSA_ERR_INVALID_ARG, "%s: scaleBlock %d is not a power of two in 1..128", fn, p->scaleBlock);
  } else if (p->kvScale || p->scaleBlock) {
    return fail(QSA_ERR_INVALID_ARG, "%s: a 16-bit pool has no kvScale (NULL) and no scaleBlock (0)", fn);
  }
  if (p->headDim != 64 && p->headDim != 128)
    return fail(QSA_ERR_UNSUPPORTED, "%s: headDim %d not 64 or 128", fn, p->headDim);
  if (p->rotDim % 16)
    return fail(QSA_ERR_UNSUPPORTED, "%s: rotDim %d is not a multiple of 16", fn, p->rotDim);
  if (p->poolHeadDim % (kv8 ? 16 : 8))
    return fail(QSA_ERR_UNSUPPORTED, "%s: poolHeadDim %d: pool rows must be whole 16-byte chunks", fn, p->poolHeadDim);
  if (p->numQHeads > 1024 || p->numKVHeads > 1024)
    return fail(QSA_ERR_UNSUPPORTED, "%s: numQHeads or numKVHeads above 1024", fn);
  if (!aligned(p->qkv, 16) || !aligned(p->qOut, 16) || !aligned(p->kOut, 16) || !aligned(p->vOut, 16) ||
      !aligned(p->kvPool, 16) || !aligned(p->kvScale, 4) || !aligned(p->pageTable, 4) ||
      !aligned(p->contextLengths, 4) || !aligned(p->newLengths, 4) || !aligned(p->qNormW, 4) ||
      !aligned(p->kNormW, 4) || !aligned(p->status, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: qkv, qOut, kOut, vOut and kvPool must be 16-byte aligned, the others 4", fn);
  if (static_cast<long long>(p->batchSize) * p->seqLen > 0x7fffffffLL ||
      static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numFlatPages) * qsa::kTokensPerPageHost > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize * seqLen, maxPagesPerSeq or numFlatPages too large", fn);
  const cudaError_t e = qsa::launch_append_kv(*p, last_rope_freqs(p->ropeTheta, p->rotDim), bf16, kv8);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

qsa_status_t sparse_paged_kv8_entry(const QsaSparsePagedKv8Params* p, const char* fn, bool bf16) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->qPtr || !p->kvPool || !p->kvScale || !p->pageTable || !p->indices || !p->contextLengths || !p->oPtr)
    return fail(QSA_ERR_INVALID_ARG, "%s: a tensor pointer is NULL", fn);
  if (p->batchSize < 1 || p->seqLen < 1 || p->numQHeads < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->topK < 1 ||
      p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->numQHeads % p->numKVHeads) return fail(QSA_ERR_INVALID_ARG, "%s: numQHeads %% numKVHeads != 0", fn);
  if (p->poolHeadDim < p->headDim) return fail(QSA_ERR_INVALID_ARG, "%s: poolHeadDim < headDim", fn);
  if (!power_of_two(p->scaleBlock) || p->scaleBlock > qsa::kTokensPerPageHost)
    return fail(QSA_ERR_INVALID_ARG, "%s: scaleBlock %d is not a power of two in 1..128", fn, p->scaleBlock);
  if (!qsa_sparse_prefill_can_implement(p->numQHeads, p->numKVHeads, p->headDim))
    return fail(QSA_ERR_UNSUPPORTED, "%s: needs headDim 128 and a GQA group of at most 16", fn);
  if (p->poolHeadDim % 16)
    return fail(QSA_ERR_UNSUPPORTED, "%s: poolHeadDim %d is not a multiple of 16", fn, p->poolHeadDim);
  if (p->topK > (1 << 24)) return fail(QSA_ERR_UNSUPPORTED, "%s: topK > %d", fn, 1 << 24);
  if (!aligned(p->qPtr, 16) || !aligned(p->kvPool, 16) || !aligned(p->oPtr, 16) || !aligned(p->kvScale, 4) ||
      !aligned(p->pageTable, 4) || !aligned(p->indices, 4) || !aligned(p->contextLengths, 4) ||
      !aligned(p->newLengths, 4) || !aligned(p->status, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: q, kvPool and o must be 16-byte aligned, the others 4", fn);
  if (static_cast<long long>(p->batchSize) * p->seqLen > 0x7fffffffLL ||
      static_cast<long long>(p->batchSize) * p->seqLen * p->numKVHeads > 0x7fffffffLL ||
      static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numFlatPages) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numKVHeads) * p->poolHeadDim > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize * seqLen * numKVHeads, maxPagesPerSeq, numFlatPages or a pool row "
                                     "too large", fn);
  const cudaError_t e = qsa::launch_sparse_paged_kv8(*p, bf16);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

// Whether rows of `len` elements, heads headStride and tokens tokenStride apart, lie apart from each other.
bool rows_apart(long long tokens, long long heads, long long len, int64_t tokenStride, int64_t headStride) {
  if (heads == 1) return tokens == 1 || tokenStride >= len;
  if (tokens == 1) return headStride >= len;
  // (heads and tokens below 2^31, so that the products stay below 2^63 for the strides that the first tests let through)
  if (headStride >= len && headStride <= tokenStride / (heads - 1) && tokenStride >= (heads - 1) * headStride + len) return true;
  return tokenStride >= len && tokenStride <= headStride / (tokens - 1) && headStride >= (tokens - 1) * tokenStride + len;
}

qsa_status_t rotary_entry(const QsaRotaryParams* p, const char* fn, int elem) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->x || !p->y || !p->positions || !p->invFreq) return fail(QSA_ERR_INVALID_ARG, "%s: a pointer is NULL", fn);
  if (p->numTokens < 1 || p->numHeads < 1 || p->headDim < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->rotDim < 2 || (p->rotDim & 1) || p->rotDim > p->headDim)
    return fail(QSA_ERR_INVALID_ARG, "%s: rotDim %d must be even, >= 2 and <= headDim", fn, p->rotDim);
  if (p->xTokenStride < 0 || p->xHeadStride < 0 || p->yTokenStride < 0 || p->yHeadStride < 0)
    return fail(QSA_ERR_INVALID_ARG, "%s: a stride is negative", fn);
  if (!rows_apart(p->numTokens, p->numHeads, p->headDim, p->yTokenStride, p->yHeadStride))
    return fail(QSA_ERR_INVALID_ARG, "%s: rows of y overlap under its strides", fn);
  if (p->x == p->y && ((p->numTokens > 1 && p->xTokenStride != p->yTokenStride) ||
                       (p->numHeads > 1 && p->xHeadStride != p->yHeadStride)))
    return fail(QSA_ERR_INVALID_ARG, "%s: in place, x and y need the same strides", fn);
  if (!std::isfinite(p->magnitude)) return fail(QSA_ERR_INVALID_ARG, "%s: magnitude is not finite", fn);
  if (p->rotDim > 2 * qsa::kRotaryMaxPairs)
    return fail(QSA_ERR_UNSUPPORTED, "%s: rotDim %d > %d", fn, p->rotDim, 2 * qsa::kRotaryMaxPairs);
  const size_t size = elem == 2 ? 4 : 2;
  if (!aligned(p->x, size) || !aligned(p->y, size) || !aligned(p->positions, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: x and y must be aligned to their elements, positions to 4 bytes", fn);
  // (two factors below 2^31 first, so that nothing overflows)
  if (static_cast<long long>(p->numTokens) * p->numHeads > 0x7fffffffLL ||
      static_cast<long long>(p->numTokens) * p->numHeads * p->headDim > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: numTokens * numHeads * headDim must stay below 2^31", fn);
  if (p->numHeads > 65535 || p->headDim > 65535)
    return fail(QSA_ERR_UNSUPPORTED, "%s: numHeads %d or headDim %d > 65535", fn, p->numHeads, p->headDim);
  qsa::RotaryTurns rt;
  for (int i = 0; i < p->rotDim / 2; ++i) {
    double x = p->invFreq[i] / 6.283185307179586;
    if (!std::isfinite(x)) return fail(QSA_ERR_INVALID_ARG, "%s: a frequency is not finite", fn);
    x -= std::floor(x);
    // a negative frequency's fraction may round to a whole turn
    rt.turn[i] = x >= 1.0 ? 0 : static_cast<unsigned long long>(x * 18446744073709551616.0);
  }
  const cudaError_t e = qsa::launch_rotary(*p, rt, elem);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

qsa_status_t store_kv4_entry(const QsaStoreKv4Params* p, const char* fn, bool bf16) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->k || !p->v || !p->contextLengths || !p->kvPool || !p->pageTable)
    return fail(QSA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
  if (p->batchSize < 1 || p->seqLen < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->numFlatPages < 1 ||
      p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  const long long row = static_cast<long long>(p->numKVHeads) * p->headDim;
  const bool several = p->batchSize > 1 || p->seqLen > 1;
  if (several && (p->kTokenStride < row || p->vTokenStride < row))
    return fail(QSA_ERR_INVALID_ARG, "%s: a token stride is below numKVHeads * headDim", fn);
  if (p->poolRowBytes < QSA_KV4_ROW_BYTES)
    return fail(QSA_ERR_INVALID_ARG, "%s: poolRowBytes < %d", fn, QSA_KV4_ROW_BYTES);
  if (p->headDim != 128) return fail(QSA_ERR_UNSUPPORTED, "%s: headDim %d is not 128", fn, p->headDim);
  if (p->poolRowBytes % 16 || (several && (p->kTokenStride % 8 || p->vTokenStride % 8)))
    return fail(QSA_ERR_UNSUPPORTED, "%s: poolRowBytes and token strides must be whole 16-byte chunks", fn);
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->kOut, 16) || !aligned(p->vOut, 16) ||
      !aligned(p->kvPool, 16) || !aligned(p->contextLengths, 4) || !aligned(p->newLengths, 4) ||
      !aligned(p->pageTable, 4) || !aligned(p->status, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: k, v, kOut, vOut and kvPool must be 16-byte aligned, the others 4", fn);
  if (static_cast<long long>(p->batchSize) * p->seqLen > 0x7fffffffLL ||
      static_cast<long long>(p->batchSize) * p->seqLen * p->numKVHeads > 0x7ffffffLL ||
      static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numFlatPages) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numKVHeads) * p->poolRowBytes > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize * seqLen * numKVHeads, maxPagesPerSeq, numFlatPages or a pool row "
                                     "too large", fn);
  const cudaError_t e = qsa::launch_store_kv4(*p, bf16);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

// What the two readers of a 4-bit pool by lists check alike.
template <typename P>
qsa_status_t check_paged_kv4(const P* p, const char* fn) {
  if (p->batchSize < 1 || p->seqLen < 1 || p->numQHeads < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->topK < 1 ||
      p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->numQHeads % p->numKVHeads) return fail(QSA_ERR_INVALID_ARG, "%s: numQHeads %% numKVHeads != 0", fn);
  if (p->poolRowBytes < QSA_KV4_ROW_BYTES)
    return fail(QSA_ERR_INVALID_ARG, "%s: poolRowBytes < %d", fn, QSA_KV4_ROW_BYTES);
  if (!qsa_sparse_prefill_can_implement(p->numQHeads, p->numKVHeads, p->headDim))
    return fail(QSA_ERR_UNSUPPORTED, "%s: needs headDim 128 and a GQA group of at most 16", fn);
  if (p->poolRowBytes % 16)
    return fail(QSA_ERR_UNSUPPORTED, "%s: poolRowBytes %d is not a multiple of 16", fn, p->poolRowBytes);
  if (p->topK > (1 << 24)) return fail(QSA_ERR_UNSUPPORTED, "%s: topK > %d", fn, 1 << 24);
  if (!aligned(p->qPtr, 16) || !aligned(p->kvPool, 16) || !aligned(p->pageTable, 4) || !aligned(p->indices, 4) ||
      !aligned(p->contextLengths, 4) || !aligned(p->newLengths, 4) || !aligned(p->lse, 4) || !aligned(p->status, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: q and kvPool must be 16-byte aligned, the others 4", fn);
  if (static_cast<long long>(p->batchSize) * p->seqLen > 0x7fffffffLL ||
      static_cast<long long>(p->batchSize) * p->seqLen * p->numKVHeads > 0x7fffffffLL ||
      static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numFlatPages) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numKVHeads) * p->poolRowBytes > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize * seqLen * numKVHeads, maxPagesPerSeq, numFlatPages or a pool row "
                                     "too large", fn);
  return QSA_OK;
}

qsa_status_t sparse_paged_kv4_entry(const QsaSparsePagedKv4Params* p, const char* fn, bool bf16) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->qPtr || !p->kvPool || !p->pageTable || !p->indices || !p->contextLengths || !p->oPtr)
    return fail(QSA_ERR_INVALID_ARG, "%s: a tensor pointer is NULL", fn);
  const qsa_status_t s = check_paged_kv4(p, fn);
  if (s != QSA_OK) return s;
  if (!aligned(p->oPtr, 16)) return fail(QSA_ERR_UNSUPPORTED, "%s: o must be 16-byte aligned", fn);
  const cudaError_t e = qsa::launch_sparse_paged_kv4(*p, bf16);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

qsa_status_t sparse_weights_kv4_entry(const QsaSparseWeightsKv4Params* p, const char* fn, bool bf16) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->qPtr || !p->kvPool || !p->pageTable || !p->indices || !p->contextLengths || !p->lse || !p->weights)
    return fail(QSA_ERR_INVALID_ARG, "%s: a tensor pointer is NULL", fn);
  if (p->totalLen < 0 || (p->total == nullptr) != (p->totalLen == 0))
    return fail(QSA_ERR_INVALID_ARG, "%s: total needs totalLen >= 1, without it totalLen is 0", fn);
  const qsa_status_t s = check_paged_kv4(p, fn);
  if (s != QSA_OK) return s;
  if (!aligned(p->weights, 4) || !aligned(p->total, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: weights and total must be 4-byte aligned", fn);
  if (p->totalLen > (1 << 24)) return fail(QSA_ERR_UNSUPPORTED, "%s: totalLen > %d", fn, 1 << 24);
  const cudaError_t e = qsa::launch_sparse_weights_kv4(*p, bf16);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

}  // namespace

extern "C" {

const char* qsa_status_string(qsa_status_t s) {
  switch (s) {
    case QSA_OK: return "QSA_OK";
    case QSA_ERR_INVALID_ARG: return "QSA_ERR_INVALID_ARG";
    case QSA_ERR_UNSUPPORTED: return "QSA_ERR_UNSUPPORTED";
    case QSA_ERR_WORKSPACE: return "QSA_ERR_WORKSPACE";
    case QSA_ERR_CUDA: return "QSA_ERR_CUDA";
  }
  return "QSA_ERR_UNKNOWN";
}

const char* qsa_last_error_message(void) { return g_last_error.c_str(); }

qsa_status_t qsa_last_device_error(const void* workspace, void* stream, int32_t* out) {
  if (!workspace || !out) return fail(QSA_ERR_INVALID_ARG, "qsa_last_device_error: workspace or out is NULL");
  const cudaError_t e = cudaMemcpyAsync(out, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "qsa_last_device_error");
}

void qsa_debug_set_wait_limit_ns(uint64_t ns) { qsa::set_decode_wait_limit_ns(ns); }

int32_t qsa_indexer_prefill_max_blocks(void) { return qsa::kPrefillMaxSeqLen; }
int32_t qsa_indexer_prefill_max_seq_len(void) { return qsa::kPrefillMaxSeqLen; }

size_t qsa_indexer_prefill_workspace_size(int32_t B, int32_t S, int32_t di, int32_t ratio) {
  if (B < 1 || S < 1 || di < 1 || ratio < 1) return 0;
  return qsa::indexer_prefill_workspace_bytes(B, S, di, ratio);
}

size_t qsa_indexer_decode_workspace_size(int32_t B, int32_t maxPagesPerSeq, int32_t ratio, int32_t budget) {
  if (B < 1 || maxPagesPerSeq < 1 || ratio < 1 || qsa::kTokensPerPageHost % ratio != 0 || budget < 1) return 0;
  return qsa::indexer_decode_workspace_bytes(B, maxPagesPerSeq, ratio, budget);
}

size_t qsa_sparse_decode_partial_o_elems(int32_t B, int32_t Hkv, int32_t D) {
  if (B < 1 || Hkv < 1 || D < 1) return 0;
  return static_cast<size_t>(B) * Hkv * 8 * 16 * D;
}
size_t qsa_sparse_decode_partial_stats_elems(int32_t B, int32_t Hkv) {
  if (B < 1 || Hkv < 1) return 0;
  return static_cast<size_t>(B) * Hkv * 8 * 2 * 16;
}
size_t qsa_sparse_decode_counter_elems(int32_t B, int32_t Hkv) {
  if (B < 1 || Hkv < 1) return 0;
  return static_cast<size_t>(B) * Hkv;
}
int32_t qsa_sparse_decode_max_splits(void) { return 8; }
int32_t qsa_sparse_decode_partial_rows(void) { return 16; }

int32_t qsa_sparse_prefill_can_implement(int32_t Hq, int32_t Hkv, int32_t D) {
  return Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && Hq / Hkv <= 16 && D == 128;
}
int32_t qsa_sparse_decode_can_implement(int32_t Hq, int32_t Hkv, int32_t D, int32_t poolHeadDim) {
  return qsa_sparse_prefill_can_implement(Hq, Hkv, D) && poolHeadDim >= D && poolHeadDim % 8 == 0;
}

qsa_status_t qsa_indexer_prefill(const QsaIndexerPrefillParams* p) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill: params is NULL");
  if (!p->idxQ || !p->idxK || !p->qNormW || !p->kNormW || !p->contextLengths || !p->indices)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill: a tensor pointer is NULL");
  if (p->batchSize < 1 || p->seqLen < 1)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill: batchSize/seqLen must be >= 1");
  qsa_status_t s = check_indexer_shape(p->numHeads, p->headDim, p->rotDim, p->compressRatio, p->budget, p->topK,
                                       p->ropeTheta, p->rmsNormEps);
  if (s != QSA_OK) return s;
  if (p->batchSize > 65535) return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_prefill: batchSize > 65535");
  if (p->seqLen > qsa::kPrefillMaxSeqLen)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_prefill: seqLen %d > %d", p->seqLen, qsa::kPrefillMaxSeqLen);
  if (static_cast<long long>(p->batchSize) * p->seqLen > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_prefill: batchSize*seqLen exceeds 2^31 - 1 rows");
  const size_t need = qsa::indexer_prefill_workspace_bytes(p->batchSize, p->seqLen, p->headDim, p->compressRatio);
  if (!p->workspace || p->workspaceBytes < need || !aligned(p->workspace, 256))
    return fail(QSA_ERR_WORKSPACE, "qsa_indexer_prefill: workspace needs %zu bytes, 256-byte aligned", need);
  const cudaError_t e = qsa::launch_indexer_prefill(*p, rope_freqs(p->ropeTheta, p->rotDim));
  return e == cudaSuccess ? ok() : cuda_fail(e, "qsa_indexer_prefill");
}

qsa_status_t qsa_indexer_decode(const QsaIndexerDecodeParams* p) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_decode: params is NULL");
  if (!p->idxQ || !p->idxK || !p->qNormW || !p->kNormW || !p->kvPool || !p->pageTable || !p->contextLengths ||
      !p->indices)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_decode: a tensor pointer is NULL");
  if (p->batchSize < 1 || p->numKVHeads < 1 || p->kvHeadDim < 1 || p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_decode: batchSize/numKVHeads/kvHeadDim/numFlatPages/"
                                     "maxPagesPerSeq must be >= 1");
  if (p->poolHeadDim < p->kvHeadDim + p->headDim)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_decode: poolHeadDim %d < kvHeadDim + headDim", p->poolHeadDim);
  qsa_status_t s = check_indexer_shape(p->numHeads, p->headDim, p->rotDim, p->compressRatio, p->budget, p->topK,
                                       p->ropeTheta, p->rmsNormEps);
  if (s != QSA_OK) return s;
  if (qsa::kTokensPerPageHost % p->compressRatio != 0)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_decode: compressRatio %d does not divide the 128-token page",
                p->compressRatio);
  if (p->compressRatio < 4 || p->compressRatio > 16)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: compressRatio %d outside 4..16 (a page's key tails are "
                                     "one swizzled TMA tile of 8..32 rows)", p->compressRatio);
  if (p->budget > 4096)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: budget %d > 4096", p->budget);
  if (p->batchSize > qsa::kDecodeMaxBatch)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: batchSize > %d", qsa::kDecodeMaxBatch);
  if (p->kvHeadDim % 8 || p->poolHeadDim % 8 || !aligned(p->kvPool, 16))
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: kvHeadDim and poolHeadDim must be multiples of 8 and "
                                     "kvPool 16-byte aligned (TMA rows)");
  if (static_cast<long long>(p->maxPagesPerSeq) * 128 > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: maxPagesPerSeq too large");
  if (static_cast<long long>(p->maxPagesPerSeq) * (qsa::kTokensPerPageHost / p->compressRatio) > (1LL << 21))
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: more than 2097152 blocks per sequence");
  const size_t need = qsa::indexer_decode_workspace_bytes(p->batchSize, p->maxPagesPerSeq, p->compressRatio, p->budget);
  if (!p->workspace || p->workspaceBytes < need || !aligned(p->workspace, 256))
    return fail(QSA_ERR_WORKSPACE, "qsa_indexer_decode: workspace needs %zu bytes, 256-byte aligned", need);
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(QSA_ERR_CUDA, "qsa_indexer_decode: cuTensorMapEncodeTiled is unavailable");
  // Strided view of the key tails: [numFlatPages][128/r block-start rows][headDim] starting at column kvHeadDim
  // of head 0 ("KV pool contract": block g's key in the V-row tail of token r*g).
  const int bpp = qsa::kTokensPerPageHost / p->compressRatio;
  const size_t row_bytes = static_cast<size_t>(p->numKVHeads) * p->poolHeadDim * 2;
  CUtensorMap map;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(p->headDim), static_cast<cuuint64_t>(bpp),
                        static_cast<cuuint64_t>(p->numFlatPages)};
  cuuint64_t strides[2] = {row_bytes * p->compressRatio, row_bytes * qsa::kTokensPerPageHost};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(bpp), 1};  // one 128-byte swizzled half per copy
  cuuint32_t estr[3] = {1, 1, 1};
  void* base = static_cast<char*>(p->kvPool) + static_cast<size_t>(p->kvHeadDim) * 2;
  const CUresult r = enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_decode: tensor map rejected (CUresult %d)", r);
  const cudaError_t e = qsa::launch_indexer_decode(*p, rope_freqs(p->ropeTheta, p->rotDim), map);
  return e == cudaSuccess ? ok() : cuda_fail(e, "qsa_indexer_decode");
}

qsa_status_t qsa_sparse_prefill(const QsaSparsePrefillParams* p) {
  return sparse_prefill_entry(p, "qsa_sparse_prefill", false);
}
qsa_status_t qsa_sparse_prefill_bf16(const QsaSparsePrefillParams* p) {
  return sparse_prefill_entry(p, "qsa_sparse_prefill_bf16", true);
}
qsa_status_t qsa_sparse_prefill_tcgen05(const QsaSparsePrefillParams* p) {
  return sparse_prefill_entry(p, "qsa_sparse_prefill_tcgen05", false, true);
}
qsa_status_t qsa_sparse_prefill_tcgen05_bf16(const QsaSparsePrefillParams* p) {
  return sparse_prefill_entry(p, "qsa_sparse_prefill_tcgen05_bf16", true, true);
}

qsa_status_t qsa_rope_qkv(const QsaRopeQkvParams* p) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "qsa_rope_qkv: params is NULL");
  if (!p->qkv || !p->qNormW || !p->kNormW || !p->contextLengths || !p->qOut)
    return fail(QSA_ERR_INVALID_ARG, "qsa_rope_qkv: a required pointer is NULL");
  if (p->batchSize < 1 || p->seqLen < 1 || p->numQHeads < 1 || p->numKVHeads < 1)
    return fail(QSA_ERR_INVALID_ARG, "qsa_rope_qkv: sizes must be >= 1");
  if (p->headDim != 64 && p->headDim != 128)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: headDim %d not 64 or 128", p->headDim);
  if (p->rotDim < 0 || p->rotDim > p->headDim || (p->rotDim & 1) || !(p->ropeTheta > 0.f) || !(p->rmsNormEps >= 0.f))
    return fail(QSA_ERR_INVALID_ARG, "qsa_rope_qkv: rotDim must be even and <= headDim; theta > 0, eps >= 0");
  if (static_cast<long long>(p->numQHeads + 2LL * p->numKVHeads) * p->headDim * 2 > qsa::kRopeMaxRowBytes)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: (numQHeads + 2 numKVHeads) * headDim * 2 exceeds %d bytes",
                qsa::kRopeMaxRowBytes);
  if (p->rotDim % 16)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: rotDim %d is not a multiple of 16 (rotation partners are "
                                     "exchanged as whole 8-element chunks)", p->rotDim);
  if (!aligned(p->qkv, 16) || !aligned(p->qOut, 16) || !aligned(p->kOut, 16) || !aligned(p->vOut, 16) ||
      !aligned(p->kvPool, 16))
    return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: qkv, qOut, kOut, vOut and kvPool must be 16-byte aligned");
  if (static_cast<long long>(p->batchSize) * p->seqLen > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: batchSize*seqLen exceeds the grid");
  if (p->kvPool) {
    if (!p->pageTable || p->poolHeadDim < p->headDim || p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
      return fail(QSA_ERR_INVALID_ARG, "qsa_rope_qkv: kvPool needs pageTable, poolHeadDim >= headDim and page counts");
    if (p->poolHeadDim % 8)
      return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: poolHeadDim %d is not a multiple of 8 (16-byte row writes)",
                  p->poolHeadDim);
    if (static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL)
      return fail(QSA_ERR_UNSUPPORTED, "qsa_rope_qkv: maxPagesPerSeq too large");
  }
  const cudaError_t e = qsa::launch_rope_qkv(*p, rope_freqs(p->ropeTheta, p->rotDim));
  return e == cudaSuccess ? ok() : cuda_fail(e, "qsa_rope_qkv");
}

qsa_status_t qsa_indexer_prefill_handoff(const QsaIndexerHandoffParams* p) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill_handoff: params is NULL");
  if (!p->idxK || !p->contextLengths || !p->workspace || !p->kvPool || !p->pageTable)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill_handoff: a pointer is NULL");
  if (p->batchSize < 1 || p->seqLen < 1 || p->compressRatio < 1 || p->numKVHeads < 1 || p->kvHeadDim < 1 ||
      p->numFlatPages < 1 || p->maxPagesPerSeq < 1)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill_handoff: sizes must be >= 1");
  if (p->headDim != 64 && p->headDim != 128)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_prefill_handoff: headDim %d not 64 or 128", p->headDim);
  if (p->poolHeadDim < p->kvHeadDim + p->headDim)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill_handoff: poolHeadDim %d < kvHeadDim + headDim",
                p->poolHeadDim);
  if (p->kvHeadDim % 8 || p->poolHeadDim % 8 || !aligned(p->kvPool, 16) || !aligned(p->idxK, 16))
    return fail(QSA_ERR_UNSUPPORTED, "qsa_indexer_prefill_handoff: kvHeadDim and poolHeadDim must be multiples of 8 "
                                     "and idxK / kvPool 16-byte aligned (16-byte copies)");
  if (static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost < p->seqLen ||
      static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL)
    return fail(QSA_ERR_INVALID_ARG, "qsa_indexer_prefill_handoff: maxPagesPerSeq must cover seqLen");
  const size_t need = qsa::indexer_prefill_workspace_bytes(p->batchSize, p->seqLen, p->headDim, p->compressRatio);
  if (p->workspaceBytes < need || !aligned(p->workspace, 256))
    return fail(QSA_ERR_WORKSPACE, "qsa_indexer_prefill_handoff: the prefill workspace has %zu bytes, 256-byte "
                                   "aligned, for this shape", need);
  const cudaError_t e = qsa::launch_indexer_handoff(*p);
  return e == cudaSuccess ? ok() : cuda_fail(e, "qsa_indexer_prefill_handoff");
}

qsa_status_t qsa_append_kv(const QsaAppendKvParams* p) { return append_kv_entry(p, "qsa_append_kv", false, false); }
qsa_status_t qsa_append_kv_bf16(const QsaAppendKvParams* p) {
  return append_kv_entry(p, "qsa_append_kv_bf16", true, false);
}
qsa_status_t qsa_append_kv8(const QsaAppendKvParams* p) { return append_kv_entry(p, "qsa_append_kv8", false, true); }
qsa_status_t qsa_append_kv8_bf16(const QsaAppendKvParams* p) {
  return append_kv_entry(p, "qsa_append_kv8_bf16", true, true);
}
qsa_status_t qsa_sparse_paged_kv8(const QsaSparsePagedKv8Params* p) {
  return sparse_paged_kv8_entry(p, "qsa_sparse_paged_kv8", false);
}
qsa_status_t qsa_sparse_paged_kv8_bf16(const QsaSparsePagedKv8Params* p) {
  return sparse_paged_kv8_entry(p, "qsa_sparse_paged_kv8_bf16", true);
}

qsa_status_t qsa_rotary(const QsaRotaryParams* p) { return rotary_entry(p, "qsa_rotary", 0); }
qsa_status_t qsa_rotary_bf16(const QsaRotaryParams* p) { return rotary_entry(p, "qsa_rotary_bf16", 1); }
qsa_status_t qsa_rotary_f32(const QsaRotaryParams* p) { return rotary_entry(p, "qsa_rotary_f32", 2); }

qsa_status_t qsa_rotary_frequencies(int32_t scaling, int32_t rot, double theta, double factor, double length,
                                    double lowTurns, double highTurns, double* out) {
  const char* fn = "qsa_rotary_frequencies";
  if (!out) return fail(QSA_ERR_INVALID_ARG, "%s: invFreq is NULL", fn);
  if (scaling < QSA_ROTARY_PLAIN || scaling > QSA_ROTARY_RAMP)
    return fail(QSA_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, scaling);
  if (rot < (scaling == QSA_ROTARY_BASE ? 4 : 2) || (rot & 1))
    return fail(QSA_ERR_INVALID_ARG, "%s: rotDim %d must be even and >= 2 (base scaling: 4)", fn, rot);
  if (!(theta > 1.0) || !std::isfinite(theta)) return fail(QSA_ERR_INVALID_ARG, "%s: theta must be finite and > 1", fn);
  if (scaling != QSA_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(QSA_ERR_INVALID_ARG, "%s: factor must be finite and >= 1", fn);
  if (scaling >= QSA_ROTARY_BLEND && (!(length >= 1.0) || !std::isfinite(length) || !(lowTurns > 0.0) ||
                                      !(highTurns > lowTurns) || !std::isfinite(highTurns)))
    return fail(QSA_ERR_INVALID_ARG, "%s: needs originalLength >= 1 and 0 < lowTurns < highTurns", fn);
  const double turn = 6.283185307179586;
  const double base = scaling == QSA_ROTARY_BASE ? theta * std::pow(factor, rot / (rot - 2.0)) : theta;
  // the (fractional) pair that turns n times in the original length
  auto pair_of = [&](double n) { return 0.5 * rot * std::log(length / (turn * n)) / std::log(theta); };
  const double first = scaling == QSA_ROTARY_RAMP ? std::floor(pair_of(highTurns)) : 0.0;
  const double last = scaling == QSA_ROTARY_RAMP ? std::ceil(pair_of(lowTurns)) : 0.0;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    double keep = 1.0;  // the share of the unscaled frequency
    if (scaling == QSA_ROTARY_LINEAR) keep = 0.0;
    if (scaling == QSA_ROTARY_BLEND) keep = (length * f / turn - lowTurns) / (highTurns - lowTurns);
    if (scaling == QSA_ROTARY_RAMP) keep = (last - i) / (last - first);  // last > first: floor(a) < ceil(b) for a < b
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    out[i] = keep * f + (1.0 - keep) * f / (keep == 1.0 ? 1.0 : factor);
  }
  return ok();
}

qsa_status_t qsa_store_kv4(const QsaStoreKv4Params* p) { return store_kv4_entry(p, "qsa_store_kv4", false); }
qsa_status_t qsa_store_kv4_bf16(const QsaStoreKv4Params* p) { return store_kv4_entry(p, "qsa_store_kv4_bf16", true); }
qsa_status_t qsa_sparse_paged_kv4(const QsaSparsePagedKv4Params* p) {
  return sparse_paged_kv4_entry(p, "qsa_sparse_paged_kv4", false);
}
qsa_status_t qsa_sparse_paged_kv4_bf16(const QsaSparsePagedKv4Params* p) {
  return sparse_paged_kv4_entry(p, "qsa_sparse_paged_kv4_bf16", true);
}
qsa_status_t qsa_sparse_weights_kv4(const QsaSparseWeightsKv4Params* p) {
  return sparse_weights_kv4_entry(p, "qsa_sparse_weights_kv4", false);
}
qsa_status_t qsa_sparse_weights_kv4_bf16(const QsaSparseWeightsKv4Params* p) {
  return sparse_weights_kv4_entry(p, "qsa_sparse_weights_kv4_bf16", true);
}

qsa_status_t qsa_evict_kv4(const QsaEvictKv4Params* p) {
  const char* fn = "qsa_evict_kv4";
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (!p->kvPool || !p->pageTable || !p->contextLengths || !p->total || !p->kept || !p->keptLengths)
    return fail(QSA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
  if (p->batchSize < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->numFlatPages < 1 || p->maxPagesPerSeq < 1 ||
      p->totalLen < 1 || p->budget < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: sizes must be >= 1", fn);
  if (p->sinks < 0 || p->recent < 0 || static_cast<long long>(p->sinks) + p->recent > p->budget)
    return fail(QSA_ERR_INVALID_ARG, "%s: sinks and recent must be >= 0 and together at most the budget", fn);
  if (p->poolRowBytes < QSA_KV4_ROW_BYTES)
    return fail(QSA_ERR_INVALID_ARG, "%s: poolRowBytes < %d", fn, QSA_KV4_ROW_BYTES);
  if (p->keptLengths == p->contextLengths)
    return fail(QSA_ERR_INVALID_ARG, "%s: keptLengths must not be contextLengths (which other heads still read)", fn);
  if (p->headDim != 128) return fail(QSA_ERR_UNSUPPORTED, "%s: headDim %d is not 128", fn, p->headDim);
  if (p->poolRowBytes % 16)
    return fail(QSA_ERR_UNSUPPORTED, "%s: poolRowBytes %d is not a multiple of 16", fn, p->poolRowBytes);
  if (!aligned(p->kvPool, 16) || !aligned(p->pageTable, 4) || !aligned(p->contextLengths, 4) || !aligned(p->total, 4) ||
      !aligned(p->kept, 4) || !aligned(p->keptLengths, 4) || !aligned(p->totalOut, 4) || !aligned(p->status, 4))
    return fail(QSA_ERR_UNSUPPORTED, "%s: kvPool must be 16-byte aligned, the others 4", fn);
  if (static_cast<long long>(p->batchSize) * p->numKVHeads > 0x7ffffffLL ||
      static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numFlatPages) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->numKVHeads) * p->poolRowBytes > 0x7fffffffLL || p->totalLen > (1 << 24) ||
      p->budget > (1 << 24))
    return fail(QSA_ERR_UNSUPPORTED, "%s: batchSize * numKVHeads, maxPagesPerSeq, numFlatPages, totalLen, budget or a "
                                     "pool row too large", fn);
  const cudaError_t e = qsa::launch_evict_kv4(*p);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

int32_t qsa_gather_scratch_pages(int32_t topK) { return topK < 1 ? 0 : qsa::gather_scratch_pages(topK); }

size_t qsa_gather_scratch_elems(int32_t B, int32_t Hkv, int32_t D, int32_t topK) {
  if (B < 1 || Hkv < 1 || D < 1 || topK < 1) return 0;
  return 2 * static_cast<size_t>(B) * qsa::gather_scratch_pages(topK) * qsa::kTokensPerPageHost * Hkv * D;
}

qsa_status_t qsa_gather_selected(const QsaGatherParams* p) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "qsa_gather_selected: params is NULL");
  if (!p->kvPool || !p->pageTable || !p->indices || !p->contextLengths || !p->scratch || !p->scratchPageTable ||
      !p->scratchIndices || !p->scratchLengths)
    return fail(QSA_ERR_INVALID_ARG, "qsa_gather_selected: a pointer is NULL");
  if (p->batchSize < 1 || p->numKVHeads < 1 || p->headDim < 1 || p->poolHeadDim < 1 || p->numFlatPages < 1 ||
      p->maxPagesPerSeq < 1 || p->topK < 1)
    return fail(QSA_ERR_INVALID_ARG, "qsa_gather_selected: sizes must be >= 1");
  if (p->poolHeadDim < p->headDim) return fail(QSA_ERR_INVALID_ARG, "qsa_gather_selected: poolHeadDim < headDim");
  if (p->headDim % 8 || p->poolHeadDim % 8 || p->numKVHeads * (p->headDim / 8) > qsa::gather_max_row_chunks())
    return fail(QSA_ERR_UNSUPPORTED, "qsa_gather_selected: headDim and poolHeadDim must be multiples of 8 and "
                                     "numKVHeads * headDim at most %d", qsa::gather_max_row_chunks() * 8);
  if (!aligned(p->kvPool, 16) || !aligned(p->scratch, 16))
    return fail(QSA_ERR_UNSUPPORTED, "qsa_gather_selected: kvPool and scratch must be 16-byte aligned");
  if (static_cast<long long>(p->maxPagesPerSeq) * qsa::kTokensPerPageHost > 0x7fffffffLL ||
      static_cast<long long>(p->batchSize) * p->topK > 0x7fffffffLL)
    return fail(QSA_ERR_UNSUPPORTED, "qsa_gather_selected: maxPagesPerSeq or batchSize * topK too large");
  const cudaError_t e = qsa::launch_gather(*p);
  return e == cudaSuccess ? ok() : cuda_fail(e, "qsa_gather_selected");
}

qsa_status_t qsa_sparse_decode(const QsaSparseDecodeParams* p) {
  return sparse_decode_entry(p, "qsa_sparse_decode", false);
}
qsa_status_t qsa_sparse_decode_bf16(const QsaSparseDecodeParams* p) {
  return sparse_decode_entry(p, "qsa_sparse_decode_bf16", true);
}

}  // extern "C"
