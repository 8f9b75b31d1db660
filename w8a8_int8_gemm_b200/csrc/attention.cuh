// attention.cuh -- what the two attention kernels share: their arguments, the
// packed documents, the masks as one limit per query, and the scores.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace w8a8 {

struct AttnParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  float* lse;  // [tokens_q, heads_q] or null
  const int32_t* cu_q;
  const int32_t* cu_k;  // document starts, or null: documents of equal length
  const int32_t* prefix;
  const float* slopes;
  int64_t ldq, hsq, ldk, hsk, ldv, hsv, ldo, hso;
  int tokens_q, tokens_k, docs;
  int heads_q, heads_k, group;  // group = heads_q / heads_k
  bool causal;
  float scale, cap;
  // With a cap, computed on the host to spare the kernels' registers: the cap in units of log2, the factor from a product
  // of q and k to a score in units of the cap, a quarter of the cap as such a product, and kTanhNear as a polynomial in
  // the product with the cap's factor in it.  (-1 where its coefficients, the cap times up to the fifth power of the
  // factor, leave binary32.)
  float cap_log2e, inv_cap, near, near_k[3];
  uint64_t timeout_ns;
};

// {64 values, tokens, heads} boxes of 64 x box_rows x 1 of a bf16 [tokens, heads, D] tensor, 128-byte swizzle.
inline bool encode_heads(CUtensorMap* map, const void* base, int D, int64_t tokens, int64_t heads, int64_t ld,
                         int64_t hs, int box_rows) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(tokens),
                              static_cast<cuuint64_t>(heads)};
  // (the stride of a dimension of one is free)
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * (tokens > 1 ? ld : D)),
                                 static_cast<cuuint64_t>(2 * (heads > 1 ? hs : D))};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_attention_rows(const AttnParams& p, int head_dim, int sms, cudaStream_t stream);
double rows_cost(const AttnParams& p, int sms, int* best_splits);
cudaError_t launch_attention_tiles(const AttnParams& p, int head_dim, cudaStream_t stream);

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// tanh(y) = y * sum_n k[n] y^2n, least squares on Chebyshev nodes: relative error 7e-7 (evaluated in binary32) for
// |y| <= 1 with kTanh (device code) and |y| <= 1/4 with kTanhNear (from which the host makes AttnParams::near_k).
constexpr float kTanhNear[3] = {9.9999960187e-1f, -3.3321876803e-1f, 1.2841111966e-1f};

#ifdef __CUDACC__

__device__ constexpr float kTanh[6] = {9.9999936384e-1f, -3.3328806676e-1f, 1.3279611505e-1f,
                                       -5.1555843877e-2f, 1.6687155235e-2f, -3.0449762314e-3f};

// One document: its tokens in the packed streams and its masks.
struct Doc {
  int q0, lq, k0, lk;
  int shift;   // query i stands at key place i + shift (the last query at the last key)
  int prefix;  // keys every query sees
};

// Start of document d in a stream of `tokens` tokens; whatever cu holds, the
// result is in [0, tokens], so no index built from it leaves the stream.
__device__ __forceinline__ int doc_start(const int32_t* cu, int d, int docs, int tokens) {
  if (cu == nullptr) return d * (tokens / docs);
  return min(max(__ldg(cu + d), 0), tokens);
}

// Work slots of `rows` rows (query tokens times `per` rows each) are numbered
// over the documents without a table: document d's slots begin at
// floor(start_d * per / rows) + d, which leaves room for every document's
// slots (a document of n rows needs at most floor((s + n)/rows) - floor(s/rows)
// + 1 of them) and at most one unused slot per document.
__device__ __forceinline__ int slot_begin(int start, int d, int per, int rows) {
  return static_cast<int>(static_cast<int64_t>(start) * per / rows) + d;
}

// The document of a slot, and the slot's first row in it (negative, or past
// the document's rows, in an unused slot): the last document that begins at
// or before the slot, 32 candidates at a time.  All lanes of the warp call it
// and return the same.  Up to 31 documents take one round of loads, a lane
// each, for everything there is to know.
__device__ __forceinline__ Doc slot_doc(const AttnParams& p, int slot, int per, int rows, int& row0) {
  const int lane = threadIdx.x & 31;
  Doc r;
  int d = 0;
  if (p.docs < 32) {
    const int q = doc_start(p.cu_q, min(lane, p.docs), p.docs, p.tokens_q);
    const int k = doc_start(p.cu_k, min(lane, p.docs), p.docs, p.tokens_k);
    const int prefix = p.prefix != nullptr ? __ldg(p.prefix + min(lane, p.docs - 1)) : 0;
    const int begin = slot_begin(q, lane, per, rows);
    d = max(0, __popc(__ballot_sync(0xFFFFFFFFu, lane < p.docs && begin <= slot)) - 1);
    row0 = (slot - __shfl_sync(0xFFFFFFFFu, begin, d)) * rows;
    r.q0 = __shfl_sync(0xFFFFFFFFu, q, d);
    r.lq = __shfl_sync(0xFFFFFFFFu, q, d + 1);
    r.k0 = __shfl_sync(0xFFFFFFFFu, k, d);
    r.lk = __shfl_sync(0xFFFFFFFFu, k, d + 1);
    r.prefix = __shfl_sync(0xFFFFFFFFu, prefix, d);
  } else {
    int n = p.docs;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int at = d + lane * step;
      const bool before =
          at < d + n && slot_begin(doc_start(p.cu_q, at, p.docs, p.tokens_q), at, per, rows) <= slot;
      const int skip = (max(1, __popc(__ballot_sync(0xFFFFFFFFu, before))) - 1) * step;
      d += skip;
      n = min(step, n - skip);
    }
    r.q0 = doc_start(p.cu_q, d, p.docs, p.tokens_q);
    r.lq = doc_start(p.cu_q, d + 1, p.docs, p.tokens_q);
    r.k0 = doc_start(p.cu_k, d, p.docs, p.tokens_k);
    r.lk = doc_start(p.cu_k, d + 1, p.docs, p.tokens_k);
    r.prefix = p.prefix != nullptr ? __ldg(p.prefix + d) : 0;
    row0 = (slot - slot_begin(r.q0, d, per, rows)) * rows;
  }
  r.lq = max(0, r.lq - r.q0);
  r.lk = max(0, r.lk - r.k0);
  r.shift = r.lk - r.lq;
  r.prefix = min(max(r.prefix, 0), r.lk);
  return r;
}

// Every mask here leaves query i the keys j < limit: all of the document's, or
// those up to its own place and the prefix.
__device__ __forceinline__ int key_limit(const AttnParams& p, const Doc& d, int i) {
  return p.causal ? min(max(i + d.shift + 1, d.prefix), d.lk) : d.lk;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * log2(e) * tanh(y), y = s * scale / cap, to a relative 1e-6: within the cap (|y| <= 1, two scores at a time) by
// the polynomial, beyond it as 1 - 2 / (1 + exp(2y)).  (That is off by 5e-7 of the cap: beyond the cap no more than
// that of the score, but all that is left of a score far inside a large cap.)
__device__ __forceinline__ uint64_t capped_within(uint64_t y, float cap_log2e) {
  const uint64_t u = mul2(y, y);
  uint64_t t = both(kTanh[5]);
#pragma unroll
  for (int n = 4; n >= 0; --n) t = fma2(t, u, both(kTanh[n]));
  return mul2(mul2(t, y), both(cap_log2e));
}

__device__ __forceinline__ float capped_beyond(float y, float cap_log2e) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2(y * (2.0f * kLog2e))));
  return fmaf(-2.0f * cap_log2e, r, cap_log2e);
}

// Both, for N scores in units of the cap; `beyond` where one of them may lie beyond it.
template <int N>
__device__ __forceinline__ void capped(float (&y)[N], bool beyond, float cap_log2e) {
  float s[N];
#pragma unroll
  for (int x = 0; x < N; x += 2) unpair(capped_within(pair(y[x], y[x + 1]), cap_log2e), s[x], s[x + 1]);
  if (beyond) {
#pragma unroll
    for (int x = 0; x < N; ++x) {
      if (!(fabsf(y[x]) <= 1.0f)) s[x] = capped_beyond(y[x], cap_log2e);
    }
  }
#pragma unroll
  for (int x = 0; x < N; ++x) y[x] = s[x];
}

#endif  // __CUDACC__

}  // namespace w8a8
