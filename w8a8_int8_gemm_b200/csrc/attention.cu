// attention.cu -- w8a8_attention: argument checks and the choice of kernel.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w8a8.h"
#include "attention.cuh"
#include "internal.h"

using namespace w8a8;

namespace {

struct View {
  const void* ptr;
  int64_t tokens, ld, heads, hs;
};

bool strides_ok(const View& v, int64_t dim) {
  if (v.ld < 0 || v.hs < 0 || v.ld > kMaxStride || v.hs > kMaxStride) return false;
  return (v.tokens <= 1 || v.ld >= dim) && (v.heads <= 1 || v.hs >= dim);
}

}  // namespace

extern "C" w8a8_status w8a8_attention(const w8a8_attention_desc* a, w8a8_stream_t stream) {
  if (a == nullptr) return W8A8_ERR_INVALID_ARG;
  constexpr int64_t kMaxTokens = int64_t{1} << 30;
  if (a->tokens_q < 0 || a->tokens_k < 0 || a->tokens_q > kMaxTokens || a->tokens_k > kMaxTokens) {
    return W8A8_ERR_INVALID_ARG;
  }
  if (a->docs < 1 || a->docs > (1 << 24) || a->heads_k < 1 || a->heads_q < a->heads_k || a->heads_q > 65536 ||
      a->heads_q % a->heads_k != 0 || (a->head_dim != 64 && a->head_dim != 128)) {
    return W8A8_ERR_INVALID_ARG;
  }
  if ((a->cu_q == nullptr && a->tokens_q % a->docs != 0) || (a->cu_k == nullptr && a->tokens_k % a->docs != 0)) {
    return W8A8_ERR_INVALID_ARG;
  }
  if (a->causal != 0 && a->causal != 1) return W8A8_ERR_INVALID_ARG;
  if (a->kernel < W8A8_ATTENTION_AUTO || a->kernel > W8A8_ATTENTION_TILES) return W8A8_ERR_INVALID_ARG;
  if (a->prefix != nullptr && !a->causal) return W8A8_ERR_INVALID_ARG;
  // (scale / cap stays within binary32, and a cap's error within the scores')
  if (!(a->scale >= 1.0e-12f && a->scale <= 1.0e6f)) return W8A8_ERR_INVALID_ARG;
  if (!(a->cap == 0.0f || (a->cap >= 1.0e-6f && a->cap <= 1.0e6f))) return W8A8_ERR_INVALID_ARG;
  if (a->tokens_q == 0) return W8A8_OK;
  const View views[4] = {{a->q, a->tokens_q, a->ldq, a->heads_q, a->hsq},
                         {a->k, a->tokens_k, a->ldk, a->heads_k, a->hsk},
                         {a->v, a->tokens_k, a->ldv, a->heads_k, a->hsv},
                         {a->out, a->tokens_q, a->ldo, a->heads_q, a->hso}};
  for (const View& v : views) {
    if (v.tokens == 0) continue;  // no keys: k and v are not used
    if (v.ptr == nullptr || !strides_ok(v, a->head_dim)) return W8A8_ERR_INVALID_ARG;
  }
  if (!rows_disjoint(a->tokens_q, a->ldo, a->heads_q, a->hso, a->head_dim)) return W8A8_ERR_INVALID_ARG;
  for (const View& v : views) {
    if (v.tokens == 0) continue;
    if (!aligned16(v.ptr) || v.ld % 8 != 0 || v.hs % 8 != 0) return W8A8_ERR_ALIGNMENT;
  }
  const uintptr_t words = reinterpret_cast<uintptr_t>(a->cu_q) | reinterpret_cast<uintptr_t>(a->cu_k) |
                          reinterpret_cast<uintptr_t>(a->prefix) | reinterpret_cast<uintptr_t>(a->slopes) |
                          reinterpret_cast<uintptr_t>(a->lse);
  if ((words & 3u) != 0) return W8A8_ERR_ALIGNMENT;
  int sms = 0;
  const w8a8_status st = check_current_device(&sms);
  if (st != W8A8_OK) return st;

  AttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.prefix = a->prefix;
  p.slopes = a->slopes;
  p.ldq = a->ldq;
  p.hsq = a->hsq;
  p.ldk = a->ldk;
  p.hsk = a->hsk;
  p.ldv = a->ldv;
  p.hsv = a->hsv;
  p.ldo = a->ldo;
  p.hso = a->hso;
  p.tokens_q = static_cast<int>(a->tokens_q);
  p.tokens_k = static_cast<int>(a->tokens_k);
  p.docs = a->docs;
  p.heads_q = a->heads_q;
  p.heads_k = a->heads_k;
  p.group = a->heads_q / a->heads_k;
  p.causal = a->causal != 0;
  p.scale = a->scale;
  p.cap = a->cap;
  p.cap_log2e = p.inv_cap = p.near = p.near_k[0] = p.near_k[1] = p.near_k[2] = 0.0f;
  if (a->cap > 0.0f) {
    p.cap_log2e = a->cap * kLog2e;
    p.inv_cap = a->scale / a->cap;
    const float square = p.inv_cap * p.inv_cap;
    float f = p.cap_log2e * p.inv_cap;
    p.near = p.inv_cap <= 1.0f && f * square * square >= 0x1p-120f ? 0.25f / p.inv_cap : -1.0f;
    for (int i = 0; i < 3; ++i, f *= square) p.near_k[i] = kTanhNear[i] * f;
  }
  p.timeout_ns = wait_timeout_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // The kernel that takes less for documents of the average length.  The tile kernel needs about 5 us beside an item's
  // tiles of 80 keys, which take 0.9 us with up to 128 queries and 1.1 us with more.  (Measured, row kernel against
  // tile kernel: one document of 2304 keys, 24 heads, 16 queries 13 | 32 us, 64 queries 23 | 32, 128 queries 45 | 33;
  // 16 000 keys, 8 key/value heads of 4: 128 rows 65 | 183, 512 rows 214 | 184.)
  int splits;
  const double by_rows = rows_cost(p, sms, &splits);
  const int64_t queries = (a->tokens_q + a->docs - 1) / a->docs;
  const int64_t items = (queries + 255) / 256 * a->docs * a->heads_q;
  const double tiles = static_cast<double>(a->tokens_k / a->docs) / 80.0;
  const double by_tiles = static_cast<double>((items + sms - 1) / sms) * (5.0 + tiles * (queries > 128 ? 1.1 : 0.9));
  const bool by_row_kernel =
      a->kernel == W8A8_ATTENTION_AUTO ? by_rows <= by_tiles : a->kernel == W8A8_ATTENTION_ROWS;
  if (by_row_kernel) return status_of(launch_attention_rows(p, a->head_dim, sms, s));
  return status_of(launch_attention_tiles(p, a->head_dim, s));
}
