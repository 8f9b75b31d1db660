// attention_rows.cu -- attention for few queries: a token per sequence over
// its cache, drafted tokens, short documents.
//
// The 16 rows of an mma.sync tile are 16 (token, head) pairs that share a
// key/value head (row r of a document is token r / group, head r % group of
// the group), so shared heads read their keys and values once.  The kernel is
// bound by reading K and V: with 16 rows the products are a tenth of the time
// the bytes take, and 5th-generation tensor cores (128 rows at least) would
// pass empty rows.  The keys of a slot of 16 rows are dealt in tiles of 64 to
// the CTAs of a cluster, which join their partial softmaxes (maximum, sum,
// weighted values) through distributed shared memory: no workspace, no second
// launch, and a fixed order of additions.
//
// One thread of a CTA loads tiles of K and V through a ring (TMA, 128-byte
// swizzle), three tiles ahead; four warps take 16 keys each of every tile
// (ldmatrix).  Two CTAs share an SM, so that one streams while the other
// starts or joins: 190 KB in flight per SM.  (Loads straight to the fragments'
// registers, one step ahead, kept 64 KB in flight with one CTA per SM, which
// left 16 sequences with 192 000 cached tokens, 32 heads over 8 of 128, at 237
// us; now 128-131 us, 6.0 TB/s, 0.92 of the measured copy rate.)
//
// P is split into two bf16 parts (p = hi + lo, 16 bits in all): the second
// product is free here, and the output then carries one bf16 rounding, its
// own.  Scores, maxima, sums and weighted values are binary32.
#include <cuda.h>

#include "attention.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

#include <cstring>

namespace w8a8 {
namespace {

constexpr int kWarps = 4;            // consumers; one more warp loads
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kTileK = 16 * kWarps;  // keys of a tile
constexpr int kStages = 3;
constexpr int kRows = 16;
constexpr int kMaxSplits = 8;
constexpr int kBlock = kTileK * 128;  // bytes of 64 values of a tile's keys

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 blocks of 16-bit values from shared memory (row i of block b at the address of lane 8 b + i).
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {  // transposed
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ float low_part(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_part(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Shared memory: the ring (a stage: K, then V, in blocks of 64 values), which the partial results reuse when the last
// tile is done, and what lies behind it.
template <int D>
__host__ __device__ constexpr int stage_bytes() {
  return 2 * (D / 64) * kBlock;
}
template <int D>
constexpr int smem_bytes() {
  return 1024 + kStages * stage_bytes<D>();
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 2)
    attention_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const AttnParams p, const int splits, int* err) {
  constexpr int kBlocks = D / 64;
  constexpr int kStage = stage_bytes<D>();
  constexpr int kPartRow = D + 8;  // floats of a row of partial results, padded against bank conflicts
  static_assert(kWarps * kRows * kPartRow * 4 <= kStages * kStage, "partial results fit the ring");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // [warp][row][kPartRow], scaled to the CTA's maximum; [0] becomes their sum
  float* part = reinterpret_cast<float*>(smem);
  __shared__ float sh_m[kWarps][kRows], sh_l[kWarps][kRows], cta_m[kRows], cta_l[kRows];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;

  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int g = lane >> 2, t = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % splits;  // the CTA's rank in its cluster
  const int unit = static_cast<int>(blockIdx.x) / splits;
  const int kv_head = unit % p.heads_k;
  const int slot = unit / p.heads_k;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    abort_word = 0;
    fence_mbar_init();
  }
  int row0;
  const Doc doc = slot_doc(p, slot, p.group, kRows, row0);
  const int rows = min(kRows, doc.lq * p.group - row0);  // rows of this slot
  if (rows <= 0 || row0 < 0) return;  // an unused slot (the whole cluster's)
  // Keys any row of the slot sees (limits grow with the token), and this CTA's tiles of them: every splits-th.
  const int keys = max(0, key_limit(p, doc, (row0 + rows - 1) / p.group));
  const int all_tiles = (keys + kTileK - 1) / kTileK;
  const int tiles = (all_tiles - split + splits - 1) / splits;
  __syncthreads();

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float o[D / 8][4] = {};  // product n: columns 8 n + 2 t, + 1 of rows g (0, 1) and g + 8 (2, 3)
  if (warp == kWarps) {
    if (elect_one()) {
      int fills = 0;
      for (; fills < tiles; ++fills) {
        const int stage = fills % kStages;
        if (!mbar_wait_bounded(&empty[stage], static_cast<uint32_t>((fills / kStages) & 1) ^ 1u, abort_flag,
                               p.timeout_ns, err, kSiteAttnLoad)) {
          break;
        }
        mbar_arrive_expect_tx(&full[stage], kStage);
        const int y = doc.k0 + (split + fills * splits) * kTileK;
        uint8_t* at = smem + stage * kStage;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) tma_load_3d(at + b * kBlock, &tm_k, &full[stage], 64 * b, y, kv_head);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          tma_load_3d(at + (kBlocks + b) * kBlock, &tm_v, &full[stage], 64 * b, y, kv_head);
        }
      }
      // Every load must have landed before the ring is used for anything else (on the normal path they have).
      for (int f = max(0, fills - kStages); f < fills; ++f) {
        mbar_wait_drain(&full[f % kStages], static_cast<uint32_t>((f / kStages) & 1), p.timeout_ns, err);
      }
    }
    __syncwarp();
  } else {
    // Rows g and g + 8 of this lane: token in the document, key limit, place.
    int limit[2], place[2];
    float slope[2];
    uint32_t qf[D / 16][4];  // A fragments: (row g | g + 8) x (values 16 x + 2 t | 16 x + 8 + 2 t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row0 + g + 8 * h;
      const bool live = g + 8 * h < rows;
      const int i = r / p.group;
      const int head = kv_head * p.group + r % p.group;
      limit[h] = live ? key_limit(p, doc, i) : 0;
      place[h] = i + doc.shift;
      slope[h] = (BIAS && live) ? __ldg(p.slopes + head) * kLog2e : 0.0f;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (doc.q0 + i) * p.ldq + head * p.hsq) + t;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        qf[x][h] = live ? __ldg(q + 8 * x) : 0u;
        qf[x][2 + h] = live ? __ldg(q + 8 * x + 4) : 0u;
      }
    }
    const float c_scale = p.scale * kLog2e;
    // ldmatrix addresses: block b's row i is lane 8 b + i's.  K: blocks are keys 0-7 | 8-15 x values 0-7 | 8-15 of a
    // step of 16 values (row = key).  V, transposed: keys 0-7 | 8-15 x values 0-7 | 8-15.
    const uint32_t k_row = 16 * warp + (lane & 7) + ((lane >> 4) << 3), k_chunk = (lane >> 3) & 1;
    const uint32_t v_row = 16 * warp + (lane & 15), v_chunk = lane >> 4;
    const uint32_t base = smem_u32(smem);

    for (int f = 0; f < tiles; ++f) {
      const int stage = f % kStages;
      if (!warp_wait(&full[stage], static_cast<uint32_t>((f / kStages) & 1), abort_flag, p.timeout_ns, err,
                     kSiteAttnOperand)) {
        break;
      }
      const uint32_t at = base + stage * kStage;
      const int key0 = (split + f * splits) * kTileK + 16 * warp;
      float s[2][4] = {};
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        uint32_t b[4];  // keys 0-7: values 0-7, 8-15; keys 8-15: the same
        ldmatrix4(b, at + (x / 4) * kBlock + k_row * 128 + (((2 * (x % 4) + k_chunk) ^ (k_row & 7)) << 4));
        mma_bf16(s[0], qf[x][0], qf[x][1], qf[x][2], qf[x][3], b[0], b[1]);
        mma_bf16(s[1], qf[x][0], qf[x][1], qf[x][2], qf[x][3], b[2], b[3]);
      }

      if constexpr (CAP) {
        float far = 0.0f;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
#pragma unroll
          for (int x = 0; x < 4; ++x) far = fmaxf(far, fabsf(s[a][x] *= p.inv_cap));
        }
        float y[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
        capped(y, far > 1.0f, p.cap_log2e);
#pragma unroll
        for (int x = 0; x < 8; ++x) s[x / 4][x % 4] = y[x];
        __syncwarp();
      }
      // Scores in units of log2, masked by the rows' limits; s[a][2h + e]: row h, key 8a + 2t + e.
      float top[2] = {m[0], m[1]};
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int h = x >> 1;
          const int j = key0 + 8 * a + 2 * t + (x & 1);
          float y = CAP ? s[a][x] : s[a][x] * c_scale;
          if (BIAS) y -= slope[h] * fabsf(static_cast<float>(place[h] - j));
          s[a][x] = j < limit[h] ? y : -INFINITY;
          top[h] = fmaxf(top[h], s[a][x]);
        }
      }
      float shrink[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 2));
        const float from = top[h] == -INFINITY ? 0.0f : top[h];
        shrink[h] = ex2(m[h] - from);
        m[h] = top[h];
        l[h] *= shrink[h];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[a][2 * h + e] = ex2(s[a][2 * h + e] - from);
            l[h] += s[a][2 * h + e];
          }
        }
      }
      if (__any_sync(0xFFFFFFFFu, shrink[0] != 1.0f || shrink[1] != 1.0f)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= shrink[0];
          o[n][1] *= shrink[0];
          o[n][2] *= shrink[1];
          o[n][3] *= shrink[1];
        }
      }
      uint32_t hi[4], lo[4];  // A fragment: (row g | g + 8) x (keys of a = 0 | 1)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = s[a][2 * h], p1 = s[a][2 * h + 1];
          const uint32_t w = pack_bf16(p0, p1);
          hi[2 * a + h] = w;
          lo[2 * a + h] = pack_bf16(p0 - low_part(w), p1 - high_part(w));
        }
      }
      // Keys that no row sees weigh nothing, whatever memory holds there.
      const int left = keys - key0;  // of the 16 keys
      const uint32_t keep0 = 2 * t + 1 < left ? 0xFFFFFFFFu : 2 * t < left ? 0xFFFFu : 0u;
      const uint32_t keep1 = 2 * t + 9 < left ? 0xFFFFFFFFu : 2 * t + 8 < left ? 0xFFFFu : 0u;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        uint32_t b[4];  // values 0-7: keys 0-7, 8-15; values 8-15: the same
        ldmatrix4_t(b, at + (kBlocks + x / 4) * kBlock + v_row * 128 + (((2 * (x % 4) + v_chunk) ^ (v_row & 7)) << 4));
        if (left < 16) {
          b[0] &= keep0;
          b[1] &= keep1;
          b[2] &= keep0;
          b[3] &= keep1;
        }
        mma_bf16(o[2 * x], hi[0], hi[1], hi[2], hi[3], b[0], b[1]);
        mma_bf16(o[2 * x], lo[0], lo[1], lo[2], lo[3], b[0], b[1]);
        mma_bf16(o[2 * x + 1], hi[0], hi[1], hi[2], hi[3], b[2], b[3]);
        mma_bf16(o[2 * x + 1], lo[0], lo[1], lo[2], lo[3], b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
    }

    // The warp's sums over the four lanes of a row.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
      if (t == 0) sh_m[warp][g + 8 * h] = m[h];
    }
  }
  __syncthreads();  // (the ring is free)
  if (warp < kWarps) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = sh_m[0][g + 8 * h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh_m[w][g + 8 * h]);
      const float f = ex2(m[h] - (top == -INFINITY ? 0.0f : top));
      if (t == 0) sh_l[warp][g + 8 * h] = l[h] * f;
      if (warp == 0 && t == 0) cta_m[g + 8 * h] = top;
      float* to = part + (warp * kRows + g + 8 * h) * kPartRow + 2 * t;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<float2*>(to + 8 * n) = make_float2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
    float4* at = reinterpret_cast<float4*>(part + e / (D / 4) * kPartRow + e % (D / 4) * 4);
    float4 sum = *at;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 x = at[w * kRows * kPartRow / 4];
      sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
    }
    *at = sum;
  }
  if (threadIdx.x < kRows) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh_l[w][threadIdx.x];
    cta_l[threadIdx.x] = sum;
  }
  if (splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }

  // Each CTA of the cluster joins and writes its share of the slot's rows x values, two values at a time.
  const uint32_t part_addr = smem_u32(part);
  const uint32_t m_addr = smem_u32(&cta_m[0]);
  const uint32_t l_addr = smem_u32(&cta_l[0]);
  for (int e = 2 * (split * kThreads + static_cast<int>(threadIdx.x)); e < rows * D; e += 2 * splits * kThreads) {
    const int r = e / D, col = e % D;
    // (unrolled, so that the remote loads overlap)
    float cm[kMaxSplits], cl[kMaxSplits], c0[kMaxSplits], c1[kMaxSplits];
#pragma unroll
    for (int c = 0; c < kMaxSplits; ++c) {
      cm[c] = -INFINITY;
      cl[c] = c0[c] = c1[c] = 0.0f;
      if (c < splits) {
        cm[c] = ld_cluster_f32(map_to_cta(m_addr + 4 * r, c));
        cl[c] = ld_cluster_f32(map_to_cta(l_addr + 4 * r, c));
        const uint32_t a = map_to_cta(part_addr + 4 * (r * kPartRow + col), c);
        c0[c] = ld_cluster_f32(a);
        c1[c] = ld_cluster_f32(a + 4);
      }
    }
    float top = cm[0];
#pragma unroll
    for (int c = 1; c < kMaxSplits; ++c) top = fmaxf(top, cm[c]);
    const float from = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
    for (int c = 0; c < kMaxSplits; ++c) {
      const float f = ex2(cm[c] - from);
      sum = fmaf(f, cl[c], sum);
      x0 = fmaf(f, c0[c], x0);
      x1 = fmaf(f, c1[c], x1);
    }
    const int i = (row0 + r) / p.group;
    const int head = kv_head * p.group + (row0 + r) % p.group;
    const int64_t token = doc.q0 + i;
    // No key left, or none with a weight (scores of -inf): 0 (and a logarithm of -inf).
    const bool any = sum != 0.0f;
    const float inv = any ? 1.0f / sum : 0.0f;
    *reinterpret_cast<uint32_t*>(p.out + token * p.ldo + head * p.hso + col) =
        any ? pack_bf16(x0 * inv, x1 * inv) : 0u;
    if (p.lse != nullptr && col == 0) {
      p.lse[token * p.heads_q + head] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
    }
  }
  if (splits > 1) cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const AttnParams& p, int splits, cudaStream_t stream) {
  CUtensorMap tm_k, tm_v;
  std::memset(&tm_k, 0, sizeof tm_k);
  std::memset(&tm_v, 0, sizeof tm_v);
  if (p.tokens_k > 0 && (!encode_heads(&tm_k, p.k, D, p.tokens_k, p.heads_k, p.ldk, p.hsk, kTileK) ||
                         !encode_heads(&tm_v, p.v, D, p.tokens_k, p.heads_k, p.ldv, p.hsv, kTileK))) {
    return cudaErrorInvalidValue;
  }
  int* err = nullptr;
  cudaError_t e = error_word_address(&err);
  if (e != cudaSuccess) return e;
  auto kernel = attention_rows_kernel<D, CAP, BIAS>;
  const int smem = smem_bytes<D>();
  static std::atomic<uint64_t> set{0};
  e = allow_shared_memory(kernel, smem, set);
  if (e != cudaSuccess) return e;
  const int64_t slots = static_cast<int64_t>(p.tokens_q) * p.group / kRows + p.docs;
  const int64_t blocks = slots * p.heads_k * splits;
  if (blocks > 2147483647) return cudaErrorInvalidValue;
  cudaLaunchConfig_t lc;
  std::memset(&lc, 0, sizeof lc);
  lc.gridDim = dim3(static_cast<unsigned>(blocks));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = static_cast<size_t>(smem);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(splits);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  lc.attrs = &attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, kernel, tm_k, tm_v, p, splits, err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// What the row kernel takes for documents of the average length, in us, and the CTAs per slot that take least.  A CTA
// needs about 5 us beside its tiles and 1 us a tile of 64 keys, and two share an SM.  (Measured with 1, 2, 4 and 8
// CTAs a slot: 16 sequences of 12 000 keys, 8 key/value heads: 149, 79, 86, 101 us; 16 of 2 000: 24, 19, 25, 36; 64 of
// 512, 4 rows each: 36, 50, 79, 149; one of 2304, 24 heads: 25, 16, 11, 11.)
double rows_cost(const AttnParams& p, int sms, int* best_splits) {
  const int64_t rows = (static_cast<int64_t>(p.tokens_q) * p.group + p.docs - 1) / p.docs;
  const int64_t units = (rows + kRows - 1) / kRows * p.docs * p.heads_k;
  const int64_t tiles = (p.tokens_k / p.docs + kTileK - 1) / kTileK;
  double best = 0.0;
  for (int splits = 1; splits <= kMaxSplits; splits *= 2) {
    const int64_t rounds = (units * splits + 2 * sms - 1) / (2 * sms);
    const double cost = static_cast<double>(rounds) * (5.0 + static_cast<double>((tiles + splits - 1) / splits));
    if (splits == 1 || cost < best) {
      best = cost;
      *best_splits = splits;
    }
  }
  return best;
}

cudaError_t launch_attention_rows(const AttnParams& p, int head_dim, int sms, cudaStream_t stream) {
  int splits = 1;
  rows_cost(p, sms, &splits);
  const bool cap = p.cap > 0.0f, bias = p.slopes != nullptr;
  if (head_dim == 64) {
    if (cap) return bias ? launch<64, true, true>(p, splits, stream) : launch<64, true, false>(p, splits, stream);
    return bias ? launch<64, false, true>(p, splits, stream) : launch<64, false, false>(p, splits, stream);
  }
  if (cap) return bias ? launch<128, true, true>(p, splits, stream) : launch<128, true, false>(p, splits, stream);
  return bias ? launch<128, false, true>(p, splits, stream) : launch<128, false, false>(p, splits, stream);
}

}  // namespace w8a8
