// attention_rows.cu -- attention for few queries: a token per sequence over
// its cache, drafted tokens, short documents.
//
// The 16 rows of an mma.sync tile are 16 (token, head) pairs that share a
// key/value head (row r of a document is token r / group, head r % group of
// the group), so shared heads read their keys and values once.  The kernel is
// bound by reading K and V: with 16 rows the products are a tenth of the time
// the bytes take, and 5th-generation tensor cores (128 rows at least) would
// pass empty rows.  The keys of a slot of 16 rows are dealt in steps of 16 to
// the 8 warps of the CTAs of a cluster, which join their partial softmaxes
// (maximum, sum, weighted values) through distributed shared memory: no
// workspace, no second launch, and a fixed order of additions.
//
// K and V go from global memory straight to the fragments, 16 bytes a load:
// the order of the head dimension inside a product is free as long as Q's
// fragments follow it, and so is the order of the output's columns.  A lane
// holds 8 successive values of a key (two k-steps of Q K^T), and 8 successive
// values of four keys of V (one column of 8 products P V; pairs of keys are
// packed by byte permutes).  The next step's keys are loaded when this step's
// scores are done with their registers, its values after this step's P V.
//
// P is split into two bf16 parts (p = hi + lo, 16 bits in all): the second
// product is free here, and the output then carries one bf16 rounding, its
// own.  Scores, maxima, sums and weighted values are binary32.
#include "attention.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

#include <cstring>

namespace w8a8 {
namespace {

constexpr int kWarps = 8;
constexpr int kStep = 16;  // keys of a warp's step
constexpr int kRows = 16;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float low_part(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_part(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

template <int D>
struct Shared {
  float part[kWarps][kRows][D];   // a warp's weighted values, scaled to the CTA's maximum; [0] holds the CTA's sum
  float m[kWarps][kRows];
  float l[kWarps][kRows];
  float cta_m[kRows];
  float cta_l[kRows];
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(32 * kWarps, 1) attention_rows_kernel(const AttnParams p, const int splits) {
  constexpr int kChunks = D / 32;  // 16-byte chunks of a key per lane
  constexpr int kHalves = D / 64;  // 16-byte chunks of a value per lane
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem_raw);

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % splits;  // the CTA's rank in its cluster
  const int unit = static_cast<int>(blockIdx.x) / splits;
  const int kv_head = unit % p.heads_k;
  const int slot = unit / p.heads_k;

  const int d = slot_doc(p, slot, p.group, kRows);
  const Doc doc = load_doc(p, d);
  const int row0 = (slot - slot_begin(p, d, p.group, kRows)) * kRows;
  const int rows = min(kRows, doc.lq * p.group - row0);  // rows of this slot
  if (rows <= 0 || row0 < 0) return;  // an unused slot (the whole cluster's)

  // Rows g and g + 8 of this lane: token in the document, key limit, place.
  int limit[2];
  int place[2];
  float slope[2];
  uint4 qf[2][kChunks];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row0 + g + 8 * h;
    const bool live = g + 8 * h < rows;
    const int i = r / p.group;
    const int head = kv_head * p.group + r % p.group;
    limit[h] = live ? key_limit(p, doc, i) : 0;
    place[h] = i + doc.shift;
    slope[h] = (BIAS && live) ? __ldg(p.slopes + head) * kLog2e : 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      qf[h][c] = make_uint4(0, 0, 0, 0);
      if (live) {
        qf[h][c] = __ldg(reinterpret_cast<const uint4*>(p.q + (doc.q0 + i) * p.ldq + head * p.hsq + c * 32 + t * 8));
      }
    }
  }
  // Keys any row of the slot sees (limits grow with the token).
  const int keys = max(0, key_limit(p, doc, (row0 + rows - 1) / p.group));

  const __nv_bfloat16* kbase = p.k + doc.k0 * p.ldk + kv_head * p.hsk + t * 8;
  const __nv_bfloat16* vbase = p.v + doc.k0 * p.ldv + kv_head * p.hsv + g * 8;
  uint4 kf[2][kChunks];       // keys 8a + g of the step
  uint4 vf[4][kHalves];       // keys 2t, 2t + 1, 2t + 8, 2t + 9
  auto load_k = [&](int key0) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int j = key0 + 8 * a + g;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        kf[a][c] = make_uint4(0, 0, 0, 0);
        if (j < keys) kf[a][c] = __ldg(reinterpret_cast<const uint4*>(kbase + j * p.ldk + c * 32));
      }
    }
  };
  auto load_v = [&](int key0) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int j = key0 + 2 * t + (b & 1) + 8 * (b >> 1);
#pragma unroll
      for (int c = 0; c < kHalves; ++c) {
        vf[b][c] = make_uint4(0, 0, 0, 0);  // keys out of range weigh nothing, whatever memory holds there
        if (j < keys) vf[b][c] = __ldg(reinterpret_cast<const uint4*>(vbase + j * p.ldv + c * 64));
      }
    }
  };

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float o[kHalves * 8][4] = {};  // product n: column (lane / 4) * 8 + n % 8 + 64 (n / 8) of the head at row g / g + 8
  const float c_scale = p.scale * kLog2e;
  const float c_tanh = CAP ? 2.0f * kLog2e * p.scale / p.cap : 0.0f;
  const float c_cap = CAP ? p.cap * kLog2e : 0.0f;

  const int stride = splits * kWarps * kStep;
  int key0 = (split * kWarps + warp) * kStep;
  if (key0 < keys) {
    load_k(key0);
    load_v(key0);
  }
  for (; key0 < keys; key0 += stride) {
    float s[2][4] = {};
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          mma_bf16(s[a], word(qf[0][c], 2 * h), word(qf[1][c], 2 * h), word(qf[0][c], 2 * h + 1),
                   word(qf[1][c], 2 * h + 1), word(kf[a][c], 2 * h), word(kf[a][c], 2 * h + 1));
        }
      }
    }
    if (key0 + stride < keys) load_k(key0 + stride);

    // Scores in units of log2, masked by the rows' limits; s[a][2h + e]: row h, key 8a + 2t + e.
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int h = x >> 1;
        const int j = key0 + 8 * a + 2 * t + (x & 1);
        float y = CAP ? capped(s[a][x], c_tanh, c_cap) : s[a][x] * c_scale;
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
      const float base = top[h] == -INFINITY ? 0.0f : top[h];
      shrink[h] = ex2(m[h] - base);
      m[h] = top[h];
      l[h] *= shrink[h];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[a][2 * h + e] = ex2(s[a][2 * h + e] - base);
          l[h] += s[a][2 * h + e];
        }
      }
    }
    if (__any_sync(0xFFFFFFFFu, shrink[0] != 1.0f || shrink[1] != 1.0f)) {
#pragma unroll
      for (int n = 0; n < kHalves * 8; ++n) {
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
#pragma unroll
    for (int c = 0; c < kHalves; ++c) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const uint32_t sel = (n & 1) ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(word(vf[0][c], n >> 1), word(vf[1][c], n >> 1), sel);
        const uint32_t b1 = __byte_perm(word(vf[2][c], n >> 1), word(vf[3][c], n >> 1), sel);
        mma_bf16(o[8 * c + n], hi[0], hi[1], hi[2], hi[3], b0, b1);
        mma_bf16(o[8 * c + n], lo[0], lo[1], lo[2], lo[3], b0, b1);
      }
    }
    if (key0 + stride < keys) load_v(key0 + stride);
  }

  // The warp's sums over the four lanes of a row, then the CTA's maximum.
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
    if (t == 0) sh.m[warp][g + 8 * h] = m[h];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float top = sh.m[0][g + 8 * h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh.m[w][g + 8 * h]);
    const float f = ex2(m[h] - (top == -INFINITY ? 0.0f : top));
    if (t == 0) sh.l[warp][g + 8 * h] = l[h] * f;
    if (warp == 0 && t == 0) sh.cta_m[g + 8 * h] = top;
#pragma unroll
    for (int c = 0; c < kHalves; ++c) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        // columns 2t and 2t + 1 of product n are values (2t) * 8 + n and (2t + 1) * 8 + n of the half
        sh.part[warp][g + 8 * h][64 * c + 16 * t + n] = o[8 * c + n][2 * h] * f;
        sh.part[warp][g + 8 * h][64 * c + 16 * t + 8 + n] = o[8 * c + n][2 * h + 1] * f;
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kRows * D; e += 32 * kWarps) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh.part[w][e / D][e % D];
    sh.part[0][e / D][e % D] = sum;
  }
  if (threadIdx.x < kRows) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh.l[w][threadIdx.x];
    sh.cta_l[threadIdx.x] = sum;
  }
  if (splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }

  // Each CTA of the cluster joins and writes its share of the slot's rows x values, two values at a time.
  const uint32_t part_addr = smem_u32(&sh.part[0][0][0]);
  const uint32_t m_addr = smem_u32(&sh.cta_m[0]);
  const uint32_t l_addr = smem_u32(&sh.cta_l[0]);
  for (int e = 2 * (split * 32 * kWarps + static_cast<int>(threadIdx.x)); e < rows * D; e += 2 * splits * 32 * kWarps) {
    const int r = e / D, col = e % D;
    float top = -INFINITY;
    for (int c = 0; c < splits; ++c) top = fmaxf(top, ld_cluster_f32(map_to_cta(m_addr + 4 * r, c)));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, x0 = 0.0f, x1 = 0.0f;
    for (int c = 0; c < splits; ++c) {
      const float f = ex2(ld_cluster_f32(map_to_cta(m_addr + 4 * r, c)) - base);
      const uint32_t a = map_to_cta(part_addr + 4 * e, c);
      sum += f * ld_cluster_f32(map_to_cta(l_addr + 4 * r, c));
      x0 += f * ld_cluster_f32(a);
      x1 += f * ld_cluster_f32(a + 4);
    }
    const int i = (row0 + r) / p.group;
    const int head = kv_head * p.group + (row0 + r) % p.group;
    const int64_t token = doc.q0 + i;
    // No key left: 0 (and a logarithm of -inf).
    const bool any = key_limit(p, doc, i) > 0;
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
  auto kernel = attention_rows_kernel<D, CAP, BIAS>;
  const int smem = static_cast<int>(sizeof(Shared<D>));
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t slots = static_cast<int64_t>(p.tokens_q) * p.group / kRows + p.docs;
  const int64_t blocks = slots * p.heads_k * splits;
  if (blocks > 2147483647) return cudaErrorInvalidValue;
  cudaLaunchConfig_t lc;
  std::memset(&lc, 0, sizeof lc);
  lc.gridDim = dim3(static_cast<unsigned>(blocks));
  lc.blockDim = dim3(32 * kWarps);
  lc.dynamicSmemBytes = static_cast<size_t>(smem);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(splits);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  lc.attrs = &attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, kernel, p, splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_rows(const AttnParams& p, int head_dim, int sms, cudaStream_t stream) {
  // CTAs per slot: enough to give every SM a few, as long as a CTA keeps two steps for each of its warps.
  const int64_t rows_per_doc = (static_cast<int64_t>(p.tokens_q) * p.group + p.docs - 1) / p.docs;
  const int64_t units = (rows_per_doc + kRows - 1) / kRows * p.docs * p.heads_k;
  const int64_t keys_per_doc = p.tokens_k / p.docs;
  int splits = 1;
  while (splits < 8 && units * splits < 4 * sms && keys_per_doc >= 2 * splits * 2 * kWarps * kStep) splits *= 2;
  const bool cap = p.cap > 0.0f, bias = p.slopes != nullptr;
  if (head_dim == 64) {
    if (cap) return bias ? launch<64, true, true>(p, splits, stream) : launch<64, true, false>(p, splits, stream);
    return bias ? launch<64, false, true>(p, splits, stream) : launch<64, false, false>(p, splits, stream);
  }
  if (cap) return bias ? launch<128, true, true>(p, splits, stream) : launch<128, true, false>(p, splits, stream);
  return bias ? launch<128, false, true>(p, splits, stream) : launch<128, false, false>(p, splits, stream);
}

}  // namespace w8a8
