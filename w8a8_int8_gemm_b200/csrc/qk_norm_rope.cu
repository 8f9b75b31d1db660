// qk_norm_rope.cu -- norms of queries and keys and their position rotation.
//
// For every token m and head h of Q and of K, with D = head_dim values x[i]:
//   n[i] = x[i] * rsqrt(sum_j x[j]^2 / D + eps) * w[i]                 (RMS norm; w = 1 where no weight is given)
//   the first R = rot_dim values turn in pairs (a, b) by the table's row of the token:
//   a' = n[a] cos[t] - n[b] sin[t],   b' = n[b] cos[t] + n[a] sin[t],   t = 0 .. R/2 - 1,
//   with (a, b) = (t, t + R/2) (W8A8_ROPE_HALVES) or (2t, 2t + 1) (W8A8_ROPE_PAIRS).
// Everything between the bf16 load and the bf16 store is binary32; the store
// is the one rounding.
//
// What bounds it: memory (2 bytes read and 2 written per value, plus 4 R
// bytes of table per token).  Separate norm and rotation kernels would move
// every value twice.  So: L = D/8 lanes (rounded up to a power of two) hold a
// head, 8 values (one 16-byte load) per lane; the sum of squares is a shuffle
// reduction over the L lanes, and a rotated pair lies in one lane (pairs) or
// in two lanes of the same head (halves: one shuffle per value).  A warp
// holds 32/L heads at a time and kSteps times that many of one token in all,
// loaded together so that 64 bytes per lane are in flight, and reads the
// token's table row once for them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w8a8.h"
#include "internal.h"

namespace w8a8 {
namespace {

constexpr int kSteps = 4;
constexpr int kWarps = 8;

struct QkParams {
  const __nv_bfloat16* x[2];  // q, k
  __nv_bfloat16* y[2];
  const __nv_bfloat16* w[2];  // weights or null
  int64_t ld[2], hs[2], ld_y[2], hs_y[2];
  const float* cos;
  const float* sin;
  const int32_t* positions;
  int64_t M, table_rows;
  int heads[2];
  int D, R;
  int units;  // warps per token
  float eps, inv_d;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// L: lanes per head (2 .. 32).  PAIRS: the rotation's pairing.
template <int L, bool PAIRS>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const QkParams p) {
  constexpr int kPerStep = 32 / L;            // heads of one step
  constexpr int kTable = PAIRS ? 4 : 8;       // table entries of a lane
  const int lane = threadIdx.x & 31;
  const int sub = lane % L;                   // place in the head: values 8 sub .. 8 sub + 7
  const int grp = lane / L;
  const bool in_head = 8 * sub < p.D;
  const int half_lanes = p.R / 16;            // halves: lanes of the first half of the rotated values
  const bool turns = 8 * sub < p.R;
  const bool upper = !PAIRS && sub >= half_lanes;  // holds the b of its pairs
  const int mate = grp * L + (upper ? sub - half_lanes : sub + half_lanes);
  const int entry = PAIRS ? 4 * sub : 8 * (upper ? sub - half_lanes : sub);
  const int all_heads = p.heads[0] + p.heads[1];

  uint4 wv[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    wv[j] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);  // ones
    if (p.w[j] != nullptr && in_head) wv[j] = __ldg(reinterpret_cast<const uint4*>(p.w[j] + 8 * sub));
  }

  const int64_t total = p.M * p.units;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < total;
       unit += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t m = unit / p.units;
    const int head0 = static_cast<int>(unit - m * p.units) * (kSteps * kPerStep) + grp;

    uint4 v[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = head0 + s * kPerStep;
      v[s] = make_uint4(0, 0, 0, 0);
      if (h < all_heads && in_head) {
        const int j = h >= p.heads[0];
        const int hj = j ? h - p.heads[0] : h;
        v[s] = *reinterpret_cast<const uint4*>(p.x[j] + m * p.ld[j] + hj * p.hs[j] + 8 * sub);
      }
    }

    float c[kTable], sn[kTable];
    if (p.cos != nullptr) {
      const int64_t row = p.positions != nullptr ? static_cast<int64_t>(__ldg(p.positions + m)) : m;
      // A position outside the table reads nothing and turns by NaN.
      const bool known = row >= 0 && row < p.table_rows;
#pragma unroll
      for (int i = 0; i < kTable; ++i) c[i] = sn[i] = __int_as_float(0x7FFFFFFF);
      if (turns && known) {
        const float4* cr = reinterpret_cast<const float4*>(p.cos + row * (p.R / 2) + entry);
        const float4* sr = reinterpret_cast<const float4*>(p.sin + row * (p.R / 2) + entry);
#pragma unroll
        for (int i = 0; i < kTable / 4; ++i) {
          const float4 a = __ldg(cr + i), b = __ldg(sr + i);
          c[4 * i] = a.x, c[4 * i + 1] = a.y, c[4 * i + 2] = a.z, c[4 * i + 3] = a.w;
          sn[4 * i] = b.x, sn[4 * i + 1] = b.y, sn[4 * i + 2] = b.z, sn[4 * i + 3] = b.w;
        }
      }
    }

#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = head0 + s * kPerStep;
      float f[8], w[8];
      unpack8(v[s], f);
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
      const float r = rsqrtf(fmaf(sq, p.inv_d, p.eps));
      const int j = h >= p.heads[0];
      unpack8(j ? wv[1] : wv[0], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
      if (p.cos != nullptr) {
        if constexpr (PAIRS) {
          if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = f[2 * i], b = f[2 * i + 1];
              f[2 * i] = a * c[i] - b * sn[i];
              f[2 * i + 1] = b * c[i] + a * sn[i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float other = __shfl_sync(0xFFFFFFFFu, f[i], mate);
            if (turns) f[i] = upper ? f[i] * c[i] + other * sn[i] : f[i] * c[i] - other * sn[i];
          }
        }
      }
      if (h < all_heads && in_head) {
        const int hj = j ? h - p.heads[0] : h;
        *reinterpret_cast<uint4*>(p.y[j] + m * p.ld_y[j] + hj * p.hs_y[j] + 8 * sub) = pack8(f);
      }
    }
  }
}

template <int L>
cudaError_t launch(const QkParams& p, bool pairs, cudaStream_t stream) {
  const int64_t blocks = (p.M * p.units + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(blocks < (int64_t{1} << 30) ? blocks : (int64_t{1} << 30));
  if (pairs) {
    qk_norm_rope_kernel<L, true><<<grid, 32 * kWarps, 0, stream>>>(p);
  } else {
    qk_norm_rope_kernel<L, false><<<grid, 32 * kWarps, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

constexpr int64_t kMaxStride = 2147483640;  // elements; keeps m * stride within 63 bits

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

}  // namespace

bool rows_disjoint(int64_t rows, int64_t ld, int64_t heads, int64_t hs, int64_t dim) {
  if (heads > 1 && rows > 1) return (hs >= dim && ld >= (heads - 1) * hs + dim) || (ld >= dim && hs >= (rows - 1) * ld + dim);
  return (heads <= 1 || hs >= dim) && (rows <= 1 || ld >= dim);
}

}  // namespace w8a8

using namespace w8a8;

extern "C" w8a8_status w8a8_qk_norm_rope(const w8a8_qk_desc* d, w8a8_stream_t stream) {
  if (d == nullptr) return W8A8_ERR_INVALID_ARG;
  if (d->M < 0 || d->M > 2147483647 || d->heads_q < 0 || d->heads_k < 0 || d->heads_q > 65536 || d->heads_k > 65536) {
    return W8A8_ERR_INVALID_ARG;
  }
  if (d->head_dim < 16 || d->head_dim > 256 || d->head_dim % 8 != 0) return W8A8_ERR_INVALID_ARG;
  if (!(d->eps >= 0.0f) || d->eps > 3.0e38f) return W8A8_ERR_INVALID_ARG;
  if (d->layout != W8A8_ROPE_HALVES && d->layout != W8A8_ROPE_PAIRS) return W8A8_ERR_INVALID_ARG;
  const bool rotate = d->cos != nullptr;
  if (rotate != (d->sin != nullptr) || (!rotate && d->positions != nullptr)) return W8A8_ERR_INVALID_ARG;
  if (rotate) {
    if (d->rot_dim < 16 || d->rot_dim > d->head_dim || d->rot_dim % 16 != 0) return W8A8_ERR_INVALID_ARG;
    if (d->table_rows < 0 || (d->positions == nullptr && d->table_rows < d->M)) return W8A8_ERR_INVALID_ARG;
  }
  const int64_t strides[8] = {d->ldq, d->hsq, d->ldk, d->hsk, d->ldq_out, d->hsq_out, d->ldk_out, d->hsk_out};
  const void* in[2] = {d->q, d->k};
  void* out[2] = {d->q_out, d->k_out};
  const void* weight[2] = {d->q_weight, d->k_weight};
  const int32_t heads[2] = {d->heads_q, d->heads_k};
  if (d->M == 0 || heads[0] + heads[1] == 0) return W8A8_OK;
  for (int j = 0; j < 2; ++j) {
    if (heads[j] == 0) continue;
    if (in[j] == nullptr || out[j] == nullptr) return W8A8_ERR_INVALID_ARG;
    const int64_t* in_s = strides + 2 * j;
    const int64_t* out_s = strides + 4 + 2 * j;
    if (!stride_ok(in_s[0]) || !stride_ok(in_s[1]) || !stride_ok(out_s[0]) || !stride_ok(out_s[1])) {
      return W8A8_ERR_INVALID_ARG;
    }
    if (!rows_disjoint(d->M, out_s[0], heads[j], out_s[1], d->head_dim)) return W8A8_ERR_INVALID_ARG;
  }
  for (int j = 0; j < 2; ++j) {
    if (heads[j] == 0) continue;
    if (!aligned16(in[j]) || !aligned16(out[j]) || !aligned16(weight[j])) return W8A8_ERR_ALIGNMENT;
    if ((strides[2 * j] | strides[2 * j + 1] | strides[4 + 2 * j] | strides[5 + 2 * j]) % 8 != 0) {
      return W8A8_ERR_ALIGNMENT;
    }
  }
  if (!aligned16(d->cos) || !aligned16(d->sin) || (reinterpret_cast<uintptr_t>(d->positions) & 3u) != 0) {
    return W8A8_ERR_ALIGNMENT;
  }
  const w8a8_status st = check_current_device();
  if (st != W8A8_OK) return st;

  QkParams p;
  for (int j = 0; j < 2; ++j) {
    p.x[j] = static_cast<const __nv_bfloat16*>(in[j]);
    p.y[j] = static_cast<__nv_bfloat16*>(out[j]);
    p.w[j] = heads[j] ? static_cast<const __nv_bfloat16*>(weight[j]) : nullptr;
    p.ld[j] = strides[2 * j];
    p.hs[j] = strides[2 * j + 1];
    p.ld_y[j] = strides[4 + 2 * j];
    p.hs_y[j] = strides[5 + 2 * j];
    p.heads[j] = heads[j];
  }
  p.cos = d->cos;
  p.sin = d->sin;
  p.positions = d->positions;
  p.M = d->M;
  p.table_rows = d->table_rows;
  p.D = d->head_dim;
  p.R = rotate ? d->rot_dim : 0;
  p.eps = d->eps;
  p.inv_d = 1.0f / static_cast<float>(d->head_dim);
  int lanes = 2;
  while (8 * lanes < d->head_dim) lanes *= 2;
  const int per_unit = kSteps * (32 / lanes);
  p.units = (heads[0] + heads[1] + per_unit - 1) / per_unit;
  const bool pairs = d->layout == W8A8_ROPE_PAIRS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (lanes) {
    case 2: return status_of(launch<2>(p, pairs, s));
    case 4: return status_of(launch<4>(p, pairs, s));
    case 8: return status_of(launch<8>(p, pairs, s));
    case 16: return status_of(launch<16>(p, pairs, s));
    default: return status_of(launch<32>(p, pairs, s));
  }
}
