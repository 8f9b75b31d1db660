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
// token's table row and the weights once for them.  The arithmetic is on
// pairs of binary32: one value at a time, with q and k mixed in a warp, the
// instructions alone took as long as the memory (51 us for 9216 tokens of 48
// heads of 128; now 43.4 us in a graph of calls, 5.3 TB/s, 0.81 of the
// measured copy rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w8a8.h"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace w8a8 {
namespace {

// 32 warps per SM in blocks of 4: 43.9 us for 9216 tokens of 48 heads of 128 (blocks of 8: 45.6, of 16: 48.6; half as
// many steps: 47.4; a quarter: 64).
constexpr int kSteps = 4;
constexpr int kWarps = 4;
constexpr int kBlocksPerSm = 8;

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
  int units, units_q;  // warps per token, and those of q among them
  float eps, inv_d;
};

// Eight bf16 values as four pairs of binary32, and back (one rounding).
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpair(f[i], a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// L: lanes per head (2 .. 32).  PAIRS: the rotation's pairing.
template <int L, bool PAIRS>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm) qk_norm_rope_kernel(const QkParams p) {
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
  const int64_t total = p.M * p.units;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < total;
       unit += static_cast<int64_t>(gridDim.x) * kWarps) {
    // (a 64-bit division only where the number of units needs it)
    const int64_t m = total <= 0x7FFFFFFF ? static_cast<int>(unit) / p.units : unit / p.units;
    int u = static_cast<int>(unit - m * p.units);
    const int j = u >= p.units_q;  // this unit's heads are of q or of k
    if (j) u -= p.units_q;
    const int head0 = u * (kSteps * kPerStep) + grp;
    const int heads = p.heads[j];
    const __nv_bfloat16* x = p.x[j] + m * p.ld[j] + 8 * sub;
    __nv_bfloat16* y = p.y[j] + m * p.ld_y[j] + 8 * sub;

    uint4 v[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = head0 + s * kPerStep;
      v[s] = make_uint4(0, 0, 0, 0);
      if (h < heads && in_head) v[s] = *reinterpret_cast<const uint4*>(x + h * p.hs[j]);
    }

    uint64_t c[kTable / 2], sn[kTable / 2];  // pairs of binary32
    if (p.cos != nullptr) {
      const int64_t row = p.positions != nullptr ? static_cast<int64_t>(__ldg(p.positions + m)) : m;
      // A position outside the table reads nothing and turns by NaN.
      const bool known = row >= 0 && row < p.table_rows;
#pragma unroll
      for (int i = 0; i < kTable / 2; ++i) c[i] = sn[i] = both(__int_as_float(0x7FFFFFFF));
      if (turns && known) {
        const ulonglong2* cr = reinterpret_cast<const ulonglong2*>(p.cos + row * (p.R / 2) + entry);
        const ulonglong2* sr = reinterpret_cast<const ulonglong2*>(p.sin + row * (p.R / 2) + entry);
#pragma unroll
        for (int i = 0; i < kTable / 4; ++i) {
          const ulonglong2 a = __ldg(cr + i), b = __ldg(sr + i);
          c[2 * i] = a.x, c[2 * i + 1] = a.y;
          sn[2 * i] = b.x, sn[2 * i + 1] = b.y;
        }
      }
    }
    uint64_t w[4];
    {
      uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);  // ones
      if (p.w[j] != nullptr && in_head) wv = __ldg(reinterpret_cast<const uint4*>(p.w[j] + 8 * sub));
      unpack8(wv, w);
    }
    if (!PAIRS && p.cos != nullptr && !upper) {
      // y[a] = n[a] cos - n[b] sin in the lower half of the pairs, n[b] cos + n[a] sin in the upper one
#pragma unroll
      for (int i = 0; i < kTable / 2; ++i) sn[i] ^= 0x8000000080000000ull;
    }

#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = head0 + s * kPerStep;
      uint64_t f[4];
      unpack8(v[s], f);
      uint64_t squares = mul2(f[0], f[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) squares = fma2(f[i], f[i], squares);
      float sq, sq1;
      unpair(squares, sq, sq1);
      sq += sq1;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
      const uint64_t r = both(rsqrtf(fmaf(sq, p.inv_d, p.eps)));
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], r), w[i]);
      if (p.cos != nullptr) {
        if constexpr (PAIRS) {
          if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float a, b, c0, c1, s0, s1;
              unpair(f[i], a, b);
              unpair(c[i / 2], c0, c1);
              unpair(sn[i / 2], s0, s1);
              const float ci = i & 1 ? c1 : c0, si = i & 1 ? s1 : s0;
              f[i] = pair(a * ci - b * si, b * ci + a * si);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;
            unpair(f[i], a, b);
            const uint64_t other = pair(__shfl_sync(0xFFFFFFFFu, a, mate), __shfl_sync(0xFFFFFFFFu, b, mate));
            if (turns) f[i] = fma2(other, sn[i], mul2(f[i], c[i]));
          }
        }
      }
      if (h < heads && in_head) *reinterpret_cast<uint4*>(y + h * p.hs_y[j]) = pack8(f);
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

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

}  // namespace

bool rows_disjoint(int64_t rows, int64_t ld, int64_t heads, int64_t hs, int64_t dim) {
  if (heads > 1 && rows > 1) {
    return (hs >= dim && ld >= (heads - 1) * hs + dim) || (ld >= dim && hs >= (rows - 1) * ld + dim);
  }
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
  p.units_q = (heads[0] + per_unit - 1) / per_unit;
  p.units = p.units_q + (heads[1] + per_unit - 1) / per_unit;
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
