// attention_sm100.cu -- attention for many queries, on the 5th-generation
// tensor cores.
//
// A CTA takes 256 queries of one document and head, as two sub-tiles of 128
// (the rows of a tcgen05.mma), and walks the keys 128 at a time:
//   S = Q K^T       Q and K from shared memory, S in tensor memory
//   P = 2^(S c - m) rounded to bf16, written over S in tensor memory
//   O += P V        P from tensor memory, V from shared memory
// with the running maximum m and sum of a softmax per query.  O stays in
// tensor memory: it is rescaled only when a row's maximum has grown by more
// than 2^8 since m was last set (P then reaches 2^8 at most, and the sum is
// binary32), so in most tiles no thread touches it.
//
//   warps 0-7, 8-15 softmax of sub-tile 0 / 1: a query's 128 scores of a
//                   tile belong to two threads, 64 each, which exchange
//                   their maximum through shared memory
//   warp 16         loads Q, then K and V tiles through a ring (TMA)
//   warp 17         issues the MMAs: while one sub-tile's softmax runs, the
//                   tensor cores work for the other
//   warp 18         zeroes the rows of the last V tile that lie behind the
//                   document's end (a weight of 0 times whatever is there
//                   must be 0)
//
// The tensor cores execute MMAs in the order they are issued, so S of tile
// j + 1 may overwrite P of tile j right behind O += P V, and "S full" also
// says that O holds every tile before.
//
// What bounds it: a 128 x 128 tile costs 4 D * 128 * 128 operations of the
// tensor cores (1024 cycles at D = 128, 512 at D = 64) and 128 * 128
// exponentials of the special-function units (1024 cycles).
#include <cuda.h>

#include <cstring>

#include "attention.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace w8a8 {
namespace {

constexpr int kSub = 128;             // queries of a sub-tile
constexpr int kTileQ = 2 * kSub;      // queries of a CTA
constexpr int kTileK = 128;           // keys of a tile
constexpr int kSoftmaxWarps = 16;
constexpr int kThreads = 32 * kSoftmaxWarps + 128;
constexpr int kRegsSoftmax = 104;     // 512 * 104 + 128 * 64 = 640 * 96, the registers the CTA starts with
constexpr int kRegsOther = 64;
constexpr int kBlockBytes = 128 * 128;  // 128 rows x 64 values
// A float per query and half of the keys (the softmax threads' exchange) and the barriers, in front of Q and the ring,
// which are aligned to 1024 bytes: at D = 128 all of the 227 KB.
constexpr int kExchange = 2 * 2 * kSub;
constexpr int kHeadBytes = 3 * 1024;
constexpr int kFma = 4;               // pairs of 16 whose exponentials run on the FMA units
constexpr float kGrowth = 8.0f;       // log2 of the growth of a row's maximum that rescales O

__host__ __device__ constexpr int tile_bytes(int D) { return D / 64 * kBlockBytes; }
__host__ __device__ constexpr int ring_stages(int D) { return D == 128 ? 5 : 8; }
__host__ __device__ constexpr int smem_bytes(int D) {
  return kHeadBytes + (2 + ring_stages(D)) * tile_bytes(D);
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float a) { return pair(a, a); }

// tanh(y) = y * sum_n kTanh[n] y^2n on [-1, 1]: least squares on Chebyshev nodes, relative error 7e-7 in binary32.
__device__ constexpr float kTanh[6] = {9.9999936384e-1f, -3.3328806676e-1f, 1.3279611505e-1f,
                                       -5.1555843877e-2f, 1.6687155235e-2f, -3.0449762314e-3f};

// Maximum of three; NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^x of a pair on the FMA and integer units, for x in [-126, 127] (below:
// 2^-126): x = n + f with n the nearest integer (read from the low bits of x +
// 1.5 * 2^23) and |f| <= 1/2, 2^f by a polynomial of degree 5 (the minimax fit
// of its relative error: 7.7e-8, 2.1e-7 as evaluated in binary32), and n added
// to the exponent.
__device__ __forceinline__ void ex2_pair_fma(uint64_t x, float& e0, float& e1) {
  float x0, x1;
  unpair(x, x0, x1);
  x = pair(fmaxf(x0, -126.0f), fmaxf(x1, -126.0f));
  const uint64_t shifted = add2(x, both(12582912.0f));
  const uint64_t f = fma2(add2(shifted, both(-12582912.0f)), both(-1.0f), x);
  uint64_t y = fma2(f, both(1.3277938903e-3f), both(9.6757576406e-3f));
  y = fma2(y, f, both(5.5507095981e-2f));
  y = fma2(y, f, both(2.4022114338e-1f));
  y = fma2(y, f, both(6.9314696823e-1f));
  y = fma2(y, f, both(1.0000000733f));
  float n0, n1, y0, y1;
  unpair(shifted, n0, n1);
  unpair(y, y0, y1);
  e0 = __uint_as_float(__float_as_uint(y0) + (__float_as_uint(n0) << 23));
  e1 = __uint_as_float(__float_as_uint(y1) + (__float_as_uint(n1) << 23));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const AttnParams p, const int slots, int* err) {
  constexpr int kStages = ring_stages(D);
  constexpr int kTile = tile_bytes(D);
  constexpr int kBlocks = D / 64;
  constexpr uint32_t kIdescS = make_idesc_bf16(kSub, kTileK, false);
  constexpr uint32_t kIdescO = make_idesc_bf16(kSub, D, true);
  constexpr uint32_t kTmemCols = 512;  // S0, S1 (128 columns each), O0, O1 (D each)

  extern __shared__ __align__(1024) uint8_t smem[];
  float* exchange = reinterpret_cast<float*>(smem);  // [half][sub-tile][query]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kExchange * sizeof(float));
  uint8_t* sQ = smem + kHeadBytes;
  uint8_t* ring = sQ + 2 * kTile;
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;   // [2]
  uint64_t* s_full = q_full + 2;        // [2]
  uint64_t* p_full = s_full + 2;        // [2]
  uint64_t* o_full = p_full + 2;        // [2]
  uint64_t* tail_full = o_full + 2;
  uint64_t* drain = tail_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);  // (known to be uniform)
  const int lane = threadIdx.x & 31;

  // Causal documents: the slots with the most keys first, so that the last CTAs to start are short ones.
  // Otherwise a head's slots side by side, which share its keys and values.
  const int block = static_cast<int>(blockIdx.x);
  const int head = p.causal ? block % p.heads_q : block / slots;
  const int slot = p.causal ? slots - 1 - block / p.heads_q : block % slots;
  const int d = slot_doc(p, slot, 1, kTileQ);
  const Doc doc = load_doc(p, d);
  const int row0 = (slot - slot_begin(p, d, 1, kTileQ)) * kTileQ;
  const int rows = min(kTileQ, doc.lq - row0);
  if (rows <= 0 || row0 < 0) return;  // an unused slot
  const int kv_head = head / p.group;
  // Key tiles of each sub-tile (limits grow with the query).
  auto key_tiles = [&](int s) {
    const int n = min(kSub, rows - s * kSub);
    return n <= 0 ? 0 : (max(0, key_limit(p, doc, row0 + s * kSub + n - 1)) + kTileK - 1) / kTileK;
  };
  const int n0 = key_tiles(0), n1 = key_tiles(1);
  const int tiles = max(n0, n1);
  const int tail_rows = doc.lk - (tiles - 1) * kTileK;  // rows of the last V tile that are the document's
  const bool tail = tiles > 0 && tail_rows < kTileK;

  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need it; a kernel without static shared memory has it
    if (threadIdx.x == 0) record_timeout(err, kSiteAttnLoad);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kSoftmaxWarps / 2);
      mbar_init(&o_full[s], 1);
    }
    mbar_init(tail_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16 && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 17) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kSoftmaxWarps) {
    reg_lower<kRegsOther>();
    // One thread each: a warp that votes, elects and converges around every wait spends most of a tile's time on
    // that (measured: 4 300 cycles a tile of 256 x 128 x 128, of which the issuing warp was idle in none).
    const auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
      return mbar_wait_bounded(bar, parity, abort_flag, p.timeout_ns, err, site);
    };
    if (warp == 16 && elect_one()) {
      // ------------------------------------------------------------ loader
      const uint64_t keep = l2_policy_evict_last();
      const uint64_t once = l2_policy_evict_first();
      int fills = 0;
      const auto load_q = [&](int s) {
        mbar_arrive_expect_tx(&q_full[s], kTile);
        for (int b = 0; b < kBlocks; ++b) {
          tma_load_3d_hint(sQ + s * kTile + b * kBlockBytes, &tm_q, &q_full[s], 64 * b, doc.q0 + row0 + s * kSub, head,
                           once);
        }
      };
      if (n0 > 0) load_q(0);
      if (n1 > 0) load_q(1);
      int stage = 0;
      uint32_t phase = 1;
      for (int f = 0; f < 2 * tiles; ++f) {
        if (!wait(&empty[stage], phase, kSiteAttnLoad)) break;
        // (a last V tile that ends inside goes to warp 18 first, which fills the slot)
        uint64_t* landed = tail && f == 2 * tiles - 1 ? tail_full : &full[stage];
        mbar_arrive_expect_tx(landed, kTile);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          tma_load_3d_hint(ring + stage * kTile + b * kBlockBytes, (f & 1) ? &tm_v : &tm_k, landed, 64 * b,
                           doc.k0 + (f >> 1) * kTileK, kv_head, keep);
        }
        ++fills;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // Every load must have landed before the CTA ends (on the normal path they have).
      for (int f = max(0, fills - kStages); f < fills; ++f) {
        if (tail && f == 2 * tiles - 1) {
          mbar_wait_drain(tail_full, 0, p.timeout_ns, err);
          continue;
        }
        mbar_wait_drain(&full[f % kStages], static_cast<uint32_t>((f / kStages) & 1), p.timeout_ns, err);
      }
      if (n0 > 0) mbar_wait_drain(&q_full[0], 0, p.timeout_ns, err);
      if (n1 > 0) mbar_wait_drain(&q_full[1], 0, p.timeout_ns, err);
    } else if (warp == 17 && elect_one()) {
      // -------------------------------------------------------- MMA issuer
      bool ok = true;
      // Matrix descriptors: the high words are constant, the low ones hold the address (in units of 16 bytes).
      const uint64_t desc_k = make_smem_desc_k_sw128(0), desc_v = make_smem_desc_n_sw128(0, kBlockBytes);
      const uint32_t q_addr = smem_u32(sQ) >> 4, ring_addr = smem_u32(ring) >> 4;
      constexpr uint32_t kTile16 = kTile / 16, kBlock16 = kBlockBytes / 16;
      // S_s = Q_s K^T with K in ring slot `stage`
      const auto scores = [&](int s, int stage) {
        const uint64_t qd = desc_k + (q_addr + s * kTile16), kd = desc_k + (ring_addr + stage * kTile16);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t off = (x / 4) * kBlock16 + 2 * (x % 4);
          mma_bf16_ss(tmem + s * kTileK, qd + off, kd + off, kIdescS, x > 0);
        }
        mma_commit(&s_full[s]);
      };
      if (tiles > 0) ok = wait(&full[0], 0, kSiteAttnOperand);
#pragma unroll 1
      for (int s = 0; ok && s < 2; ++s) {
        if ((s == 0 ? n0 : n1) == 0) continue;
        ok = wait(&q_full[s], 0, kSiteAttnOperand);
        if (ok) scores(s, 0);
      }
      if (ok && tiles > 0) mma_commit(&empty[0]);
      int v_stage = 1;
      uint32_t v_phase = 0;
      for (int j = 0; ok && j < tiles; ++j) {
        int k_stage = v_stage + 1;  // of tile j + 1
        uint32_t k_phase = v_phase;
        if (k_stage == kStages) {
          k_stage = 0;
          k_phase ^= 1u;
        }
        ok = wait(&full[v_stage], v_phase, kSiteAttnOperand) &&
             (j + 1 == tiles || wait(&full[k_stage], k_phase, kSiteAttnOperand));
        if (!ok) break;
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          const int n = s == 0 ? n0 : n1;
          if (j >= n) continue;
          ok = wait(&p_full[s], static_cast<uint32_t>(j & 1), kSiteAttnWeights);
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t vd = desc_v + (ring_addr + v_stage * kTile16);
#pragma unroll
          for (int x = 0; x < kTileK / 16; ++x) {
            mma_bf16_ts(tmem + 2 * kTileK + s * D, tmem + s * kTileK + 8 * x, vd + 128 * x, kIdescO,
                        (x > 0 || j > 0) ? 1u : 0u);
          }
          if (j + 1 < n) {
            scores(s, k_stage);
          } else {
            mma_commit(&o_full[s]);
          }
        }
        if (!ok) break;
        mma_commit(&empty[v_stage]);
        if (j + 1 < tiles) mma_commit(&empty[k_stage]);
        v_stage = k_stage + 1;
        v_phase = k_phase;
        if (v_stage == kStages) {
          v_stage = 0;
          v_phase ^= 1u;
        }
      }
      // No MMA may still run when tensor memory is freed.
      mma_commit(drain);
      mbar_wait_drain(drain, 0, p.timeout_ns, err);
    } else if (warp == 18 && tail) {
      // ------------------------------------------------ end of the document
      const int stage = (2 * tiles - 1) % kStages;
      if (warp_wait(tail_full, 0, abort_flag, p.timeout_ns, err, kSiteAttnOperand)) {
        uint8_t* v = ring + stage * kTile;
        for (int x = tail_rows * 8 + lane; x < kTileK * 8; x += 32) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) *reinterpret_cast<uint4*>(v + b * kBlockBytes + x * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    reg_raise<kRegsSoftmax>();
    const int s = warp >> 3;
    const int part = (warp >> 2) & 1;  // keys 64 part .. 64 part + 63 of every tile
    const int quarter = warp & 3;
    const uint32_t partners = 1 + (warp >> 3) * 4 + quarter;  // named barrier of the two warps of 32 queries
    const int my_rows = min(kSub, rows - s * kSub);  // <= 0: nothing in this sub-tile
    const int n = s == 0 ? n0 : n1;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + s * kTileK;
    const uint32_t t_o = tmem + lanes + 2 * kTileK + s * D;
    const int in_sub = quarter * 32 + lane;
    const int i = row0 + s * kSub + in_sub;  // the thread's query
    const int limit = in_sub < my_rows ? max(0, key_limit(p, doc, i)) : 0;
    const int least = my_rows > 0 ? key_limit(p, doc, row0 + s * kSub) : 0;  // the sub-tile's smallest limit
    constexpr bool kChange = CAP || BIAS;  // scores need more than the factor c
    const float c = p.scale * kLog2e;
    const float inv_cap = CAP ? p.scale / p.cap : 0.0f;
    const float c_tanh = 2.0f * kLog2e * inv_cap;
    const float c_cap = CAP ? p.cap * kLog2e : 0.0f;
    const float slope = BIAS ? __ldg(p.slopes + head) * kLog2e : 0.0f;
    const int place = i + doc.shift;
    const int first_place = row0 + s * kSub + doc.shift;  // of the sub-tile's queries

    // 32 scores of a tile, from key key0 of the document on: cap, bias and mask; their maximum.
    auto first_pass = [&](uint32_t (&v)[32], int key0, bool masked) {
      if constexpr (CAP) {
        // Scores within the cap on either side (all of them, unless the scores are far beyond it) take the
        // polynomial for tanh; others two special functions each.
        float far = 0.0f;
#pragma unroll
        for (int x = 0; x < 32; x += 2) far = max3(far, fabsf(__uint_as_float(v[x])), fabsf(__uint_as_float(v[x + 1])));
        if (__all_sync(0xFFFFFFFFu, far * inv_cap <= 1.0f)) {
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const uint64_t y = mul2(pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), both(inv_cap));
            const uint64_t u = mul2(y, y);
            uint64_t t = fma2(u, both(kTanh[5]), both(kTanh[4]));
            t = fma2(t, u, both(kTanh[3]));
            t = fma2(t, u, both(kTanh[2]));
            t = fma2(t, u, both(kTanh[1]));
            t = fma2(t, u, both(kTanh[0]));
            float a0, a1;
            unpair(mul2(t, mul2(y, both(c_cap))), a0, a1);
            v[x] = __float_as_uint(a0);
            v[x + 1] = __float_as_uint(a1);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(capped(__uint_as_float(v[x]), c_tanh, c_cap));
        }
      }
      if constexpr (BIAS) {
        const float f = CAP ? 1.0f : c;
        const float first = static_cast<float>(key0 - place);  // distance of the first key, signed
        if (key0 + 31 <= first_place) {
          // No key lies ahead of any query of the sub-tile: the bias is linear in the key.
          const float at0 = slope * first;
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            v[x] = __float_as_uint(fmaf(__uint_as_float(v[x]), f, fmaf(slope, static_cast<float>(x), at0)));
          }
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            v[x] = __float_as_uint(fmaf(__uint_as_float(v[x]), f, -slope * fabsf(first + static_cast<float>(x))));
          }
        }
      }
      if (masked) {
        const int left = limit - key0;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if (x >= left) v[x] = 0xFF800000u;  // -inf
        }
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 32; x += 4) {
        top[0] = max3(top[0], __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
        top[1] = max3(top[1], __uint_as_float(v[x + 2]), __uint_as_float(v[x + 3]));
      }
      return fmax_nan(top[0], top[1]);
    };

    // The value of the thread with the other 64 keys of this query.  One barrier is enough: a thread writes its
    // next value when the MMAs that wait for its partner's weights are done, so after the partner read this one.
    float* const mine = exchange + (part * 2 + s) * kSub + in_sub;
    const float* const other = exchange + ((part ^ 1) * 2 + s) * kSub + in_sub;
    const auto partner = [&](float x) {
      *mine = x;
      named_barrier_sync(partners, 64);
      return *other;
    };

    float m = -INFINITY;  // in units of log2
    float l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = warp_wait(&s_full[s], static_cast<uint32_t>(j & 1), abort_flag, p.timeout_ns, err, kSiteAttnScores);
      if (!ok) break;
      tc_fence_after_sync();
      const bool masked = (j + 1) * kTileK > least;
      const int key0 = j * kTileK + 64 * part;
      uint32_t va[32], vb[32];
      tmem_load_32cols_async(t_s + 64 * part, va);
      tmem_load_32cols_async(t_s + 64 * part + 32, vb);
      tmem_wait_load(va);
      tmem_wait_load(vb);
      float top = fmax_nan(first_pass(va, key0, masked), first_pass(vb, key0 + 32, masked));
      // The partner's maximum.  (Behind the barrier both have read their scores, and P may be written over them.)
      tc_fence_before_sync();
      top = fmax_nan(top, partner(top));
      tc_fence_after_sync();
      if (!kChange) top *= c;  // c > 0
      if (j == 0) {
        m = top;
      } else {
        const bool grow = !(top <= m + kGrowth);  // (a NaN reaches O and l, and stays there)
        if (__any_sync(0xFFFFFFFFu, grow)) {      // (the same in both warps)
          const float f = grow ? ex2(m - top) : 1.0f;
          if (grow) m = top;
          l *= f;
#pragma unroll 1
          for (int b = 0; b < D / 32; ++b) {
            uint32_t o[16];
            tmem_load_16cols(t_o + D / 2 * part + 16 * b, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_store_16cols(t_o + D / 2 * part + 16 * b, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.0f : m;
      const uint64_t c2 = both(kChange ? 1.0f : c), minus = both(-base);
      uint64_t sums[2] = {both(0.0f), both(0.0f)};
      // Weights of 32 keys.  In whole tiles kFma of every 16 pairs take their exponentials on the FMA units; masked
      // tiles need 2^-inf = 0.
      auto weights = [&](const uint32_t (&v)[32], int b, bool mixed) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const uint64_t y = pair(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
          const uint64_t e = kChange ? add2(y, minus) : fma2(y, c2, minus);
          float a0, a1;
          if (mixed && x * kFma / 16 != (x + 1) * kFma / 16) {
            ex2_pair_fma(e, a0, a1);
          } else {
            unpair(e, a0, a1);
            a0 = ex2(a0);
            a1 = ex2(a1);
          }
          sums[x & 1] = add2(sums[x & 1], pair(a0, a1));
          w[x] = pack_bf16(a0, a1);  // the weights' one rounding; their sum is that of the unrounded ones
        }
        tmem_store_16cols(t_s + 32 * part + 16 * b, w);
      };
      if (kFma == 0 || masked) {
        weights(va, 0, false);
        weights(vb, 1, false);
      } else {
        weights(va, 0, true);
        weights(vb, 1, true);
      }
      tmem_wait_store();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s]);
      float s0, s1;
      unpair(add2(sums[0], sums[1]), s0, s1);
      l += s0 + s1;
    }

    // ------------------------------------------------------------- epilogue
    if (ok && n > 0) ok = warp_wait(&o_full[s], 0, abort_flag, p.timeout_ns, err, kSiteAttnOut);
    if (!ok) named_barrier_arrive(partners, 64);  // the partner may stand at its barrier: it will see the abort next
    if (ok && my_rows > 0) {
      tc_fence_after_sync();
      l += partner(l);
      const bool any = limit > 0;
      const float inv = any ? 1.0f / l : 0.0f;
      // The warp's 32 rows x D/2 values through shared memory (its part of the sub-tile's Q, which no MMA reads any
      // more), so that they leave in whole segments of D bytes.
      constexpr int kVec = D / 16;  // 16-byte vectors of a row
      uint8_t* stage = sQ + s * kTile + (part * 4 + quarter) * 32 * D;
#pragma unroll 1
      for (int b = 0; b < D / 32; ++b) {
        uint32_t o[16];
        if (n > 0) {
          tmem_load_16cols(t_o + D / 2 * part + 16 * b, o);
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float a0 = __uint_as_float(o[8 * x + 2 * y]) * inv, a1 = __uint_as_float(o[8 * x + 2 * y + 1]) * inv;
            w[y] = any ? pack_bf16(a0, a1) : 0u;
          }
          *reinterpret_cast<uint4*>(stage + lane * D + (((2 * b + x) ^ (lane & (kVec - 1))) * 16)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      const int64_t token0 = doc.q0 + row0 + s * kSub + quarter * 32;
      const int valid = min(32, my_rows - quarter * 32);
#pragma unroll 4
      for (int e = lane; e < 32 * kVec; e += 32) {
        const int r = e / kVec, x = e % kVec;
        if (r < valid) {
          const uint4 w = *reinterpret_cast<const uint4*>(stage + r * D + ((x ^ (r & (kVec - 1))) * 16));
          *reinterpret_cast<uint4*>(p.out + (token0 + r) * p.ldo + head * p.hso + D / 2 * part + x * 8) = w;
        }
      }
      if (p.lse != nullptr && part == 0 && in_sub < my_rows) {
        p.lse[(token0 + lane) * p.heads_q + head] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (*abort_flag) {
    // A wait ran out: give copies already issued time to land before the shared memory they target is released.
    if (threadIdx.x == 0) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
    __syncthreads();
  }
  if (warp == 17) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// {64 values, tokens, heads} boxes of 64 x 128 x 1 of a bf16 [tokens, heads, D] tensor, 128-byte swizzle.
bool encode_heads(CUtensorMap* map, const void* base, int D, int64_t tokens, int64_t heads, int64_t ld, int64_t hs) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(tokens),
                              static_cast<cuuint64_t>(heads)};
  // (the stride of a dimension of one is free)
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * (tokens > 1 ? ld : D)),
                                 static_cast<cuuint64_t>(2 * (heads > 1 ? hs : D))};
  const cuuint32_t box[3] = {64, 128, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap tm_q, tm_k, tm_v;
  std::memset(&tm_q, 0, sizeof tm_q);
  // No keys: no tile of them is ever loaded, and the maps describe q.
  const bool none = p.tokens_k == 0;
  bool ok = encode_heads(&tm_q, p.q, D, p.tokens_q, p.heads_q, p.ldq, p.hsq);
  tm_k = tm_v = tm_q;
  if (!none) {
    ok = ok && encode_heads(&tm_k, p.k, D, p.tokens_k, p.heads_k, p.ldk, p.hsk) &&
         encode_heads(&tm_v, p.v, D, p.tokens_k, p.heads_k, p.ldv, p.hsv);
  }
  if (!ok) return cudaErrorInvalidValue;
  int* err = nullptr;
  cudaError_t e = error_word_address(&err);
  if (e != cudaSuccess) return e;
  auto kernel = attention_tiles_kernel<D, CAP, BIAS>;
  constexpr int smem = smem_bytes(D);
  static_assert(smem <= 232448 && kExchange * 4 + (2 * ring_stages(D) + 10) * 8 + 8 <= kHeadBytes, "shared memory");
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t slots = p.tokens_q / kTileQ + p.docs;
  if (slots * p.heads_q > 2147483647) return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(slots * p.heads_q), kThreads, smem, stream>>>(tm_q, tm_k, tm_v, p,
                                                                              static_cast<int>(slots), err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_tiles(const AttnParams& p, int head_dim, cudaStream_t stream) {
  const bool cap = p.cap > 0.0f, bias = p.slopes != nullptr;
  if (head_dim == 64) {
    if (cap) return bias ? launch<64, true, true>(p, stream) : launch<64, true, false>(p, stream);
    return bias ? launch<64, false, true>(p, stream) : launch<64, false, false>(p, stream);
  }
  if (cap) return bias ? launch<128, true, true>(p, stream) : launch<128, true, false>(p, stream);
  return bias ? launch<128, false, true>(p, stream) : launch<128, false, false>(p, stream);
}

}  // namespace w8a8
