// attention_sm100.cu -- attention for many queries, on the 5th-generation
// tensor cores.
//
// A work item is 256 queries of one document and head, as two sub-tiles of
// 128 (the rows of a tcgen05.mma); its keys are walked a tile at a time:
//   S = Q K^T       Q and K from shared memory, S in tensor memory
//   P = 2^(S c - m) rounded to bf16, in tensor memory
//   O += P V        P from tensor memory, V from shared memory
// with the running maximum m and sum of a softmax per query.  O stays in
// tensor memory: it is rescaled only when a row's maximum has grown by more
// than 2^8 since m was last set (P then reaches 2^8 at most, and the sum is
// binary32), so in most tiles no thread touches it.
//
//   warps 0-7, 8-15 softmax of sub-tile 0 / 1: a query's scores of a tile
//                   belong to two threads, half of the keys each, which
//                   exchange their maxima through shared memory
//   warp 16         loads Q, then K and V tiles through a ring (TMA)
//   warps 17, 18    one thread each issues the MMAs of sub-tile 0 / 1.  (Two,
//                   because it takes a lone thread about 7 cycles per
//                   instruction beside the softmax warps: one thread for
//                   both sub-tiles needed 2 360 cycles a tile of 80 keys.)
//   warp 19         zeroes the rows of the last V tile that lie behind the
//                   document's end (a weight of 0 times whatever is there
//                   must be 0)
//
// The grid has a CTA per item.  A CTA that runs takes over ones that have not
// started (cluster launch control), so that an item's first loads and scores
// run beside the epilogue of the one before, and the hardware's dynamic order
// stays: items dealt out in a fixed way left some SMs an item more than
// others (487 us against 422 at 2 x 4608 tokens, 24 heads of 128).
//
// S and P have columns of their own, so that S of the next tile is computed
// while the softmax of this one runs, and the softmax warps never wait for a
// product that waits for them.  With the O's of two sub-tiles in the 512
// columns of tensor memory that leaves tiles of 128 keys at D = 64 and of 80
// at D = 128.  (Tiles of 128 keys with P written over S, as D = 128 would
// allow, took 3 250 cycles per 256 x 128 scores: the softmax of a sub-tile,
// 1 950 cycles, and its two products, 1 250, one after the other.)
//
// What bounds it, per 256 queries x 128 keys: the tensor cores, 4 D * 256 *
// 128 operations (2048 cycles at D = 128; Q K^T reads its operands at the
// limit of shared memory and takes 1.2 times its share), and the softmax:
// 2048 cycles of the special-function units for the exponentials alone.
// Measured, in graphs of calls: 2 x 4608 tokens, 24 heads of 128: 412 us, 1.27
// PFLOP/s, 0.76 of the measured bf16 rate (484 us in a loop of seconds, where
// the board's power cap sets the clock); 2 x 4095 tokens, 16 heads of 128,
// causal, with slopes: 162 us; 9 ragged prompts of 911 tokens on average, cap
// and prefix, 16 heads of 64 over 4: 68 us.
#include <cuda.h>

#include <cstring>

#include "attention.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace w8a8 {
namespace {

constexpr int kSub = 128;             // queries of a sub-tile
constexpr int kTileQ = 2 * kSub;      // queries of a CTA
__host__ __device__ constexpr int tile_keys(int D) { return D == 128 ? 80 : 128; }
constexpr int kSoftmaxWarps = 16;
constexpr int kThreads = 32 * kSoftmaxWarps + 128;
constexpr int kRegsSoftmax = 104;     // 512 * 104 + 128 * 64 = 640 * 96, the registers the CTA starts with
constexpr int kRegsOther = 64;
constexpr float kGrowth = 8.0f;       // log2 of the growth of a row's maximum that rescales O

// Blocks of 64 values (128 bytes) x rows: Q in sub-tiles of 128 rows, K and V in tiles of tile_keys rows.
__host__ __device__ constexpr int q_bytes(int D) { return D / 64 * kSub * 128; }
__host__ __device__ constexpr int tile_bytes(int D) { return D / 64 * tile_keys(D) * 128; }
__host__ __device__ constexpr int ring_stages(int D) { return D == 128 ? 6 : 8; }
// The softmax threads' exchange (two tiles' buffers of a float per half of the keys, sub-tile and query) and the
// barriers, in front of Q and the ring, which are aligned to 1024 bytes.
constexpr int kExchange = 2 * 2 * 2 * kSub;
constexpr int kHeadBytes = 5 * 1024;
constexpr int kStagingBytes = 2048;  // of a softmax warp's output
__host__ __device__ constexpr int smem_bytes(int D) {
  return kHeadBytes + 2 * q_bytes(D) + ring_stages(D) * tile_bytes(D) + kSoftmaxWarps * kStagingBytes;
}

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

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const AttnParams p, const int slots, int* err) {
  constexpr int kTileK = tile_keys(D);
  constexpr int kHalf = kTileK / 2;  // keys of a softmax thread
  constexpr int kStages = ring_stages(D);
  constexpr int kQ = q_bytes(D);
  constexpr int kTile = tile_bytes(D);
  constexpr int kBlocks = D / 64;
  constexpr int kQBlock = kSub * 128, kBlock = kTileK * 128;
  constexpr uint32_t kIdescS = make_idesc_bf16(kSub, kTileK, false);
  constexpr uint32_t kIdescO = make_idesc_bf16(kSub, D, true);
  // Columns of tensor memory: S and P of sub-tile s at s * kSpan, O behind them.
  constexpr uint32_t kTmemCols = 512;
  constexpr uint32_t kSpan = D == 128 ? 128 : 192;
  constexpr uint32_t kColO = 2 * kSpan;
  static_assert(kTileK + kTileK / 2 <= kSpan && kColO + 2 * D <= kTmemCols, "tensor memory");

  extern __shared__ __align__(1024) uint8_t smem[];
  float* exchange = reinterpret_cast<float*>(smem);  // [tile parity][half of the keys][sub-tile][query]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kExchange * sizeof(float));
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;   // [2]
  uint64_t* q_free = q_full + 2;        // [2] the item's last scores done
  uint64_t* s_full = q_free + 2;        // [2] scores ready
  uint64_t* s_free = s_full + 2;        // [2] scores read
  uint64_t* p_full = s_free + 2;        // [2] weights ready
  uint64_t* o_full = p_full + 2;        // [2] product with V done: O complete so far, P free
  // [2] a last V tile that ends inside has landed, and warp 19 has filled it: two in turn, so that the loader may be an
  // item ahead of warp 19.  (Without the second wait it could be two ahead, and complete a phase that warp 19 has not
  // seen: an item's Q waits for the last scores of its own sub-tile alone, and items without sub-tile 0, whose first
  // queries see no key, do not wait for those without sub-tile 1.)
  uint64_t* tail_full = o_full + 2;
  uint64_t* tail_free = tail_full + 2;
  uint64_t* drain = tail_free + 2;      // [2]
  uint64_t* item_full = drain + 2;      // [2] the next item is known
  uint64_t* item_free = item_full + 2;  // [2] ... and read by every warp
  uint8_t* answer = smem + kHeadBytes - 32;  // [2][16]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_free + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* sQ = smem + kHeadBytes;
  uint8_t* ring = sQ + 2 * kQ;
  uint8_t* staging = ring + kStages * kTile;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);  // (known to be uniform)
  const int lane = threadIdx.x & 31;

  // A work item, the same for every warp (all lanes call it).  Causal documents: the slots with the most keys first, so
  // that the last items are short ones.  Otherwise a head's slots side by side, which share its keys and values.
  struct Item {
    Doc doc;
    int head, row0, rows;  // rows <= 0: an unused slot
    int n0, n1, tiles;     // key tiles of each sub-tile (limits grow with the query) and of the item
    int tail_rows;         // rows of the last V tile that are the document's
    bool tail;             // ... and not all of them
  };
  // A warp that has nothing to do in an item, or waits for its end, waits as long as the item takes, some 1 us a tile:
  // its limit grows with the tiles.  (If the others stop, they find out within their own limits and raise the flag.)
  int item_tiles = 0;
  const auto item_limit = [&] { return p.timeout_ns + 100000ull * static_cast<uint64_t>(item_tiles); };
  const auto item_of = [&](int x) {
    Item it;
    it.head = p.causal ? x % p.heads_q : x / slots;
    const int slot = p.causal ? slots - 1 - x / p.heads_q : x % slots;
    it.doc = slot_doc(p, slot, 1, kTileQ, it.row0);
    it.rows = it.row0 < 0 ? 0 : min(kTileQ, it.doc.lq - it.row0);
    const auto key_tiles = [&](int s) {
      const int n = min(kSub, it.rows - s * kSub);
      return n <= 0 ? 0 : (max(0, key_limit(p, it.doc, it.row0 + s * kSub + n - 1)) + kTileK - 1) / kTileK;
    };
    it.n0 = key_tiles(0);
    it.n1 = key_tiles(1);
    it.tiles = item_tiles = max(it.n0, it.n1);
    it.tail_rows = it.doc.lk - (it.tiles - 1) * kTileK;
    it.tail = it.tiles > 0 && it.tail_rows < kTileK;
    return it;
  };
  // The items of this CTA, one after the other, in every warp: the first is the CTA's own, the next ones come into two
  // buffers in turn.
  int item = static_cast<int>(blockIdx.x), taken = 0;
  const auto next_item = [&](bool ok) {  // all lanes; -1 behind the last one, or if !ok
    if (!ok) return -1;
    ++taken;
    const int b = taken & 1;
    const bool got = mbar_wait_bounded(&item_full[b], static_cast<uint32_t>((taken - 1) >> 1) & 1u, abort_flag,
                                       item_limit(), err, kSiteAttnItem);
    if (!__all_sync(0xFFFFFFFFu, got)) return -1;
    const int x = launch_cancelled(answer + 16 * b);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[b]);
    return x;
  };

  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need it; a kernel without static shared memory has it
    if (threadIdx.x == 0) record_timeout(err, kSiteAttnLoad);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // both issuers
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tail_full[s], 1);
      mbar_init(&tail_free[s], 1);
      mbar_init(&drain[s], 1);
      mbar_init(&item_full[s], 1);
      mbar_init(&item_free[s], kThreads / 32);
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], kSoftmaxWarps / 2);
      mbar_init(&p_full[s], kSoftmaxWarps / 2);
      mbar_init(&o_full[s], 1);
    }
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
    // One thread each loads and issues: a warp that votes, elects and converges around every wait spends most of a
    // tile's time on that.
    const auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
      return mbar_wait_bounded(bar, parity, abort_flag, p.timeout_ns, err, site);
    };
    bool ok = true;
    if (warp == 16) {
      // ------------------------------------------------------------ loader
      const uint64_t keep = l2_policy_evict_last();
      const uint64_t once = l2_policy_evict_first();
      int stage = 0;
      uint32_t phase = 1, q_phase[2] = {1, 1};
      int tails = 0;
      for (; item >= 0; item = next_item(ok)) {
        const Item it = item_of(item);
        if (elect_one()) {
          const int kv_head = it.head / p.group;
          const auto load_q = [&](int s) {
            ok = ok && wait(&q_free[s], q_phase[s], kSiteAttnLoad);
            if (!ok) return;
            q_phase[s] ^= 1u;
            mbar_arrive_expect_tx(&q_full[s], kQ);
            for (int b = 0; b < kBlocks; ++b) {
              tma_load_3d_hint(sQ + s * kQ + b * kQBlock, &tm_q, &q_full[s], 64 * b, it.doc.q0 + it.row0 + s * kSub,
                               it.head, once);
            }
          };
          const auto load = [&](const CUtensorMap* map, int tile, uint64_t* landed) {
            ok = ok && wait(&empty[stage], phase, kSiteAttnLoad);
            if (!ok) return;
            if (landed == nullptr) landed = &full[stage];
            mbar_arrive_expect_tx(landed, kTile);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
              tma_load_3d_hint(ring + stage * kTile + b * kBlock, map, landed, 64 * b, it.doc.k0 + tile * kTileK,
                               kv_head, keep);
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          };
          // Fills in the order of their use: K of tile 0, then K of tile j + 1 and V of tile j.
          if (it.tiles > 0) load(&tm_k, 0, nullptr);
          if (it.n0 > 0) load_q(0);
          if (it.n1 > 0) load_q(1);
          for (int j = 0; ok && j < it.tiles; ++j) {
            if (j + 1 < it.tiles) load(&tm_k, j + 1, nullptr);
            // (a last V tile that ends inside goes to warp 19 first, which fills the slot)
            const bool tail = it.tail && j + 1 == it.tiles;
            const int t = tails & 1;
            if (tail && tails >= 2) {
              ok = ok && wait(&tail_free[t], static_cast<uint32_t>((tails - 2) >> 1) & 1u, kSiteAttnLoad);
            }
            load(&tm_v, j, tail ? &tail_full[t] : nullptr);
          }
          tails += it.tail;
          // The item after this one, asked for with the last loads of this one (earlier, and items are dealt out before
          // it is known who is done first).  Its buffer has been read by every warp.
          const int asked = taken + 1, b = asked & 1;
          ok = ok && (asked <= 2 || wait(&item_free[b], static_cast<uint32_t>((asked - 3) >> 1) & 1u, kSiteAttnItem));
          if (ok) {
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&item_full[b], 16);
            launch_cancel_async(answer + 16 * b, &item_full[b]);
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
    } else if (warp == 17 || warp == 18) {
      // -------------------------------------------------------- MMA issuer
      const int s = warp - 17;
      // Matrix descriptors: the high words are constant, the low ones hold the address (in units of 16 bytes).
      const uint64_t desc_q = make_smem_desc_k_sw128(smem_u32(sQ + s * kQ));
      const uint64_t desc_k = make_smem_desc_k_sw128(smem_u32(ring));
      const uint64_t desc_v = make_smem_desc_n_sw128(smem_u32(ring), kBlock);
      const uint32_t t_s = tmem + s * kSpan, t_o = tmem + kColO + s * D;
      int stage = 0;
      uint32_t phase = 0, q_phase = 0;
      uint32_t s_phase = 1, p_phase = 0;  // of s_free (one phase behind s_full) and p_full
      for (; item >= 0; item = next_item(ok)) {
        const Item it = item_of(item);
        if (elect_one()) {
          const int n = s == 0 ? it.n0 : it.n1;
          const auto wait_fill = [&] { ok = ok && wait(&full[stage], phase, kSiteAttnOperand); };
          const auto release = [&] {  // the ring slot is free when the MMAs issued so far are done
            mma_commit(&empty[stage]);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          };
          const auto scores = [&](int j) {  // S = Q K^T
            ok = ok && wait(&s_free[s], s_phase, kSiteAttnWeights);
            if (!ok) return;
            s_phase ^= 1u;
            tc_fence_after_sync();
            const uint64_t kd = desc_k + stage * (kTile / 16);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              mma_bf16_ss(t_s, desc_q + ((x / 4) * (kQBlock / 16) + 2 * (x % 4)),
                          kd + ((x / 4) * (kBlock / 16) + 2 * (x % 4)), kIdescS, x > 0);
            }
            mma_commit(&s_full[s]);
            if (j + 1 == n) mma_commit(&q_free[s]);
          };
          // Step j: the scores of tile j, then the product of tile j - 1.
#pragma unroll 1
          for (int j = 0; ok && j <= it.tiles && it.tiles > 0; ++j) {
            if (j < it.tiles) {
              wait_fill();
              if (ok && j == 0 && n > 0) {
                ok = wait(&q_full[s], q_phase, kSiteAttnOperand);
                q_phase ^= 1u;
              }
              if (j < n) scores(j);
              if (!ok) break;
              release();
            }
            if (j == 0) continue;
            wait_fill();
            if (j - 1 < n) {
              ok = ok && wait(&p_full[s], p_phase, kSiteAttnWeights);
              if (!ok) break;
              p_phase ^= 1u;
              tc_fence_after_sync();
              const uint64_t vd = desc_v + stage * (kTile / 16);
#pragma unroll
              for (int x = 0; x < kTileK / 16; ++x) {
                mma_bf16_ts(t_o, t_s + kTileK + 8 * x, vd + 128 * x, kIdescO, (x > 0 || j > 1) ? 1u : 0u);
              }
              mma_commit(&o_full[s]);
            }
            if (ok) release();
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
      // No MMA may still run when tensor memory is freed.
      if (elect_one()) {
        mma_commit(&drain[s]);
        mbar_wait_drain(&drain[s], 0, p.timeout_ns, err);
      }
    } else {
      // ------------------------------------------------ ends of documents
      int fills = 0, tails = 0;
      for (; item >= 0; item = next_item(ok)) {
        const Item it = item_of(item);
        fills = (fills + 2 * it.tiles) % kStages;  // the ring slot behind the item's last V tile
        if (!it.tail) continue;
        ok = warp_wait(&tail_full[tails & 1], static_cast<uint32_t>(tails >> 1) & 1u, abort_flag, item_limit(), err,
                       kSiteAttnOperand);
        if (!ok) continue;
        const int stage = (fills + kStages - 1) % kStages;
        uint8_t* v = ring + stage * kTile;
        for (int e = it.tail_rows * 8 + lane; e < kTileK * 8; e += 32) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) *reinterpret_cast<uint4*>(v + b * kBlock + e * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[stage]);
          mbar_arrive(&tail_free[tails & 1]);
        }
        ++tails;
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    reg_raise<kRegsSoftmax>();
    const int s = warp >> 3;
    const int part = (warp >> 2) & 1;  // keys kHalf * part .. of every tile
    const int quarter = warp & 3;
    const uint32_t partners = 1 + (warp >> 3) * 4 + quarter;  // named barrier of the two warps of 32 queries
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + s * kSpan + kHalf * part;
    const uint32_t t_p = tmem + lanes + s * kSpan + kTileK + kHalf / 2 * part;
    const uint32_t t_o = tmem + lanes + kColO + s * D + D / 2 * part;
    const int in_sub = quarter * 32 + lane;
    constexpr bool kChange = CAP || BIAS;  // scores need more than the factor c
    const float c = p.scale * kLog2e;
    bool ok = true;
    uint32_t s_phase = 0, o_phase = 0;  // of s_full and o_full
    int turn = 0;                       // of the exchange buffers

    for (; item >= 0; item = next_item(ok)) {
      const Item it = item_of(item);
      const Doc& doc = it.doc;
      const int head = it.head, row0 = it.row0;
      const int my_rows = min(kSub, it.rows - s * kSub);  // <= 0: nothing in this sub-tile
      if (my_rows <= 0) continue;
      const int n = s == 0 ? it.n0 : it.n1;
      const int i = row0 + s * kSub + in_sub;  // the thread's query
      const int limit = in_sub < my_rows ? max(0, key_limit(p, doc, i)) : 0;
      const int least = key_limit(p, doc, row0 + s * kSub);  // the sub-tile's smallest limit
      const float slope = BIAS ? __ldg(p.slopes + head) * kLog2e : 0.0f;
      const int place = i + doc.shift;
      const int first_place = row0 + s * kSub + doc.shift;  // of the sub-tile's queries

      // The cap, on a thread's scores of a tile, from key key0 of the document on.  Scores within the cap on either side
      // (all of them, unless the scores are far beyond it) take a polynomial for tanh: 4 operations for two scores within
      // a quarter of the cap, in s^2 with the scale and the cap in its coefficients; 8 within the cap.  Where there are
      // others, each score takes the form that fits it.  The choice is the thread's, over the keys that its query sees:
      // other queries, hidden keys and other documents must not change a query's bits.
      const auto cap_pass = [&](auto& va, auto& vb, int key0, bool masked) {
        const auto farthest = [](const auto& v, float far) {
          constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
          for (int x = 0; x < N; x += 2) {
            far = max3(far, fabsf(__uint_as_float(v[x])), fabsf(__uint_as_float(v[x + 1])));
          }
          return far;
        };
        const auto hide = [](auto& v, int left) {
          constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
          for (int x = 0; x < N; ++x) {
            if (x >= left) v[x] = 0u;
          }
        };
        float far = farthest(vb, farthest(va, 0.0f));
        if (masked && !__all_sync(0xFFFFFFFFu, far <= p.near)) {
          hide(va, limit - key0);
          hide(vb, limit - key0 - 32);
          far = farthest(vb, farthest(va, 0.0f));
        }
        if (far <= p.near) {  // (a NaN among the scores compares false)
          const uint64_t k0 = both(p.near_k[0]), k1 = both(p.near_k[1]), k2 = both(p.near_k[2]);
          const auto nearby = [&](auto& v) {
            constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
            for (int x = 0; x < N; x += 2) {
              const uint64_t y = pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), u = mul2(y, y);
              float a0, a1;
              unpair(mul2(fma2(fma2(k2, u, k1), u, k0), y), a0, a1);
              v[x] = __float_as_uint(a0);
              v[x + 1] = __float_as_uint(a1);
            }
          };
          nearby(va);
          nearby(vb);
        } else {
          // (one stretch of code within and beyond the cap, a few scores at a time: with one for each, 604 us against
          // 534 for 4608 tokens, 24 heads of 128 and a cap of 3, three times the scores' deviation)
          const bool beyond = !(far * p.inv_cap <= 1.0f);
          const auto rest = [&](auto& v) {
            constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
            for (int at = 0; at < N; at += 8) {
              float y[8];
#pragma unroll
              for (int x = 0; x < 8; x += 2) {
                const uint64_t two = pair(__uint_as_float(v[at + x]), __uint_as_float(v[at + x + 1]));
                unpair(mul2(two, both(p.inv_cap)), y[x], y[x + 1]);
              }
              capped(y, beyond, p.cap_log2e);
#pragma unroll
              for (int x = 0; x < 8; ++x) v[at + x] = __float_as_uint(y[x]);
            }
          };
          rest(va);
          rest(vb);
        }
        __syncwarp();
      };

      // Scores of a tile, from key key0 of the document on: bias and mask; their maximum.
      const auto first_pass = [&](auto& v, int key0, bool masked) {
        constexpr int N = sizeof(v) / sizeof(v[0]);
        if constexpr (BIAS) {
          const float f = CAP ? 1.0f : c;
          const float first = static_cast<float>(key0 - place);  // distance of the first key, signed
          if (key0 + N - 1 <= first_place) {
            // No key lies ahead of any query of the sub-tile: the bias is linear in the key.
            const float at0 = slope * first;
#pragma unroll
            for (int x = 0; x < N; ++x) {
              v[x] = __float_as_uint(fmaf(__uint_as_float(v[x]), f, fmaf(slope, static_cast<float>(x), at0)));
            }
          } else {
#pragma unroll
            for (int x = 0; x < N; ++x) {
              v[x] = __float_as_uint(fmaf(__uint_as_float(v[x]), f, -slope * fabsf(first + static_cast<float>(x))));
            }
          }
        }
        if (masked) {
          const int left = limit - key0;
#pragma unroll
          for (int x = 0; x < N; ++x) {
            if (x >= left) v[x] = 0xFF800000u;  // -inf
          }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < N; x += 4) {
          top[0] = max3(top[0], __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
          top[1] = max3(top[1], __uint_as_float(v[x + 2]), __uint_as_float(v[x + 3]));
        }
        return fmax_nan(top[0], top[1]);
      };

      // The value of the thread with the other half of this query's keys.  One barrier is enough with two buffers in
      // turn: a buffer is written again behind the next tile's barrier, where the partner has read it.  (A warp that
      // aborts arrives once more, and its partner looks at the flag before it comes back: none is left waiting.)
      const auto partner = [&](float x) {
        float* const at = exchange + (turn & 1) * (4 * kSub) + s * kSub + in_sub;
        ++turn;
        at[part * 2 * kSub] = x;
        named_barrier_sync(partners, 64);
        return at[(part ^ 1) * 2 * kSub];
      };
      const auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
        const bool done = mbar_wait_bounded(bar, parity, abort_flag, p.timeout_ns, err, site);
        return __all_sync(0xFFFFFFFFu, done && !*abort_flag);
      };

      float m = -INFINITY;  // in units of log2
      float l = 0.0f;
      for (int j = 0; j < n; ++j) {
        ok = wait(&s_full[s], s_phase, kSiteAttnScores);
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after_sync();
        const bool masked = (j + 1) * kTileK > least;
        const int key0 = j * kTileK + kHalf * part;
        uint32_t va[32], vb[kHalf - 32];
        tmem_load_cols_async(t_s, va);
        tmem_load_cols_async(t_s + 32, vb);
        tmem_wait_loads(va);
        tmem_wait_loads(vb);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[s]);
        if constexpr (CAP) cap_pass(va, vb, key0, masked);
        float top = fmax_nan(first_pass(va, key0, masked), first_pass(vb, key0 + 32, masked));
        top = fmax_nan(top, partner(top));
        if (!kChange) top *= c;  // c > 0
        // P and O are free when the last tile's product is done.  (To wait here, rather than behind the exponentials,
        // keeps the two sub-tiles out of step: 427 us against 448 for 2 x 4608 tokens, 24 heads of 128.  When both
        // compute exponentials at the same time, both come to wait at the same time.)
        if (j > 0) {
          ok = wait(&o_full[s], o_phase, kSiteAttnOut);
          if (!ok) break;
          o_phase ^= 1u;
          tc_fence_after_sync();
        }
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
              tmem_load_16cols(t_o + 16 * b, o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_store_cols(t_o + 16 * b, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        const uint64_t c2 = both(kChange ? 1.0f : c), minus = both(-base);
        uint64_t sums[2] = {both(0.0f), both(0.0f)};
        // Weights of 2 N keys.  (A part of the exponentials as polynomials on the FMA units, to relieve the
        // special-function units, made it slower: 438 us against 427 with an eighth of them, 453 with three eighths,
        // at 2 x 4608 tokens, 24 heads of 128.  Two warps per scheduler do not hide the polynomial's latency.)
        const auto weights = [&](const uint32_t* v, auto& w) {
          constexpr int N = sizeof(w) / sizeof(w[0]);
#pragma unroll
          for (int x = 0; x < N; ++x) {
            const uint64_t y = pair(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
            const uint64_t e = kChange ? add2(y, minus) : fma2(y, c2, minus);
            float a0, a1;
            unpair(e, a0, a1);
            a0 = ex2(a0);
            a1 = ex2(a1);
            sums[x & 1] = add2(sums[x & 1], pair(a0, a1));
            w[x] = pack_bf16(a0, a1);  // the weights' one rounding; their sum is that of the unrounded ones
          }
        };
        uint32_t wa[16], wb[kHalf / 2 - 16];
        weights(va, wa);
        weights(vb, wb);
        tmem_store_cols(t_p, wa);
        tmem_store_cols(t_p + 16, wb);
        tmem_wait_store();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[s]);
        float s0, s1;
        unpair(add2(sums[0], sums[1]), s0, s1);
        l += s0 + s1;
      }

      // ------------------------------------------------------------- epilogue
      if (ok && n > 0) {
        ok = wait(&o_full[s], o_phase, kSiteAttnOut);
        o_phase ^= 1u;
      }
      if (!ok) break;
      tc_fence_after_sync();
      if (n > 0) l += partner(l);
      const bool any = l != 0.0f;  // (a key that is seen, with a score above -inf)
      const float inv = any ? 1.0f / l : 0.0f;
      const int64_t token = doc.q0 + i;
      // The warp's 32 rows x D/2 values, 32 columns at a time through shared memory, so that they leave in segments
      // of 64 bytes (16 bytes a thread, each in a row of its own, keep the load/store units busy for 4 000 cycles an
      // item).
      uint8_t* stage = staging + warp * kStagingBytes;
      const int64_t token0 = doc.q0 + row0 + s * kSub + quarter * 32;
      const int valid = my_rows - quarter * 32;
#pragma unroll 1
      for (int b = 0; b < D / 64; ++b) {
        uint32_t o[32];
        if (n > 0) {
          tmem_load_32cols(t_o + 32 * b, o);
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0u;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float a0 = __uint_as_float(o[8 * y + 2 * z]) * inv, a1 = __uint_as_float(o[8 * y + 2 * z + 1]) * inv;
            w[z] = any ? pack_bf16(a0, a1) : 0u;
          }
          *reinterpret_cast<uint4*>(stage + (4 * lane + (y ^ ((lane >> 1) & 3))) * 16) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int r = 8 * y + (lane >> 2), z = lane & 3;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + (4 * r + (z ^ ((r >> 1) & 3))) * 16);
          if (r < valid) {
            *reinterpret_cast<uint4*>(p.out + (token0 + r) * p.ldo + head * p.hso + D / 2 * part + 32 * b + 8 * z) = w;
          }
        }
        __syncwarp();
      }
      if (p.lse != nullptr && part == 0 && in_sub < my_rows) {
        p.lse[token * p.heads_q + head] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    if (!ok) named_barrier_arrive(partners, 64);  // the partner may stand at its barrier: it will see the abort next
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

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap tm_q, tm_k, tm_v;
  std::memset(&tm_q, 0, sizeof tm_q);
  // No keys: no tile of them is ever loaded, and the maps describe q.
  const bool none = p.tokens_k == 0;
  bool ok = encode_heads(&tm_q, p.q, D, p.tokens_q, p.heads_q, p.ldq, p.hsq, kSub);
  tm_k = tm_v = tm_q;
  if (!none) {
    ok = ok && encode_heads(&tm_k, p.k, D, p.tokens_k, p.heads_k, p.ldk, p.hsk, tile_keys(D)) &&
         encode_heads(&tm_v, p.v, D, p.tokens_k, p.heads_k, p.ldv, p.hsv, tile_keys(D));
  }
  if (!ok) return cudaErrorInvalidValue;
  int* err = nullptr;
  cudaError_t e = error_word_address(&err);
  if (e != cudaSuccess) return e;
  auto kernel = attention_tiles_kernel<D, CAP, BIAS>;
  constexpr int smem = smem_bytes(D);
  static_assert(smem <= 232448, "shared memory");
  static_assert(kExchange * 4 + (2 * ring_stages(D) + 22) * 8 + 8 <= kHeadBytes - 32, "barriers before the answers");
  static std::atomic<uint64_t> set{0};
  e = allow_shared_memory(kernel, smem, set);
  if (e != cudaSuccess) return e;
  const int64_t slots = p.tokens_q / kTileQ + p.docs;
  const int64_t items = slots * p.heads_q;
  if (items > 2147483647) return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(items), kThreads, smem, stream>>>(tm_q, tm_k, tm_v, p, static_cast<int>(slots), err);
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
