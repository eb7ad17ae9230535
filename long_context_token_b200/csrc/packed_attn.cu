// Causal attention over packed prompts on the 5th-generation tensor cores.
//
// A work item is one sequence, one K/V head and 2 x 128 query rows: a row is a (token, head
// of the group) pair, tokens outer, so the query heads that share a K/V head share its tiles
// and a short prompt still fills the MMA's 128 rows.  Persistent CTAs, one per SM, take items
// from a counter, each sequence's longest ones first.  Per 128-key block j and tile t:
//
//   S_t[128 x 128]  = Q_t . K_j^T            (smem x smem, D/16 MMAs)
//   P_t             = 2^(S_t c - m)          (softmax warps, one thread per row)
//   O_t[128 x D]   += P_t . V_j              (P_t from TMEM, 128/16 MMAs)
//
//   warps 0..3, 4..7  softmax of tile 0, 1: a thread owns a row, so the row's maximum and
//               sum need no shuffle.  The reference m moves only when a logit passes it by
//               more than 8 (log2 units); O is then rescaled in TMEM, which is safe once
//               S_t(j) is complete because P_t(j-1) . V ran before it.  P replaces S in TMEM
//               (two 16-bit weights per column).
//   warp 8      MMA issuer: Q.K of block j + 1 is issued after P.V of block j of the same
//               tile, so each tile's softmax runs under the other tile's MMAs.
//   warp 9      work items and TMA loads: Q (2 x 128 rows), K and V blocks in one ring.
//
// Weights are rounded to the inputs' 16-bit type for the second product, as the MMA needs;
// the row sums, references and O stay in float32.
#include <string.h>

#include "paged.cuh"
#include "sm100.cuh"
#include "tc_common.cuh"

namespace hs2 {

using namespace sm100;

namespace {

constexpr int kRows = 128;         // query rows per tile (the MMA's M)
constexpr int kKeys = 128;         // keys per block (the MMA's N, then its K extent)
constexpr int kSoftmaxThreads = 256;
constexpr int kPackedThreads = kSoftmaxThreads + 64;
constexpr float kMoveAt = 8.0f;    // log2 units by which a logit may pass the reference
constexpr float kLn2 = 0.69314718055994531f;

struct Item {
  int n[2];      // key blocks of each tile (0: none)
  int tokens[2];  // query tokens of each tile
  int q_row;     // first query token (row of q)
  int pos;       // its position in its sequence
  int k_row;     // first key (row of k)
  int lk;        // keys of the sequence
  int head;      // K/V head
  int valid;     // 0: no more items
};

template <int D>
struct PackedSmem {
  static constexpr uint32_t kBox = kRows * 128;       // 128 rows x 64 elements
  static constexpr uint32_t kTile = D / 64 * kBox;    // 128 rows x D
  static constexpr int kStages = 5;
  static constexpr uint32_t kQOff = 0;                // two tiles
  static constexpr uint32_t kRingOff = 2 * kTile;
  static constexpr uint32_t kItemOff = kRingOff + kStages * kTile;  // two slots
  static constexpr uint32_t kBarOff = kItemOff + 2 * 64;
  static constexpr uint32_t kBars = 2 * kStages + 13;
  static constexpr uint32_t kSlotOff = kBarOff + kBars * 8;
  static constexpr uint32_t kBytes = kSlotOff + 16 + 1024;
  static_assert(sizeof(Item) <= 64 && kBytes <= 227 * 1024, "shared memory budget");
};

// K-major operand (Q or K tile, boxes of 64 elements, 128-byte swizzle): K step kk of 16.
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile, int kk) {
  return smem_desc(tile + (uint32_t)(kk >> 2) * (kRows * 128u) + (uint32_t)(kk & 3) * 32u, 16, 1024,
                   kSwizzle128B);
}
// V tile as the MN-major B operand (N = D, K = keys): K step kk covers keys [16kk, 16kk + 16).
__device__ __forceinline__ uint64_t v_desc(uint32_t tile, int kk) {
  return smem_desc(tile + (uint32_t)kk * 16u * 128u, kRows * 128u, 1024, kSwizzle128B);
}

__device__ __forceinline__ void zero16(uint8_t* p) {
  *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
}

}  // namespace

// Walks the sequences for the producer warp: work items are numbered sequence by sequence,
// within one by query block (last first), then K/V head.  Item numbers only grow, so the
// cursor only moves forward, 32 sequences at a time.
struct ItemCursor {
  int b0 = 0;           // first sequence of the current 32
  uint32_t base = 0;    // items before it
  int lq = 0, lk = 0, q0 = 0, k0 = 0;  // this lane's sequence
  uint32_t count = 0, before = 0;      // its items, and the items before it in the 32
  uint32_t total = 0;   // items of the 32

  __device__ void load(const PackedAttnParams& p, int tokens_per_item, int lane) {
    lq = lk = 0;
    if (b0 + lane < p.batch) {
      const int a = __ldg(p.cu_q + b0 + lane), b = __ldg(p.cu_q + b0 + lane + 1);
      const int c = __ldg(p.cu_k + b0 + lane), d = __ldg(p.cu_k + b0 + lane + 1);
      if (a < 0 || b < a || b > p.n_q || c < 0 || d < c || d > p.n_k)
        set_status(p.status, HS2_ERR_BAD_LENGTH);
      q0 = min(max(a, 0), p.n_q);
      k0 = min(max(c, 0), p.n_k);
      lq = max(min(b, p.n_q) - q0, 0);
      lk = max(min(d, p.n_k) - k0, 0);
    }
    count = (uint32_t)((lq + tokens_per_item - 1) / tokens_per_item) * (uint32_t)p.h_kv;
    uint32_t incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    before = incl - count;
    total = __shfl_sync(0xffffffffu, incl, 31);
  }

  // Item number -> item (valid 0 behind the last).  All lanes together, the same number.
  __device__ Item find(const PackedAttnParams& p, uint32_t item, int tpt, int lane) {
    while (item - base >= total) {
      if (b0 + 32 >= p.batch) {
        Item none = {};
        return none;
      }
      base += total;
      b0 += 32;
      load(p, 2 * tpt, lane);
    }
    const uint32_t at = item - base;
    const uint32_t owner = __ballot_sync(0xffffffffu, at >= before && at - before < count);
    const int src = __ffs(owner) - 1;
    const int s_lq = __shfl_sync(0xffffffffu, lq, src), s_lk = __shfl_sync(0xffffffffu, lk, src);
    const int s_q0 = __shfl_sync(0xffffffffu, q0, src), s_k0 = __shfl_sync(0xffffffffu, k0, src);
    const uint32_t in = at - __shfl_sync(0xffffffffu, before, src);
    const int blocks = (s_lq + 2 * tpt - 1) / (2 * tpt);
    const int blk = blocks - 1 - (int)(in / (uint32_t)p.h_kv);
    Item it;
    it.valid = 1;
    it.head = (int)(in % (uint32_t)p.h_kv);
    const int tok0 = blk * 2 * tpt;  // within the sequence
    it.q_row = s_q0 + tok0;
    it.k_row = s_k0;
    it.lk = s_lk;
    it.pos = s_lk - s_lq + tok0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      it.tokens[t] = min(max(s_lq - tok0 - t * tpt, 0), tpt);
      const int last = it.pos + t * tpt + it.tokens[t] - 1;  // the tile's last token sees [0, last]
      it.n[t] = it.tokens[t] > 0 && last >= 0 ? last / kKeys + 1 : 0;
    }
    return it;
  }
};

template <int D, typename T>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, PackedAttnParams p) {
  using L = PackedSmem<D>;
  constexpr int NS = L::kStages;
  constexpr bool kBf16 = !std::is_same<T, __half>::value;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* qs = smem + L::kQOff;
  uint8_t* ring = smem + L::kRingOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* full = bars;
  uint64_t* empty = bars + NS;
  uint64_t* q_full = bars + 2 * NS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;   // [2] tile's logits complete
  uint64_t* p_full = q_full + 4;   // [2] tile's weights written
  uint64_t* o_full = q_full + 6;   // [2] tile's output complete
  uint64_t* it_full = q_full + 8;  // [2] item slot written
  uint64_t* it_empty = q_full + 10;  // [2] item slot read
  uint64_t* drained = q_full + 12;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlotOff);
  auto item_slot = [&](int i) { return reinterpret_cast<Item*>(smem + L::kItemOff + 64 * (i & 1)); };

  const int warp = threadIdx.x >> 5, lane = (int)lane_id();
  const int tpt = kRows / p.group;  // query tokens per tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drained, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(p_full + t, kRows);
      mbar_init(o_full + t, 1);
      mbar_init(it_full + t, 1);
      mbar_init(it_empty + t, kSoftmaxThreads + 1);
    }
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S0, S1: 128 columns each; O0, O1: at 256, 256 + 128
  griddep_wait();
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity)) {
      ok = false;
      set_status(p.status, HS2_ERR_DEVICE_TIMEOUT);
    }
  };

  if (warp == 9) {
    // ------------------------------------------------------------ items and loads
    ItemCursor cur;
    cur.load(p, 2 * tpt, lane);
    const uint64_t keep = policy_evict_last();  // other CTAs read the same K and V
    const uint64_t once = policy_evict_first();
    uint32_t slot = 0;  // ring position (slots filled so far)
    uint32_t q_loads = 0;
    for (int i = 0; ok; ++i) {
      uint32_t number = blockIdx.x;
      if (i > 0) {
        if (lane == 0) number = gridDim.x + atomicAdd(p.sync, 1u);
        number = __shfl_sync(0xffffffffu, number, 0);
      }
      const Item it = cur.find(p, number, tpt, lane);
      wait(it_empty + (i & 1), ((i >> 1) & 1) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        *item_slot(i) = it;
        mbar_arrive(it_full + (i & 1));
      }
      if (!it.valid) break;
      const int blocks = max(it.n[0], it.n[1]);
      if (lane == 0 && blocks > 0) {
        auto fill = [&](const CUtensorMap* m, int x, int y, int z, int boxes) {
          const uint32_t s = slot % NS;
          wait(empty + s, ((slot / NS) & 1) ^ 1);
          if (!ok) return;
          mbar_arrive_expect_tx(full + s, L::kTile);
          for (int c = 0; c < boxes; ++c)
            tma_load_3d(ring + s * L::kTile + c * L::kBox, m, full + s, x + 64 * c, y, z, keep);
          ++slot;
        };
        fill(&tmap_k, 0, it.head, it.k_row, D / 64);
        wait(q_empty, (q_loads & 1) ^ 1);
        if (ok) {
          // (only tiles with tokens; rows behind the group's heads x tokens stay stale)
          const int tiles = it.tokens[1] > 0 ? 2 : 1;
          const uint32_t bytes = (uint32_t)(tpt * p.group) * D * 2;
          mbar_arrive_expect_tx(q_full, tiles * bytes);
          for (int t = 0; t < tiles; ++t)
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(qs + t * L::kTile + c * L::kBox, &tmap_q, q_full, 64 * c,
                          it.head * p.group, it.q_row + t * tpt, once);
          ++q_loads;
        }
        for (int j = 0; j < blocks && ok; ++j) {
          if (j > 0) fill(&tmap_k, 0, it.head, it.k_row + j * kKeys, D / 64);
          if (ok) fill(&tmap_v, 0, it.head, it.k_row + j * kKeys, D / 64);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0) {
      // No load may outlive the CTA (they were all consumed unless a wait gave up).
      for (uint32_t s = slot > NS ? slot - NS : 0; s < slot; ++s)
        mbar_wait(full + s % NS, (s / NS) & 1);
      if (q_loads) mbar_wait(q_full, (q_loads - 1) & 1);
      // The last CTA to take its items puts the counters back.
      if (atomicAdd(p.sync + 1, 1u) == gridDim.x - 1) {
        p.sync[0] = 0;
        p.sync[1] = 0;
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_qk = idesc_f16(kRows, kKeys, kBf16, false, false);
    constexpr uint32_t id_pv = idesc_f16(kRows, D, kBf16, false, true);
    const uint32_t q_addr = smem_u32(qs);
    uint32_t slot = 0, q_loads = 0;
    uint32_t n_p[2] = {0, 0};  // weights consumed of each tile
    for (int i = 0; ok; ++i) {
      wait(it_full + (i & 1), (i >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Item it = *item_slot(i);
      __syncwarp();
      if (lane == 0) mbar_arrive(it_empty + (i & 1));
      if (!it.valid) break;
      const int blocks = max(it.n[0], it.n[1]);
      if (blocks == 0) continue;
      auto qk = [&](int t, uint32_t k_addr) {
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ss(tmem + t * kKeys, rows_desc(q_addr + t * L::kTile, kk), rows_desc(k_addr, kk),
                       id_qk, kk > 0 ? 1u : 0u);
          mma_commit(s_full + t);
        }
      };
      auto pv = [&](int t, uint32_t v_addr, int steps, int j) {
        wait(p_full + t, n_p[t] & 1);
        ++n_p[t];
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        if (lane == 0) {
          for (int kk = 0; kk < steps; ++kk)
            mma_f16_ts(tmem + 2 * kKeys + t * kKeys, tmem + t * kKeys + kk * 8, v_desc(v_addr, kk),
                       id_pv, (j > 0 || kk > 0) ? 1u : 0u);
          if (j == it.n[t] - 1) mma_commit(o_full + t);
        }
      };
      // Logits of both tiles for the block in ring slot `slot`.
      auto next_k = [&]() -> uint32_t {
        wait(full + slot % NS, (slot / NS) & 1);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        return smem_u32(ring + (slot % NS) * L::kTile);
      };
      wait(q_full, q_loads & 1);
      ++q_loads;
      uint32_t k_addr = next_k();
      if (!ok) break;
      if (it.n[0] > 0) qk(0, k_addr);
      if (it.n[1] > 0) qk(1, k_addr);
      if (lane == 0) {
        mma_commit(empty + slot % NS);
        if (blocks == 1) mma_commit(q_empty);
      }
      ++slot;
      for (int j = 0; j < blocks && ok; ++j) {
        const uint32_t v_slot = slot;
        const uint32_t v_addr = next_k();
        ++slot;
        if (!ok) break;
        // The sequence's last block: MMA steps past its keys are left out, and the rows of
        // the last step that belong to other sequences are cleared (their weights are 0,
        // but 0 times an infinity or NaN is not).
        const int live = min(it.lk - j * kKeys, kKeys);
        const int steps = (live + 15) >> 4;
        if (live & 15) {
          const int rows = 16 - (live & 15);
          uint8_t* base = ring + (v_slot % NS) * L::kTile + live * 128;
          for (int e = lane; e < rows * 8 * (D / 64); e += 32)
            zero16(base + (e >> 3) % rows * 128 + (e >> 3) / rows * L::kBox + (e & 7) * 16);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (j < it.n[0]) pv(0, v_addr, steps, j);
        uint32_t k_slot = 0;
        if (j + 1 < blocks && ok) {
          k_slot = slot;
          k_addr = next_k();
          ++slot;
          if (ok && j + 1 < it.n[0]) qk(0, k_addr);
        }
        if (j < it.n[1] && ok) pv(1, v_addr, steps, j);
        if (lane == 0) mma_commit(empty + v_slot % NS);
        if (j + 1 < blocks && ok) {
          if (j + 1 < it.n[1]) qk(1, k_addr);
          if (lane == 0) {
            mma_commit(empty + k_slot % NS);
            if (j + 2 == blocks) mma_commit(q_empty);
          }
        }
      }
    }
    if (lane == 0) {  // nothing of this CTA's is in flight when the TMEM goes
      mma_commit(drained);
      mbar_wait(drained, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * kKeys, to = tmem + lanes + 2 * kKeys + t * kKeys;
    const int tok = r / p.group, hh = r - tok * p.group;
    const float c = p.scale_log2;
    uint32_t n_s = 0, n_o = 0;
    for (int i = 0; ok; ++i) {
      wait(it_full + (i & 1), (i >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Item it = *item_slot(i);
      mbar_arrive(it_empty + (i & 1));
      if (!it.valid) break;
      const bool live = tok < it.tokens[t];
      const int seen = live ? it.pos + t * tpt + tok + 1 : 0;  // keys [0, seen) are visible
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < it.n[t]; ++j) {
        wait(s_full + t, n_s & 1);
        ++n_s;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[kKeys];
#pragma unroll
        for (int e = 0; e < kKeys; e += 32) tmem_ld32(ts + e, s + e);
        tmem_wait_ld();
        const int lim = seen - j * kKeys;
        if (lim < kKeys) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e)
            if (e >= lim) s[e] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kKeys; e += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mx[u] = fmaxf(fmaxf(mx[u], __uint_as_float(s[e + 2 * u])), __uint_as_float(s[e + 2 * u + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool move = top - m > kMoveAt;  // false while top is -inf
        if (__any_sync(0xffffffffu, move)) {
          float alpha = 1.f;
          if (move) {
            alpha = ex2_ftz(m - top);  // 0 while m is -inf
            m = top;
            l *= alpha;
          }
          if (j > 0) {
#pragma unroll 1
            for (int e = 0; e < D; e += 16) {
              uint32_t o[16];
              tmem_ld16(to + e, o);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
              tmem_st16(to + e, o);
            }
          }
        }
        const float ref = -finite_ref(m);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < kKeys; e += 2) {
          const float a = ex2_ftz(fmaf(__uint_as_float(s[e]), c, ref));
          const float b = ex2_ftz(fmaf(__uint_as_float(s[e + 1]), c, ref));
          sum[e & 2] += a;
          sum[(e & 2) + 1] += b;
          s[e >> 1] = pack2<T>(a, b);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st32(ts, s);
        tmem_st32(ts + 32, s + 32);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + t);
      }
      if (!ok) break;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const size_t row = (size_t)(it.q_row + t * tpt + tok) * p.h_q + it.head * p.group + hh;
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * (D * 2));
      if (it.n[t] > 0) {
        wait(o_full + t, n_o & 1);
        ++n_o;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < D; e += 32) {
          uint32_t o[32];
          tmem_ld32(to + e, o);
          tmem_wait_ld();
          if (live) {
#pragma unroll
            for (int u = 0; u < 32; u += 8) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = l > 0.f ? pack2<T>(__uint_as_float(o[u + 2 * x]) * inv,
                                          __uint_as_float(o[u + 2 * x + 1]) * inv)
                               : 0u;
              out[(e + u) >> 3] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        tc_fence_before();
      } else if (live) {
#pragma unroll
        for (int e = 0; e < D / 8; ++e) out[e] = make_uint4(0, 0, 0, 0);
      }
      if (live && p.lse) p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
    __threadfence();  // the results are visible before the next kernel may start
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
  griddep_launch_dependents();
}

template <int D, typename T>
static cudaError_t launch_packed(const PackedAttnParams& p, cudaStream_t st) {
  const CUtensorMapDataType dt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int tpt = kRows / p.group;
  auto stride = [](int n, int64_t s) { return n > 1 ? (uint64_t)s : uint64_t(16); };
  CUtensorMap tq, tk, tv;
  const uint64_t qd[3] = {D, (uint64_t)p.h_q, (uint64_t)p.n_q};
  const uint64_t qst[2] = {stride(p.h_q, p.q_head), stride(p.n_q, p.q_tok)};
  const uint32_t qb[3] = {64, (uint32_t)p.group, (uint32_t)tpt};
  const uint64_t kd[3] = {D, (uint64_t)p.h_kv, (uint64_t)(p.n_k ? p.n_k : 1)};
  const uint64_t kst[2] = {stride(p.h_kv, p.kv_head), stride(p.n_k, p.kv_tok)};
  const uint32_t kb[3] = {64, 1, kKeys};
  // (without keys nothing is loaded; the maps still need an address)
  if (!make_tmap_nd(&tq, p.q, dt, 3, qd, qst, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_nd(&tk, p.n_k ? p.k : p.q, dt, 3, kd, kst, kb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_nd(&tv, p.n_k ? p.v : p.q, dt, 3, kd, kst, kb, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto* kernel = packed_attn_kernel<D, T>;
  constexpr uint32_t smem = PackedSmem<D>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // At most this many items: full blocks of every sequence, and one partial block each.
  const long long items = ((long long)p.n_q / (2 * tpt) + p.batch) * p.h_kv;
  const int sms = device_sm_count();
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  return launch_pdl(kernel, dim3(grid), dim3(kPackedThreads), smem, st, tq, tk, tv, p);
}

cudaError_t launch_packed_attn(const PackedAttnParams& p, int head_dim, int dtype, cudaStream_t s) {
  if (head_dim == 128)
    return dtype == HS2_KV_F16 ? launch_packed<128, __half>(p, s) : launch_packed<128, __nv_bfloat16>(p, s);
  return dtype == HS2_KV_F16 ? launch_packed<64, __half>(p, s) : launch_packed<64, __nv_bfloat16>(p, s);
}

}  // namespace hs2
