// Causal attention over packed prompts on the 5th-generation tensor cores.
//
// A work item is one sequence, one K/V head and 2 x 128 query rows: a row is a (token, head
// of the group) pair, tokens outer, so the query heads that share a K/V head share its tiles
// and a short prompt still fills the MMA's 128 rows.  Persistent CTAs, one per SM, take items
// from a counter, those with the most keys first.  Keys go in steps i of 64; per step and tile t:
//
//   S_t[128 x 64]   = Q_t . K_i^T            (smem x smem, D/16 MMAs)
//   P_t             = 2^(S_t c - m)          (softmax warps, one thread per row)
//   O_t[128 x D]   += P_t . V_i              (P_t from TMEM, 4 MMAs)
//
//   warps 0..3, 4..7  softmax of tile 0, 1: a thread owns a row, so the row's maximum and
//               sum need no shuffle.  The reference m moves only when a logit passes it by
//               more than 8 (log2 units); O is then rescaled in TMEM, after P(i-1) . V.
//               P replaces S in TMEM (two 16-bit weights per column).  The two tiles' warps
//               on a scheduler form their exponentials in turn.
//   warps 8, 11 MMA issuers of tile 0, 1: each tile has two S buffers, and Q.K of step i + 1
//               is issued before P.V of step i, so the softmax of a tile need not wait for
//               its own products.
//   warp 9      work items and TMA loads: Q (2 x 128 rows), 128-key K and V blocks in a ring.
//   warp 10     clears V rows of other sequences in a sequence's last block.
//
// What bounds it: the exponentials.  A step's 128 x 64 weights take a scheduler's warp 512
// cycles of its special-function unit and about 740 with what cannot hide behind it, so two
// tiles take 1480 cycles a step, in which the tensor pipe works 1090.  On a B200, one prompt
// of 16384 tokens (16 heads, 2 K/V heads, d 128, bfloat16): 840 us, 1309 TFLOP/s, 0.79 of the
// measured burst rate of a library product (up to 890 us on a warm GPU); 975 us when the call
// repeats until the power cap lowers the clock (0.80 of the measured sustained rate).  What
// was measured on the way to this shape, on that prompt: 128-key steps with one S buffer per
// tile 1040 us; the MMAs of both tiles from one warp 942; without taking turns 878; two
// threads per row 904.  At d 64 the exponentials and the step's fixed costs are the same for half
// the products: one prompt of 16384 tokens 760 us, 2.3 times its floor.
//
// Keys are never split: an item walks all keys that its rows see on one SM.  Few queries after a
// long prefix leave the other SMs idle: 64 tokens of 16 heads (one K/V head) at the end of 131072
// keys take 1380 us, 33 times their floor; 512 tokens at the end of 16000 (two K/V heads) 168, 4.2
// times.
//
// Weights are rounded to the inputs' 16-bit type for the second product, as the MMA needs
// (float16 ones scaled so that the largest lies in [2^7, 2^15]); the row sums, references and O
// stay in float32 (O of long sequences in two parts: see drain).
#include <string.h>

#include "paged.cuh"
#include "sm100.cuh"
#include "tc_common.cuh"

namespace hs2 {

using namespace sm100;

namespace {

constexpr int kRows = 128;         // query rows per tile (the MMA's M)
constexpr int kKeys = 128;         // keys per loaded block
constexpr int kStep = 64;          // keys per step (the MMA's N, then its K extent)
constexpr int kSoftmaxThreads = 256;
constexpr int kPackedThreads = kSoftmaxThreads + 128;
// Keys of a sequence: warps that wait for an item's end (the cleaner, and tile 1's softmax in
// items of one tile) would give up after mbar_wait's limit, about 150 million keys.
constexpr int kMaxKeys = 1 << 26;
constexpr int kOneTileUpTo = 1;    // see launch_packed
constexpr int kDrainSteps = 256;   // steps between which O leaves the tensor cores' sum
constexpr float kMoveAt = 8.0f;    // log2 units by which a logit may pass the reference
constexpr float kLn2 = 0.69314718055994531f;

constexpr uint32_t kNothing = 0xfffffffeu, kNoMore = 0xffffffffu;  // to the cleaner

struct Item {
  int n[2];      // key steps of each tile (0: none)
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
  static constexpr uint32_t kBars = 2 * kStages + 30;
  static constexpr uint32_t kSlotOff = kBarOff + kBars * 8;
  static constexpr uint32_t kBytes = kSlotOff + 16 + 1024;
  static_assert(sizeof(Item) <= 64 && kBytes <= 227 * 1024, "shared memory budget");
};

// K-major operand (Q or K tile, boxes of 64 elements, 128-byte swizzle), K step kk of 16, and
// V tile as the MN-major B operand (N = D, K = keys), keys [16kk, 16kk + 16): descriptors of
// step 0, and what to add for step kk (the address field counts 16-byte units).
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile) {
  return smem_desc(tile, 16, 1024, kSwizzle128B);
}
__host__ __device__ constexpr uint64_t rows_step(int kk) {
  return (uint64_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4);
}
__device__ __forceinline__ uint64_t v_desc(uint32_t tile) {
  return smem_desc(tile, kRows * 128u, 1024, kSwizzle128B);
}
__host__ __device__ constexpr uint64_t v_step(int kk) { return (uint64_t)(kk * 16 * 128 >> 4); }

// 2^x of two numbers of up to about 100 on the multiply-add pipes: x = n + f with n the nearest
// integer, 2^f by the polynomial of degree 4 with the least relative error on [-1/2, 1/2]
// (2.6e-6, from the Remez exchange), times 2^n.  Of each kPairsOf pairs of
// weights kPairsByFma are formed this way, to relieve the special-function units: one in
// eight (none 862 us on the prompt above, one 841, two 855, three 865, four 887: the
// multiply-add pipes and the issue slots are not free either; 8192 tokens at d 64, 16 heads on 2:
// none 210, one 205, two 207).
constexpr int kPairsOf = 8, kPairsByFma = 1;
__device__ __forceinline__ float2 exp2_fma(float2 x) {
  // (Below -126.5 the factor 2^n is 0, so a masked key weighs nothing; a NaN stays one.)
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-127.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-127.f));
  // 1.5 x 2^23 + 127: the low bits of its sum with x are n + 127, the exponent of 2^n.
  const float2 magic = make_float2(12583039.f, 12583039.f);
  const float2 minus = make_float2(-12583039.f, -12583039.f), one = make_float2(-1.f, -1.f);
  const float2 t = add2(x, magic);
  const float2 f = fma2(add2(t, minus), one, x);
  auto both = [](float v) { return make_float2(v, v); };
  float2 y = fma2(both(0x1.3997d6p-7f), f, both(0x1.ca1444p-5f));
  y = fma2(y, f, both(0x1.ec06dap-3f));
  y = fma2(y, f, both(0x1.62e0dcp-1f));
  y = fma2(y, f, both(0x1.ffffe8p-1f));
  return mul2(y, make_float2(__uint_as_float(__float_as_uint(t.x) << 23),
                             __uint_as_float(__float_as_uint(t.y) << 23)));
}

// A row's outputs so far leave the tensor cores' sum for `kept`, which is first weighed by w (0
// at the first time, when it holds nothing); and come back to it, weighed likewise.  A sum in
// TMEM is cut, not rounded: each product of an MMA by up to 2^-25 of the sum, so a sum over n
// keys lost n 2^-27 of itself (0.7 % at 1048576) before it was drained every kDrainSteps steps.
template <int D>
__device__ __noinline__ void drain(uint32_t to, float* kept, float w) {
#pragma unroll 1
  for (int e = 0; e < D; e += 16) {
    uint32_t o[16];
    tmem_ld16(to + e, o);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 16; ++u)
      kept[e + u] = w > 0.f ? fmaf(kept[e + u], w, __uint_as_float(o[u])) : __uint_as_float(o[u]);
  }
}
template <int D>
__device__ __noinline__ void restore(uint32_t to, const float* kept, float w) {
#pragma unroll 1
  for (int e = 0; e < D; e += 16) {
    uint32_t o[16];
    tmem_ld16(to + e, o);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(fmaf(kept[e + u], w, __uint_as_float(o[u])));
    tmem_st16(to + e, o);
  }
  tmem_wait_st();
}

}  // namespace

// Walks the sequences for the producer warp.  Work items are numbered 32 sequences at a time,
// within them by their number of key blocks, largest first, so that the last items to be
// handed out are the shortest.  Item numbers only grow, so the cursor only moves forward.
struct ItemCursor {
  int b0 = 0;             // first sequence of the current 32
  uint32_t base = 0;      // items before it
  uint32_t total = 0;     // items of the 32
  int level = 0;          // the current number of key blocks
  uint32_t above = 0;     // items of the 32 with more key blocks, and with at least as many
  uint32_t upto = 0;
  int lq = 0, lk = 0, q0 = 0, k0 = 0;  // this lane's sequence
  int blocks = 0;         // its query blocks
  int done = 0, have = 0;  // of them, those with more key blocks than `level`, at least as many

  // How many of this lane's query blocks (the last ones) have at least n key blocks.
  __device__ int at_least(int n, int tokens_per_item) const {
    // the block's last token sits at lk - lq + (tokens up to it) - 1 >= (n - 1) * kKeys
    const int need = n > 0 ? (n - 1) * kKeys + 1 - lk + lq : 0;
    if (need <= 0) return blocks;
    return need > lq ? 0 : blocks - (need - 1) / tokens_per_item;
  }

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
      if (lk > kMaxKeys) {
        set_status(p.status, HS2_ERR_BAD_LENGTH);
        lk = kMaxKeys;
      }
    }
    blocks = (lq + tokens_per_item - 1) / tokens_per_item;
    total = __reduce_add_sync(0xffffffffu, (uint32_t)blocks) * (uint32_t)p.h_kv;
    level = __reduce_max_sync(0xffffffffu, blocks > 0 ? (lk + kKeys - 1) / kKeys : 0);
    done = 0;
    have = at_least(level, tokens_per_item);
    above = 0;
    upto = __reduce_add_sync(0xffffffffu, (uint32_t)have) * (uint32_t)p.h_kv;
  }

  // Item number -> item (valid 0 behind the last).  All lanes together, the same number.
  __device__ Item find(const PackedAttnParams& p, uint32_t number, int tpt, int tiles, int lane) {
    while (number - base >= total) {
      if (b0 + 32 >= p.batch) {
        Item none = {};
        return none;
      }
      base += total;
      b0 += 32;
      load(p, tiles * tpt, lane);
    }
    const uint32_t at = number - base;
    while (at >= upto) {  // (ends: with level 0, upto is total)
      --level;
      done = have;
      above = upto;
      have = at_least(level, tiles * tpt);
      upto = __reduce_add_sync(0xffffffffu, (uint32_t)have) * (uint32_t)p.h_kv;
    }
    const uint32_t mine = (uint32_t)(have - done) * (uint32_t)p.h_kv;  // this level's
    uint32_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    before -= mine;
    const uint32_t in = at - above;
    const int src = __ffs(__ballot_sync(0xffffffffu, in >= before && in - before < mine)) - 1;
    auto of = [&](int x) { return __shfl_sync(0xffffffffu, x, src); };
    const int s_lq = of(lq), s_lk = of(lk), s_q0 = of(q0), s_k0 = of(k0);
    const uint32_t nth = in - (uint32_t)of((int)before);
    const int blk = of(blocks) - 1 - of(done) - (int)(nth / (uint32_t)p.h_kv);
    Item it;
    it.valid = 1;
    it.head = (int)(nth % (uint32_t)p.h_kv);
    const int tok0 = blk * tiles * tpt;  // within the sequence
    it.q_row = s_q0 + tok0;
    it.k_row = s_k0;
    it.lk = s_lk;
    it.pos = s_lk - s_lq + tok0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      it.tokens[t] = t < tiles ? min(max(s_lq - tok0 - t * tpt, 0), tpt) : 0;
      const int last = it.pos + t * tpt + it.tokens[t] - 1;  // the tile's last token sees [0, last]
      it.n[t] = it.tokens[t] > 0 && last >= 0 ? last / kStep + 1 : 0;
    }
    return it;
  }
};

// kDrain: sequences may have more than kDrainSteps steps.
template <int D, typename T, bool kDrain>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, PackedAttnParams p) {
  using L = PackedSmem<D>;
  constexpr int NS = L::kStages;
  constexpr bool kBf16 = !std::is_same<T, __half>::value;
  // Float16 weights are 2^7 times 2^(x - m): at most 2^15, as m lags by at most 8.  Without the
  // factor those below 2^-25 of the reference vanished from the output but not from the sum.
  constexpr float kLift = kBf16 ? 0.f : 7.f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* qs = smem + L::kQOff;
  uint8_t* ring = smem + L::kRingOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* full = bars;
  uint64_t* empty = bars + NS;
  uint64_t* q_full = bars + 2 * NS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;     // [2 tiles][2 buffers] logits complete
  uint64_t* p_full = q_full + 6;     // [2 tiles][2 buffers] weights written
  // [2 tiles][2 buffers] a step's product is in the tile's output.  (One barrier per buffer:
  // who waits for a step has seen the one before the last, so a parity tells its phases apart.)
  uint64_t* o_done = q_full + 10;
  uint64_t* it_full = q_full + 14;   // [2] item slot written
  uint64_t* it_empty = q_full + 16;  // [2] item slot read
  uint64_t* v_dirty = q_full + 18;   // rows of a V block to clear, and cleared
  uint64_t* v_clean = q_full + 19;
  uint64_t* drained = q_full + 20;   // [2]
  uint64_t* turn = q_full + 22;      // [2 tiles][4 warps] this warp may form its exponentials
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlotOff);
  uint32_t* unclean = tmem_slot + 1;  // ring offset of the rows to clear
  auto item_slot = [&](int i) { return reinterpret_cast<Item*>(smem + L::kItemOff + 64 * (i & 1)); };

  // (shuffled: the compiler then knows that a warp takes one role as a whole)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = (int)lane_id();
  const int tpt = kRows / p.group;  // query tokens per tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 2);  // both tiles' MMAs
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(v_dirty, 2);
    mbar_init(v_clean, 1);
    for (int t = 0; t < 4; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(p_full + t, kRows);
      mbar_init(o_done + t, 1);
      mbar_init(turn + t, 1);
      mbar_init(turn + 4 + t, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(drained + t, 1);
      mbar_init(it_full + t, 1);
      mbar_init(it_empty + t, kSoftmaxThreads + 2);
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
  const uint32_t tmem = *tmem_slot;  // two S buffers of 64 columns per tile; O0, O1 at 256, 256 + 128
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
    cur.load(p, p.tiles * tpt, lane);
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
      const Item it = cur.find(p, number, tpt, p.tiles, lane);
      wait(it_empty + (i & 1), ((i >> 1) & 1) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        *item_slot(i) = it;
        mbar_arrive(it_full + (i & 1));
      }
      if (!it.valid) break;
      const int blocks = (max(it.n[0], it.n[1]) * kStep + kKeys - 1) / kKeys;
      if (lane == 0 && blocks > 0 && !p.stall_test) {
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
  } else if (warp == 8 || warp == 11) {
    // ------------------------------------------------------------ MMA issuers
    // One warp per tile, so that no tile's products queue behind a wait for the other's
    // weights.  The whole warp walks the loop and one elected thread issues: descriptors and
    // TMEM addresses then are warp-uniform values, which the MMA takes as they are.  (From a
    // branch of a single thread each MMA cost about 115 cycles to issue, twice its run time.)
    const int t = warp == 8 ? 0 : 1;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t td = tm + t * 2 * kStep, to = tm + 4 * kStep + t * 128;  // S buffers, O
    constexpr uint32_t id_qk = idesc_f16(kRows, kStep, kBf16, false, false);
    constexpr uint32_t id_pv = idesc_f16(kRows, D, kBf16, false, true);
    const uint64_t qd = rows_desc(smem_u32(qs) + t * L::kTile);
    uint32_t slot = 0, q_loads = 0, n_clean = 0;
    uint32_t n_s = 0, n_p = 0;  // products issued, of all items
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      wait(bar, parity);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto qk = [&](uint64_t kd) {
      const uint32_t buf = n_s++ & 1, d = td + buf * kStep;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(d, qd + rows_step(kk), kd + rows_step(kk), id_qk, kk > 0 ? 1u : 0u);
        mma_commit(s_full + 2 * t + buf);
      }
      __syncwarp();
    };
    auto pv = [&](uint64_t vd, int live, bool first) {
      const uint32_t n = n_p++, buf = n & 1, w = td + buf * kStep;
      wait_all(p_full + 2 * t + buf, (n >> 1) & 1);
      tc_fence_after();
      if (!ok) return;  // (the caller's loops end with it)
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          if (kk * 16 < live)  // (MMA steps past the sequence's keys are left out)
            mma_f16_ts(to, w + kk * 8, vd + v_step(kk), id_pv, kk > 0 ? 1u : first ? 0u : 1u);
        mma_commit(o_done + 2 * t + buf);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) mma_commit(bar);
      __syncwarp();
    };
    auto next = [&]() -> uint32_t {  // the next ring slot, when it is filled
      const uint32_t s = slot % NS;
      wait_all(full + s, (slot / NS) & 1);
      tc_fence_after();
      ++slot;
      return s;
    };
    constexpr uint64_t kHalf = (uint64_t)(kStep * 128 >> 4);  // rows 64.. of a K or V block
    for (int i = 0; ok; ++i) {
      wait_all(it_full + (i & 1), (i >> 1) & 1);
      if (!ok) break;
      const Item* it = item_slot(i);
      const int n = __shfl_sync(0xffffffffu, it->n[t], 0);
      const int steps = max(n, __shfl_sync(0xffffffffu, it->n[1 - t], 0));  // the blocks to release
      const int lk = __shfl_sync(0xffffffffu, it->lk, 0);
      const int valid = __shfl_sync(0xffffffffu, it->valid, 0);
      if (lane == 0) mbar_arrive(it_empty + (i & 1));
      if (!valid) break;
      if (steps == 0) continue;
      wait_all(q_full, q_loads & 1);
      ++q_loads;
      uint32_t ks = next(), vs = 0;
      if (!ok) break;
      uint64_t kd = rows_desc(smem_u32(ring + ks * L::kTile)), vd = 0;
      if (n > 0) qk(kd);
      if (steps == 1) {
        commit(empty + ks);
        commit(q_empty);
      }
      for (int j = 0; j < steps && ok; ++j) {
        // step j of P.V behind step j + 1 of Q.K
        const bool more = j + 1 < steps;
        if ((j & 1) && more) {
          ks = next();
          kd = rows_desc(smem_u32(ring + ks * L::kTile));
        }
        if (j + 1 < n && ok) qk(kd + ((j + 1) & 1 ? kHalf : 0));
        if (more && ok && (!(j & 1) || j + 2 == steps)) {  // (its second half, or the last step)
          commit(empty + ks);
          if (j + 2 == steps) commit(q_empty);
        }
        if (!(j & 1)) {
          vs = next();
          vd = v_desc(smem_u32(ring + vs * L::kTile));
          if (!ok) break;
          if (j + 2 >= steps) {  // the item's last V block
            // In the sequence's last block the last MMA step's rows that belong to other
            // sequences are cleared.  (The cleaner hears of every item from both warps, so
            // that its waits are short and neither warp can pass a phase of its answers
            // unseen; an answer without rows is only waited for an item later.)
            const int live = lk - j * kStep;
            const bool dirty = live < kKeys && (live & 15);
            if (n_clean > 0) wait_all(v_clean, (n_clean - 1) & 1);
            if (lane == 0) {
              if (t == 0) *unclean = dirty ? vs * L::kTile + live * 128 : kNothing;
              mbar_arrive(v_dirty);
            }
            ++n_clean;
            if (dirty) wait_all(v_clean, (n_clean - 1) & 1);
          }
        }
        if (j < n && ok) pv(vd + (j & 1 ? kHalf : 0), lk - j * kStep, kDrain ? j % kDrainSteps == 0 : j == 0);
        if ((j & 1) || !more) commit(empty + vs);
      }
    }
    if (n_clean > 0) wait_all(v_clean, (n_clean - 1) & 1);
    if (lane == 0) {
      if (t == 0) *unclean = kNoMore;
      mbar_arrive(v_dirty);
    }
    commit(drained + t);  // nothing of this CTA's is in flight when the TMEM goes
    mbar_wait(drained + t, 0);
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ cleaner
    // Clears the rows of a V tile's last MMA step that lie behind its sequence's end: their
    // weights are 0, but 0 times another sequence's infinity or NaN is not.
    for (uint32_t n = 0; ok; ++n) {
      wait(v_dirty, n & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t from = *reinterpret_cast<volatile uint32_t*>(unclean);
      if (from == kNoMore) break;
      const int rows = from == kNothing ? 0 : 16 - (int)((from / 128) & 15);
      for (int e = lane; e < rows * 8 * (D / 64); e += 32)
        *reinterpret_cast<uint4*>(ring + from + (e >> 3) % rows * 128 + (e >> 3) / rows * L::kBox +
                                  (e & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_clean);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 2 * kStep, to = tmem + lanes + 4 * kStep + t * 128;
    const int tok = r / p.group, hh = r - tok * p.group;
    const float c = p.scale_log2;
    uint32_t n = 0;  // steps of this tile, of all items
    // Warps w and w + 4 (one of each tile) share a scheduler and its special-function unit.
    // They form their exponentials in turn, tile 0 first: one then loads, compares and stores
    // while the other keeps that unit busy.  Rounds count the longer tile's steps, so that both
    // take part in each.
    uint64_t* const my_turn = turn + warp;
    uint64_t* const other_turn = turn + (warp ^ 4);
    uint32_t round = 0;
    auto take_turn = [&]() {
      if (p.tiles == 2 && (t == 1 || round > 0)) wait(my_turn, (t == 1 ? round : round - 1) & 1);
    };
    auto pass_turn = [&]() {
      __syncwarp();
      if (p.tiles == 2 && lane == 0) mbar_arrive(other_turn);
      ++round;
    };
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
      float kept[D], m_kept = -INFINITY;  // what was drained from O (in local memory), its reference
      const int steps = it.n[t];
      const int rounds = p.tiles == 2 ? max(it.n[0], it.n[1]) : 0;
      for (int j = 0; j < steps; ++j, ++n) {
        const uint32_t buf = n & 1, tb = ts + buf * kStep;
        if (kDrain && j % kDrainSteps == 0 && j > 0) {  // (the step's P.V then begins O anew)
          wait(o_done + 2 * t + ((n - 1) & 1), ((n - 1) >> 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          drain<D>(to, kept, j > kDrainSteps ? ex2_ftz(m_kept - finite_ref(m)) : 0.f);
          m_kept = m;
        }
        wait(s_full + 2 * t + buf, (n >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[kStep];
        tmem_ld32(tb, s);
        tmem_ld32(tb + 32, s + 32);
        tmem_wait_ld();
        const int lim = seen - j * kStep;
        if (lim < kStep) {
#pragma unroll
          for (int e = 0; e < kStep; ++e)
            if (e >= lim) s[e] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kStep; e += 8)
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
            wait(o_done + 2 * t + ((n - 1) & 1), ((n - 1) >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
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
        take_turn();
        const float ref = kLift - finite_ref(m);
        const float2 c2 = make_float2(c, c), ref2 = make_float2(ref, ref);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < kStep; e += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, ref2);
          const bool by_fma = e / 2 % kPairsOf >= kPairsOf - kPairsByFma;
          const float2 w = by_fma ? exp2_fma(x) : make_float2(ex2_ftz(x.x), ex2_ftz(x.y));
          sum[e / 2 & 1] = add2(sum[e / 2 & 1], w);
          s[e >> 1] = pack2<T>(w.x, w.y);
        }
        pass_turn();
        tmem_st32(tb, s);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + 2 * t + buf);
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
      }
      for (int j = steps; j < rounds && ok; ++j) {
        take_turn();
        ok = __all_sync(0xffffffffu, ok);
        pass_turn();
      }
      if (!ok) break;
      const bool any = seen > 0;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // (0: every logit is -inf)
      const size_t row = (size_t)(it.q_row + t * tpt + tok) * p.h_q + it.head * p.group + hh;
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * (D * 2));
      if (steps > 0) {
        wait(o_done + 2 * t + ((n - 1) & 1), ((n - 1) >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (kDrain && steps > kDrainSteps) restore<D>(to, kept, ex2_ftz(m_kept - finite_ref(m)));
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
                w[x] = any ? pack2<T>(__uint_as_float(o[u + 2 * x]) * inv,
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
      if (live && p.lse) p.lse[row] = any ? (m - kLift + log2f(l)) * kLn2 : -INFINITY;
    }
    __threadfence();  // the results are visible before the next kernel may start
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
  griddep_launch_dependents();
}

template <int D, typename T, bool kDrain>
static cudaError_t launch_packed_k(const PackedAttnParams& p, cudaStream_t st) {
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
  auto* kernel = packed_attn_kernel<D, T, kDrain>;
  constexpr uint32_t smem = PackedSmem<D>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // At most this many items: full blocks of every sequence, and one partial block each.  Items
  // of one tile while they all find an SM of their own: a step of one tile takes 0.8 of the
  // time of a step of two (2000 tokens of 8 heads: 30.6 us against 36.7), but beyond one wave
  // two tiles per item are better (nine short prompts, 244 such items: 13.2 against 12.4;
  // 4000 tokens of 16 heads, 504: 84.8 against 60.5).
  const int sms = device_sm_count();
  auto items_of = [&](int tiles) { return ((long long)p.n_q / (tiles * tpt) + p.batch) * p.h_kv; };
  PackedAttnParams q = p;
  q.tiles = items_of(1) <= kOneTileUpTo * sms ? 1 : 2;
  const long long items = items_of(q.tiles);
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  return launch_pdl(kernel, dim3(grid), dim3(kPackedThreads), smem, st, tq, tk, tv, q);
}

// Calls without room for a sequence of more than kDrainSteps steps take the kernel that never
// drains: 12.7 us against 13.1 for nine short prompts, 58.2 against 58.9 for five after prefixes,
// 979 against 984 for one of 16384.
template <int D, typename T>
static cudaError_t launch_packed(const PackedAttnParams& p, cudaStream_t st) {
  return p.n_k > kDrainSteps * kStep ? launch_packed_k<D, T, true>(p, st) : launch_packed_k<D, T, false>(p, st);
}

cudaError_t launch_packed_attn(const PackedAttnParams& p, int head_dim, int dtype, cudaStream_t s) {
  if (head_dim == 128)
    return dtype == HS2_KV_F16 ? launch_packed<128, __half>(p, s) : launch_packed<128, __nv_bfloat16>(p, s);
  return dtype == HS2_KV_F16 ? launch_packed<64, __half>(p, s) : launch_packed<64, __nv_bfloat16>(p, s);
}

}  // namespace hs2
