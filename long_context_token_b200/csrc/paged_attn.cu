// Attention of one new token per sequence over a paged cache (grouped heads).
//
// Per key and K/V head the kernel reads two rows (K and V) and spends 4 D flop on each of
// the group's queries, so memory bounds it up to groups of about 64; the work is laid out
// to stream pages without a pause.  The 32-key tiles of all (sequence, K/V head) pairs form
// one line, cut into equal runs, one per persistent CTA (one CTA per SM), so ragged batches
// and single long sequences both fill the GPU.
//
//   4 producer warps  take the run's tiles in turn: page table look-ups (a window of 32
//                  entries ahead), one TMA load per page and tensor into a ring of 128 KB,
//                  float32 scales of an FP8 cache by 4-byte asynchronous copies.  (One warp
//                  spends about 600 cycles on a tile, 1200 with scales: too slow alone.)
//   8 warps        attention with mma.sync m16n8k16, transposed: S^T = K Q^T with 16
//                  keys as the rows and 8 heads as the columns, O^T += V^T P^T, so a group
//                  of 7 or 8 heads wastes nothing and P goes from accumulator to operand
//                  by a transposing move within the warp.  The tensor work is a few per
//                  cent of the time, and fragments in registers need no TMEM round trip per
//                  tile, so tcgen05 would only lengthen each tile's chain.  A warp takes a
//                  whole tile for 8 or 16 heads; warps with the same heads take tiles in
//                  turn and keep their own references, sums and outputs, joined through
//                  shared memory when a (sequence, head) pair ends.
//
// The softmax reference moves only when a logit passes it by more than 8 (log2 units), so a
// tile has no shuffles.  A weight is rounded once, to the type of the second product: bfloat16,
// or float16 scaled so that the largest lies in [2^7, 2^15], half a step each down to 2^-21 of
// it and 2^-32 of it below.  (A second bfloat16 term for each weight, as the contiguous layers
// keep, brings results from 0.0024 of their size to 0.0017, their own rounding, and costs 3 % of
// the time with 16 heads per K/V head, 8 % with 128; it is left out.)  An FP8 row's scale is folded into its weight: w = 2^(x - m) * s_v,
// with m following max(x + log2 s_v) over the rows of V that are not all zeros, so w is rounded
// to float16 relative to the largest weight however the scales vary; E4M3 codes are exact in float16.  A bfloat16
// query against codes is brought to float16 by a power of two per head, exactly down to
// 2^-29 of its largest element.
//
// A pair cut between CTAs leaves partial results (m, l, o) in the workspace; the CTAs that
// arrive last join them, in CTA order and fixed groups, so the result does not depend on timing.
//
// What bounds it: memory while the runs last (7 TB/s of rows in the steady state), and 6 to
// 10 us of latencies around them: the run and the first pages (3 us), the join within the CTA,
// the arrival and the join of the parts (4 us).  On a B200, 8 x 131072 bfloat16 keys of one
// K/V head under 16 query heads: 91 us, 5.9 TB/s, 0.90 of the measured copy rate; 64
// sequences of 1 .. 8191 FP8 keys, 8 K/V heads under 64: 96 us, 5.2 TB/s, 0.80.  Groups of 32
// and more heads are bound by the products and conversions, which every 16 heads repeat: one
// sequence of 1048576 FP8 keys under 64 heads takes 188 us, 4.5 times its bytes' time, one of
// 131072 57 us (11 times), 64 of 8192 under 128 heads 178 us (8 times).
#include <atomic>

#include "paged.cuh"
#include "sm100.cuh"
#include "tc_common.cuh"

namespace hs2 {

using namespace sm100;

namespace {

constexpr int kTileKeys = 32;
constexpr int kConsumers = 256;
constexpr int kProducerWarps = 4;
constexpr int kPagedThreads = kConsumers + 32 * kProducerWarps;
// Registers per thread: launched with 168 (65536 / 384, in eights), 64512 in all.  With two
// 8-head tiles per warp the consumers then take 208 and the producers keep 88: 256 x 208 +
// 128 x 88 = 64512 (the launcher checks the kernel's count).
constexpr int kLaunchRegs = 168, kConsumerRegs = 208, kProducerRegs = 88;
constexpr int kJoinAtOnce = 512;  // rows (heads x partial results) that one CTA joins alone
constexpr int kDrainTiles = 512;  // tiles that a warp adds up before its outputs leave the registers
// A run is at least a tile for each warp.  (4096 bfloat16 keys, 16 heads on one: 12.6 us with 8,
// 13.7 with 4, 12.9 with 16; 16384 keys: 15.1, 16.1, 16.8; 1024 keys: 11.3, 10.3, 12.8.)
constexpr int kMinTiles = 8;
constexpr float kMoveAt = 8.0f;
constexpr float kNoScale = -64.f;  // log2 that stands for a V scale of 0 (and any below 2^-64)
constexpr float kLn2 = 0.69314718055994531f;

// NT: 8-head tiles per warp.
template <int D, bool kFp8, int NT>
struct PagedSmem {
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  static constexpr int kTile = kTileKeys * kRowBytes;  // K or V
  static constexpr int kScales = kFp8 ? 2 * kTileKeys * 4 : 0;
  // 128 KB of rows.  A multiple of 8 (and of the producer warps): warps that take tiles in
  // turn then always find theirs in the same stages, so they wait for every phase of those
  // stages' barriers.  (A parity wait that skips a phase passes too early when the skipped
  // phase's data is late.)
  static constexpr int kStages = 128 * 1024 / (2 * kTile);
  // A pair's own cost, in tiles: 128 KB of rows, at most 16 tiles (128 sequences of 1 .. 600
  // bfloat16 keys, 64 heads on 8, d 128: 40.5 us with 8 tiles, 53.8 with 4, 59.0 with 2; of
  // 1 .. 3000 FP8 keys, 32 on 4, d 64: 42.5 with 16, 46.0 with 32).
  static constexpr int kExtra = 128 * 1024 / (2 * kTile) > 16 ? 16 : 128 * 1024 / (2 * kTile);
  static constexpr uint32_t kScaleOff = kStages * 2 * kTile;
  static constexpr uint32_t kRedOff = kScaleOff + kStages * kScales;
  static constexpr uint32_t kRedFloats = 8 * 8 * NT * D;  // [8 warps][8 NT heads][D]
  static constexpr uint32_t kMlOff = kRedOff + kRedFloats * 4;  // [8 warps][8 NT heads] (m, l)
  static constexpr uint32_t kBarOff = kMlOff + 8 * 8 * NT * 8;
  static constexpr uint32_t kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr uint32_t kBytes = kMiscOff + 64 + 1024;
  static_assert(kBytes <= 227 * 1024 && kStages % 8 == 0 && kStages % kProducerWarps == 0,
                "shared memory budget");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four E4M3 codes as two float16 pairs: the low two, the high two.
__device__ __forceinline__ void cvt_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A (sequence, K/V head) pair's part of the run, the same walk for all warps.  A pair takes
// `extra` + tiles units of the line: starting and joining it costs a CTA about as long as
// `extra` tiles, so that a run of many short sequences gets fewer tiles.  A pair of at most
// `extra` tiles is not cut between runs.
struct Segment {
  int b, h, len, t0, nt, tiles;  // tiles [t0, t0 + nt) of the pair's `tiles`
  int first;                     // the line's unit at which the pair's tiles start
};

__device__ __forceinline__ int pair_tiles(const PagedAttnParams& p, int b, bool report) {
  return (paged_len(p.c, b, report) + kTileKeys - 1) / kTileKeys;
}

template <int kExtra>
struct Walk {
  int at, end;   // the rest of the run, in the line's units
  int b;         // sequence
  int b_first;   // the line's unit at which it starts
  __device__ bool next(const PagedAttnParams& p, Segment& s) {
    while (at < end) {
      const int len = paged_len(p.c, b, false);
      const int tiles = (len + kTileKeys - 1) / kTileKeys, units = tiles > 0 ? tiles + kExtra : 0;
      if (at >= b_first + units * p.c.h_kv) {  // (also over empty sequences)
        b_first += units * p.c.h_kv;
        ++b;
        continue;
      }
      s.b = b;
      s.len = len;
      s.tiles = tiles;
      const int in = at - b_first;
      s.h = in / units;
      const int from = in - s.h * units, to = min(units, from + (end - at));
      if (tiles <= kExtra) {  // not cut: all of it where it starts (joining parts costs more)
        s.t0 = 0;
        s.nt = from == 0 ? tiles : 0;
      } else {
        s.t0 = max(from - kExtra, 0);
        s.nt = max(to - kExtra, 0) - s.t0;
      }
      s.first = at - from + kExtra;
      at += to - from;
      if (s.nt > 0) return true;
    }
    return false;
  }
};

// Warps that share a key tile, each with 8 or 16 heads of the group.
__host__ __device__ __forceinline__ int head_tiles(int group) {
  return group <= 16 ? 1 : group <= 32 ? 2 : group <= 64 ? 4 : 8;
}

// Joins n partial results, in the order of their CTAs: part i is in slot 0 of CTA
// first + i * step, part 0 in slot 1 if that CTA begins the pair.  The result becomes the
// finished rows (out_rows, lse) or, with out_rows null, takes the place of part 0.
// Warp `warp` of 8 takes heads warp, warp + 8, ...; per 32 parts lane c holds the weight of
// part c, and the lanes share the head's elements, the first of which are on their way
// before the weights are known.  (A call of its own: inlined, its registers made the main
// loop spill.)
template <int D, typename Q>
__device__ __noinline__ void join_parts(float* partials, int part_floats, int first, int step,
                                        bool begins, int n, int group, int warp,
                                        uint8_t* out_rows, float* lse) {
  constexpr int E = D / 32;
  using Piece = typename std::conditional<E == 4, float4, float2>::type;
  const int lane = (int)lane_id();
  auto part = [&](int i) {
    return partials + (size_t)(2 * (first + i * step) + (i == 0 && begins ? 1 : 0)) * part_floats;
  };
  for (int hr = warp; hr < group; hr += 8) {
    float mm = -INFINITY, ll = 0.f, v[E] = {};
    for (int from = 0; from < n; from += 32) {
      const int k = min(n - from, 32);
      Piece u[8];
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < k)
            u[i] = __ldcg(reinterpret_cast<const Piece*>(part(from + c + i) + hr * D + lane * E));
      };
      fetch(0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < k) ml = __ldcg(reinterpret_cast<const float2*>(part(from + lane) + group * D + 2 * hr));
      const float top = fmaxf(mm, warp_max(ml.x)), ref = finite_ref(top);  // (-inf: all logits are)
      const float keep = ex2_ftz(mm - ref), w = ex2_ftz(ml.x - ref);
      ll = fmaf(ll, keep, warp_sum(w * ml.y));
      mm = top;
#pragma unroll
      for (int x = 0; x < E; ++x) v[x] *= keep;
      for (int c = 0; c < k; c += 8) {
        if (c > 0) fetch(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, (c + i) & 31);
          if (c + i < k) {
            const float* x = reinterpret_cast<const float*>(&u[i]);
#pragma unroll
            for (int y = 0; y < E; ++y) v[y] = fmaf(wi, x[y], v[y]);
          }
        }
      }
    }
    if (out_rows) {
      const float inv = ll != 0.f ? 1.f / ll : 0.f;  // (a NaN stays one)
      uint32_t* out = reinterpret_cast<uint32_t*>(out_rows + (size_t)hr * (D * 2)) + lane * (E / 2);
#pragma unroll
      for (int x = 0; x < E / 2; ++x) out[x] = pack2<Q>(v[2 * x] * inv, v[2 * x + 1] * inv);
      if (lse && lane == 0) lse[hr] = ll != 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    } else {
      // (this warp has read all of the head's parts)
      float* to = part(0);
#pragma unroll
      for (int x = 0; x < E; ++x) to[hr * D + lane * E + x] = v[x];
      if (lane == 0) *reinterpret_cast<float2*>(to + group * D + 2 * hr) = make_float2(mm, ll);
    }
  }
}

}  // namespace

// kDrain: a warp may have more than kDrainTiles tiles of a pair.
template <int D, typename Q, bool kFp8, int NT, bool kDrain>
__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, PagedAttnParams p) {
  using L = PagedSmem<D, kFp8, NT>;
  constexpr int NS = L::kStages;
  constexpr int RB = L::kRowBytes;
  constexpr bool kBf16 = !kFp8 && !std::is_same<Q, __half>::value;  // the MMAs' type
  constexpr bool kScaleQ = kFp8 && !std::is_same<Q, __half>::value;
  // Float16 weights are 2^7 times 2^(x - m): at most 2^15, as m lags by at most 8.  Without the
  // factor those below 2^-25 of the reference vanished from the output but not from the sum.
  constexpr float kLift = kBf16 ? 0.f : 7.f;
  constexpr int KS = D / 16;  // MMA steps along D
  constexpr int HT = 8 * NT;  // heads of a warp
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* red = reinterpret_cast<float*>(smem + L::kRedOff);
  float2* red_ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + NS;
  int* misc = reinterpret_cast<int*>(smem + L::kMiscOff);  // 0..3 the run, 4..11 scan, 12 flag

  const int warp = threadIdx.x >> 5, lane = (int)lane_id();
  // Warps that share the heads of a tile of the group, and warps per key tile.
  const int mt = NT == 1 ? 1 : head_tiles(p.group);
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, kFp8 ? 33 : 1);
      mbar_init(empty + s, mt);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == kConsumers) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  griddep_wait();

  // ---- the run: a prefix sum of the sequences' units, 256 threads of `each` sequences
  {
    const int each = (p.c.batch + 255) / 256;
    int mine = 0;
    const int b_lo = min((int)threadIdx.x * each, p.c.batch), b_hi = min(b_lo + each, p.c.batch);
    if (warp < 8)
      for (int b = b_lo; b < b_hi; ++b) {
        const int n = pair_tiles(p, b, blockIdx.x == 0);
        mine += n > 0 ? n + L::kExtra : 0;
      }
    mine *= p.c.h_kv;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (warp < 8 && lane == 31) misc[4 + warp] = incl;
    if (threadIdx.x == 0) misc[2] = misc[3] = 0;
    __syncthreads();
    int before = incl - mine, total = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += misc[4 + w];
      total += misc[4 + w];
    }
    const int per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinTiles);
    const int begin = (int)min((long long)blockIdx.x * per, (long long)total);
    if (threadIdx.x == 0) {
      misc[0] = per;
      misc[1] = (int)min((long long)begin + per, (long long)total);
    }
    if (warp < 8 && begin >= before && begin < before + mine) {
      int b = b_lo;
      for (;; ++b) {
        const int n = pair_tiles(p, b, false), units = (n > 0 ? n + L::kExtra : 0) * p.c.h_kv;
        if (begin < before + units) break;
        before += units;
      }
      misc[2] = b;
      misc[3] = before;
    }
    __syncthreads();
  }
  const int per = misc[0];
  Walk<L::kExtra> walk;
  walk.end = misc[1];
  walk.at = (int)min((long long)blockIdx.x * per, (long long)walk.end);
  walk.b = misc[2];
  walk.b_first = misc[3];
  bool ok = true;
  // A wait that gives up is recorded; the loops then run to their end without waiting (every
  // access stays in bounds, the results are undefined), so that no barrier misses a warp.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity)) {
      ok = false;
      set_status(p.c.status, HS2_ERR_DEVICE_TIMEOUT);
    }
  };
  Segment s;

  if (warp >= 8) {
    // ------------------------------------------------------------ producers
    reg_dec<kProducerRegs>();
    const int me = warp - 8;
    const int shift = p.c.page_shift, in_page = (1 << shift) - 1;
    const int rows = min(1 << shift, kTileKeys);  // rows of one load
    const uint32_t box_bytes = (uint32_t)rows * RB;
    uint32_t slot = 0;  // this run's tiles so far
    uint32_t mine = 0;  // of them, this warp's last one + 1 (0: none)
    while (ok && !p.stall_test && walk.next(p, s)) {
      const int32_t* table = p.c.pages + (size_t)s.b * p.c.max_pages;
      const int last_page = (s.len - 1) >> shift;
      auto load_pages = [&](int from) {
        int id = 0;
        if (from + lane <= last_page) {
          id = __ldg(table + from + lane);
          if (id < 0 || id >= p.c.num_pages) {
            set_status(p.c.status, HS2_ERR_INDEX_OUT_OF_RANGE);
            id = 0;
          }
        }
        return id;
      };
      // (a tile's pages never straddle two windows: both start at whole tiles)
      int base = (s.t0 * kTileKeys) >> shift;
      int ids = load_pages(base), ids_next = load_pages(base + 32);
      for (int t = s.t0; t < s.t0 + s.nt; ++t, ++slot) {
        if ((int)(slot % kProducerWarps) != me) continue;
        const int key0 = t * kTileKeys, keys = min(s.len - key0, kTileKeys);
        const int n = (keys + rows - 1) / rows;  // loads per tensor, at most 4
        while (((key0 + (n - 1) * rows) >> shift) >= base + 32) {
          base += 32;
          ids = ids_next;
          ids_next = load_pages(base + 32);
        }
        const uint32_t st = slot % NS;
        wait(empty + st, ((slot / NS) & 1) ^ 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full + st, 2 * n * box_bytes);
        __syncwarp();
        const int i = lane & 15, key = key0 + min(i, n - 1) * rows;
        const int id = __shfl_sync(0xffffffffu, ids, (key >> shift) - base);
        if (i < n) {
          const uint32_t dst = smem_u32(smem + st * 2 * L::kTile) + (lane < 16 ? 0 : L::kTile) +
                               i * box_bytes;
          tma_load_5d(dst, lane < 16 ? &tmap_k : &tmap_v, full + st, 0, key & in_page, 0, s.h, id);
        }
        if constexpr (kFp8) {
          const uint32_t dst = smem_u32(smem + L::kScaleOff + st * L::kScales) + lane * 4;
          const int k = key0 + min(lane, keys - 1);
          const int pg = __shfl_sync(0xffffffffu, ids, (k >> shift) - base);
          if (lane < keys) {
            const int64_t at = pg * p.c.sc_page + s.h * p.c.sc_head + (k & in_page) * p.c.sc_row;
            cp_async_4(dst, p.c.k_scale + at);
            cp_async_4(dst + kTileKeys * 4, p.c.v_scale + at);
          }
          cp_async_arrive(full + st);
        }
        mine = slot + 1;
      }
    }
    // No load may outlive the CTA: this warp's last fill of each of its stages.
    for (uint32_t x = mine; x > 0 && mine - x < NS; x -= min(x, (uint32_t)kProducerWarps))
      mbar_wait(full + (x - 1) % NS, ((x - 1) / NS) & 1);
  } else {
    // ------------------------------------------------------------ consumers
    reg_inc<kConsumerRegs>();
    // Empty sequences have no tiles: their rows are written here, spread over the CTAs.
    for (int b = blockIdx.x; b < p.c.batch; b += gridDim.x) {
      if (paged_len(p.c, b, false) > 0) continue;
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (size_t)b * p.h_q * D * 2);
      for (int e = threadIdx.x; e < p.h_q * (D / 8); e += kConsumers) o[e] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int e = threadIdx.x; e < p.h_q; e += kConsumers) p.lse[(size_t)b * p.h_q + e] = -INFINITY;
    }
    const int m_tile = warp % mt, turn = warp / mt, turns = 8 / mt;
    const int c4 = lane & 3, r8 = lane >> 2;
    // Byte offset within a tile of 16-byte chunk `c` of key `r`, in the layout TMA wrote: an
    // even chunk added to c only flips address bits 4..6 (and, in rows of 256 bytes, adds
    // half a load), so one offset per lane and 16 keys serves all chunks.
    const int rshift = min(p.c.page_shift, 5);  // rows of one load, log2
    const uint32_t half = 128u << rshift;       // rows of 256 bytes: from a row's half to the other
    auto at = [&](int r, int c) -> uint32_t {
      if constexpr (RB == 256)
        return ((uint32_t)(r >> rshift) << (rshift + 8)) + (uint32_t)(r & ((1 << rshift) - 1)) * 128u +
               (uint32_t)((c ^ (r & 7)) << 4);
      else if constexpr (RB == 128)
        return (uint32_t)r * 128u + (uint32_t)((c ^ (r & 7)) << 4);
      else
        return (uint32_t)r * 64u + (uint32_t)((c ^ ((r >> 1) & 3)) << 4);
    };
    auto chunk = [&](uint32_t a, int c) -> uint32_t {  // a + even chunk c
      if constexpr (RB == 256) return (a ^ (uint32_t)((c & 7) << 4)) + (c >= 8 ? half : 0u);
      return a ^ (uint32_t)(c << 4);
    };
    // This lane's rows and first chunks in ldmatrix of K (rows by 8s, then chunks) and V (16-bit:
    // chunks, then rows by 8s, so that the transposed fragment is V^T; codes: as K).
    uint32_t k_at[2], v_at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k_at[i] = at(16 * i + (((lane >> 3) & 1) << 3) + (lane & 7), lane >> 4);
      v_at[i] = kFp8 ? k_at[i] : at(16 * i + ((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1);
    }
    uint32_t slot = 0;
    // The 16-byte pieces of a pair's query rows (zeros behind the group's heads).
    const int pieces = mt * HT * (D / 8);
    auto q_piece = [&](const Segment& g, int e) {
      const int row = e / (D / 8), c = e % (D / 8);
      return row < p.group ? __ldg(reinterpret_cast<const uint4*>(
                                 p.q + (int64_t)g.b * p.q_seq +
                                 (int64_t)(g.h * p.group + row) * p.q_head + c * 16))
                           : make_uint4(0, 0, 0, 0);
    };
    auto put_piece = [&](int e, uint4 x) {
      const int row = e / (D / 8), c = e % (D / 8);
      reinterpret_cast<uint4*>(red)[row * (D / 8) + (c ^ (row & 7))] = x;
    };
    Segment after;
    bool have = walk.next(p, s), more;
    uint4 piece = make_uint4(0, 0, 0, 0);
    if (have && (int)threadIdx.x < pieces) piece = q_piece(s, threadIdx.x);
    for (; have; s = after, have = more) {
      // ---- queries, as the MMA's K x N operand: head r8 of each 8-head tile.  The pair's rows
      // go through the result buffer once for all warps, a row's 16-byte pieces xored with it.
      if ((int)threadIdx.x < pieces) put_piece(threadIdx.x, piece);
      for (int e = threadIdx.x + kConsumers; e < pieces; e += kConsumers) put_piece(e, q_piece(s, e));
      named_bar_sync(1, kConsumers);
      uint32_t qb[KS][NT][2];
      {
        const uint32_t qs = smem_u32(red) + (m_tile * HT) * (D * 2);
        auto piece_at = [&](int row, int c) -> uint32_t {
          return qs + row * (D * 2) + ((c ^ (row & 7)) << 4);
        };
        if constexpr (kFp8) {  // a step's 16 elements in the order of the codes' registers
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                           : "=r"(qb[k][n][0]), "=r"(qb[k][n][1])
                           : "r"(piece_at(n * 8 + r8, 2 * k + (c4 >> 1)) + (c4 & 1) * 8));
        } else if constexpr (NT == 2) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t w[4];
            ldsm4(piece_at(((lane >> 4) << 3) + (lane & 7), 2 * k + ((lane >> 3) & 1)), w);
            qb[k][0][0] = w[0], qb[k][0][1] = w[1], qb[k][1][0] = w[2], qb[k][1][1] = w[3];
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t w[4];
            ldsm4(piece_at(lane & 7, 2 * k + (lane >> 3)), w);
            qb[k][0][0] = w[0], qb[k][0][1] = w[1], qb[k + 1][0][0] = w[2], qb[k + 1][0][1] = w[3];
          }
        }
      }
      named_bar_sync(1, kConsumers);  // (the buffer is the results' again)
      float f[NT][2];  // factors of the logits of heads 2 c4 and 2 c4 + 1
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float g = 1.f;  // 1 / the power of two that this thread's head is multiplied by
        if constexpr (kScaleQ) {
          float top = 0.f;  // over the finite elements: an infinity stays one under any factor but 0
          auto size = [](float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.f; };
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 x = unpack2<Q>(qb[k][n][u]);
              top = fmaxf(top, fmaxf(size(x.x), size(x.y)));
            }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // The largest element lands in [2^14, 2^15): float16 keeps bfloat16's bits down to
          // 2^-14, its exponents down to 2^-24.
          const int e = top > 0.f ? min(14 - ilogbf(top), 100) : 0;
          const float by = exp2f((float)e);
          g = exp2f((float)-e);
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 x = unpack2<Q>(qb[k][n][u]);
              qb[k][n][u] = pack2<__half>(x.x * by, x.y * by);
            }
        }
        f[n][0] = p.scale_log2 * __shfl_sync(0xffffffffu, g, 8 * c4);
        f[n][1] = p.scale_log2 * __shfl_sync(0xffffffffu, g, 8 * c4 + 4);
      }
      float m[NT][2], l[NT][2];
      float o[KS][NT][4];  // 16 elements of D x 8 heads each
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) o[j][n][u] = 0.f;
      }

      // The outputs so far leave the MMAs' sum for this warp's part of the result buffer, which is
      // weighed by the move of the reference since (kept in red_ml); last: and come back to it.
      // (An MMA's sum is cut, not rounded: each of its products by up to 2^-25 of the sum, so a
      // sum over n keys lost n 2^-27 of itself.)
      int done = 0;  // tiles of this warp
      auto drain = [&](bool last) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = warp * HT + n * 8 + 2 * c4 + e;
            const bool first = done == kDrainTiles && !last;
            const float w = first ? 0.f : ex2_ftz(red_ml[row].x - finite_ref(m[n][e]));
            float* to = red + row * D;
            const int swz = c4 << 3;
            auto add = [&](float* at, float& x) {
              x = first ? x : fmaf(*at, w, x);
              if (!last) {
                *at = x;
                x = 0.f;
              }
            };
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              add(to + ((16 * j + (kFp8 ? 2 : 1) * r8) ^ swz), o[j][n][e]);
              add(to + ((16 * j + (kFp8 ? 2 * r8 + 1 : 8 + r8)) ^ swz), o[j][n][2 + e]);
            }
            __syncwarp();
            if (!last && r8 == 0) red_ml[row].x = m[n][e];
          }
        __syncwarp();
      };

      // The pair after this one, found (and its queries fetched) while this one's tiles come.
      more = walk.next(p, after);
      if (more && (int)threadIdx.x < pieces) piece = q_piece(after, threadIdx.x);

      for (int t = s.t0; t < s.t0 + s.nt; ++t, ++slot) {
        if ((int)(slot & (turns - 1)) != turn) continue;
        const uint32_t st = slot % NS;
        wait(full + st, (slot / NS) & 1);
        const uint32_t kt = smem_u32(smem + st * 2 * L::kTile), vt = kt + L::kTile;
        const float* ks = reinterpret_cast<const float*>(smem + L::kScaleOff + st * L::kScales);
        const int left = s.len - t * kTileKeys;  // keys of the tile (32 or more: all)
        // ---- logits: rows i * 16 + r8 (+ 8) are keys, columns heads
        float sc[2][NT][4] = {};
        const uint32_t ka[2] = {kt + k_at[0], kt + k_at[1]}, va[2] = {vt + v_at[0], vt + v_at[1]};
        if constexpr (!kFp8) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a[4];
              ldsm4(chunk(ka[i], 2 * k), a);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<kBf16>(sc[i][n], a, qb[k][n][0], qb[k][n][1]);
            }
        } else {
#pragma unroll
          for (int k = 0; k < KS; k += 2)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t w[4];
              ldsm4(chunk(ka[i], k), w);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t a[4];
                cvt_e4m3x4(w[2 * u], a[0], a[2]);
                cvt_e4m3x4(w[2 * u + 1], a[1], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma16816<false>(sc[i][n], a, qb[k + u][n][0], qb[k + u][n][1]);
              }
            }
        }
        // ---- logits in log2 units; keys past the sequence's end drop out
        float vs[2][2], ref_by[2][2];  // FP8: V's scales of the thread's keys and their log2
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = 16 * i + 8 * u + r8;
            float kk = 1.f;
            if constexpr (kFp8) {
              kk = ks[key];
              vs[i][u] = ks[kTileKeys + key];
              ref_by[i][u] = fmaxf(lg2(vs[i][u]), kNoScale);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float2 x = make_float2(sc[i][n][2 * u], sc[i][n][2 * u + 1]);
              if constexpr (kFp8) x = mul2(x, make_float2(kk, kk));
              x = mul2(x, make_float2(f[n][0], f[n][1]));
              sc[i][n][2 * u] = x.x;
              sc[i][n][2 * u + 1] = x.y;
            }
          }
        if (left < kTileKeys) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (16 * i + 8 * u + r8 >= left) {
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[i][n][2 * u] = sc[i][n][2 * u + 1] = -INFINITY;
                if constexpr (kFp8) vs[i][u] = ref_by[i][u] = 0.f;
              }
        }
        float top[NT][2];
        auto any_moves = [&]() {
          bool move = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                x[u] = sc[u >> 1][n][2 * (u & 1) + e];
                if constexpr (kFp8) x[u] += ref_by[u >> 1][u & 1];
              }
              top[n][e] = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
              move = move || top[n][e] - m[n][e] > kMoveAt;
            }
          return (bool)__any_sync(0xffffffffu, move);
        };
        bool moves = any_moves();
        if (kFp8 && moves) {
          // A row of zeros in V adds nothing whatever its scale (1, from hs2_paged_kv_write): it
          // must not take the reference along, so it counts as one with scale 0.
          uint32_t bits = 0;
#pragma unroll
          for (int c = 0; c < RB / 16; ++c) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(vt + at(lane, c)));
            bits |= w[0] | w[1] | w[2] | w[3];
          }
          const uint32_t zero = __ballot_sync(0xffffffffu, (bits & 0x7f7f7f7fu) == 0);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (zero >> (16 * i + 8 * u + r8) & 1) {
                vs[i][u] = 0.f;
                ref_by[i][u] = kNoScale;
              }
          if (zero) moves = any_moves();
        }
        if (moves) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = top[n][e];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
              x = fmaxf(x, m[n][e]);
              const float a = ex2_ftz(m[n][e] - finite_ref(x));
              m[n][e] = x;
              l[n][e] *= a;
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                o[j][n][e] *= a;
                o[j][n][2 + e] *= a;
              }
            }
        }
        // ---- weights, transposed into the second product's K x N operand
        using W = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float n0 = kLift - finite_ref(m[n][0]), n1 = kLift - finite_ref(m[n][1]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float a = ex2_ftz(sc[i][n][2 * u] + n0), b = ex2_ftz(sc[i][n][2 * u + 1] + n1);
              l[n][0] += a;
              l[n][1] += b;
              if constexpr (kFp8) {
                a *= vs[i][u];
                b *= vs[i][u];
              }
              pb[i][n][u] = transpose8x8(pack2<W>(a, b));
            }
        }
        // ---- O^T += V^T P^T
        auto pv = [&](auto tail) {
          // In the last tile, V's rows past the end are cleared (they may hold anything, and
          // 0 times an infinity is not 0).
          auto live = [&](int key) -> uint32_t {
            return (key < left ? 0xffffu : 0u) | (key + 1 < left ? 0xffff0000u : 0u);
          };
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v0 = live(16 * i + 2 * c4), v1 = live(16 * i + 8 + 2 * c4);
            auto cut = [&](uint32_t (&a)[4]) {
              if constexpr (decltype(tail)::value) {
                a[0] &= v0;
                a[1] &= v0;
                a[2] &= v1;
                a[3] &= v1;
              }
            };
            if constexpr (!kFp8) {
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                uint32_t a[4];
                ldsm4t(chunk(va[i], 2 * j), a);
                cut(a);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<kBf16>(o[j][n], a, pb[i][n][0], pb[i][n][1]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < KS; j += 2) {
                uint32_t w[4];
                ldsm4t(chunk(va[i], j), w);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  // rows 0..7 are a chunk's even elements, rows 8..15 its odd ones
                  uint32_t a[4];
                  cvt_e4m3x4(__byte_perm(w[2 * u], 0, 0x3120), a[0], a[1]);
                  cvt_e4m3x4(__byte_perm(w[2 * u + 1], 0, 0x3120), a[2], a[3]);
                  cut(a);
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma16816<false>(o[j + u][n], a, pb[i][n][0], pb[i][n][1]);
                }
              }
            }
          }
        };
        if (left >= kTileKeys)
          pv(std::false_type{});
        else
          pv(std::true_type{});
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st);
        if (kDrain && ++done % kDrainTiles == 0) drain(false);
      }
      if (kDrain && done >= kDrainTiles) drain(true);

      // ---- the pair's results of all warps, joined through shared memory
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[n][e];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
          const int row = warp * HT + n * 8 + 2 * c4 + e;
          if (r8 == 0) red_ml[row] = make_float2(m[n][e] - kLift, x);
          // (elements xored with the head, to spread the heads over the banks)
          float* to = red + row * D;
          const int swz = c4 << 3;
#pragma unroll
          for (int j = 0; j < KS; ++j)
            if constexpr (!kFp8) {
              to[(16 * j + r8) ^ swz] = o[j][n][e];
              to[(16 * j + 8 + r8) ^ swz] = o[j][n][2 + e];
            } else {
              *reinterpret_cast<float2*>(to + ((16 * j + 2 * r8) ^ swz)) =
                  make_float2(o[j][n][e], o[j][n][2 + e]);
            }
        }
      named_bar_sync(1, kConsumers);
      const bool whole = s.nt == s.tiles;
      const size_t head0 = (size_t)s.b * p.h_q + s.h * p.group;  // row of the pair's first head
      const int part_floats = paged_part_floats(p.group, D);
      // Partial results: slot 2c holds CTA c's part of a pair that began before it, slot
      // 2c + 1 its part of one that it begins and does not end.
      auto part_of = [&](int c, bool begins) {
        return p.partials + (size_t)(2 * c + (begins ? 1 : 0)) * part_floats;
      };
      float* part = part_of(blockIdx.x, s.t0 == 0);
      auto emit = [&](int hr, int d, float4 v, float m, float l) {  // a finished row's four elements
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint2 w = make_uint2(pack2<Q>(v.x * inv, v.y * inv), pack2<Q>(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (head0 + hr) * (D * 2) + d * 2) = w;
        if (d == 0 && p.lse) p.lse[head0 + hr] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      };
      auto join = [&](auto warps_of_a_head) {
        constexpr int N = decltype(warps_of_a_head)::value;
        for (int e = threadIdx.x; e < p.group * (D / 4); e += kConsumers) {
          const int hr = e / (D / 4), d = e % (D / 4) * 4;
          const int swz = ((hr >> 1) & 3) << 3;
          float2 ml[N];
          float4 u[N];
#pragma unroll
          for (int x = 0; x < N; ++x) {
            const int row = hr + x * (8 / N) * HT;  // 8 / N head tiles
            ml[x] = red_ml[row];
            u[x] = *reinterpret_cast<const float4*>(red + row * D + (d ^ swz));
          }
          float mm = ml[0].x;
#pragma unroll
          for (int x = 1; x < N; ++x) mm = fmaxf(mm, ml[x].x);
          float ll = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < N; ++x) {
            const float w = ex2_ftz(ml[x].x - finite_ref(mm));  // 0 for a warp that saw no key
            ll = fmaf(w, ml[x].y, ll);
            v.x = fmaf(w, u[x].x, v.x);
            v.y = fmaf(w, u[x].y, v.y);
            v.z = fmaf(w, u[x].z, v.z);
            v.w = fmaf(w, u[x].w, v.w);
          }
          if (whole) {
            emit(hr, d, v, mm, ll);
          } else {
            *reinterpret_cast<float4*>(part + hr * D + d) = v;
            if (d == 0) *reinterpret_cast<float2*>(part + p.group * D + 2 * hr) = make_float2(mm, ll);
          }
        }
      };
      if (NT == 1 || mt == 1)
        join(std::integral_constant<int, 8>{});
      else if (mt == 2)
        join(std::integral_constant<int, 4>{});
      else if (mt == 4)
        join(std::integral_constant<int, 2>{});
      else
        join(std::integral_constant<int, 1>{});
      named_bar_sync(1, kConsumers);  // the buffers are read; the partial result is written
      if (!whole) {
        // The n parts of the pair are joined by the CTA that arrives last; with more than
        // kJoinAtOnce rows in them first in groups of r neighbours, each by the last CTA of the
        // group, and then the groups' results by the last of those.  (One CTA alone took 15 us
        // longer over the 148 parts of a sequence of 131072 keys under 16 heads, 64 us longer
        // under 64.)
        const int c0 = s.first / per, n = (s.first + s.tiles - 1) / per - c0 + 1;
        const int r = n * p.group <= kJoinAtOnce ? n : (int)ceilf(sqrtf((float)n)), groups = (n + r - 1) / r;
        const int g = ((int)blockIdx.x - c0) / r, g0 = c0 + g * r, members = min(r, n - g * r);
        // Whether this CTA is the last of `of` to count up `counter`.
        auto last_of = [&](uint32_t* counter, int of) {
          if (threadIdx.x == 0) {
            const bool last = atom_add_acq_rel_gpu(counter, 1u) == (uint32_t)(of - 1);
            if (last) *counter = 0;
            misc[12] = last;
          }
          named_bar_sync(1, kConsumers);
          const bool last = misc[12];
          named_bar_sync(1, kConsumers);  // (misc is free again, all writes before are done)
          return last;
        };
        uint8_t* out_rows = static_cast<uint8_t*>(p.out) + head0 * (D * 2);
        float* lse_rows = p.lse ? p.lse + head0 : nullptr;
        // (Counters by CTA: one that begins a group of two or more neither begins nor ends
        // another pair's group, and one CTA begins at most one pair that it does not end.)
        bool last = members == 1 || last_of(p.counters + g0, members);
        if (last && groups > 1) {
          if (members > 1) {
            join_parts<D, Q>(p.partials, part_floats, g0, 1, g == 0, members, p.group, warp, nullptr, nullptr);
            named_bar_sync(1, kConsumers);
          }
          last = last_of(p.counters + kPagedMaxCtas + c0, groups);
        }
        if (last)
          join_parts<D, Q>(p.partials, part_floats, c0, groups > 1 ? r : 1, true, groups > 1 ? groups : n,
                           p.group, warp, out_rows, lse_rows);
      }
    }
    __threadfence();  // the results are visible before the next kernel may start
  }
  __syncthreads();
  griddep_launch_dependents();
}

template <int D, typename Q, bool kFp8, int NT, bool kDrain>
static cudaError_t launch_paged_k(const PagedAttnParams& p, unsigned grid, cudaStream_t st) {
  using L = PagedSmem<D, kFp8, NT>;
  const int page = 1 << p.c.page_shift, inner = L::kRowBytes >= 128 ? 128 : L::kRowBytes;
  const int elt = kFp8 ? 1 : 2;
  auto stride = [](int n, int64_t s) { return n > 1 ? (uint64_t)s : uint64_t(16); };
  // A row as (halves of) 128 bytes, the rows of a page, heads, pages.
  const uint64_t dims[5] = {(uint64_t)(inner / elt), (uint64_t)page, (uint64_t)(L::kRowBytes / inner),
                            (uint64_t)p.c.h_kv, (uint64_t)p.c.num_pages};
  const uint64_t strides[4] = {(uint64_t)p.c.row_stride, 128, stride(p.c.h_kv, p.c.head_stride),
                               stride(p.c.num_pages, p.c.page_stride)};
  const uint32_t box[5] = {(uint32_t)(inner / elt), (uint32_t)(page < kTileKeys ? page : kTileKeys),
                           (uint32_t)(L::kRowBytes / inner), 1, 1};
  const CUtensorMapDataType dt = kFp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const CUtensorMapSwizzle sw = inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUtensorMap tk, tv;
  if (!make_tmap_nd(&tk, p.c.k, dt, 5, dims, strides, box, sw) ||
      !make_tmap_nd(&tv, p.c.v, dt, 5, dims, strides, box, sw))
    return cudaErrorInvalidValue;
  auto* kernel = paged_attn_kernel<D, Q, kFp8, NT, kDrain>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  // With fewer registers at launch the consumers would wait for more for good.  (The tests hold
  // the build to the number; this is for builds that nobody tested.)
  static std::atomic<bool> checked{false};  // (two threads may both check)
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    const cudaError_t q = cudaFuncGetAttributes(&a, kernel);
    if (q != cudaSuccess) return q;
    if (a.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  return launch_pdl(kernel, dim3(grid), dim3(kPagedThreads), L::kBytes, st, tk, tv, p);
}

template <int D, typename Q, bool kFp8, int NT>
static cudaError_t launch_paged(const PagedAttnParams& p, cudaStream_t st) {
  const long long tiles = (((long long)p.c.max_pages << p.c.page_shift) + kTileKeys - 1) / kTileKeys;
  const long long pairs = (long long)p.c.batch * p.c.h_kv, runs = (pairs * tiles + kMinTiles - 1) / kMinTiles;
  const int sms = device_sm_count() < kPagedMaxCtas ? device_sm_count() : kPagedMaxCtas;
  const unsigned grid = (unsigned)(runs < sms ? runs : sms);
  // The most tiles of one pair that a CTA can meet: all of a sequence that fills its pages, or a
  // run of a batch of such.  While no warp's share is above kDrainTiles (131072 keys in a CTA of up
  // to 16 heads a pair, 16384 of more than 64), the kernel need not drain: 12.85 us against 13.16
  // for one sequence of 4096 bfloat16 keys, 101 against 103 for 64 of 1 .. 8191 FP8 keys.
  const long long run = (pairs * (tiles + PagedSmem<D, kFp8, NT>::kExtra) + grid - 1) / grid;
  const bool drain = (tiles < run ? tiles : run) > (long long)kDrainTiles * (8 / head_tiles(p.group));
  return drain ? launch_paged_k<D, Q, kFp8, NT, true>(p, grid, st)
               : launch_paged_k<D, Q, kFp8, NT, false>(p, grid, st);
}

// Groups of up to 8 heads take the kernel with one head tile per warp: half the products
// and registers of the one with two, which serves larger groups without reading a tile's
// rows from shared memory once per 8 heads.
template <int D, typename Q, bool kFp8>
static cudaError_t launch_paged_n(const PagedAttnParams& p, cudaStream_t st) {
  return p.group <= 8 ? launch_paged<D, Q, kFp8, 1>(p, st) : launch_paged<D, Q, kFp8, 2>(p, st);
}

template <int D>
static cudaError_t launch_paged_d(const PagedAttnParams& p, bool fp8, bool half, cudaStream_t s) {
  return fp8 ? (half ? launch_paged_n<D, __half, true>(p, s) : launch_paged_n<D, __nv_bfloat16, true>(p, s))
             : (half ? launch_paged_n<D, __half, false>(p, s) : launch_paged_n<D, __nv_bfloat16, false>(p, s));
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, int head_dim, int cache_dtype, int q_dtype,
                              cudaStream_t s) {
  const bool fp8 = cache_dtype == HS2_KV_FP8_E4M3, half = q_dtype == HS2_KV_F16;
  return head_dim == 128 ? launch_paged_d<128>(p, fp8, half, s) : launch_paged_d<64>(p, fp8, half, s);
}

}  // namespace hs2
