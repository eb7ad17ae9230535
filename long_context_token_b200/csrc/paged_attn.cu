// Attention of one new token per sequence over a paged cache (grouped heads).
//
// Per key and K/V head the kernel reads two rows (K and V) and spends 4 D flop on each of
// the group's queries, so memory bounds it up to groups of about 64; the work is laid out
// to stream pages without a pause.  The 64-key tiles of all (sequence, K/V head) pairs form
// one line, cut into equal runs, one per persistent CTA (one CTA per SM), so ragged batches
// and single long sequences both fill the GPU.
//
//   producer warp  page table look-ups (a window of 32 entries ahead) and one TMA load per
//                  page and tensor into a ring of tiles (160 KB in flight per SM); float32
//                  scales of an FP8 cache by 4-byte asynchronous copies.
//   8 warps        flash decoding with mma.sync m16n8k16: 16 query heads of the group are
//                  the rows, 16 keys a step.  The tensor work is a few per cent of the
//                  time, and fragments in registers need no TMEM round trip per 64 keys,
//                  so tcgen05 would only lengthen each tile's chain.  The warps split the
//                  head tiles first, then the keys; each keeps its own reference, sums and
//                  outputs, joined through shared memory when a (sequence, head) pair ends.
//
// The softmax reference moves only when a logit passes it by more than 8 (log2 units), so a
// step has no shuffles.  An FP8 row's scale is folded into its weight: w = 2^(x - m) * s_v,
// with m following max(x + log2 s_v), so w <= 2^8 is rounded to float16 relative to the
// largest weight however the scales vary; E4M3 codes are exact in float16.  A bfloat16
// query against codes is brought to float16 by a power of two per head, exactly down to
// 2^-29 of its largest element.
//
// A pair cut between CTAs leaves partial results (m, l, o) in the workspace; the CTA that
// arrives last joins them in CTA order, so the result does not depend on timing.
#include "paged.cuh"
#include "sm100.cuh"
#include "tc_common.cuh"

namespace hs2 {

using namespace sm100;

namespace {

constexpr int kTileKeys = 64;
constexpr int kConsumers = 256;
constexpr int kPagedThreads = kConsumers + 32;
constexpr int kMinTiles = 2;  // a run is at least this many tiles
constexpr float kMoveAt = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <int D, bool kFp8>
struct PagedSmem {
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  static constexpr int kTile = kTileKeys * kRowBytes;  // K or V
  static constexpr int kScales = kFp8 ? 2 * kTileKeys * 4 : 0;
  static constexpr int kFit = 160 * 1024 / (2 * kTile + kScales);
  // Even: where two groups of warps take alternate tiles, each stage then always belongs to
  // the same group, which so waits for every phase of its barrier.  (A parity wait that skips
  // a phase passes too early when the skipped phase's data is late.)
  static constexpr int kStages = kFit > 16 ? 16 : kFit / 2 * 2;
  static constexpr uint32_t kScaleOff = kStages * 2 * kTile;
  static constexpr uint32_t kRedOff = kScaleOff + kStages * kScales;
  static constexpr uint32_t kMlOff = kRedOff + 8 * 16 * D * 4;  // [8 warps][16][2]
  static constexpr uint32_t kBarOff = kMlOff + 8 * 16 * 8;
  static constexpr uint32_t kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr uint32_t kBytes = kMiscOff + 128 + 1024;
  static_assert(kBytes <= 227 * 1024 && kStages % 2 == 0, "shared memory budget");
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
__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t two) {
  const __half2 h = e4m3x2_to_half2(two & 0xffffu);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One run of the tile line: where a CTA starts and how far it goes.
struct Run {
  long long total, per, begin, end;  // tiles
  int b;                             // sequence of tile `begin`
  long long b_first;                 // the line's tile at which that sequence starts
};

// A (sequence, K/V head) pair's part of the run, the same walk for all warps.
struct Segment {
  int b, h, len, t0, nt, tiles;  // tiles [t0, t0 + nt) of the pair's `tiles`
  long long first;               // the line's tile at which the pair starts
};

struct Walk {
  long long at, end, b_first;
  int b;
  __device__ bool next(const PagedAttnParams& p, Segment& s) {
    if (at >= end) return false;
    int len = paged_len(p.c, b, false);
    int tiles = (len + kTileKeys - 1) / kTileKeys;
    while (at >= b_first + (long long)tiles * p.c.h_kv) {  // (also over empty sequences)
      b_first += (long long)tiles * p.c.h_kv;
      ++b;
      len = paged_len(p.c, b, false);
      tiles = (len + kTileKeys - 1) / kTileKeys;
    }
    s.b = b;
    s.len = len;
    s.tiles = tiles;
    const long long in = at - b_first;
    s.h = (int)(in / tiles);
    s.t0 = (int)(in - (long long)s.h * tiles);
    s.first = b_first + (long long)s.h * tiles;
    s.nt = (int)min((long long)(tiles - s.t0), end - at);
    at += s.nt;
    return true;
  }
};

}  // namespace

template <int D, typename Q, bool kFp8>
__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, PagedAttnParams p) {
  using L = PagedSmem<D, kFp8>;
  constexpr int NS = L::kStages;
  constexpr int RB = L::kRowBytes;
  constexpr bool kBf16 = !kFp8 && !std::is_same<Q, __half>::value;  // the MMAs' type
  constexpr bool kScaleQ = kFp8 && !std::is_same<Q, __half>::value;
  constexpr int KS = D / 16;  // MMA steps along D
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* red = reinterpret_cast<float*>(smem + L::kRedOff);
  float2* red_ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + NS;
  long long* misc = reinterpret_cast<long long*>(smem + L::kMiscOff);  // [0..3] the run, [4..] scan
  int* flag = reinterpret_cast<int*>(smem + L::kMiscOff + 120);

  const int warp = threadIdx.x >> 5, lane = (int)lane_id();
  const int mt = p.group <= 16 ? 1 : p.group <= 32 ? 2 : p.group <= 64 ? 4 : 8;  // head tiles
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, kFp8 ? 33 : 1);
      mbar_init(empty + s, mt == 1 ? 4 : 8);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == kConsumers) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  griddep_wait();

  // ---- the run: a prefix sum of the sequences' tiles, kConsumers threads of `each` sequences
  {
    long long* sums = misc + 4;  // [8]
    const int each = (p.c.batch + kConsumers - 1) / kConsumers;
    long long mine = 0;
    const int b_lo = min((int)threadIdx.x * each, p.c.batch), b_hi = min(b_lo + each, p.c.batch);
    if (warp < 8)
      for (int b = b_lo; b < b_hi; ++b)
        mine += (paged_len(p.c, b, blockIdx.x == 0) + kTileKeys - 1) / kTileKeys;
    mine *= p.c.h_kv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (warp < 8 && lane == 31) sums[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    long long per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinTiles) per = kMinTiles;
    const long long begin = (long long)blockIdx.x * per;
    if (threadIdx.x == 0) {
      misc[0] = per;
      misc[1] = min(begin + per, total);
      misc[2] = 0;
      misc[3] = 0;
    }
    __syncthreads();
    if (warp < 8 && begin >= before && begin < before + mine) {
      int b = b_lo;
      for (;; ++b) {
        const long long n =
            (long long)((paged_len(p.c, b, false) + kTileKeys - 1) / kTileKeys) * p.c.h_kv;
        if (begin < before + n) break;
        before += n;
      }
      misc[2] = b;
      misc[3] = before;
    }
    __syncthreads();
  }
  const long long per = misc[0];
  Walk walk;
  walk.at = (long long)blockIdx.x * per;
  walk.end = misc[1];
  walk.b = (int)misc[2];
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

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    const int shift = p.c.page_shift;
    const int rows = min(1 << shift, kTileKeys);  // rows of one load
    const uint32_t box_bytes = (uint32_t)rows * RB;
    uint32_t slot = 0;
    while (ok && walk.next(p, s)) {
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
      int base = (s.t0 * kTileKeys) >> shift;
      int ids = load_pages(base), ids_next = load_pages(base + 32);
      for (int t = s.t0; t < s.t0 + s.nt; ++t, ++slot) {
        const int key0 = t * kTileKeys, keys = min(s.len - key0, kTileKeys);
        const int n = (keys + rows - 1) / rows;  // loads per tensor, at most 8
        if (((key0 + (n - 1) * rows) >> shift) >= base + 32) {
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
          tma_load_5d(dst, lane < 16 ? &tmap_k : &tmap_v, full + st, 0, key & ((1 << shift) - 1), 0,
                      s.h, id);
        }
        if constexpr (kFp8) {
          const uint32_t dst = smem_u32(smem + L::kScaleOff + st * L::kScales);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = lane + 32 * u, k = key0 + min(r, keys - 1);
            const int pg = __shfl_sync(0xffffffffu, ids, (k >> shift) - base);
            if (r < keys) {
              const int64_t at = pg * p.c.sc_page + s.h * p.c.sc_head + (k & ((1 << shift) - 1)) * p.c.sc_row;
              cp_async_4(dst + r * 4, p.c.k_scale + at);
              cp_async_4(dst + (kTileKeys + r) * 4, p.c.v_scale + at);
            }
          }
          cp_async_arrive(full + st);
        }
      }
    }
    // No load may outlive the CTA.
    for (uint32_t x = slot > NS ? slot - NS : 0; x < slot; ++x) mbar_wait(full + x % NS, (x / NS) & 1);
  } else {
    // ------------------------------------------------------------ consumers
    // Empty sequences have no tiles: their rows are written here, spread over the CTAs.
    for (int b = blockIdx.x; b < p.c.batch; b += gridDim.x) {
      if (paged_len(p.c, b, false) > 0) continue;
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (size_t)b * p.h_q * D * 2);
      for (int e = threadIdx.x; e < p.h_q * (D / 8); e += kConsumers) o[e] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int e = threadIdx.x; e < p.h_q; e += kConsumers) p.lse[(size_t)b * p.h_q + e] = -INFINITY;
    }
    const int m_tile = warp % mt, slice = warp / mt, slices = 8 / mt;
    const int blocks = mt <= 2 ? 1 : mt / 2;  // 16-key steps of a tile per warp
    const int c4 = lane & 3, r0 = lane >> 2;
    const int rshift = min(p.c.page_shift, 6);  // rows of one load, log2
    // Byte offset within a tile of 16-byte chunk `c` of key `r`, in the layout TMA wrote.
    auto at = [&](int r, int c) -> uint32_t {
      if constexpr (RB == 256)
        return ((uint32_t)(r >> rshift) << (rshift + 8)) + ((uint32_t)(c >> 3) << (rshift + 7)) +
               (uint32_t)(r & ((1 << rshift) - 1)) * 128u + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
      else if constexpr (RB == 128)
        return (uint32_t)r * 128u + (uint32_t)((c ^ (r & 7)) << 4);
      else
        return (uint32_t)r * 64u + (uint32_t)((c ^ ((r >> 1) & 3)) << 4);
    };
    uint32_t slot = 0;
    while (walk.next(p, s)) {
      // ---- queries: rows r0 and r0 + 8 of this warp's head tile
      uint32_t qa[KS][4];
      float f0 = 1.f, f1 = 1.f;  // 1 / the power of two that a query row was multiplied by
      {
        const int h0 = m_tile * 16 + r0;
        const uint8_t* q0 = p.q + (int64_t)s.b * p.q_seq + (int64_t)(s.h * p.group + h0) * p.q_head;
        const uint8_t* q1 = q0 + 8 * p.q_head;
        const bool v0 = h0 < p.group, v1 = h0 + 8 < p.group;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          // FP8: a step's 16 elements in the order of the codes' registers (4 per thread)
          const int e0 = 16 * k + (kFp8 ? 4 * c4 : 2 * c4), e1 = kFp8 ? e0 + 2 : e0 + 8;
          qa[k][0] = v0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 2 * e0)) : 0u;
          qa[k][1] = v1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + 2 * e0)) : 0u;
          qa[k][2] = v0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 2 * e1)) : 0u;
          qa[k][3] = v1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + 2 * e1)) : 0u;
        }
        if constexpr (kScaleQ) {
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float2 x = unpack2<Q>(qa[k][u]);
              float& a = u & 1 ? a1 : a0;
              a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
            a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
          }
          // The largest element lands in [2^14, 2^15): float16 keeps bfloat16's bits down to
          // 2^-14, its exponents down to 2^-24.
          auto to14 = [](float a, float& inverse) {
            int e = a > 0.f ? 14 - ilogbf(a) : 0;
            e = min(e, 100);  // (at least 14 - 127)
            inverse = exp2f((float)-e);
            return exp2f((float)e);
          };
          const float g0 = to14(a0, f0), g1 = to14(a1, f1);
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float2 x = unpack2<Q>(qa[k][u]);
              const float g = u & 1 ? g1 : g0;
              qa[k][u] = pack2<__half>(x.x * g, x.y * g);
            }
        }
      }
      f0 *= p.scale_log2;
      f1 *= p.scale_log2;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float o[D / 8][4];
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[n][u] = 0.f;

      for (int t = s.t0; t < s.t0 + s.nt; ++t, ++slot) {
        if (mt == 1 && (int)(slot & 1) != slice >> 2) continue;  // tiles alternate
        const uint32_t st = slot % NS;
        wait(full + st, (slot / NS) & 1);
        const uint32_t kt = smem_u32(smem + st * 2 * L::kTile), vt = kt + L::kTile;
        const float* ks = reinterpret_cast<const float*>(smem + L::kScaleOff + st * L::kScales);
        const int keys = min(s.len - t * kTileKeys, kTileKeys);
        const int blk0 = mt == 1 ? slice & 3 : slice * blocks;
        for (int blk = blk0; blk < blk0 + blocks; ++blk) {
          const int key = blk * 16;
          const int left = keys - key;  // keys of this step
          if (left <= 0) break;
          // ---- logits of 16 keys: two 8-key column tiles
          float sc[2][4] = {};
          {
            const int r = key + ((lane >> 4) << 3) + (lane & 7);
            if constexpr (!kFp8) {
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                uint32_t b[4];
                ldsm4(kt + at(r, 2 * k + ((lane >> 3) & 1)), b);
                mma16816<kBf16>(sc[0], qa[k], b[0], b[1]);
                mma16816<kBf16>(sc[1], qa[k], b[2], b[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < KS; k += 2) {
                uint32_t b[4];
                ldsm4(kt + at(r, k + ((lane >> 3) & 1)), b);
                mma16816<false>(sc[0], qa[k], cvt_e4m3x2(b[0]), cvt_e4m3x2(b[0] >> 16));
                mma16816<false>(sc[1], qa[k], cvt_e4m3x2(b[2]), cvt_e4m3x2(b[2] >> 16));
                mma16816<false>(sc[0], qa[k + 1], cvt_e4m3x2(b[1]), cvt_e4m3x2(b[1] >> 16));
                mma16816<false>(sc[1], qa[k + 1], cvt_e4m3x2(b[3]), cvt_e4m3x2(b[3] >> 16));
              }
            }
          }
          // ---- weights; column n * 8 + 2 c4 + e is a key
          float vs[4], ref_by[4];  // FP8: V's scale of the thread's four keys and its log2
          if constexpr (kFp8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int k = key + (u >> 1) * 8 + 2 * c4 + (u & 1);
              const float kk = ks[k];
              vs[u] = ks[kTileKeys + k];
              ref_by[u] = fmaxf(lg2(vs[u]), -64.f);
              sc[u >> 1][u & 1] *= kk;
              sc[u >> 1][2 + (u & 1)] *= kk;
            }
          }
          const bool partial = left < 16;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sc[n][e] *= f0;
              sc[n][2 + e] *= f1;
              if (partial && n * 8 + 2 * c4 + e >= left) {
                sc[n][e] = -INFINITY;
                sc[n][2 + e] = -INFINITY;
                if constexpr (kFp8) {
                  vs[2 * n + e] = 0.f;
                  ref_by[2 * n + e] = 0.f;
                }
              }
            }
          float t0, t1;
          if constexpr (kFp8) {
            t0 = fmaxf(fmaxf(sc[0][0] + ref_by[0], sc[0][1] + ref_by[1]),
                       fmaxf(sc[1][0] + ref_by[2], sc[1][1] + ref_by[3]));
            t1 = fmaxf(fmaxf(sc[0][2] + ref_by[0], sc[0][3] + ref_by[1]),
                       fmaxf(sc[1][2] + ref_by[2], sc[1][3] + ref_by[3]));
          } else {
            t0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
            t1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
          }
          if (__any_sync(0xffffffffu, t0 - m0 > kMoveAt || t1 - m1 > kMoveAt)) {
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
              t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
            }
            t0 = fmaxf(t0, m0);
            t1 = fmaxf(t1, m1);
            const float a0 = ex2_ftz(m0 - finite_ref(t0)), a1 = ex2_ftz(m1 - finite_ref(t1));
            m0 = t0;
            m1 = t1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][0] *= a0;
              o[n][1] *= a0;
              o[n][2] *= a1;
              o[n][3] *= a1;
            }
          }
          const float n0 = -finite_ref(m0), n1 = -finite_ref(m1);
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sc[n][e] = ex2_ftz(sc[n][e] + n0);
              sc[n][2 + e] = ex2_ftz(sc[n][2 + e] + n1);
              l0 += sc[n][e];
              l1 += sc[n][2 + e];
              if constexpr (kFp8) {
                sc[n][e] *= vs[2 * n + e];
                sc[n][2 + e] *= vs[2 * n + e];
              }
            }
          using W = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
          const uint32_t pa[4] = {pack2<W>(sc[0][0], sc[0][1]), pack2<W>(sc[0][2], sc[0][3]),
                                  pack2<W>(sc[1][0], sc[1][1]), pack2<W>(sc[1][2], sc[1][3])};
          // ---- o += weights x V; rows past the sequence's end are cleared (they may hold
          // anything, and 0 times an infinity is not 0)
          const int i0 = 2 * c4;
          const uint32_t v0 = !partial ? ~0u : (i0 < left ? 0xffffu : 0u) | (i0 + 1 < left ? 0xffff0000u : 0u);
          const uint32_t v1 = !partial ? ~0u : (i0 + 8 < left ? 0xffffu : 0u) | (i0 + 9 < left ? 0xffff0000u : 0u);
          const int r = key + (((lane >> 3) & 1) << 3) + (lane & 7);
          if constexpr (!kFp8) {
#pragma unroll
            for (int n = 0; n < D / 8; n += 2) {
              uint32_t b[4];
              ldsm4t(vt + at(r, n + (lane >> 4)), b);
              if (partial) {
                b[0] &= v0;
                b[1] &= v1;
                b[2] &= v0;
                b[3] &= v1;
              }
              mma16816<kBf16>(o[n], pa, b[0], b[1]);
              mma16816<kBf16>(o[n + 1], pa, b[2], b[3]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < D / 16; n += 2) {  // chunks of 16: even and odd elements apart
              uint32_t b[4];
              ldsm4t(vt + at(r, n + (lane >> 4)), b);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t e0 = cvt_e4m3x2(__byte_perm(b[2 * u], 0, 0x4420)), e1 = cvt_e4m3x2(__byte_perm(b[2 * u + 1], 0, 0x4420));
                uint32_t d0 = cvt_e4m3x2(__byte_perm(b[2 * u], 0, 0x4431)), d1 = cvt_e4m3x2(__byte_perm(b[2 * u + 1], 0, 0x4431));
                if (partial) {
                  e0 &= v0;
                  d0 &= v0;
                  e1 &= v1;
                  d1 &= v1;
                }
                mma16816<false>(o[2 * (n + u)], pa, e0, e1);
                mma16816<false>(o[2 * (n + u) + 1], pa, d0, d1);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st);
      }

      // ---- the pair's results of all warps, joined through shared memory
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, x);
        l1 += __shfl_xor_sync(0xffffffffu, l1, x);
      }
      if (c4 == 0) {
        red_ml[warp * 16 + r0] = make_float2(m0, l0);
        red_ml[warp * 16 + r0 + 8] = make_float2(m1, l1);
      }
      {
        // (16-byte chunks xored with the row, r0 = row mod 8, to spread rows over the banks)
        float* w0 = red + (warp * 16 + r0) * D;
        float* w1 = w0 + 8 * D;
        if constexpr (!kFp8) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const int f = (8 * n + 2 * c4) ^ (r0 << 2);
            *reinterpret_cast<float2*>(w0 + f) = make_float2(o[n][0], o[n][1]);
            *reinterpret_cast<float2*>(w1 + f) = make_float2(o[n][2], o[n][3]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            const int f = (16 * n + 4 * c4) ^ (r0 << 2);
            *reinterpret_cast<float4*>(w0 + f) =
                make_float4(o[2 * n][0], o[2 * n + 1][0], o[2 * n][1], o[2 * n + 1][1]);
            *reinterpret_cast<float4*>(w1 + f) =
                make_float4(o[2 * n][2], o[2 * n + 1][2], o[2 * n][3], o[2 * n + 1][3]);
          }
        }
      }
      named_bar_sync(1, kConsumers);
      const bool whole = s.nt == s.tiles;
      const size_t head0 = (size_t)s.b * p.h_q + s.h * p.group;  // row of the pair's first head
      const int part_stride = paged_part_floats(p.group, D);
      const int my_slot = 2 * blockIdx.x + (s.t0 == 0 && s.first != (long long)blockIdx.x * per ? 1 : 0);
      float* part = p.partials + (size_t)my_slot * part_stride;
      auto emit = [&](int hr, int d, float4 v, float m, float l) {  // a finished row's four elements
        const float inv = l > 0.f ? 1.f / l : 0.f;
        uint2 w = make_uint2(pack2<Q>(v.x * inv, v.y * inv), pack2<Q>(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (head0 + hr) * (D * 2) + d * 2) = w;
        if (d == 0 && p.lse) p.lse[head0 + hr] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      };
      for (int e = threadIdx.x; e < p.group * (D / 4); e += kConsumers) {
        const int hr = e / (D / 4), d = e % (D / 4) * 4;
        float m = -INFINITY;
        for (int x = 0; x < slices; ++x)
          m = fmaxf(m, red_ml[((hr >> 4) + mt * x) * 16 + (hr & 15)].x);
        float l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < slices; ++x) {
          const int row = ((hr >> 4) + mt * x) * 16 + (hr & 15);
          const float2 ml = red_ml[row];
          const float w = ex2_ftz(ml.x - finite_ref(m));  // 0 for a warp that saw no key
          const float4 u = *reinterpret_cast<const float4*>(red + row * D + (d ^ ((row & 7) << 2)));
          l = fmaf(w, ml.y, l);
          v.x = fmaf(w, u.x, v.x);
          v.y = fmaf(w, u.y, v.y);
          v.z = fmaf(w, u.z, v.z);
          v.w = fmaf(w, u.w, v.w);
        }
        if (whole) {
          emit(hr, d, v, m, l);
        } else {
          *reinterpret_cast<float4*>(part + hr * D + d) = v;
          if (d == 0) *reinterpret_cast<float2*>(part + p.group * D + 2 * hr) = make_float2(m, l);
        }
      }
      if (!whole) {
        const int c0 = (int)(s.first / per), c1 = (int)((s.first + s.tiles - 1) / per);
        uint32_t* counter = p.counters + (size_t)s.b * p.c.h_kv + s.h;
        __threadfence();
        named_bar_sync(1, kConsumers);
        if (threadIdx.x == 0) {
          const bool last = atomicAdd(counter, 1u) == (uint32_t)(c1 - c0);
          if (last) *counter = 0;
          *flag = last;
        }
        named_bar_sync(1, kConsumers);
        if (*flag) {
          __threadfence();
          auto slot_of = [&](int c) {
            return p.partials + (size_t)(2 * c + (c == c0 && s.first != (long long)c * per ? 1 : 0)) * part_stride;
          };
          for (int e = threadIdx.x; e < p.group * (D / 4); e += kConsumers) {
            const int hr = e / (D / 4), d = e % (D / 4) * 4;
            float m = -INFINITY;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c)
              m = fmaxf(m, __ldcg(slot_of(c) + p.group * D + 2 * hr));
            float l = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              const float* q = slot_of(c);
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(q + p.group * D + 2 * hr));
              const float4 u = __ldcg(reinterpret_cast<const float4*>(q + hr * D + d));
              const float w = ex2_ftz(ml.x - finite_ref(m));
              l = fmaf(w, ml.y, l);
              v.x = fmaf(w, u.x, v.x);
              v.y = fmaf(w, u.y, v.y);
              v.z = fmaf(w, u.z, v.z);
              v.w = fmaf(w, u.w, v.w);
            }
            emit(hr, d, v, m, l);
          }
        }
      } else {
        named_bar_sync(1, kConsumers);  // the buffers are read before the next pair's results
      }
    }
    __threadfence();  // the results are visible before the next kernel may start
  }
  __syncthreads();
  griddep_launch_dependents();
}

template <int D, typename Q, bool kFp8>
static cudaError_t launch_paged(const PagedAttnParams& p, cudaStream_t st) {
  using L = PagedSmem<D, kFp8>;
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
  auto* kernel = paged_attn_kernel<D, Q, kFp8>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const int tiles = (p.c.max_pages * page + kTileKeys - 1) / kTileKeys;
  const long long runs = ((long long)p.c.batch * p.c.h_kv * tiles + kMinTiles - 1) / kMinTiles;
  const int sms = device_sm_count() < kPagedMaxCtas ? device_sm_count() : kPagedMaxCtas;
  const unsigned grid = (unsigned)(runs < sms ? runs : sms);
  return launch_pdl(kernel, dim3(grid), dim3(kPagedThreads), L::kBytes, st, tk, tv, p);
}

template <int D>
static cudaError_t launch_paged_d(const PagedAttnParams& p, bool fp8, bool half, cudaStream_t s) {
  return fp8 ? (half ? launch_paged<D, __half, true>(p, s) : launch_paged<D, __nv_bfloat16, true>(p, s))
             : (half ? launch_paged<D, __half, false>(p, s) : launch_paged<D, __nv_bfloat16, false>(p, s));
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, int head_dim, int cache_dtype, int q_dtype,
                              cudaStream_t s) {
  const bool fp8 = cache_dtype == HS2_KV_FP8_E4M3, half = q_dtype == HS2_KV_F16;
  return head_dim == 128 ? launch_paged_d<128>(p, fp8, half, s) : launch_paged_d<64>(p, fp8, half, s);
}

}  // namespace hs2
