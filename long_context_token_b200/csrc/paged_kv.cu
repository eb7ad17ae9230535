// Moving rows in and out of a paged cache: hs2_paged_kv_write (16-bit rows copied, FP8 rows
// quantised with their own scale) and hs2_paged_kv_read (the way back, dequantised).
//
// Both only move bytes: per row of d elements 2d bytes on the packed side and 2d (16-bit)
// or d + 4 (E4M3 code and float32 scale) in the pages.  A CTA takes a run of tokens: one
// thread per token first looks up the token's sequence, position and page (four dependent
// loads), once for all its heads.  Then a thread moves 16 elements of the K row and of the V
// row of a (token, head) pair at a time and loads the next pair before it converts and
// stores this one; an E4M3 row is a whole number of 16-byte pieces.
//
// A division per element bound the writing of FP8 rows (145 us where it now takes 82), so the
// quotients of a row, which share their divisor, are formed from its reciprocal and corrected
// twice by their remainder: Markstein's method ("Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990), which gives the correctly rounded quotient from one
// within a unit in the last place and the correctly rounded reciprocal.
//
// What bounds them: memory, and about 5 us of look-ups and tail.  On a B200: 65K tokens of 8
// heads (d 128, bfloat16) into an FP8 cache 82 us, 4.9 TB/s, 0.75 of the measured copy rate;
// 67K tokens back 75 us, 5.5 TB/s, 0.84; a single token 2.2 us.  16-bit rows, 61512 tokens: 90 us
// in and 89 out, 0.85 and 0.86.  The order of a page's rows and heads makes no difference: pages
// with the heads of a token side by side, as the threads walk them, take 76.6 us where pages
// with a head's tokens side by side take 77.3.
#include "paged.cuh"

namespace hs2 {

constexpr int kMoveThreads = 256;
constexpr int kMaxTokensPerCta = 512;
// (Three, which end the spills of the FP8 write: 79.5 us to write 61512 tokens of 8 heads, 72.8 to
// read them back; with four 77.3 and 69.6.)
constexpr int kMoveCtasPerSm = 4;

struct TokenSlot {
  int page;  // -1: nothing to move for this token
  int row;
};

// Page and row of packed token t, or page -1 (padding, or an error that is recorded).
template <bool kWrite>
__device__ __forceinline__ TokenSlot token_slot(const PagedMoveParams& p, int t) {
  TokenSlot s = {-1, 0};
  int b, first, n;
  if (p.cu) {
    b = find_sequence(p.cu, p.c.batch, t);
    first = __ldg(p.cu + b);
    n = __ldg(p.cu + b + 1) - first;
    if (t < first || t - first >= n) return s;  // padding behind the last sequence
  } else {
    b = t / p.uniform;
    first = b * p.uniform;
    n = p.uniform;
  }
  const int L = __ldg(p.c.lens + b), cap = p.c.max_pages << p.c.page_shift;
  long long pos = t - first;
  bool ok = L >= 0 && L <= cap;
  if (kWrite) {
    ok = ok && L >= n;
    pos += L - n;
  } else {
    if (p.start) pos += __ldg(p.start + b);
    ok = ok && pos >= 0 && pos < L;
  }
  if (!ok) {
    set_status(p.c.status, HS2_ERR_BAD_LENGTH);
    return s;
  }
  const int page = __ldg(p.c.pages + (size_t)b * p.c.max_pages + (size_t)(pos >> p.c.page_shift));
  if (page < 0 || page >= p.c.num_pages) {
    set_status(p.c.status, HS2_ERR_INDEX_OUT_OF_RANGE);
    return s;
  }
  s.page = page;
  s.row = (int)(pos & ((1 << p.c.page_shift) - 1));
  return s;
}

// Two E4M3 codes, rounded to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3_pair(float2 y) {
  return __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
}
// -x / s, correctly rounded, from nr = -1 / s rounded: the product is within 1.5 units in the
// last place, so within one after the first correction and rounded correctly after the
// second.  (The negated quotient keeps the sign of zeros through the corrections.)  Every
// remainder that matters is exact while s is finite and at least 2^-60; other rows are
// divided out.
__device__ __forceinline__ float2 minus_quotient(float2 x, float2 s, float2 nr) {
  float2 y = mul2(x, nr);
  y = fma2(fma2(y, s, x), nr, y);
  return fma2(fma2(y, s, x), nr, y);
}
// The larger magnitudes of two 16-bit pairs, element by element.
template <typename T>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&a)),
                              __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
  } else {
    const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}

// D: head_dim; T: the packed rows' type; kFp8: the cache holds E4M3 codes and scales.
template <int D, typename T, bool kFp8, bool kWrite>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtasPerSm) paged_move_kernel(PagedMoveParams p) {
  __shared__ TokenSlot slots[kMaxTokensPerCta];
  constexpr int kLanes = D / 16;  // threads of one pair of rows, 16 elements each
  constexpr int kStep = kMoveThreads / kLanes;
  // A thread's 16 elements are 8 of each half of a row, so that every access of a row's
  // threads together covers whole 32-byte sectors: a 16-byte piece of each half, or 8 bytes
  // of codes.
  constexpr int kRowHalf = D * (kFp8 ? 1 : 2) / 2, kPackedHalf = D;  // bytes
  using Cell = typename std::conditional<kFp8 && !kWrite, uint2, uint4>::type;  // as read
  constexpr int kReadHalf = kWrite ? kPackedHalf : kRowHalf;
  griddep_wait();
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.n_tokens - t0);
  for (int t = threadIdx.x; t < nt; t += kMoveThreads) slots[t] = token_slot<kWrite>(p, t0 + t);
  __syncthreads();
  const int c = threadIdx.x % kLanes, h_kv = p.c.h_kv;
  const int step_i = kStep / h_kv, step_h = kStep - step_i * h_kv;
  int i = (int)(threadIdx.x / kLanes) / h_kv, h = (int)(threadIdx.x / kLanes) - i * h_kv;

  struct Pair {
    bool live;
    int64_t packed, paged, scale;  // offsets of the rows (this thread's piece) and of the scale
    Cell k[2], v[2];
    float ks, vs;
  };
  auto fetch = [&](Pair& x) {  // the pair (i, h), and on to this thread's next one
    x.live = i < nt;
    if (x.live) {
      const TokenSlot s = slots[i];
      x.live = s.page >= 0;
      if (x.live) {
        x.packed = (int64_t)(t0 + i) * p.token_stride + h * p.head_stride + c * 16;
        x.paged = s.page * p.c.page_stride + h * p.c.head_stride + s.row * p.c.row_stride +
                  c * (kFp8 ? 8 : 16);
        if constexpr (kFp8) x.scale = s.page * p.c.sc_page + h * p.c.sc_head + s.row * p.c.sc_row;
        const uint8_t* k = kWrite ? p.k_src + x.packed : p.c.k + x.paged;
        const uint8_t* v = kWrite ? p.v_src + x.packed : p.c.v + x.paged;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x.k[u] = *reinterpret_cast<const Cell*>(k + u * kReadHalf);
          x.v[u] = *reinterpret_cast<const Cell*>(v + u * kReadHalf);
        }
        if constexpr (kFp8 && !kWrite) {
          x.ks = p.c.k_scale[x.scale];
          x.vs = p.c.v_scale[x.scale];
        }
      }
    }
    i += step_i;
    h += step_h;
    if (h >= h_kv) {
      h -= h_kv;
      ++i;
    }
  };
  auto quantise = [&](const Cell (&w)[2], uint8_t* row, float* scale, uint32_t mask) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = absmax2<T>(top, u[e]);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      top = absmax2<T>(top, __shfl_xor_sync(mask, top, o));
    const float2 both = unpack2<T>(top);
    const float amax = fmaxf(both.x, both.y);
    const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    const float nr = -__frcp_rn(s);
    const float2 s2 = make_float2(s, s), nr2 = make_float2(nr, nr);
    uint32_t code[4];
    if (s >= 0x1p-60f && s < INFINITY) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        code[e] = (e4m3_pair(minus_quotient(unpack2<T>(u[2 * e]), s2, nr2)) |
                   (e4m3_pair(minus_quotient(unpack2<T>(u[2 * e + 1]), s2, nr2)) << 16)) ^ 0x80808080u;
    } else {  // tiny rows, and rows with an infinity
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = unpack2<T>(u[2 * e]), z = unpack2<T>(u[2 * e + 1]);
        code[e] = e4m3_pair(make_float2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s))) |
                  (e4m3_pair(make_float2(__fdiv_rn(z.x, s), __fdiv_rn(z.y, s))) << 16);
      }
    }
    *reinterpret_cast<uint2*>(row) = make_uint2(code[0], code[1]);
    *reinterpret_cast<uint2*>(row + kRowHalf) = make_uint2(code[2], code[3]);
    if (c == 0) *scale = s;
  };
  auto widen = [&](const Cell (&w)[2], float s, uint8_t* row) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 x = __half22float2(e4m3x2_to_half2((u[e >> 1] >> (16 * (e & 1))) & 0xffffu));
      o[e] = pack2<T>(x.x * s, x.y * s);
    }
    *reinterpret_cast<uint4*>(row) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(row + kPackedHalf) = make_uint4(o[4], o[5], o[6], o[7]);
  };
  auto put = [&](const Pair& x) {
    if (!x.live) return;  // (the threads of a pair are live together)
    uint8_t* k = kWrite ? p.c.k + x.paged : p.k_dst + x.packed;
    uint8_t* v = kWrite ? p.c.v + x.paged : p.v_dst + x.packed;
    if constexpr (!kFp8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        *reinterpret_cast<uint4*>(k + u * kRowHalf) = x.k[u];
        *reinterpret_cast<uint4*>(v + u * kRowHalf) = x.v[u];
      }
    } else if constexpr (kWrite) {
      const uint32_t mask = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
      quantise(x.k, k, p.c.k_scale + x.scale, mask);
      quantise(x.v, v, p.c.v_scale + x.scale, mask);
    } else {
      widen(x.k, x.ks, k);
      widen(x.v, x.vs, v);
    }
  };
  Pair a, b;
  fetch(a);
  for (int u = threadIdx.x / kLanes; u < nt * h_kv; u += 2 * kStep) {
    fetch(b);
    put(a);
    fetch(a);
    put(b);
  }
  __threadfence();  // the rows are visible before the next kernel may start
  griddep_launch_dependents();
}

template <bool kWrite>
static cudaError_t launch_move(PagedMoveParams p, int head_dim, int cache_dtype, int row_dtype,
                               cudaStream_t s) {
  // One run of tokens for every CTA that fits the GPU: the look-ups' latency is paid once.
  const int ctas = kMoveCtasPerSm * device_sm_count();
  const int per = (p.n_tokens + ctas - 1) / ctas;
  p.tokens_per_cta = per > kMaxTokensPerCta ? kMaxTokensPerCta : per;
  const dim3 grid((p.n_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta), block(kMoveThreads);
  const bool fp8 = cache_dtype == HS2_KV_FP8_E4M3, half = row_dtype == HS2_KV_F16;
  // 16-bit rows are copied as they are, whichever of the two types they hold.
  if (head_dim == 128)
    return !fp8   ? launch_pdl(paged_move_kernel<128, __half, false, kWrite>, grid, block, 0, s, p)
           : half ? launch_pdl(paged_move_kernel<128, __half, true, kWrite>, grid, block, 0, s, p)
                  : launch_pdl(paged_move_kernel<128, __nv_bfloat16, true, kWrite>, grid, block, 0, s, p);
  return !fp8   ? launch_pdl(paged_move_kernel<64, __half, false, kWrite>, grid, block, 0, s, p)
         : half ? launch_pdl(paged_move_kernel<64, __half, true, kWrite>, grid, block, 0, s, p)
                : launch_pdl(paged_move_kernel<64, __nv_bfloat16, true, kWrite>, grid, block, 0, s, p);
}

cudaError_t launch_paged_write(const PagedMoveParams& p, int head_dim, int cache_dtype,
                               int row_dtype, cudaStream_t s) {
  return launch_move<true>(p, head_dim, cache_dtype, row_dtype, s);
}
cudaError_t launch_paged_read(const PagedMoveParams& p, int head_dim, int cache_dtype,
                              int row_dtype, cudaStream_t s) {
  return launch_move<false>(p, head_dim, cache_dtype, row_dtype, s);
}

}  // namespace hs2
