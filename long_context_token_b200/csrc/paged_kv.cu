// Moving rows in and out of a paged cache: hs2_paged_kv_write (16-bit rows copied, FP8 rows
// quantised with their own scale) and hs2_paged_kv_read (the way back, dequantised).
//
// Both only move bytes: per row of d elements 2d bytes on the packed side and 2d (16-bit)
// or d + 4 (E4M3 code and float32 scale) in the pages.  A CTA takes a run of tokens: one
// thread per token first looks up the token's sequence, position and page (four dependent
// loads), then all threads move the run's rows, 16 bytes of the packed side per thread, so
// a row is one to two 128-byte lines and the lookups are paid once per token, not per head.
#include "paged.cuh"

namespace hs2 {

constexpr int kMoveThreads = 256;
constexpr int kMaxTokensPerCta = 32;

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

// D: head_dim; T: the packed rows' type; kFp8: the cache holds E4M3 codes and scales.
template <int D, typename T, bool kFp8, bool kWrite>
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(PagedMoveParams p) {
  __shared__ TokenSlot slots[kMaxTokensPerCta];
  constexpr int kLanes = D / 8;  // threads of one row, 16 bytes each
  griddep_wait();
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.n_tokens - t0);
  if (threadIdx.x < nt) slots[threadIdx.x] = token_slot<kWrite>(p, t0 + threadIdx.x);
  __syncthreads();
  const int c = threadIdx.x % kLanes;
  const int rows = nt * p.c.h_kv * 2;  // (token, head, K or V)
  // (every group of kLanes threads goes through the same number of rows or stops as one)
  for (int r = threadIdx.x / kLanes; r < rows; r += kMoveThreads / kLanes) {
    const int th = r >> 1, i = th / p.c.h_kv, h = th - i * p.c.h_kv;
    const bool is_v = r & 1;
    const TokenSlot s = slots[i];
    if (s.page < 0) continue;
    uint8_t* row = (is_v ? p.c.v : p.c.k) + s.page * p.c.page_stride + h * p.c.head_stride +
                   s.row * p.c.row_stride;
    const int64_t packed = (int64_t)(t0 + i) * p.token_stride + h * p.head_stride + c * 16;
    float* sc = kFp8 ? (is_v ? p.c.v_scale : p.c.k_scale) + s.page * p.c.sc_page +
                           h * p.c.sc_head + s.row * p.c.sc_row
                     : nullptr;
    if constexpr (kWrite) {
      const uint4 w = *reinterpret_cast<const uint4*>((is_v ? p.v_src : p.k_src) + packed);
      if constexpr (!kFp8) {
        *reinterpret_cast<uint4*>(row + c * 16) = w;
      } else {
        const float2 x[4] = {unpack2<T>(w.x), unpack2<T>(w.y), unpack2<T>(w.z), unpack2<T>(w.w)};
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
        const uint32_t mask = ((kLanes == 32 ? 0u : 1u << kLanes) - 1u)
                              << ((threadIdx.x & 31) / kLanes * kLanes);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
        const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
        uint32_t code[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          code[e] = __nv_cvt_float2_to_fp8x2(
              make_float2(__fdiv_rn(x[e].x, scale), __fdiv_rn(x[e].y, scale)), __NV_SATFINITE,
              __NV_E4M3);
        *reinterpret_cast<uint2*>(row + c * 8) =
            make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
        if (c == 0) *sc = scale;
      }
    } else {
      uint4 w;
      if constexpr (!kFp8) {
        w = *reinterpret_cast<const uint4*>(row + c * 16);
      } else {
        const uint2 code = *reinterpret_cast<const uint2*>(row + c * 8);
        const float scale = *sc;
        const uint32_t two[4] = {code.x & 0xffffu, code.x >> 16, code.y & 0xffffu, code.y >> 16};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = __half22float2(e4m3x2_to_half2(two[e]));
          o[e] = pack2<T>(x.x * scale, x.y * scale);
        }
        w = make_uint4(o[0], o[1], o[2], o[3]);
      }
      *reinterpret_cast<uint4*>((is_v ? p.v_dst : p.k_dst) + packed) = w;
    }
  }
  __threadfence();  // the rows are visible before the next kernel may start
  griddep_launch_dependents();
}

template <bool kWrite>
static cudaError_t launch_move(PagedMoveParams p, int head_dim, int cache_dtype, int row_dtype,
                               cudaStream_t s) {
  // About four CTAs per SM before a CTA takes a second token.
  int per = p.n_tokens / (4 * device_sm_count());
  p.tokens_per_cta = per < 1 ? 1 : per > kMaxTokensPerCta ? kMaxTokensPerCta : per;
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
