// Shared declarations of the paged cache and packed prompt operators: parameter blocks,
// element types, and the lookup of a packed token's sequence and of a position's row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hs2_internal.cuh"

namespace hs2 {

// Workspace of the paged calls: the status word, two arrival counters per CTA of paged_attn
// (of the group of CTAs that it begins, and of the groups of the pair that it begins; 0
// between calls), then the CTAs' partial results, two each.  The places do not depend on the sizes of a call, so one workspace
// serves calls of different shapes.
constexpr int kPagedMaxCtas = kSmCountBound;
constexpr size_t kPagedCounterOff = 256;
constexpr size_t kPagedPartialOff = kPagedCounterOff + (2 * kPagedMaxCtas * 4 + 255) / 256 * 256;
// Floats of one partial result: o [group][head_dim], then (m, l) of each head.
__host__ __device__ constexpr int paged_part_floats(int group, int head_dim) {
  return (group * (head_dim + 2) + 3) / 4 * 4;
}

struct PagedView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* pages;
  const int32_t* lens;
  int64_t page_stride, head_stride, row_stride;  // bytes
  int64_t sc_page, sc_head, sc_row;              // floats
  int batch, max_pages, num_pages, page_shift, h_kv;
  uint32_t* status;
};

struct PagedMoveParams {  // hs2_paged_kv_write / hs2_paged_kv_read
  PagedView c;
  const uint8_t* k_src;  // write: the new rows
  const uint8_t* v_src;
  uint8_t* k_dst;  // read: the packed rows
  uint8_t* v_dst;
  const int32_t* cu;     // [batch + 1], or null: `uniform` tokens each
  const int32_t* start;  // read: first position of each sequence, or null
  int64_t token_stride, head_stride;  // bytes
  int n_tokens, uniform, tokens_per_cta;
};

struct PagedAttnParams {
  PagedView c;
  const uint8_t* q;
  int64_t q_seq, q_head;  // bytes
  int h_q, group;
  float scale_log2;  // sm_scale * log2(e)
  void* out;
  float* lse;
  uint32_t* counters;
  float* partials;
  int stall_test;  // hs2_debug_stall_waits: the producers issue no loads
};

// Workspace of hs2_packed_attn: the status word, then at kPackedSyncOff the next work item
// and the number of CTAs that are done (both 0 between calls).
constexpr size_t kPackedSyncOff = 256;

struct PackedAttnParams {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t q_tok, q_head, kv_tok, kv_head;  // bytes
  int n_q, n_k, batch, h_q, h_kv, group;
  int tiles;  // 128-row tiles per work item, 1 or 2
  float scale_log2;
  void* out;
  float* lse;
  uint32_t* status;
  uint32_t* sync;
  int stall_test;  // hs2_debug_stall_waits: no loads are issued
};

cudaError_t launch_paged_write(const PagedMoveParams& p, int head_dim, int cache_dtype,
                               int row_dtype, cudaStream_t s);
cudaError_t launch_paged_read(const PagedMoveParams& p, int head_dim, int cache_dtype,
                              int row_dtype, cudaStream_t s);
cudaError_t launch_paged_attn(const PagedAttnParams& p, int head_dim, int cache_dtype,
                              int q_dtype, cudaStream_t s);
cudaError_t launch_packed_attn(const PackedAttnParams& p, int head_dim, int dtype, cudaStream_t s);

#ifdef __CUDACC__

// Two 16-bit elements packed in a register, widened.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// ... and rounded to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t w;
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    w = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    w = *reinterpret_cast<const uint32_t*>(&h);
  }
  return w;
}
// Element-wise products and sums of two float32 at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 c;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(c))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return c;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 c;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(c))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return c;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 d) {
  float2 c;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(c))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(d)));
  return c;
}
// Two E4M3 codes (the low 16 bits) as float16, exactly.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return *reinterpret_cast<const __half2*>(&r);
}

// Length of sequence b of a paged cache, clamped to what its page table can hold.
__device__ __forceinline__ int paged_len(const PagedView& c, int b, bool report) {
  const int L = __ldg(c.lens + b);
  const int cap = c.max_pages << c.page_shift;
  if (L < 0 || L > cap) {
    if (report) set_status(c.status, HS2_ERR_BAD_LENGTH);
    return L < 0 ? 0 : cap;
  }
  return L;
}

// The last sequence b in [0, batch) whose cu[b] is at most t (cu[0] <= t).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

#endif  // __CUDACC__

}  // namespace hs2
