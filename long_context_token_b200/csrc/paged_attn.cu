// Attention of one new token per sequence over a paged cache: one warp per (sequence, query
// head) walks the keys with a running maximum and sum; each lane holds D / 32 elements.
#include "paged.cuh"

namespace hs2 {

constexpr int kWarps = 4;

// Q: the queries' type (and the cache's, unless kFp8).
template <int D, typename Q, bool kFp8>
__global__ void __launch_bounds__(32 * kWarps) paged_attn_kernel(PagedAttnParams p) {
  griddep_wait();
  constexpr int E = D / 32;  // 2 or 4 elements per lane
  const int lane = threadIdx.x & 31;
  const long long bh = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (bh >= (long long)p.c.batch * p.h_q) return;
  const int b = (int)(bh / p.h_q), h = (int)(bh - (long long)b * p.h_q), hk = h / p.group;
  const int L = paged_len(p.c, b, h == 0 && lane == 0);
  float q[E], o[E];
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(p.q + b * p.q_seq + h * p.q_head) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    const float2 x = unpack2<Q>(qw[e]);
    q[2 * e] = x.x;
    q[2 * e + 1] = x.y;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < L; ++j) {
    int page = __ldg(p.c.pages + (size_t)b * p.c.max_pages + (j >> p.c.page_shift));
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0) set_status(p.c.status, HS2_ERR_INDEX_OUT_OF_RANGE);
      page = 0;
    }
    const int r = j & ((1 << p.c.page_shift) - 1);
    const int64_t off = page * p.c.page_stride + hk * p.c.head_stride + r * p.c.row_stride;
    const int64_t so = page * p.c.sc_page + hk * p.c.sc_head + r * p.c.sc_row;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      float2 a, c;
      if constexpr (kFp8) {
        a = __half22float2(e4m3x2_to_half2(reinterpret_cast<const uint16_t*>(p.c.k + off)[lane * (E / 2) + e]));
        c = __half22float2(e4m3x2_to_half2(reinterpret_cast<const uint16_t*>(p.c.v + off)[lane * (E / 2) + e]));
        const float ks = p.c.k_scale[so], vs = p.c.v_scale[so];
        a.x *= ks, a.y *= ks, c.x *= vs, c.y *= vs;
      } else {
        a = unpack2<Q>(reinterpret_cast<const uint32_t*>(p.c.k + off)[lane * (E / 2) + e]);
        c = unpack2<Q>(reinterpret_cast<const uint32_t*>(p.c.v + off)[lane * (E / 2) + e]);
      }
      k[2 * e] = a.x, k[2 * e + 1] = a.y, v[2 * e] = c.x, v[2 * e + 1] = c.y;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s) * p.scale_log2;
    const float m2 = fmaxf(m, s), keep = exp2f(m - m2), w = exp2f(s - m2);
    m = m2;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * v[e];
  }
  const float inv = L > 0 ? 1.f / l : 0.f;
  uint32_t* out = static_cast<uint32_t*>(p.out) + bh * (D / 2) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = pack2<Q>(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (p.lse && lane == 0) p.lse[bh] = L > 0 ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, int head_dim, int cache_dtype, int q_dtype,
                              cudaStream_t s) {
  const dim3 grid((unsigned)(((long long)p.c.batch * p.h_q + kWarps - 1) / kWarps)), block(32 * kWarps);
  const bool fp8 = cache_dtype == HS2_KV_FP8_E4M3, half = q_dtype == HS2_KV_F16;
  if (head_dim == 128)
    return fp8 ? (half ? launch_pdl(paged_attn_kernel<128, __half, true>, grid, block, 0, s, p)
                       : launch_pdl(paged_attn_kernel<128, __nv_bfloat16, true>, grid, block, 0, s, p))
               : (half ? launch_pdl(paged_attn_kernel<128, __half, false>, grid, block, 0, s, p)
                       : launch_pdl(paged_attn_kernel<128, __nv_bfloat16, false>, grid, block, 0, s, p));
  return fp8 ? (half ? launch_pdl(paged_attn_kernel<64, __half, true>, grid, block, 0, s, p)
                     : launch_pdl(paged_attn_kernel<64, __nv_bfloat16, true>, grid, block, 0, s, p))
             : (half ? launch_pdl(paged_attn_kernel<64, __half, false>, grid, block, 0, s, p)
                     : launch_pdl(paged_attn_kernel<64, __nv_bfloat16, false>, grid, block, 0, s, p));
}

}  // namespace hs2
