// Causal attention over packed prompts: one warp per (query token, head) walks the keys it
// sees with a running maximum and sum; each lane holds D / 32 elements.
#include "paged.cuh"

namespace hs2 {

constexpr int kWarps = 4;

template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarps) packed_attn_kernel(PackedAttnParams p) {
  griddep_wait();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += 32 * kWarps)
      if (__ldg(p.cu_q + b + 1) < __ldg(p.cu_q + b) || __ldg(p.cu_k + b + 1) < __ldg(p.cu_k + b))
        set_status(p.status, HS2_ERR_BAD_LENGTH);
  const long long th = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (th >= (long long)p.n_q * p.h_q) return;
  const int t = (int)(th / p.h_q), h = (int)(th - (long long)t * p.h_q);
  const int b = find_sequence(p.cu_q, p.batch, t);
  int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > p.n_q || k0 < 0 || k1 < k0 || k1 > p.n_k) {
    if (lane == 0) set_status(p.status, HS2_ERR_BAD_LENGTH);
    q1 = min(q1, p.n_q);
    k0 = max(k0, 0);
    k1 = min(k1, p.n_k);
  }
  if (t < q0 || t >= q1) return;  // padding
  const int lq = q1 - q0, lk = max(k1 - k0, 0);
  const int n = lk - lq + (t - q0) + 1;  // visible keys (<= 0: none)
  const int64_t kv = (int64_t)k0 * p.kv_tok + (h / p.group) * p.kv_head;
  float q[E], o[E];
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(p.q + t * p.q_tok + h * p.q_head) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    const float2 x = unpack2<T>(qw[e]);
    q[2 * e] = x.x, q[2 * e + 1] = x.y;
    o[2 * e] = 0.f, o[2 * e + 1] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(p.k + kv + j * p.kv_tok) + lane * (E / 2);
    const uint32_t* vr = reinterpret_cast<const uint32_t*>(p.v + kv + j * p.kv_tok) + lane * (E / 2);
    float s = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 a = unpack2<T>(kr[e]), c = unpack2<T>(vr[e]);
      s = fmaf(q[2 * e], a.x, fmaf(q[2 * e + 1], a.y, s));
      v[2 * e] = c.x, v[2 * e + 1] = c.y;
    }
    s = warp_sum(s) * p.scale_log2;
    const float m2 = fmaxf(m, s), keep = exp2f(m - m2), w = exp2f(s - m2);
    m = m2;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * v[e];
  }
  const float inv = n > 0 ? 1.f / l : 0.f;
  uint32_t* out = static_cast<uint32_t*>(p.out) + th * (D / 2) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (p.lse && lane == 0) p.lse[th] = n > 0 ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

cudaError_t launch_packed_attn(const PackedAttnParams& p, int head_dim, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)(((long long)p.n_q * p.h_q + kWarps - 1) / kWarps)), block(32 * kWarps);
  if (head_dim == 128)
    return dtype == HS2_KV_F16 ? launch_pdl(packed_attn_kernel<128, __half>, grid, block, 0, s, p)
                               : launch_pdl(packed_attn_kernel<128, __nv_bfloat16>, grid, block, 0, s, p);
  return dtype == HS2_KV_F16 ? launch_pdl(packed_attn_kernel<64, __half>, grid, block, 0, s, p)
                             : launch_pdl(packed_attn_kernel<64, __nv_bfloat16>, grid, block, 0, s, p);
}

}  // namespace hs2
