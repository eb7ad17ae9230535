// Host side of the paged cache and packed prompt calls of the C ABI: argument validation,
// workspace layout and launches.  Nothing here allocates device memory.
#include <math.h>

#include "paged.cuh"

namespace hs2 {

// Tokens times heads stay below this, so that counts rounded up to whole blocks fit an int.
constexpr int kMaxRows = (1 << 30) + ((1 << 30) - 4096);

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool is_16bit(int dtype) { return dtype == HS2_KV_BF16 || dtype == HS2_KV_F16; }

// Strides of rows of `elt`-byte elements: non-negative multiples of 16 bytes, below the 2^40
// bytes that end a tensor map's strides.
static bool good_stride(int64_t elements, int elt) {
  return elements >= 0 && elements < (int64_t(1) << 38) && elements * elt % 16 == 0;
}

// A stride that an axis of n elements can be walked with (the tensor maps take no 0).
static bool walks(int n, int64_t stride) { return n <= 1 || stride > 0; }

static hs2_status check_paged(const hs2_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v || !kv->pages || !kv->lens) return HS2_ERR_INVALID_ARGUMENT;
  if (kv->head_dim != 64 && kv->head_dim != 128) return HS2_ERR_UNSUPPORTED;
  const bool fp8 = kv->dtype == HS2_KV_FP8_E4M3;
  if (!fp8 && !is_16bit(kv->dtype)) return HS2_ERR_UNSUPPORTED;
  if (fp8 != (kv->k_scale != nullptr) || fp8 != (kv->v_scale != nullptr))
    return HS2_ERR_INVALID_ARGUMENT;
  if (kv->batch < 1 || kv->max_pages < 1 || kv->num_pages < 1 || kv->n_kv_heads < 1)
    return HS2_ERR_INVALID_ARGUMENT;
  if (kv->page_size < 8 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)))
    return HS2_ERR_UNSUPPORTED;
  if (kv->batch > 65535 || kv->n_kv_heads > 1024 ||
      (long long)kv->max_pages * kv->page_size >= (1ll << 31) - 64 ||
      ((long long)kv->max_pages * kv->page_size / 32 + 17) * kv->batch * kv->n_kv_heads >= (1ll << 31) - 1024)
    return HS2_ERR_UNSUPPORTED;
  const int elt = fp8 ? 1 : 2;
  if (!aligned16(kv->k) || !aligned16(kv->v) || !good_stride(kv->page_stride, elt) ||
      !good_stride(kv->head_stride, elt) || !good_stride(kv->row_stride, elt) ||
      kv->row_stride < kv->head_dim || !walks(kv->num_pages, kv->page_stride) ||
      !walks(kv->n_kv_heads, kv->head_stride))
    return HS2_ERR_INVALID_ARGUMENT;
  if (fp8 && (((uintptr_t)kv->k_scale | (uintptr_t)kv->v_scale) & 3u || kv->scale_page_stride < 0 ||
              kv->scale_head_stride < 0 || kv->scale_row_stride < 0))
    return HS2_ERR_INVALID_ARGUMENT;
  return HS2_OK;
}

static bool check_heads(int h_q, int h_kv) {
  return h_q >= 1 && h_q % h_kv == 0 && h_q / h_kv <= 128;
}

constexpr float kLog2e = 1.4426950408889634f;
static bool check_scale(float s) { return isfinite(s * kLog2e) && s > 0.f; }

static size_t paged_bytes(const hs2_paged_kv* kv, int h_q) {
  if (!h_q) return kPagedCounterOff;
  return kPagedPartialOff +
         (size_t)2 * kPagedMaxCtas * paged_part_floats(h_q / kv->n_kv_heads, kv->head_dim) * 4;
}

static PagedView paged_view(const hs2_paged_kv* kv, void* ws) {
  PagedView c;
  const int elt = kv->dtype == HS2_KV_FP8_E4M3 ? 1 : 2;
  c.k = static_cast<uint8_t*>(kv->k);
  c.v = static_cast<uint8_t*>(kv->v);
  c.k_scale = kv->k_scale;
  c.v_scale = kv->v_scale;
  c.pages = kv->pages;
  c.lens = kv->lens;
  c.page_stride = kv->page_stride * elt;
  c.head_stride = kv->head_stride * elt;
  c.row_stride = kv->row_stride * elt;
  c.sc_page = kv->scale_page_stride;
  c.sc_head = kv->scale_head_stride;
  c.sc_row = kv->scale_row_stride;
  c.batch = kv->batch;
  c.max_pages = kv->max_pages;
  c.num_pages = kv->num_pages;
  c.page_shift = __builtin_ctz((unsigned)kv->page_size);
  c.h_kv = kv->n_kv_heads;
  c.status = static_cast<uint32_t*>(ws);
  return c;
}

// Checks shared by the two row-moving calls.
static hs2_status check_move(const hs2_paged_kv* kv, const void* k_rows, const void* v_rows,
                             int dtype, int64_t token_stride, int64_t head_stride, int n_tokens,
                             const int32_t* cu, const void* ws, size_t ws_bytes) {
  const hs2_status st = check_paged(kv);
  if (st != HS2_OK) return st;
  if (!is_16bit(dtype)) return HS2_ERR_UNSUPPORTED;
  if (kv->dtype != HS2_KV_FP8_E4M3 && kv->dtype != dtype) return HS2_ERR_INVALID_ARGUMENT;
  if (n_tokens < 0 || !ws || !aligned16(ws) || !good_stride(token_stride, 2) ||
      !good_stride(head_stride, 2))
    return HS2_ERR_INVALID_ARGUMENT;
  if (n_tokens && (!k_rows || !v_rows || !aligned16(k_rows) || !aligned16(v_rows)))
    return HS2_ERR_INVALID_ARGUMENT;
  if (!cu && n_tokens % kv->batch) return HS2_ERR_INVALID_ARGUMENT;
  if (n_tokens >= kMaxRows / kv->n_kv_heads) return HS2_ERR_UNSUPPORTED;
  if (ws_bytes < paged_bytes(kv, 0)) return HS2_ERR_WORKSPACE_TOO_SMALL;
  return HS2_OK;
}

}  // namespace hs2

using namespace hs2;

extern "C" {

size_t hs2_paged_workspace_bytes(const hs2_paged_kv* kv, int h_q) {
  if (check_paged(kv) != HS2_OK || (h_q != 0 && !check_heads(h_q, kv->n_kv_heads))) return 0;
  return paged_bytes(kv, h_q);
}

hs2_status hs2_paged_kv_write(const void* k_new, const void* v_new, int dtype,
                              int64_t token_stride, int64_t head_stride, int n_tokens,
                              const int32_t* cu_new, const hs2_paged_kv* kv, void* workspace,
                              size_t ws_bytes, hs2_stream_t stream) {
  const hs2_status st = check_move(kv, k_new, v_new, dtype, token_stride, head_stride, n_tokens,
                                   cu_new, workspace, ws_bytes);
  if (st != HS2_OK || n_tokens == 0) return st;
  PagedMoveParams p = {};
  p.c = paged_view(kv, workspace);
  p.k_src = static_cast<const uint8_t*>(k_new);
  p.v_src = static_cast<const uint8_t*>(v_new);
  p.cu = cu_new;
  p.token_stride = token_stride * 2;
  p.head_stride = head_stride * 2;
  p.n_tokens = n_tokens;
  p.uniform = n_tokens / kv->batch;
  const cudaError_t e = launch_paged_write(p, kv->head_dim, kv->dtype, dtype, stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "paged cache write launch");
}

hs2_status hs2_paged_kv_read(const hs2_paged_kv* kv, const int32_t* cu, const int32_t* start,
                             int n_tokens, void* k_out, void* v_out, int dtype,
                             int64_t token_stride, int64_t head_stride, void* workspace,
                             size_t ws_bytes, hs2_stream_t stream) {
  if (!cu) return HS2_ERR_INVALID_ARGUMENT;
  const hs2_status st = check_move(kv, k_out, v_out, dtype, token_stride, head_stride, n_tokens,
                                   cu, workspace, ws_bytes);
  if (st != HS2_OK || n_tokens == 0) return st;
  PagedMoveParams p = {};
  p.c = paged_view(kv, workspace);
  p.k_dst = static_cast<uint8_t*>(k_out);
  p.v_dst = static_cast<uint8_t*>(v_out);
  p.cu = cu;
  p.start = start;
  p.token_stride = token_stride * 2;
  p.head_stride = head_stride * 2;
  p.n_tokens = n_tokens;
  const cudaError_t e = launch_paged_read(p, kv->head_dim, kv->dtype, dtype, stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "paged cache read launch");
}

hs2_status hs2_paged_attn(const void* q, int dtype, int h_q, int64_t q_seq_stride,
                          int64_t q_head_stride, const hs2_paged_kv* kv, float sm_scale, void* out,
                          float* lse, void* workspace, size_t ws_bytes, hs2_stream_t stream) {
  const hs2_status st = check_paged(kv);
  if (st != HS2_OK) return st;
  if (!is_16bit(dtype) || !check_heads(h_q, kv->n_kv_heads)) return HS2_ERR_UNSUPPORTED;
  if (kv->dtype != HS2_KV_FP8_E4M3 && kv->dtype != dtype) return HS2_ERR_INVALID_ARGUMENT;
  if (!q || !out || !workspace || !aligned16(q) || !aligned16(out) || !aligned16(workspace) ||
      !good_stride(q_seq_stride, 2) || !good_stride(q_head_stride, 2) || !check_scale(sm_scale) ||
      ((uintptr_t)lse & 3u))
    return HS2_ERR_INVALID_ARGUMENT;
  if (ws_bytes < paged_bytes(kv, h_q)) return HS2_ERR_WORKSPACE_TOO_SMALL;
  PagedAttnParams p = {};
  p.c = paged_view(kv, workspace);
  p.q = static_cast<const uint8_t*>(q);
  p.q_seq = q_seq_stride * 2;
  p.q_head = q_head_stride * 2;
  p.h_q = h_q;
  p.group = h_q / kv->n_kv_heads;
  p.scale_log2 = sm_scale * kLog2e;
  p.out = out;
  p.lse = lse;
  p.counters = ws_ptr<uint32_t>(workspace, kPagedCounterOff);
  p.partials = ws_ptr<float>(workspace, kPagedPartialOff);
  p.stall_test = g_stall_test == 1;
  const cudaError_t e = launch_paged_attn(p, kv->head_dim, kv->dtype, dtype, stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "paged attention launch");
}

size_t hs2_packed_workspace_bytes(void) { return 512; }

hs2_status hs2_packed_attn(const hs2_packed* a, float sm_scale, void* out, float* lse,
                           void* workspace, size_t ws_bytes, hs2_stream_t stream) {
  if (!a || !a->cu_q || !a->cu_k) return HS2_ERR_INVALID_ARGUMENT;
  if (a->head_dim != 64 && a->head_dim != 128) return HS2_ERR_UNSUPPORTED;
  if (!is_16bit(a->dtype)) return HS2_ERR_UNSUPPORTED;
  if (a->batch < 1 || a->n_q < 0 || a->n_k < 0 || a->n_kv_heads < 1)
    return HS2_ERR_INVALID_ARGUMENT;
  if (a->n_kv_heads > 1024 || !check_heads(a->h_q, a->n_kv_heads) || a->batch > 65535 ||
      a->n_q >= kMaxRows / a->h_q || a->n_k >= kMaxRows / a->n_kv_heads)
    return HS2_ERR_UNSUPPORTED;
  if (!check_scale(sm_scale) || !good_stride(a->q_token_stride, 2) ||
      !good_stride(a->q_head_stride, 2) || !good_stride(a->kv_token_stride, 2) ||
      !good_stride(a->kv_head_stride, 2) || ((uintptr_t)lse & 3u))
    return HS2_ERR_INVALID_ARGUMENT;
  if (!walks(a->n_q, a->q_token_stride) || !walks(a->h_q, a->q_head_stride) ||
      !walks(a->n_k, a->kv_token_stride) || !walks(a->n_kv_heads, a->kv_head_stride))
    return HS2_ERR_INVALID_ARGUMENT;
  if (!workspace || !aligned16(workspace)) return HS2_ERR_INVALID_ARGUMENT;
  if (ws_bytes < hs2_packed_workspace_bytes()) return HS2_ERR_WORKSPACE_TOO_SMALL;
  if (a->n_q == 0) return HS2_OK;
  if (!a->q || !out || !aligned16(a->q) || !aligned16(out)) return HS2_ERR_INVALID_ARGUMENT;
  if (a->n_k && (!a->k || !a->v || !aligned16(a->k) || !aligned16(a->v)))
    return HS2_ERR_INVALID_ARGUMENT;
  PackedAttnParams p = {};
  p.q = static_cast<const uint8_t*>(a->q);
  p.k = static_cast<const uint8_t*>(a->k);
  p.v = static_cast<const uint8_t*>(a->v);
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.q_tok = a->q_token_stride * 2;
  p.q_head = a->q_head_stride * 2;
  p.kv_tok = a->kv_token_stride * 2;
  p.kv_head = a->kv_head_stride * 2;
  p.n_q = a->n_q;
  p.n_k = a->n_k;
  p.batch = a->batch;
  p.h_q = a->h_q;
  p.h_kv = a->n_kv_heads;
  p.group = a->h_q / a->n_kv_heads;
  p.scale_log2 = sm_scale * kLog2e;
  p.out = out;
  p.lse = lse;
  p.status = static_cast<uint32_t*>(workspace);
  p.sync = ws_ptr<uint32_t>(workspace, kPackedSyncOff);
  p.stall_test = g_stall_test == 1;
  const cudaError_t e = launch_packed_attn(p, a->head_dim, a->dtype, stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "packed attention launch");
}

}  // extern "C"
