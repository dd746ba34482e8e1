// libmoe C ABI of the decode-step operators around the expert layer: validation and launches.
#include <cmath>

#include "decoder.cuh"

using namespace moe;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool activation(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16; }
// Elements of a row stride that keep a row 16-byte aligned.
bool stride_ok(int64_t stride, moe_dtype t, int64_t at_least) {
  return stride >= at_least && stride <= (int64_t(1) << 31) && stride % (t == MOE_BF16 ? 8 : 4) == 0;
}
moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status check_cache(const moe_kv_cache* c) {
  if (!c || c->n_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16 && c->dtype != MOE_E4M3) return MOE_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return MOE_ERR_INVALID_ARG;
  if (c->dtype == MOE_E4M3 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return MOE_ERR_INVALID_ARG;
  if (c->page_size % 16 != 0 || c->page_size > kMaxPageSize) return MOE_ERR_UNSUPPORTED;
  if (int64_t(c->n_pages) * c->n_kv_heads >= (int64_t(1) << 31) / c->page_size) return MOE_ERR_UNSUPPORTED;
  if (c->head_dim % 16 != 0 || c->head_dim > kMaxHeadDim || c->n_kv_heads > kMaxHeads) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

CacheDev to_dev(const moe_kv_cache* c) {
  CacheDev d;
  d.n_pages = c->n_pages;
  d.page = c->page_size;
  d.heads = c->n_kv_heads;
  d.dim = c->head_dim;
  d.e4m3 = c->dtype == MOE_E4M3;
  d.k = static_cast<uint8_t*>(c->k);
  d.v = static_cast<uint8_t*>(c->v);
  d.k_exp = c->k_exp;
  d.v_exp = c->v_exp;
  return d;
}

moe_status check_table(const int32_t* page_table, int n_seqs, int max_pages) {
  if (!page_table || !aligned4(page_table) || n_seqs <= 0 || max_pages <= 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_status_ws(const void* ws, size_t ws_bytes) {
  if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < sizeof(DevStatus) ? MOE_ERR_WORKSPACE : MOE_OK;
}

// The checks moe_kv_write and moe_kv_read share (T > 0).
moe_status check_tokens(const int32_t* seq, const int32_t* pos, int T, const int32_t* page_table, int n_seqs,
                        int max_pages, const void* ws, size_t ws_bytes) {
  if (!pos || !aligned4(pos) || !aligned4(seq)) return MOE_ERR_INVALID_ARG;
  if (!seq && T > n_seqs) return MOE_ERR_INVALID_ARG;
  const moe_status rc = check_table(page_table, n_seqs, max_pages);
  return rc != MOE_OK ? rc : check_status_ws(ws, ws_bytes);
}

moe_status check_attn_shape(const moe_kv_cache* c, int n_heads, int B) {
  const moe_status rc = check_cache(c);
  if (rc != MOE_OK) return rc;
  if (n_heads <= 0 || n_heads % c->n_kv_heads != 0 || B < 0) return MOE_ERR_INVALID_ARG;
  if (n_heads > kMaxHeads || B > kMaxSeqs) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_kv_write(const moe_kv_cache* cache, const void* k, const void* v, moe_dtype kv_dtype, int64_t k_stride,
                        int64_t v_stride, int T, const int32_t* seq, const int32_t* pos, const int32_t* page_table,
                        int n_seqs, int max_pages, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status rc = check_cache(cache);
  if (rc != MOE_OK) return rc;
  if (T < 0 || T > kMaxTokens || !activation(kv_dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const int64_t row = int64_t(cache->n_kv_heads) * cache->head_dim;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !stride_ok(k_stride, kv_dtype, row) ||
      !stride_ok(v_stride, kv_dtype, row))
    return MOE_ERR_INVALID_ARG;
  rc = check_tokens(seq, pos, T, page_table, n_seqs, max_pages, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  const PageTable pt{page_table, n_seqs, max_pages, static_cast<int*>(ws)};
  return cuda_status(launch_kv_write(to_dev(cache), pt, k, v, kv_dtype == MOE_BF16, k_stride, v_stride, T, seq, pos,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_read(const moe_kv_cache* cache, int T, const int32_t* seq, const int32_t* pos,
                       const int32_t* page_table, int n_seqs, int max_pages, void* k_out, void* v_out,
                       moe_dtype out_dtype, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status rc = check_cache(cache);
  if (rc != MOE_OK) return rc;
  if (T < 0 || T > kMaxTokens || !activation(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return MOE_ERR_INVALID_ARG;
  rc = check_tokens(seq, pos, T, page_table, n_seqs, max_pages, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  const PageTable pt{page_table, n_seqs, max_pages, static_cast<int*>(ws)};
  return cuda_status(launch_kv_read(to_dev(cache), pt, T, seq, pos, k_out, v_out, out_dtype == MOE_BF16,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_attn_workspace_bytes(const moe_kv_cache* cache, int n_heads, int B) {
  if (check_attn_shape(cache, n_heads, B) != MOE_OK) return 0;
  return attn_workspace_bytes(to_dev(cache), n_heads, B);
}

moe_status moe_attn_workspace_init(void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kAttnPartialsAt) return MOE_ERR_WORKSPACE;
  return cuda_status(cudaMemsetAsync(ws, 0, kAttnPartialsAt, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_attn_decode(const moe_kv_cache* cache, const void* q, int64_t q_stride, int n_heads, int B,
                           const int32_t* lens, const int32_t* page_table, int max_pages, float scale, int window,
                           void* out, float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status rc = check_attn_shape(cache, n_heads, B);
  if (rc != MOE_OK) return rc;
  if (!std::isfinite(scale) || window < 0) return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!q || !aligned16(q) || !stride_ok(q_stride, MOE_BF16, int64_t(n_heads) * cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  if (!lens || !aligned4(lens) || !out || !aligned16(out) || !aligned4(lse)) return MOE_ERR_INVALID_ARG;
  rc = check_table(page_table, B, max_pages);
  if (rc != MOE_OK) return rc;
  // positions and the tiles of a call are counted in 32 bits (a tile is of 32 tokens and 4 heads at least)
  const int64_t room = int64_t(max_pages) * cache->page_size, group = n_heads / cache->n_kv_heads;
  if (room > (int64_t(1) << 28) ||
      (room / 32 + 1) * B * cache->n_kv_heads >= (int64_t(1) << 31) / ((group + 3) / 4))
    return MOE_ERR_UNSUPPORTED;
  if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  AttnArgs a;
  a.cache = to_dev(cache);
  if (ws_bytes < attn_workspace_bytes(a.cache, n_heads, B)) return MOE_ERR_WORKSPACE;
  a.table = PageTable{page_table, B, max_pages, static_cast<int*>(ws)};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.n_heads = n_heads;
  a.B = B;
  a.window = window;
  a.scale = scale;
  a.lens = lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws = static_cast<char*>(ws);
  return cuda_status(launch_attn_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_block_norm(const void* y, moe_dtype y_dtype, const float* w_post, const void* gate,
                          moe_dtype gate_dtype, int64_t gate_stride, float alpha, const void* residual,
                          void* residual_out, moe_dtype r_dtype, const float* w_pre, void* x, moe_dtype x_dtype, int T,
                          int d, float eps, moe_stream_t stream) {
  if (T < 0 || T > kMaxTokens || d <= 0) return MOE_ERR_INVALID_ARG;
  if (!activation(r_dtype) || (y && !activation(y_dtype)) || (gate && !activation(gate_dtype)) ||
      (x && !activation(x_dtype)))
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(alpha) || !(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > kMaxNormDim) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!residual || (y && !residual_out) || (!y && (w_post || gate)) || (x && !w_pre) || (!y && !x))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(w_post) || !aligned16(gate) || !aligned16(residual) || !aligned16(residual_out) ||
      !aligned16(w_pre) || !aligned16(x))
    return MOE_ERR_INVALID_ARG;
  if (gate && gate_stride != 0 && !(stride_ok(gate_stride, MOE_BF16, d))) return MOE_ERR_INVALID_ARG;
  NormArgs a;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.gate_stride = gate_stride;
  a.alpha = alpha;
  a.eps = eps;
  a.inv_d = 1.0f / float(d);
  a.residual = residual;
  a.residual_out = residual_out;
  a.w_pre = w_pre;
  a.x = x;
  a.y_bf16 = y_dtype == MOE_BF16;
  a.gate_bf16 = gate_dtype == MOE_BF16;
  a.r_bf16 = r_dtype == MOE_BF16;
  a.x_bf16 = x_dtype == MOE_BF16;
  a.T = T;
  a.d = d;
  return cuda_status(launch_block_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
