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
  if (c->dtype != MOE_BF16 && c->dtype != MOE_E4M3 && c->dtype != MOE_INT4) return MOE_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return MOE_ERR_INVALID_ARG;
  if (c->dtype == MOE_INT4 && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
    return MOE_ERR_INVALID_ARG;
  if (c->page_size % 16 != 0 || c->page_size > kMaxPageSize) return MOE_ERR_UNSUPPORTED;
  if (int64_t(c->n_pages) * c->n_kv_heads >= (int64_t(1) << 31) / c->page_size) return MOE_ERR_UNSUPPORTED;
  if (c->head_dim % (c->dtype == MOE_INT4 ? 32 : 16) != 0 || c->head_dim > kMaxHeadDim || c->n_kv_heads > kMaxHeads) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

CacheScaled to_dev(const moe_kv_cache* c) {
  CacheScaled d;
  d.n_pages = c->n_pages;
  d.page = c->page_size;
  d.heads = c->n_kv_heads;
  d.dim = c->head_dim;
  d.rows = c->dtype == MOE_E4M3 ? RowKind::kE4M3 : c->dtype == MOE_INT4 ? RowKind::kInt4 : RowKind::kBf16;
  d.k = static_cast<uint8_t*>(c->k);
  d.v = static_cast<uint8_t*>(c->v);
  d.k_exp = c->k_exp;
  d.v_exp = c->v_exp;
  // a descriptor of a program built before INT4 caches ends with v_exp
  d.k_scale = d.rows == RowKind::kInt4 ? c->k_scale : nullptr;
  d.v_scale = d.rows == RowKind::kInt4 ? c->v_scale : nullptr;
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

// The checks moe_page_plan and moe_page_release share.
moe_status check_pages(const int32_t* lens, int B, const int32_t* table, int max_pages, const int32_t* free_pages,
                       const int32_t* n_free, int n_pages, int page_size, const int32_t* lens_out,
                       const int32_t* n_free_out, const void* ws, size_t ws_bytes) {
  if (B < 0 || max_pages <= 0 || n_pages <= 0 || page_size <= 0) return MOE_ERR_INVALID_ARG;
  if (B > kMaxSeqs || page_size > kMaxPageSize || int64_t(max_pages) * page_size > kMaxPagePositions ||
      n_pages > INT32_MAX / page_size)
    return MOE_ERR_UNSUPPORTED;
  if (B > 0 && (!lens || !lens_out || !table)) return MOE_ERR_INVALID_ARG;
  if (!free_pages || !n_free || !n_free_out) return MOE_ERR_INVALID_ARG;
  if (!aligned4(lens) || !aligned4(lens_out) || !aligned4(table) || !aligned4(free_pages) || !aligned4(n_free) ||
      !aligned4(n_free_out) || !ws || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  return ws_bytes < pages_workspace_bytes(B) ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status check_rope(const moe_rope_table* r, int head_dim) {
  if (!r || r->dim <= 0 || head_dim <= 0 || r->dim > head_dim || !r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7u) ||
      !std::isfinite(r->magnitude))
    return MOE_ERR_INVALID_ARG;
  if (r->dim % 8 != 0 || head_dim % 8 != 0 || head_dim > kMaxHeadDim) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

RopeDev to_dev(const moe_rope_table* r) { return RopeDev{r->turns, r->dim, r->interleaved != 0, r->magnitude}; }

constexpr double kPi = 3.14159265358979323846;

// A frequency in radians as a fraction of a turn in units of 2^-64, modulo a turn.  1 / (2 pi) in two parts and the
// product's own rounding error leave it off by about one unit for frequencies up to 1.
uint64_t turns_of(double f) {
  if (f < 0.0) return 0u - turns_of(-f);  // 1 - p would round p
  constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
  const double p = f * kHigh, rest = std::fma(f, kHigh, -p) + f * kLow;
  // p's fraction is exact, and so is that times 2^32 taken apart into its whole and its fraction
  const double whole = std::floor(p), high = (p - whole) * 4294967296.0, high_whole = std::floor(high);
  const double low = (high - high_whole) * 4294967296.0 + rest * 18446744073709551616.0;  // |low| below 2^63
  return (uint64_t(high_whole) << 32) + uint64_t(int64_t(std::llrint(low)));
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
  AttnScaledArgs a;
  const CacheScaled c = to_dev(cache);
  a.cache = c;  // (without its scales)
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
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

size_t moe_pages_workspace_bytes(int B) { return B < 0 || B > kMaxSeqs ? 0 : pages_workspace_bytes(B); }

moe_status moe_page_plan(const int32_t* lens, const int32_t* new_tokens, int B, int32_t* page_table, int max_pages,
                         const int32_t* free_pages, const int32_t* n_free, int n_pages, int page_size, int max_tokens,
                         int32_t* lens_out, int32_t* n_free_out, int32_t* starts, int32_t* seq, int32_t* pos,
                         int32_t* slot, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const moe_status rc = check_pages(lens, B, page_table, max_pages, free_pages, n_free, n_pages, page_size, lens_out,
                                    n_free_out, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (max_tokens < 0 || max_tokens > kMaxTokens) return MOE_ERR_INVALID_ARG;
  if (!aligned4(new_tokens) || !starts || !aligned4(starts)) return MOE_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!seq || !pos || !slot)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(seq) || !aligned16(pos) || !aligned16(slot)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_page_plan(PlanArgs{lens, new_tokens, B, page_table, max_pages, free_pages, n_free, n_pages,
                                               page_size, max_tokens, lens_out, n_free_out, starts, seq, pos, slot,
                                               static_cast<char*>(ws)},
                                      reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_page_release(const int32_t* lens, const uint8_t* ended, int B, const int32_t* page_table, int max_pages,
                            int32_t* free_pages, const int32_t* n_free, int n_pages, int page_size, int32_t* lens_out,
                            int32_t* n_free_out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const moe_status rc = check_pages(lens, B, page_table, max_pages, free_pages, n_free, n_pages, page_size, lens_out,
                                    n_free_out, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (B > 0 && !ended) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_page_release(ReleaseArgs{lens, ended, B, page_table, max_pages, free_pages, n_free, n_pages,
                                                     page_size, lens_out, n_free_out, static_cast<char*>(ws)},
                                         reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_rope_turns(const double* frequencies, int n, uint64_t* turns_out) {
  if (n < 0 || (n > 0 && (!frequencies || !turns_out))) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(frequencies[i]) < 2147483648.0)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) turns_out[i] = turns_of(frequencies[i]);
  return MOE_OK;
}

moe_status moe_rope_frequencies(int dim, double base, moe_rope_scaling scaling, double factor, double original, double low,
                                double high, uint64_t* turns_out, float* magnitude_out) {
  if (dim < 2 || dim % 2 != 0 || dim > kMaxHeadDim || !turns_out || !magnitude_out) return MOE_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return MOE_ERR_INVALID_ARG;
  if (scaling < MOE_ROPE_PLAIN || scaling > MOE_ROPE_BY_TURNS) return MOE_ERR_INVALID_ARG;
  if (scaling != MOE_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return MOE_ERR_INVALID_ARG;
  const bool blend = scaling == MOE_ROPE_BY_INDEX || scaling == MOE_ROPE_BY_TURNS;
  if (blend && !(original > 0.0 && low > 0.0 && low < high && std::isfinite(original) && std::isfinite(high)))
    return MOE_ERR_INVALID_ARG;
  if (scaling == MOE_ROPE_BASE && dim == 2) return MOE_ERR_INVALID_ARG;
  if (scaling == MOE_ROPE_BASE) base *= std::pow(factor, double(dim) / (dim - 2));
  if (!std::isfinite(base)) return MOE_ERR_INVALID_ARG;
  auto index_of = [&](double turns) { return dim * std::log(original / (2.0 * kPi * turns)) / (2.0 * std::log(base)); };
  const double first = blend ? std::fmax(std::floor(index_of(high)), 0.0) : 0.0;
  const double last = blend ? std::fmin(std::ceil(index_of(low)), dim - 1.0) : 0.0;
  *magnitude_out = scaling == MOE_ROPE_BY_INDEX ? float(0.1 * std::log(factor) + 1.0) : 1.0f;
  for (int i = 0; i < dim / 2; ++i) {
    double f = std::exp(-2.0 * i / dim * std::log(base)), slowed = 0.0;  // the slowed frequency's share
    if (scaling == MOE_ROPE_LINEAR) slowed = 1.0;
    if (scaling == MOE_ROPE_BY_INDEX) slowed = (i - first) / std::fmax(last - first, 0.001);
    if (scaling == MOE_ROPE_BY_TURNS) slowed = 1.0 - (original * f / (2.0 * kPi) - low) / (high - low);
    slowed = std::fmin(std::fmax(slowed, 0.0), 1.0);
    turns_out[i] = turns_of(f * (1.0 - slowed) + (slowed > 0.0 ? f / factor * slowed : 0.0));
  }
  return MOE_OK;
}

moe_status moe_rope_apply(const moe_rope_table* rope, const void* x, int64_t x_stride, void* out, int64_t out_stride,
                          moe_dtype dtype, int T, int n_heads, int head_dim, const int32_t* pos, int inverse,
                          moe_stream_t stream) {
  moe_status rc = check_rope(rope, head_dim);
  if (rc != MOE_OK) return rc;
  if (T < 0 || T > kMaxTokens || n_heads <= 0 || !activation(dtype)) return MOE_ERR_INVALID_ARG;
  if (n_heads > kMaxHeads) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int64_t row = int64_t(n_heads) * head_dim;
  if (!x || !out || !aligned16(x) || !aligned16(out) || !stride_ok(x_stride, dtype, row) ||
      !stride_ok(out_stride, dtype, row) || !pos || !aligned4(pos))
    return MOE_ERR_INVALID_ARG;
  if (x == out && x_stride != out_stride) return MOE_ERR_INVALID_ARG;
  RopeArgs a{};
  a.rope = to_dev(rope);
  a.q = HeadRows{x, x_stride, n_heads};
  a.out = out;
  a.out_stride = out_stride;
  a.dim = head_dim;
  a.T = T;
  a.inverse = inverse != 0;
  a.pos = pos;
  return cuda_status(launch_rope(a, dtype == MOE_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_rope_kv_write(const moe_rope_table* rope, const moe_kv_cache* cache, const void* q, int64_t q_stride,
                             int n_heads, void* q_out, int64_t q_out_stride, const void* k, const void* v,
                             moe_dtype dtype, int64_t k_stride, int64_t v_stride, int T, const int32_t* pos,
                             const int32_t* slot, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status rc = check_cache(cache);
  if (rc != MOE_OK) return rc;
  rc = check_rope(rope, cache->head_dim);
  if (rc != MOE_OK) return rc;
  if (T < 0 || T > kMaxTokens || n_heads <= 0 || !activation(dtype)) return MOE_ERR_INVALID_ARG;
  if (n_heads > kMaxHeads) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int64_t q_row = int64_t(n_heads) * cache->head_dim, kv_row = int64_t(cache->n_kv_heads) * cache->head_dim;
  if (!q || !q_out || !k || !v || !aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) ||
      !stride_ok(q_stride, dtype, q_row) || !stride_ok(q_out_stride, MOE_BF16, q_row) ||
      !stride_ok(k_stride, dtype, kv_row) || !stride_ok(v_stride, dtype, kv_row))
    return MOE_ERR_INVALID_ARG;
  if (q == q_out && (dtype != MOE_BF16 || q_stride != q_out_stride)) return MOE_ERR_INVALID_ARG;
  if (!pos || !aligned4(pos) || !slot || !aligned4(slot)) return MOE_ERR_INVALID_ARG;
  rc = check_status_ws(ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  RopeArgs a{};
  a.rope = to_dev(rope);
  a.q = HeadRows{q, q_stride, n_heads};
  a.k = HeadRows{k, k_stride, cache->n_kv_heads};
  a.v = HeadRows{v, v_stride, cache->n_kv_heads};
  a.out = q_out;
  a.out_stride = q_out_stride;
  a.cache = to_dev(cache);
  a.dim = cache->head_dim;
  a.T = T;
  a.pos = pos;
  a.slot = slot;
  a.status_flags = static_cast<int*>(ws);
  return cuda_status(launch_rope_kv_write(a, dtype == MOE_BF16, reinterpret_cast<cudaStream_t>(stream)));
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
