// The attention of attn_decode.cuh over bf16 and E4M3 caches, and which of its kernels a call takes.  (attn_int4.cu has
// those of INT4 caches: apart, the two compile side by side.)
#include "attn_decode.cuh"

namespace moe {
namespace {

// The kernel for a cache and a group of query heads: a segment's heads are the fewest that hold the
// group, and of a larger group as many as its registers do.
//   bf16: up to 16 (groups of 16, 64 x 8k tokens: 66 us, in two passes of 8 99; small calls, whose time
//   is the joint of the partial results, lose: 8 x 8k 21 against 16), 8 at widths above 128.
//   E4M3: up to 8 (16 spill: 29.3 us against 16.7 in two passes; a group of 8 in one pass 70 us, in two of
//   4 108), 4 at widths above 128 (8 spill: 39.0 against 28.6).
template <typename F>
auto with_shape(const CacheDev& c, int group, F f) {
  if (c.rows == RowKind::kE4M3) {
    if (c.dim <= 64) return group <= 4 ? f(Shape<RowKind::kE4M3, 64, 4>{}) : f(Shape<RowKind::kE4M3, 64, 8>{});
    if (c.dim <= 128) return group <= 4 ? f(Shape<RowKind::kE4M3, 128, 4>{}) : f(Shape<RowKind::kE4M3, 128, 8>{});
    return f(Shape<RowKind::kE4M3, 256, 4>{});
  }
  if (c.dim <= 64) return group <= 8 ? f(Shape<RowKind::kBf16, 64, 8>{}) : f(Shape<RowKind::kBf16, 64, 16>{});
  if (c.dim <= 128) return group <= 8 ? f(Shape<RowKind::kBf16, 128, 8>{}) : f(Shape<RowKind::kBf16, 128, 16>{});
  return f(Shape<RowKind::kBf16, 256, 8>{});
}

}  // namespace

size_t attn_workspace_bytes(const CacheDev& c, int n_heads, int) {
  if (c.rows == RowKind::kInt4) return attn_int4_workspace_bytes(c, n_heads);
  return kAttnPartialsAt + with_shape(c, n_heads / c.heads, [](auto shape) {
           return size_t(kMaxCtas) * 2 * decltype(shape)::kSlot * sizeof(float);
         });
}

cudaError_t launch_attn_decode(const AttnScaledArgs& a, cudaStream_t s) {
  if (a.cache.rows == RowKind::kInt4) return launch_attn_int4(a, s);
  return with_shape(a.cache, a.n_heads / a.cache.heads, [&](auto shape) { return launch<decltype(shape)>(a, s); });
}

}  // namespace moe
