// The attention of attn_decode.cuh over INT4 caches.
#include "attn_decode.cuh"

namespace moe {
namespace {

// A segment's heads as over bf16, which the products are (attn_decode.cu); and shorter tiles where no segment can be
// longer than kShortSegment tokens: the page table's width and the window are what the host knows of that.
constexpr int kShortSegment = 1024;

template <int kDim, typename F>
auto with_heads(int group, int longest, F f) {
  if (longest <= kShortSegment)
    return group <= 8 ? f(Shape<RowKind::kInt4, kDim, 8, true>{}) : f(Shape<RowKind::kInt4, kDim, 16, true>{});
  return group <= 8 ? f(Shape<RowKind::kInt4, kDim, 8>{}) : f(Shape<RowKind::kInt4, kDim, 16>{});
}
template <typename F>
auto with_shape(const CacheDev& c, int group, int longest, F f) {
  if (c.dim <= 64) return with_heads<64>(group, longest, f);
  if (c.dim <= 128) return with_heads<128>(group, longest, f);
  return f(Shape<RowKind::kInt4, 256, 8>{});
}

}  // namespace

size_t attn_int4_workspace_bytes(const CacheDev& c, int n_heads) {
  return kAttnPartialsAt + with_shape(c, n_heads / c.heads, 0, [](auto shape) {  // a partial result is as large in any tile
           return size_t(kMaxCtas) * 2 * decltype(shape)::kSlot * sizeof(float);
         });
}

cudaError_t launch_attn_int4(const AttnScaledArgs& a, cudaStream_t s) {
  const int room = a.table.max_pages * a.cache.page, longest = a.window > 0 ? std::min(a.window, room) : room;
  return with_shape(a.cache, a.n_heads / a.cache.heads, longest,
                    [&](auto shape) { return launch<decltype(shape)>(a, s); });
}

}  // namespace moe
