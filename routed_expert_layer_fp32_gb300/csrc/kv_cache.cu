// Writing keys and values into the paged cache (as bf16, or quantised to E4M3 or to 4 bits; kv_rows.cuh) and
// reading them back.
//
// Both are copies bound by memory: a row is one token's key or value of one kv head.  A group of
// kLanes lanes takes the key and value rows of kHeadsEach heads of one token, eight elements a lane of
// each.  So the place in the cache, three dependent loads away (sequence and position, then page, then
// row), is looked up once for four rows, and four rows' loads are in flight together in every lane; a
// row's largest magnitude is a few shuffles.
//
// Writing rows in 4 bits is bound by instructions more than by memory: about 23 an element, half of them the code itself
// (kv_rows.cuh).  Reading them, 9 an element, waits for memory: issuing takes about 4 of 10 us, and a lane has the
// codes, scales and exponents of four rows under way, of four, one and one bytes.  16k tokens of 4 heads of 128, 43 MB: 17 us
// to write, 10 to read back; E4M3 rows 14 and 10, bf16 rows 15 and 12.
#include "kv_rows.cuh"

namespace moe {
namespace {

constexpr int kHeadsEach = 2;

// The row (an index over [n_pages, heads, page]) of token t and head 0 in the cache; -1 for a skipped
// or refused token.  Head h's row is h * page further.
__device__ __forceinline__ int64_t cache_row(const CacheDev& c, const PageTable& pt, const int32_t* seq,
                                             const int32_t* pos, int t) {
  const int p = pos[t];
  const int s = seq ? seq[t] : t;
  if (p < 0) return -1;
  const int slot = unsigned(p) / unsigned(c.page);
  int page = -1;
  if (s >= 0 && s < pt.n_seqs && slot < pt.max_pages) page = pt.pages[int64_t(s) * pt.max_pages + slot];
  if (page < 0 || page >= c.n_pages) {
    report_bad_page(pt.status_flags);
    return -1;
  }
  return int64_t(page) * c.heads * c.page + (p - slot * c.page);
}

// INT4 is bound by what its warps issue, and is better with a few registers less and a fifth more of them (16k tokens
// written and read back 26.5 -> 25.0 us; with a quarter of the registers less again 25.9).
template <int kLanes, RowKind kRows, typename Src>
__global__ void __launch_bounds__(256, kRows == RowKind::kInt4 ? 5 : 1) k_kv_write(CacheOf<kRows> c, PageTable pt, const Src* k,
                                                  const Src* v, int64_t k_stride, int64_t v_stride, int T,
                                                  const int32_t* seq, const int32_t* pos) {
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int h0 = blockIdx.y * kHeadsEach, heads = min(kHeadsEach, c.heads - h0);
  const bool mine = t < T && lane * 8 < c.dim;
  pdl_begin();
  float kx[kHeadsEach][8], vx[kHeadsEach][8];
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) kx[j][i] = vx[j][i] = 0.0f;
    if (mine && j < heads) {
      load_vec8(k + t * k_stride + (h0 + j) * c.dim + lane * 8, kx[j]);
      load_vec8(v + t * v_stride + (h0 + j) * c.dim + lane * 8, vx[j]);
    }
  }
  const int64_t row0 = t < T ? cache_row(c, pt, seq, pos, t) : -1;
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
    const int64_t row = row0 + int64_t(h0 + j) * c.page;
    RowCode<kRows> kc, vc;
    kc.template find<kLanes>(kx[j]);
    vc.template find<kLanes>(vx[j]);
    if (row0 < 0 || j >= heads) continue;
    kc.store(c, c.k, c.k_exp, scales_of<kRows>(c, true), row, lane, 0, kx[j]);
    vc.store(c, c.v, c.v_exp, scales_of<kRows>(c, false), row, lane, 1, vx[j]);
  }
}

template <int kLanes, RowKind kRows, typename Dst>
__global__ void __launch_bounds__(256) k_kv_read(CacheOf<kRows> c, PageTable pt, int T, const int32_t* seq,
                                                 const int32_t* pos, Dst* __restrict__ k_out,
                                                 Dst* __restrict__ v_out) {
  const int t = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int h0 = blockIdx.y * kHeadsEach, heads = min(kHeadsEach, c.heads - h0);
  if (t >= T || lane * 8 >= c.dim) return;
  pdl_begin();
  const int64_t row0 = cache_row(c, pt, seq, pos, t);
  RawRow<kRows> k[kHeadsEach], v[kHeadsEach];
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
    const int64_t row = row0 + int64_t(h0 + j) * c.page;
    const bool read = row0 >= 0 && j < heads;
    k[j].load(c, c.k, c.k_exp, scales_of<kRows>(c, true), row, read, lane);
    v[j].load(c, c.v, c.v_exp, scales_of<kRows>(c, false), row, read, lane);
  }
#pragma unroll
  for (int j = 0; j < kHeadsEach; ++j) {
    if (j >= heads) continue;
    const int64_t at = (int64_t(t) * c.heads + h0 + j) * c.dim + lane * 8;
    k[j].store(k_out + at);
    v[j].store(v_out + at);
  }
}

dim3 token_grid(int T, int lanes, int heads) {
  return dim3((T + 256 / lanes - 1) / (256 / lanes), (heads + kHeadsEach - 1) / kHeadsEach);
}

}  // namespace

cudaError_t launch_kv_write(const CacheScaled& c, const PageTable& pt, const void* k, const void* v, bool bf16,
                            int64_t k_stride, int64_t v_stride, int T, const int32_t* seq, const int32_t* pos,
                            cudaStream_t s) {
  return with_lanes(c.dim, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    return with_rows(c.rows, [&](auto rows) {
      return with_source(bf16, [&](auto src) {
        using Src = decltype(src);
        return launch_pdl(k_kv_write<L, decltype(rows)::value, Src>, token_grid(T, L, c.heads), dim3(256), 0, s,
                          CacheOf<decltype(rows)::value>(c), pt, static_cast<const Src*>(k), static_cast<const Src*>(v), k_stride, v_stride, T, seq, pos);
      });
    });
  });
}

cudaError_t launch_kv_read(const CacheScaled& c, const PageTable& pt, int T, const int32_t* seq, const int32_t* pos,
                           void* k_out, void* v_out, bool bf16, cudaStream_t s) {
  return with_lanes(c.dim, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    return with_rows(c.rows, [&](auto rows) {
      return with_source(bf16, [&](auto dst) {
        using Dst = decltype(dst);
        return launch_pdl(k_kv_read<L, decltype(rows)::value, Dst>, token_grid(T, L, c.heads), dim3(256), 0, s,
                          CacheOf<decltype(rows)::value>(c), pt, T, seq, pos, static_cast<Dst*>(k_out), static_cast<Dst*>(v_out));
      });
    });
  });
}

}  // namespace moe
