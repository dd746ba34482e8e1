// Rotary positions: queries and keys turned pair by pair, alone or on the way into the paged cache.
//
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),   t = p f_i
//
// Angles.  f_i is held as a fraction of a turn in units of 2^-64, so p f_i modulo a turn is one 64-bit integer
// product, exact but for f_i's own rounding: positions of any size keep their angle, which fp32 products lose past a
// few thousand, and fp64 is slow on this GPU.  The top 32 bits are taken to the nearest quarter turn, and the rest,
// within an eighth of a turn, to sincospi.
//
// What bounds it is memory: 6 operations a pair.  So a group of kLanes lanes takes a token, eight elements a lane of
// each head, works out its elements' cosines and sines once and goes through the heads with them, the next head's
// loads ahead of the current one's arithmetic.  Where pairs are half the turned part apart a lane loads its partners'
// elements as well (they are in L1: another lane of the group loads them).  With few tokens the heads are shared out
// over more groups: jobs of one head or more, queries first, then keys, then values.
#include "kv_rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// One lane's cosines and sines: element i becomes x_i cs[i].x + partner_i cs[i].y.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int pos, float magnitude) {
  const uint64_t phase = turns * uint64_t(int64_t(pos));
  const uint32_t hi = uint32_t(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;      // of the nearest quarter turn, 0 .. 3
  const int rest = int(hi - (quarter << 30));             // within an eighth of a turn
  float s, c;
  sincospif(float(rest) * 0x1p-31f, &s, &c);              // in half turns
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  // cos(t + pi/2) = -sin t, sin(t + pi/2) = cos t
  return make_float2((quarter == 1 || quarter == 2 ? -x : x) * magnitude, (quarter >= 2 ? -y : y) * magnitude);
}

// Four elements as fp32, at a multiple of four.
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
}

// Where a lane's elements (e0 .. e0 + 7) have their partners.
struct Partners {
  bool inside;  // among the lane's own elements: interleaved pairs (eight elements are turned or none)
  int by[2];    // else how far from each block of four, 0: none (half of the turned part is a multiple of four)
  __device__ __forceinline__ Partners(const RopeDev& r, int e0) {
    const int half = r.dim / 2;
    inside = r.interleaved && e0 < r.dim;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int e = e0 + 4 * b;
      by[b] = r.interleaved || e >= r.dim ? 0 : e < half ? half : -half;
    }
  }
};

__device__ __forceinline__ void turn_of(const RopeDev& r, int pos, int e0, bool inverse, Turn& t) {
  const int half = r.dim / 2;
  const float sign = inverse ? -1.0f : 1.0f;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      t.c[i] = t.c[i + 1] = 1.0f;
      t.s[i] = t.s[i + 1] = 0.0f;
      if (e0 + i >= r.dim) continue;
      const float2 cs = cos_sin(__ldg(r.turns + (e0 + i) / 2), pos, r.magnitude);
      t.c[i] = t.c[i + 1] = cs.x;
      t.s[i] = -sign * cs.y;
      t.s[i + 1] = sign * cs.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      t.c[i] = 1.0f;
      t.s[i] = 0.0f;
      if (e >= r.dim) continue;
      const float2 cs = cos_sin(__ldg(r.turns + (e < half ? e : e - half)), pos, r.magnitude);
      t.c[i] = cs.x;
      t.s[i] = e < half ? -sign * cs.y : sign * cs.y;
    }
  }
}

// A head's eight elements with their partners.
template <typename Src>
struct Head {
  float x[8], y[8];
  __device__ __forceinline__ void load(const Src* p, const Partners& with, bool mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.0f;
    if (!mine) return;
    load_vec8(p, x);
    if (with.by[0] == with.by[1]) {
      if (with.by[0] != 0 && (with.by[0] & 7) == 0) {
        load_vec8(p + with.by[0], y);
        return;
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (with.by[b] != 0) load4(p + 4 * b + with.by[b], y + 4 * b);
  }
  __device__ __forceinline__ void turn(const Turn& t, const Partners& with) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = x[i], b = x[i + 1];
      x[i] = fmaf(a, t.c[i], (with.inside ? b : y[i]) * t.s[i]);
      x[i + 1] = fmaf(b, t.c[i + 1], (with.inside ? a : y[i + 1]) * t.s[i + 1]);
    }
  }
};

// Heads [j0, j0 + each) of the list of q's, k's and v's heads, of one token a group.
template <int kLanes, bool kCache, RowKind kRows, typename Src, typename Out>
__global__ void __launch_bounds__(kThreads) k_rope(RopeArgs a, int each) {
  const int t = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int e0 = lane * 8, all = a.q.heads + a.k.heads + a.v.heads;
  const int j0 = blockIdx.y * each, j1 = min(all, j0 + each);
  const bool here = t < a.T, mine = here && e0 < a.dim;
  const Partners with(a.rope, e0);
  pdl_begin();
  const int pos = here ? __ldg(a.pos + t) : 0;
  int64_t row0 = -1;  // of head 0 in the cache
  if constexpr (kCache) {
    if (here && j1 > a.q.heads) {
      const int slot = __ldg(a.slot + t), page = unsigned(slot) / unsigned(a.cache.page);
      if (slot >= 0) {
        if (page < a.cache.n_pages) row0 = int64_t(page) * a.cache.heads * a.cache.page + (slot - page * a.cache.page);
        else report_bad_page(a.status_flags);
      }
    }
  }
  auto load = [&](int j, Head<Src>& h) {
    const bool is_q = j < a.q.heads, is_k = !is_q && j < a.q.heads + a.k.heads;
    const HeadRows& r = is_q ? a.q : is_k ? a.k : a.v;
    const int head = is_q ? j : is_k ? j - a.q.heads : j - a.q.heads - a.k.heads;
    h.load(static_cast<const Src*>(r.x) + t * r.stride + int64_t(head) * a.dim + e0, with, mine && j < j1);
  };
  Head<Src> next;
  load(j0, next);
  Turn turn;
  if (j0 < a.q.heads + a.k.heads) turn_of(a.rope, pos, mine ? e0 : a.rope.dim, a.inverse, turn);
  for (int j = j0; j < j1; ++j) {
    Head<Src> h = next;
    load(j + 1, next);
    if (j < a.q.heads + a.k.heads) h.turn(turn, with);
    if (!kCache || j < a.q.heads) {
      __syncwarp();  // out may be x: the group's lanes have their partners' elements
      if (mine) store_vec8(static_cast<Out*>(a.out) + t * a.out_stride + int64_t(j) * a.dim + e0, h.x);
    } else if constexpr (kCache) {
      const bool is_k = j < a.q.heads + a.k.heads;
      const int head = j - a.q.heads - (is_k ? 0 : a.k.heads);
      store_row<kLanes, kRows>(a.cache, is_k ? a.cache.k : a.cache.v, is_k ? a.cache.k_exp : a.cache.v_exp,
                               is_k ? a.cache.k_scale : a.cache.v_scale, row0 + int64_t(head) * a.cache.page, row0 >= 0,
                               lane, h.x);
    }
  }
}

// Heads a group: enough groups to fill the GPU, and with more tokens fewer that work out the same angles.
int heads_each(int T, int heads, int lanes) {
  const int64_t fill = int64_t(std::max(sm_count(), 1)) * 2048 / lanes;
  return int(std::min<int64_t>(heads, std::max<int64_t>(1, int64_t(T) * heads / fill)));
}

template <int kLanes, bool kCache, RowKind kRows, typename Src, typename Out>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int heads = a.q.heads + a.k.heads + a.v.heads, each = heads_each(a.T, heads, kLanes);
  const int tokens = kThreads / kLanes;
  return launch_pdl(k_rope<kLanes, kCache, kRows, Src, Out>, dim3((a.T + tokens - 1) / tokens, (heads + each - 1) / each),
                    dim3(kThreads), 0, s, a, each);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, cudaStream_t s) {
  return with_lanes(a.dim, [&](auto lanes) {
    return with_source(bf16, [&](auto src) {
      return launch<decltype(lanes)::value, false, RowKind::kBf16, decltype(src), decltype(src)>(a, s);
    });
  });
}

cudaError_t launch_rope_kv_write(const RopeArgs& a, bool bf16, cudaStream_t s) {
  return with_lanes(a.dim, [&](auto lanes) {
    return with_rows(a.cache.rows, [&](auto rows) {
      return with_source(bf16, [&](auto src) {
        return launch<decltype(lanes)::value, true, decltype(rows)::value, decltype(src), __nv_bfloat16>(a, s);
      });
    });
  });
}

}  // namespace moe
