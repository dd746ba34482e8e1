// Rotary positions: queries and keys turned pair by pair, alone or on the way into the paged cache.
//
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),   t = p f_i
//
// Angles.  f_i is held as a fraction of a turn in units of 2^-64, so p f_i modulo a turn is one 64-bit integer
// product, exact but for f_i's own rounding: positions of any size keep their angle, which fp32 products lose past a
// few thousand, and fp64 is slow on this GPU.  The top 32 bits are taken to the nearest quarter turn, and the rest,
// within an eighth of a turn, to sincospi.
//
// What bounds it is memory: 6 operations a pair.  A group of kLanes lanes takes a token, eight elements of each head a
// lane, works out its pairs' cosines and sines once and goes through heads with them, four heads' loads ahead of the
// arithmetic.  Where the pairs are half the turned part apart, a lane has four elements of one half and their partners in
// the other, so that nothing is read twice or exchanged, and a query may be turned in place.  Rows of the cache need
// eight elements in a row (their scales and codes), so for keys and values a lane has those, and loads its keys' partners
// as well (they are in L1: another lane of the group loads them).  The heads of a token are shared out over blocks: those
// of the queries, then those of keys and values.
//
// Measured: 16k tokens of 32 heads of 128 bf16 turned 41.4 us, 97 % of the copy rate (with a row's eight elements a lane
// and partners loaded for the queries too, one head ahead, 74.7), fp32 79 us, all of it; with 4 kv heads into a bf16 cache,
// half of a head turned, 59.7 us, 84 % (two or four rows ahead 59.7 and 70.7, for their registers; two heads of keys and
// values a block 62.4); one token 2.0 us.  All of a head turned, halves paired: into a bf16 cache 61 us (82 % of the copy
// rate), E4M3 70 (68 %), 4 bits 76 (62 %); from fp32 94, 93 and 95 (80, 78 and 75 %).  The kernels of quantised rows take 73
// and 74 registers, those of fp32 sources 102, which is three and two CTAs an SM, for the queries too.
#include "kv_rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// One lane's cosines and sines: element i becomes x_i c[i] + partner_i s[i].
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

__device__ __forceinline__ void turn_of(const RopeDev& r, int pos, int e0, Turn& t) {
  const int half = r.dim / 2;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      t.c[i] = t.c[i + 1] = 1.0f;
      t.s[i] = t.s[i + 1] = 0.0f;
      if (e0 + i >= r.dim) continue;
      const float2 cs = cos_sin(__ldg(r.turns + (e0 + i) / 2), pos, r.magnitude);
      t.c[i] = t.c[i + 1] = cs.x;
      t.s[i] = -cs.y;
      t.s[i + 1] = cs.y;
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
      t.s[i] = e < half ? -cs.y : cs.y;
    }
  }
}

// A head's eight elements with their partners.
template <typename Src>
struct Head {
  float x[8], y[8];
  __device__ __forceinline__ void load(const Src* p, const Partners& with, bool turned, bool mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.0f;
    if (!mine) return;
    load_vec8(p, x);
    if (!turned) return;
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

// Four elements as they lie.
template <typename Src>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void values(float (&x)[4]) const {
    x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
  }
};
template <>
struct Quad<float> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void values(float (&x)[4]) const { x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w; }
};
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// Query heads [j0, j1) of token t.
constexpr int kAhead = 4;
template <typename Src, typename Out>
__device__ __forceinline__ void turn_queries(const RopeArgs& a, int t, int lane, int j0, int j1) {
  if (t >= a.T || lane * 8 >= a.dim) return;
  const RopeDev& r = a.rope;
  const bool turned = lane * 8 < r.dim, apart = turned && !r.interleaved;
  const int e0 = apart ? 4 * lane : 8 * lane, e1 = apart ? r.dim / 2 + 4 * lane : 8 * lane + 4;
  const Src* from = static_cast<const Src*>(a.q.x) + t * a.q.stride;
  Out* to = static_cast<Out*>(a.out) + t * a.out_stride;
  Quad<Src> next[kAhead][2];
  auto fetch = [&](int j) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (j + i < j1) {
        next[i][0].load(from + (j + i) * a.dim + e0);
        next[i][1].load(from + (j + i) * a.dim + e1);
      }
  };
  fetch(j0);
  float c[4], s[4];
  const int pos = a.pos[t];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 cs = turned ? cos_sin(__ldg(r.turns + 4 * lane + i), pos, r.magnitude) : make_float2(1.0f, 0.0f);
    c[i] = cs.x;
    s[i] = a.inverse ? -cs.y : cs.y;
  }
  for (int j = j0; j < j1; j += kAhead) {
    Quad<Src> now[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i][0] = next[i][0], now[i][1] = next[i][1];
    fetch(j + kAhead);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (j + i >= j1) break;
      float x[4], y[4];
      now[i][0].values(x);
      now[i][1].values(y);
      if (apart) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = x[k], q = y[k];
          x[k] = fmaf(p, c[k], -(q * s[k]));
          y[k] = fmaf(q, c[k], p * s[k]);
        }
      } else if (turned) {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float p = x[k], q = x[k + 1], v = y[k], w = y[k + 1];
          x[k] = fmaf(p, c[k / 2], -(q * s[k / 2]));
          x[k + 1] = fmaf(q, c[k / 2], p * s[k / 2]);
          y[k] = fmaf(v, c[2 + k / 2], -(w * s[2 + k / 2]));
          y[k + 1] = fmaf(w, c[2 + k / 2], v * s[2 + k / 2]);
        }
      }
      store4(to + (j + i) * a.dim + e0, x);
      store4(to + (j + i) * a.dim + e1, y);
    }
  }
}

// Heads [j0, j1) of the list of keys' and then values' heads of token t, into the cache; the whole warp comes here.
template <int kLanes, RowKind kRows, typename Src>
__device__ __forceinline__ void place_rows(const RopeArgs& a, int t, int lane, int j0, int j1) {
  const bool here = t < a.T, mine = here && lane * 8 < a.dim;
  const int e0 = lane * 8;
  const Partners with(a.rope, e0);
  int64_t row0 = -1;  // of head 0
  if (here) {
    const int slot = a.slot[t], page = unsigned(slot) / unsigned(a.cache.page);
    if (slot >= 0) {
      if (page < a.cache.n_pages) row0 = int64_t(page) * a.cache.heads * a.cache.page + (slot - page * a.cache.page);
      else report_bad_page(a.status_flags);
    }
  }
  auto load = [&](int j, Head<Src>& h) {
    const bool is_k = j < a.k.heads;
    const HeadRows& r = is_k ? a.k : a.v;
    h.load(static_cast<const Src*>(r.x) + t * r.stride + (is_k ? j : j - a.k.heads) * a.dim + e0, with, is_k,
           mine && j < j1);
  };
  Head<Src> next;
  load(j0, next);
  Turn turn;
  if (j0 < a.k.heads) turn_of(a.rope, here ? a.pos[t] : 0, mine ? e0 : a.rope.dim, turn);
  for (int j = j0; j < j1; ++j) {
    Head<Src> h = next;
    load(j + 1, next);
    const bool is_k = j < a.k.heads;
    if (is_k) h.turn(turn, with);
    RowCode<kRows> code;
    code.template find<kLanes>(h.x);
    if (row0 >= 0)
      code.store(a.cache, is_k ? a.cache.k : a.cache.v, is_k ? a.cache.k_exp : a.cache.v_exp,
                 is_k ? a.cache.k_scale : a.cache.v_scale, row0 + int64_t(is_k ? j : j - a.k.heads) * a.cache.page, lane, 0,
                 h.x);
  }
}

// Blocks [0, q_blocks) of the second axis take q_each query heads each, those behind them kv_each heads of keys and
// values.
template <int kLanes, bool kCache, RowKind kRows, typename Src, typename Out>
__global__ void __launch_bounds__(kThreads) k_rope(RopeArgs a, int q_blocks, int q_each, int kv_each) {
  const int t = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  pdl_begin();
  if (!kCache || blockIdx.y < q_blocks) {
    const int j0 = blockIdx.y * q_each;
    turn_queries<Src, Out>(a, t, lane, j0, min(a.q.heads, j0 + q_each));
  } else if constexpr (kCache) {
    const int j0 = (blockIdx.y - q_blocks) * kv_each;
    place_rows<kLanes, kRows, Src>(a, t, lane, j0, min(a.k.heads + a.v.heads, j0 + kv_each));
  }
}

// Heads a block: as few as fill the GPU some times over; and not fewer than share the angles' cost where there are more
// tokens than that.
int heads_each(int T, int heads, int lanes, int enough) {
  const int64_t groups = int64_t(std::max(sm_count(), 1)) * 1024 / lanes;
  return int(std::min<int64_t>(std::min(heads, enough), std::max<int64_t>(1, int64_t(T) * heads / groups)));
}

template <int kLanes, bool kCache, RowKind kRows, typename Src, typename Out>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int kv = a.k.heads + a.v.heads, q_each = heads_each(a.T, a.q.heads, kLanes, 8);
  const int kv_each = kv > 0 ? heads_each(a.T, kv, kLanes, 4) : 1;
  const int tokens = kThreads / kLanes, q_blocks = (a.q.heads + q_each - 1) / q_each;
  return launch_pdl(k_rope<kLanes, kCache, kRows, Src, Out>,
                    dim3((a.T + tokens - 1) / tokens, q_blocks + (kv + kv_each - 1) / kv_each), dim3(kThreads), 0, s, a,
                    q_blocks, q_each, kv_each);
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
