// Attention of one new token a sequence over the paged key-value cache, in one pass over the keys
// and values.
//
//   out = sum_j w_j v_j / sum_j p_j,   p_j = exp2(t_j - m),   t_j = (scale log2 e) q.k_j
//
// with the running maximum m, the sum and the accumulator in fp32.  In an E4M3 cache key j is
// 2^a_j times its codes and value j is 2^c_j times its codes: 2^a_j multiplies the score, and the
// weight of value j's codes is w_j = p_j 2^c_j.  There m is the running maximum of t_j + c_j, so
// that no w_j is above 1 and the largest is close to it: w_j is then rounded to fp16 without
// losing the rows that matter, however the rows' sizes differ.  In a bf16 cache w_j = p_j, rounded
// to bf16 (a product's operands have one type); the sum takes p_j before the rounding.
//
// What bounds it is reading the cache: 2 * group operations an element (group = query heads a kv
// head), against about 290 a byte for the tensor cores.  So the kernel is built around keeping
// copies in flight, and the products only have to keep up.
//
// Work split.  The unit is a tile of kTokens tokens of one (sequence, kv head, block of up to
// kHeads query heads), a segment; all tiles of the call in that order form one line, which is cut
// into equal parts, one for each CTA (a CTA an SM).  Mixed lengths and a single long sequence
// balance alike, and nothing about the lengths has to be known on the host.  A segment that lies
// in one part is finished by its CTA; one cut between CTAs leaves partial results (m, sum, fp32
// accumulator) in the workspace, and the CTA that writes the last of them (a counter a segment,
// back to 0 afterwards) joins them in CTA order, so the result does not depend on timing.
//
// In a CTA, one warp is the producer: it looks up pages and starts the tiles' TMA copies into a
// ring of shared-memory stages (about 190 KB of them in flight a SM).  The other warps form groups
// that take the CTA's tiles in turn; a warp has kPerWarp tokens of each of its group's tiles and
// its own m, sum and accumulator, which are joined once a segment through shared memory.  Copies
// of the next segments go on meanwhile.
//
// The products are warp MMAs (m16n8k16) with the tokens (scores) and the value elements (output)
// on the M side and the query heads on the N side, so that eight heads, not sixteen, are the unit
// that a small group is padded to; a tcgen05 product has at least 64 rows on M and its scores
// would have to travel through TMEM.  Keys and values reach the registers by ldmatrix from the
// swizzled tiles, the values transposed; E4M3 codes become fp16 on the way (exact), the queries
// fp16 after scaling by a power of two (exact but for elements 2^-38 below a head's largest).
#include "decoder.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;  // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMaxCtas = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMinExp = -100;  // least value exponent that enters m: keeps the sum inside fp32's range
static_assert(kMaxCtas <= kAttnTickets, "a counter a CTA");

template <bool kE4M3_, int kDim_, int kBlocks_>
struct Shape {
  static constexpr bool kE4M3 = kE4M3_;
  static constexpr int kDim = kDim_;        // head_dim rounded up to 64, 128 or 256 (copies fill with zeros)
  static constexpr int kBlocks = kBlocks_;  // blocks of eight query heads
  static constexpr int kHeads = 8 * kBlocks;
  static constexpr int kRow = kDim * (kE4M3 ? 1 : 2);       // bytes
  static constexpr int kSpan = kRow < 128 ? kRow : 128;     // bytes of a row in one swizzled copy
  static constexpr int kSpans = kRow / kSpan;
  static constexpr int kSpanElems = kDim / kSpans;
  // 32 KB stages (16 KB for the narrowest rows): 32 tokens a warp where a stage has room for that
  static constexpr int kPerWarp = kRow <= 128 ? 32 : 16;
  static constexpr int kGroupWarps = kRow <= 256 ? 4 : 2;
  static constexpr int kGroups = kWarps / kGroupWarps;
  static constexpr int kTokens = kPerWarp * kGroupWarps;
  static constexpr int kTile = kTokens * kRow;
  static constexpr int kExps = kE4M3 ? 2 * kTokens : 0;     // the keys' and the values' exponents
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = 192 * 1024 / kStage;
  static constexpr int kOutLd = kDim + 4;                    // row of the join buffer: no bank conflicts
  static constexpr int kSlot = kHeads * (kDim + 2);          // floats of a partial result
  struct Control {
    uint64_t full[kStages], empty[kStages];
    uint32_t valid[kStages];  // a bit for each 16 tokens of the tile: copied
    int abort;
    int b0, last;
    long long off0, scan[kWarps + 1];
    float m[kWarps][kHeads], sum[kWarps][kHeads];
    float total_m[kHeads], total_sum[kHeads];
  };
  // layout: stages, exponents, join buffer, control
  static constexpr size_t kExpsAt = size_t(kStages) * kStage;
  static constexpr size_t kOutAt = kExpsAt + size_t(kStages) * kExps;
  static constexpr size_t kControlAt = kOutAt + size_t(kHeads) * kOutLd * 4;
  static constexpr size_t kSmem = kControlAt + sizeof(Control) + 1024;  // and room to align the stages
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// ------------------------------------------------------------------ instructions ------------

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t r) {
  uint32_t t;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(r));
  return t;
}
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {  // exp2(-inf) = 0; relative error 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes (low half of `codes`) as fp16.
__device__ __forceinline__ uint32_t half2_of_codes(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes), __NV_E4M3);
  return uint32_t(h.x) | uint32_t(h.y) << 16;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float max_over_rows(float v) {  // over the lanes that share lane % 4
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum_over_rows(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void consumers_sync() { named_bar_sync(1, kWarps * 32); }

// ----------------------------------------------------------------------- the split ----------

struct Span {  // the tokens of one sequence that are seen, and their tiles
  int first, end, tile0, tiles;
};

template <typename S>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  const int room = a.table.max_pages * a.cache.page;
  Span s;
  s.end = max(0, min(__ldg(a.lens + b), room));
  s.first = a.window > 0 ? max(0, s.end - a.window) : 0;
  s.tile0 = s.first / S::kTokens;
  s.tiles = (s.end + S::kTokens - 1) / S::kTokens - s.tile0;
  return s;
}

// Walks a CTA's part of the line, segment by segment.  Producer and consumers walk alike.
template <typename S>
struct Walk {
  int b, seg, tile;  // sequence, segment in it, first tile (of the segment's) that is ours
  int take;          // how many tiles are ours
  long long pos, hi;
  Span span;

  __device__ __forceinline__ void start(const AttnArgs& a, int segs, int b0, long long off0, long long lo,
                                        long long hi_) {
    pos = lo;
    hi = hi_;
    b = b0;
    if (pos >= hi) return;
    span = span_of<S>(a, b);
    seg = int(off0 / span.tiles);
    tile = int(off0 - (long long)seg * span.tiles);
    take = int(min((long long)(span.tiles - tile), hi - pos));
  }
  __device__ __forceinline__ bool done() const { return pos >= hi; }
  __device__ __forceinline__ void next(const AttnArgs& a, int segs) {
    pos += take;
    tile = 0;
    if (pos >= hi) return;
    if (++seg == segs) {
      seg = 0;
      do span = span_of<S>(a, ++b);
      while (span.tiles == 0);  // pos < hi: a sequence with tiles follows
    }
    take = int(min((long long)span.tiles, hi - pos));
  }
};

// ------------------------------------------------------------------------- kernel -----------

template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_decode(const AttnArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  int box, int group, int head_blocks) {
  using Control = typename S::Control;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* exps = smem + S::kExpsAt;
  float* joined = reinterpret_cast<float*>(smem + S::kOutAt);
  Control* ctl = reinterpret_cast<Control*>(smem + S::kControlAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheDev& c = a.cache;
  const int segs = c.heads * head_blocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], S::kGroupWarps);
    }
    ctl->abort = 0;
    mbar_fence_init();
  }
  pdl_begin();

  // The line's length and the place where this CTA's part begins.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, int(threadIdx.x) * per), b_hi = min(a.B, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += (long long)span_of<S>(a, b).tiles * segs;
    if (blockIdx.x == 0 && __ldg(a.lens + b) > a.table.max_pages * c.page) report_bad_page(a.table.status_flags);
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) ctl->scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w <= kWarps; ++w) {
    if (w == warp) upto += total;
    total += ctl->scan[w];
  }
  const long long ctas = min((long long)gridDim.x, total);
  const bool working = blockIdx.x < ctas;
  const long long lo = working ? total * blockIdx.x / ctas : 0, hi = working ? total * (blockIdx.x + 1) / ctas : 0;
  if (lo < hi && lo >= upto - mine && lo < upto) {
    long long at = upto - mine;
    int b = b_lo;
    for (;; ++b) {
      const long long n = (long long)span_of<S>(a, b).tiles * segs;
      if (lo < at + n) break;
      at += n;
    }
    ctl->b0 = b;
    ctl->off0 = lo - at;
  }
  __syncthreads();

  Walk<S> walk;
  walk.start(a, segs, ctl->b0, ctl->off0, lo, hi);
  int it = 0;  // tiles of this CTA so far: the ring's position

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer --------------
    const int boxes = S::kTokens / box;
    const uint32_t box_bits = (1u << (box / 16)) - 1u;
    const uint32_t box_bytes = uint32_t(box) * (2 * S::kRow + (S::kE4M3 ? 2 : 0));
    bool ok = true;
    for (; ok && !walk.done(); walk.next(a, segs)) {
      const int kv = walk.seg / head_blocks;
      const int32_t* pages = a.table.pages + int64_t(walk.b) * a.table.max_pages;
      const int t_end = walk.span.tile0 + walk.tile + walk.take;
      // a box's page: looked up a tile ahead of its copies
      auto look_up = [&](int tile) {
        const int p = tile * S::kTokens + lane * box;
        return lane < boxes && tile < t_end && p < walk.span.end && p + box > walk.span.first ? __ldg(pages + p / c.page)
                                                                                             : -1;
      };
      int page = look_up(walk.span.tile0 + walk.tile);
      for (int tile = walk.span.tile0 + walk.tile; tile < t_end; ++tile, ++it) {
        const int page_next = look_up(tile + 1);
        const int p0 = tile * S::kTokens + lane * box;
        const bool wanted = lane < boxes && p0 < walk.span.end && p0 + box > walk.span.first;
        const bool good = wanted && page >= 0 && page < c.n_pages;
        if (wanted && !good) report_bad_page(a.table.status_flags);
        const uint32_t copied = __ballot_sync(0xffffffffu, good);
        const int stage = it % S::kStages;
        ok = mbar_wait(&ctl->empty[stage], ((it / S::kStages) & 1) ^ 1, &ctl->abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          uint32_t bits = 0;
          for (int i = 0; i < boxes; ++i)
            if (copied >> i & 1) bits |= box_bits << (i * (box / 16));
          ctl->valid[stage] = bits;
          mbar_arrive_expect_tx(&ctl->full[stage], __popc(copied) * box_bytes);
        }
        __syncwarp();
        const uint32_t bar = smem_u32(&ctl->full[stage]);
        const uint32_t dst = smem_u32(smem + size_t(stage) * S::kStage);
        const int jobs = 2 * boxes * S::kSpans;  // keys first
        for (int j0 = 0; j0 < jobs; j0 += 32) {
          const int j = j0 + lane;
          const int i = j % boxes, span = j / boxes % S::kSpans, is_v = j / (boxes * S::kSpans);
          const int pg = __shfl_sync(0xffffffffu, page, i);
          if (j < jobs && (copied >> i & 1)) {
            const int p = tile * S::kTokens + i * box;
            tma_load_4d(dst + is_v * S::kTile + span * (S::kTokens * S::kSpan) + i * box * S::kSpan,
                        is_v ? &map_v : &map_k, span * S::kSpanElems, p % c.page, kv, pg, bar);
          }
        }
        if constexpr (S::kE4M3) {
          const int i = lane % boxes, is_v = lane / boxes;  // boxes <= 8
          const int pg = __shfl_sync(0xffffffffu, page, i);
          if (is_v < 2 && (copied >> i & 1)) {
            const int p = tile * S::kTokens + i * box;
            const uint8_t* src = (is_v ? c.v_exp : c.k_exp) + (int64_t(pg) * c.heads + kv) * c.page + p % c.page;
            bulk_g2s(exps + stage * S::kExps + is_v * S::kTokens + i * box, src, box, &ctl->full[stage]);
          }
        }
        page = page_next;
      }
    }
    if (!ok && lane == 0) {
      // some wait ran out: this CTA's copies must land before it ends (bounded again)
      report_timeout_flag(a.table.status_flags, 40);
      const unsigned long long t0 = global_timer_ns();
      for (int i = max(0, it - S::kStages); i < it; ++i)
        while (!mbar_try_wait(&ctl->full[i % S::kStages], (i / S::kStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
    }
    return;
  }

  // ------------------------------------------------------------------ consumers -------------
  const int g = lane >> 2, t = lane & 3;
  const int wg = warp / S::kGroupWarps, row0 = (warp % S::kGroupWarps) * S::kPerWarp;
  constexpr int kMT = S::kPerWarp / 16;     // blocks of 16 tokens
  constexpr int kKS = S::kDim / 16;         // steps of 16 elements
  constexpr int kNB = S::kBlocks;
  bool timed_out = false;

  // sequences without a token: zeros
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (span_of<S>(a, b).tiles != 0) continue;
    const int n = a.n_heads * c.dim / 8;
    uint4* out = reinterpret_cast<uint4*>(a.out + int64_t(b) * a.n_heads * c.dim);
    for (int i = threadIdx.x; i < n; i += kWarps * 32) out[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int h = threadIdx.x; h < a.n_heads; h += kWarps * 32) a.lse[int64_t(b) * a.n_heads + h] = -INFINITY;
  }

  // ldmatrix addresses.  A 16-byte chunk i of row r of a tile lies at chunk i ^ (r % 8) of the row
  // (128-byte rows), or i ^ (r / 2 % 4) (64-byte rows).  `lo_row`: lanes 8-15 and 24-31 address rows
  // 8 further, lanes 16-31 the next chunk; `lo_chunk` the other way round.
  constexpr bool kNarrow = S::kSpan == 64;
  const int r8 = lane & 7;
  auto swizzle = [&](int row) { return kNarrow ? (row >> 1) & 3 : row & 7; };
  const int a_row = row0 + r8 + ((lane >> 3) & 1) * 8, a_hi = lane >> 4;
  const int v_row = S::kE4M3 ? a_row : row0 + r8 + (lane >> 4) * 8, v_hi = S::kE4M3 ? a_hi : (lane >> 3) & 1;
  const uint32_t k_off = uint32_t(a_row * S::kSpan), k_x = uint32_t((a_hi ^ swizzle(a_row)) << 4);
  const uint32_t v_off = uint32_t(v_row * S::kSpan), v_x = uint32_t((v_hi ^ swizzle(v_row)) << 4);
  // byte offset of chunks 2 i (and 2 i + 1, by lane) in a tile; rows 16 further do not change the swizzle
  constexpr int kPairs = S::kSpan / 32;
  auto chunk = [&](int i, uint32_t x) {
    return uint32_t(i / kPairs * (S::kTokens * S::kSpan)) + (uint32_t((i % kPairs) << 5) ^ x);
  };

  for (; !walk.done(); walk.next(a, segs)) {
    const int kv = walk.seg / head_blocks, hb = walk.seg % head_blocks;
    const int head0 = kv * group + hb * S::kHeads;             // first query head
    const int heads = min(S::kHeads, group - hb * S::kHeads);  // of this segment

    // the queries as B fragments: lane (g, t) has head g's elements 2t, 2t+1, 2t+8, 2t+9 of each
    // step (bf16), or 4t .. 4t+3 (E4M3: the order in which ldmatrix delivers the codes)
    uint32_t qf[kKS][kNB][2];
    float factor[kNB][2];  // scores to base-2 exponents, for heads 2t and 2t+1
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      const bool live = nb * 8 + g < heads;
      const __nv_bfloat16* q = a.q + walk.b * a.q_stride + int64_t(head0 + (live ? nb * 8 + g : 0)) * c.dim;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        const bool in = live && ks * 16 < c.dim;  // head_dim is a multiple of 16
        if constexpr (S::kE4M3) {
          const uint2 u = in ? *reinterpret_cast<const uint2*>(q + ks * 16 + 4 * t) : make_uint2(0, 0);
          qf[ks][nb][0] = u.x;
          qf[ks][nb][1] = u.y;
        } else {
          qf[ks][nb][0] = in ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 2 * t) : 0;
          qf[ks][nb][1] = in ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 2 * t + 8) : 0;
        }
      }
      factor[nb][0] = factor[nb][1] = a.scale * kLog2e;
      if constexpr (S::kE4M3) {
        // head g's queries times 2^-e, the largest between 2^14 and 2^15, as fp16
        float top = 0.0f;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[ks][nb][i] << 16)),
                                   fabsf(__uint_as_float(qf[ks][nb][i] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(113, max(-100, int(__float_as_uint(top) >> 23) - 127 - 14));
        const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[ks][nb][i] = pack_half2(__uint_as_float(qf[ks][nb][i] << 16) * down,
                                       __uint_as_float(qf[ks][nb][i] & 0xffff0000u) * down);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          factor[nb][i] *= __uint_as_float(uint32_t(127 + __shfl_sync(0xffffffffu, e, 8 * t + 4 * i)) << 23);
      }
    }

    float m[kNB][2], sum[kNB][2], acc[kKS][kNB][4];
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nb][i] = -INFINITY, sum[nb][i] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[ks][nb][i] = 0.0f;

    const int t_begin = walk.span.tile0 + walk.tile;
    for (int n = 0; n < walk.take; ++n, ++it) {
      if (it % S::kGroups != wg) continue;
      const int stage = it % S::kStages;
      if (!mbar_wait(&ctl->full[stage], (it / S::kStages) & 1, &ctl->abort)) timed_out = true;
      const uint32_t k_tile = smem_u32(smem + size_t(stage) * S::kStage), v_tile = k_tile + S::kTile;
      const int pos0 = (t_begin + n) * S::kTokens + row0;  // of this warp's first token
      const uint32_t valid = ctl->valid[stage] >> (row0 / 16);
      constexpr uint32_t kAll = (1u << kMT) - 1u;
      const bool whole = (valid & kAll) == kAll && pos0 >= walk.span.first && pos0 + S::kPerWarp <= walk.span.end;

      if ((valid & kAll) != 0) {
        // scores: tokens g and g + 8 of each block, heads 2t and 2t + 1
        float s[kMT][kNB][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          float s2[kNB][4];  // two chains of products
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][nb][i] = s2[nb][i] = 0.0f;
          const uint32_t rows = k_tile + k_off + mt * 16 * S::kSpan;
          if constexpr (S::kE4M3) {
#pragma unroll
            for (int ks = 0; ks < kKS; ks += 2) {
              uint32_t r[4];
              ldmatrix4(rows + chunk(ks / 2, k_x), r);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a0 = half2_of_codes(r[2 * h] & 0xffffu), a1 = half2_of_codes(r[2 * h + 1] & 0xffffu);
                const uint32_t a2 = half2_of_codes(r[2 * h] >> 16), a3 = half2_of_codes(r[2 * h + 1] >> 16);
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb)
                  mma<true>(h ? s2[nb] : s[mt][nb], a0, a1, a2, a3, qf[ks + h][nb][0], qf[ks + h][nb][1]);
              }
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
              uint32_t r[4];
              ldmatrix4(rows + chunk(ks, k_x), r);
#pragma unroll
              for (int nb = 0; nb < kNB; ++nb)
                mma<false>(ks & 1 ? s2[nb] : s[mt][nb], r[0], r[1], r[2], r[3], qf[ks][nb][0], qf[ks][nb][1]);
            }
          }
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][nb][i] += s2[nb][i];
        }

        // exponents: t of each (token, head), and the values' exponents
        float c_exp[kMT][2], c_unit[kMT][2];  // of tokens g and g + 8: in m, and as a factor
        float top[kNB][2];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) top[nb][0] = top[nb][1] = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + g;
            const bool seen = whole || ((valid >> mt & 1) && pos0 + r >= walk.span.first && pos0 + r < walk.span.end);
            float unit = 1.0f;
            c_exp[mt][half] = 0.0f;
            c_unit[mt][half] = 1.0f;
            if constexpr (S::kE4M3) {
              const uint8_t* e = exps + stage * S::kExps + row0 + r;
              unit = exp_value(e[0]);
              const uint32_t ve = e[S::kTokens];
              c_exp[mt][half] = float(max(int(ve) - kExpBias, kMinExp));
              c_unit[mt][half] = seen ? exp_value(ve) : 0.0f;
            }
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float& x = s[mt][nb][2 * half + i];
                x = seen ? x * (factor[nb][i] * unit) : -INFINITY;
                top[nb][i] = fmaxf(top[nb][i], x + c_exp[mt][half]);
              }
          }
        float base[kNB][2], fix[kNB][2];
        bool moved = false;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float now = fmaxf(m[nb][i], max_over_rows(top[nb][i]));
            base[nb][i] = now == -INFINITY ? 0.0f : now;  // nothing seen yet: exp2(-inf - 0) = 0
            fix[nb][i] = exp2_fast(m[nb][i] - base[nb][i]);
            moved |= now != m[nb][i];
            m[nb][i] = now;
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            sum[nb][0] *= fix[nb][0];
            sum[nb][1] *= fix[nb][1];
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
              acc[ks][nb][0] *= fix[nb][0];
              acc[ks][nb][1] *= fix[nb][1];
              acc[ks][nb][2] *= fix[nb][0];
              acc[ks][nb][3] *= fix[nb][1];
            }
          }
        }
        // weights, as the B operand of the product with the values
        uint32_t w[kMT][kNB][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float p0 = exp2_fast(s[mt][nb][2 * half] - base[nb][0]);
              const float p1 = exp2_fast(s[mt][nb][2 * half + 1] - base[nb][1]);
              sum[nb][0] += p0;
              sum[nb][1] += p1;
              w[mt][nb][half] = transpose8x8(S::kE4M3 ? pack_half2(p0 * c_unit[mt][half], p1 * c_unit[mt][half])
                                                      : pack_bf16x2(p0, p1));
            }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          if (!(valid >> mt & 1)) continue;  // nothing was copied there (all weights are 0)
          // what lies in rows that are not seen is no number: 0 there (tokens 2t, 2t+1, 2t+8, 2t+9)
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
          if (!whole)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int p = pos0 + mt * 16 + half * 8 + 2 * t;
              keep[half] = (p >= walk.span.first && p < walk.span.end ? 0xffffu : 0u) |
                           (p + 1 >= walk.span.first && p + 1 < walk.span.end ? 0xffff0000u : 0u);
            }
          const uint32_t rows = v_tile + v_off + mt * 16 * S::kSpan;
          if constexpr (S::kE4M3) {
#pragma unroll
            for (int ks = 0; ks < kKS; ks += 2) {
              uint32_t r[4];
              ldmatrix4_trans(rows + chunk(ks / 2, v_x), r);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // codes of elements 2g (bytes 0 and 2: two tokens) and 2g + 1 (bytes 1 and 3)
                const uint32_t lo = r[2 * h] & (whole ? 0xffffffffu : keep[0]);
                const uint32_t hi = r[2 * h + 1] & (whole ? 0xffffffffu : keep[1]);
                const uint32_t a0 = half2_of_codes(__byte_perm(lo, 0, 0x4420)),
                               a1 = half2_of_codes(__byte_perm(lo, 0, 0x4431)),
                               a2 = half2_of_codes(__byte_perm(hi, 0, 0x4420)),
                               a3 = half2_of_codes(__byte_perm(hi, 0, 0x4431));
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) mma<true>(acc[ks + h][nb], a0, a1, a2, a3, w[mt][nb][0], w[mt][nb][1]);
              }
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
              uint32_t r[4];
              ldmatrix4_trans(rows + chunk(ks, v_x), r);
              if (!whole) r[0] &= keep[0], r[1] &= keep[0], r[2] &= keep[1], r[3] &= keep[1];
#pragma unroll
              for (int nb = 0; nb < kNB; ++nb)
                mma<false>(acc[ks][nb], r[0], r[1], r[2], r[3], w[mt][nb][0], w[mt][nb][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[stage]);
    }

    // -------- the warps' results of this segment joined in shared memory --------
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float s = sum_over_rows(sum[nb][i]);
        if (g == 0) {
          ctl->m[warp][nb * 8 + 2 * t + i] = m[nb][i];
          ctl->sum[warp][nb * 8 + 2 * t + i] = s;
        }
      }
    consumers_sync();
    float fix[kNB][2];
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = nb * 8 + 2 * t + i;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ctl->m[w][h]);
        const float base = top == -INFINITY ? 0.0f : top;
        fix[nb][i] = exp2_fast(m[nb][i] - base);
        if (warp == 0 && g == 0) {
          float all = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) all += ctl->sum[w][h] * exp2_fast(ctl->m[w][h] - base);
          ctl->total_m[h] = top;
          ctl->total_sum[h] = all;
        }
      }
    // A part of the width a warp and round, another one each round: every element is added up over
    // the warps in a fixed order, and all warps are busy.
    constexpr int kParts = kKS < kWarps ? kKS : kWarps, kPartSteps = kKS / kParts;
#pragma unroll 1
    for (int round = 0; round < kWarps; ++round) {
      const int part = (warp + round) % kWarps;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        if (part != ks / kPartSteps) continue;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* at = joined + (nb * 8 + 2 * t + i) * S::kOutLd + ks * 16;
            const float x0 = acc[ks][nb][i] * fix[nb][i], x1 = acc[ks][nb][2 + i] * fix[nb][i];
            float* p0 = at + (S::kE4M3 ? 2 * g : g);
            float* p1 = at + (S::kE4M3 ? 2 * g + 1 : g + 8);
            if (round == 0) {
              *p0 = x0;
              *p1 = x1;
            } else {
              *p0 += x0;
              *p1 += x1;
            }
          }
      }
      consumers_sync();
    }

    // -------- finished here, or a partial result --------
    const int vecs = c.dim / 8;
    const long long seg_at = walk.pos - walk.tile;  // the segment's place on the line
    if (walk.take == walk.span.tiles) {
      for (int i = threadIdx.x; i < heads * vecs; i += kWarps * 32) {
        const int h = i / vecs, d = (i - h * vecs) * 8;
        const float all = ctl->total_sum[h], scale = all == 0.0f ? 0.0f : 1.0f / all;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = joined[h * S::kOutLd + d + j] * scale;
        store_vec8(a.out + (int64_t(walk.b) * a.n_heads + head0 + h) * c.dim + d, v);
      }
      if (a.lse && threadIdx.x < heads) {
        const float all = ctl->total_sum[threadIdx.x];
        a.lse[int64_t(walk.b) * a.n_heads + head0 + threadIdx.x] =
            all == 0.0f ? -INFINITY : ctl->total_m[threadIdx.x] * kLn2 + logf(all);
      }
    } else {
      // slot 0: a segment that began before this CTA's part; slot 1: one that begins in it
      float* slots = reinterpret_cast<float*>(a.ws + kAttnPartialsAt);
      float* slot = slots + (size_t(blockIdx.x) * 2 + (walk.tile == 0)) * S::kSlot;
      for (int i = threadIdx.x; i < heads * c.dim / 4; i += kWarps * 32) {
        const int h = i / (c.dim / 4), d = (i - h * (c.dim / 4)) * 4;
        __stcg(reinterpret_cast<float4*>(slot + 2 * S::kHeads + h * S::kDim + d),
               *reinterpret_cast<const float4*>(joined + h * S::kOutLd + d));
      }
      if (threadIdx.x < heads) {
        __stcg(slot + threadIdx.x, ctl->total_m[threadIdx.x]);
        __stcg(slot + S::kHeads + threadIdx.x, ctl->total_sum[threadIdx.x]);
      }
      __threadfence();
      consumers_sync();
      // the CTAs whose parts hold the segment's first and last tile
      const int c0 = int(((seg_at + 1) * ctas - 1) / total);
      const int c1 = int(((seg_at + walk.span.tiles) * ctas - 1) / total);
      int* counter = reinterpret_cast<int*>(a.ws + kAttnTicketsAt) + c0;
      if (threadIdx.x == 0) {
        const int before = atomicAdd(counter, 1);
        ctl->last = before == c1 - c0;
        if (before == c1 - c0) *counter = 0;
      }
      consumers_sync();
      if (ctl->last) {
        __threadfence();
        const int n = c1 - c0 + 1;
        auto slot_of = [&](int i) { return slots + (size_t(c0 + i) * 2 + (i == 0)) * S::kSlot; };
        for (int h = warp; h < heads; h += kWarps) {
          float top = -INFINITY, all = 0.0f;
          for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(slot_of(i) + h));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float base = top == -INFINITY ? 0.0f : top;
          for (int i = lane; i < n; i += 32)
            all += __ldcg(slot_of(i) + S::kHeads + h) * exp2_fast(__ldcg(slot_of(i) + h) - base);
          all = warp_sum(all);
          if (lane == 0) {
            ctl->total_m[h] = base;
            ctl->total_sum[h] = all;
            if (a.lse)
              a.lse[int64_t(walk.b) * a.n_heads + head0 + h] = all == 0.0f ? -INFINITY : base * kLn2 + logf(all);
          }
        }
        consumers_sync();
        for (int i = threadIdx.x; i < heads * c.dim / 4; i += kWarps * 32) {
          const int h = i / (c.dim / 4), d = (i - h * (c.dim / 4)) * 4;
          const float base = ctl->total_m[h], all = ctl->total_sum[h];
          float v[4] = {};
#pragma unroll 8
          for (int k = 0; k < n; ++k) {
            const float* p = slot_of(k);
            const float f = exp2_fast(__ldcg(p + h) - base);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(p + 2 * S::kHeads + h * S::kDim + d));
            v[0] = fmaf(x.x, f, v[0]);
            v[1] = fmaf(x.y, f, v[1]);
            v[2] = fmaf(x.z, f, v[2]);
            v[3] = fmaf(x.w, f, v[3]);
          }
          const float scale = all == 0.0f ? 0.0f : 1.0f / all;
          *reinterpret_cast<uint2*>(a.out + (int64_t(walk.b) * a.n_heads + head0 + h) * c.dim + d) =
              make_uint2(pack_bf16x2(v[0] * scale, v[1] * scale), pack_bf16x2(v[2] * scale, v[3] * scale));
        }
      }
    }
    consumers_sync();  // the join buffer is free again
  }
  if (timed_out && lane == 0) report_timeout_flag(a.table.status_flags, 41);
}

// -------------------------------------------------------------------------- host ------------

// [n_pages, heads, page, dim] rows, boxes of `box` tokens of one head of one page and `span` bytes.
bool cache_map(CUtensorMap* map, const void* base, const CacheDev& c, int box, int span) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t elem = c.e4m3 ? 1 : 2;
  const cuuint64_t dims[4] = {cuuint64_t(c.dim), cuuint64_t(c.page), cuuint64_t(c.heads), cuuint64_t(c.n_pages)};
  const cuuint64_t strides[3] = {c.dim * elem, cuuint64_t(c.page) * c.dim * elem,
                                 cuuint64_t(c.heads) * c.page * c.dim * elem};
  const cuuint32_t boxes[4] = {cuuint32_t(span / elem), cuuint32_t(box), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn(map, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
            dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  static const int sms = [] {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
  }();
  return sms;
}

template <typename S>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  const CacheDev& c = a.cache;
  static const cudaError_t attr =
      cudaFuncSetAttribute(k_attn_decode<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::kSmem));
  if (attr != cudaSuccess) return attr;
  // tokens a copy: the largest power of two that divides a page, up to a tile
  const int box = std::min(S::kTokens, c.page & -c.page);
  CUtensorMap mk, mv;
  if (!cache_map(&mk, c.k, c, box, S::kSpan) || !cache_map(&mv, c.v, c, box, S::kSpan)) return cudaErrorInvalidValue;
  const int group = a.n_heads / c.heads;
  return launch_pdl(k_attn_decode<S>, dim3(std::min(sm_count(), kMaxCtas)), dim3(kThreads), S::kSmem, s, a, mk, mv, box,
                    group, (group + S::kHeads - 1) / S::kHeads);
}

// The kernel for a cache and group.  Blocks of 16 query heads where a group is larger than 8: a
// second pass over the keys and values costs more than the wider products.  Not at widths above
// 128, where 16 heads' accumulators do not fit the registers.
template <typename F>
auto with_shape(const CacheDev& c, int group, F f) {
  auto by_type = [&](auto e4m3) {
    constexpr bool E = decltype(e4m3)::value;
    if (c.dim <= 64) return group <= 8 ? f(Shape<E, 64, 1>{}) : f(Shape<E, 64, 2>{});
    if (c.dim <= 128) return group <= 8 ? f(Shape<E, 128, 1>{}) : f(Shape<E, 128, 2>{});
    return f(Shape<E, 256, 1>{});
  };
  return c.e4m3 ? by_type(std::true_type{}) : by_type(std::false_type{});
}

}  // namespace

size_t attn_workspace_bytes(const CacheDev& c, int n_heads, int) {
  return kAttnPartialsAt + with_shape(c, n_heads / c.heads, [](auto shape) {
           return size_t(kMaxCtas) * 2 * decltype(shape)::kSlot * sizeof(float);
         });
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) {
  return with_shape(a.cache, a.n_heads / a.cache.heads, [&](auto shape) { return launch<decltype(shape)>(a, s); });
}

}  // namespace moe
