// Attention of one new token a sequence over the paged key-value cache, in one pass over the keys
// and values.
//
//   out = sum_j w_j v_j / sum_j p_j,   p_j = exp2(t_j - m),   t_j = (scale log2 e) q.k_j
//
// with the running maximum m, the sum and the accumulator in fp32.  In an E4M3 cache key j is
// 2^a_j times its codes and value j is 2^c_j times its codes: 2^a_j multiplies the score, and the
// weight of value j's codes is w_j = p_j 2^c_j; there m is the maximum of t_j + c_j, so that no w_j
// is above 1 and the largest is close to it, however the rows' sizes differ.  p_j itself may then be
// anything from 2^-120 (beside values of the largest size) to 2^100 (kMinExp): see kAbove and scale_sum.
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
// In a CTA, two warps are producers: they look up pages and start the tiles' TMA copies into a ring of
// shared-memory stages.  Two more lay the next segments' queries out as operands.  Eight warps
// compute, in groups that take the tiles in turn; a warp has kPerWarp tokens of each of its group's
// tiles and its own m, sum and accumulator, and at a segment's end leaves them in shared memory and
// goes on.  Four warps add up the results of the groups that had a tile of the segment, write the
// output or the partial result, and join partial results.  So neither the copies nor the products
// wait for a segment's end (with all of that in the eight warps, 128 windows of 513 tokens took
// 31.4 us, like this 22.3).  A group passes over segments without a tile of its own, so that several
// short ones are worked on at once, each group with a join buffer of its own (177 sequences of up to
// 42 tokens, 8 kv heads of 8 query heads, 192 wide, E4M3: with all eight warps at every segment's
// end and one warp for the queries 79 us, with this 43, and 48 with the E4M3 form's small weights).
// A stage, and a join buffer, belongs to one group: a barrier's wait tells only the parity of the
// phase, so whoever waits for it has to have seen each of its phases.
//
// Code is short where it can be: sixteen warps run six programs, and where segments are short the
// instruction cache does not hold them.  So a tile's whole and its masked rows go one way (two copies of
// the product code, one without masks, gained 1 % on long rows, and cost 67 us against that 43, and
// 87 against 62 for 52 mixed lengths of up to 499 tokens, groups of 12, 256 wide).
//
// Starting a copy holds a warp up for 100 to 200 cycles, enough to fall behind the memory with the 2 KB
// copies of 16-token pages if it computes anything else there: there is no division a tile, each lane
// has its own copy of every tile worked out beforehand, and the copies of a tile are shared out between
// the two warps (32 mixed lengths, E4M3: one warp 22.8 us, two 20.5).
//
// Measured (GB300, bf16 unless said, 4 kv heads of 4 query heads, 128 wide): 64 sequences of up to 16k
// tokens 200 us, 1.37 GB at the measured copy rate; one of 64k tokens 28.9 us (69 % of that rate); one
// 513-token window 7.1 us, all of it latency (the lengths, the pages, the tile, the count of partial
// results and their joint are each a trip to memory).  What a call costs beyond its bytes is about
// 10 us: 3 to 4 until the first tile is there, 4 from the last tile to the end, and the launch.
//
// The products are warp MMAs with the tokens (scores) and the value elements (output) on the M
// side and the query heads on the N side, so that eight columns are the unit that a small group is
// padded to; a tcgen05 product has at least 64 rows on M, and its scores would have to travel
// through TMEM.  Keys and values reach the registers by ldmatrix from the swizzled tiles, the
// values transposed.
//
// An INT4 cache is read as a bf16 cache of its values, which bf16 holds exactly: the computing warps make the products'
// operands of the codes, scales and exponents (Int4Operands).  There the bytes are 0.57 an element and no longer the
// bound: 64 sequences of up to 16k tokens, 4 kv heads of 8 query heads, take 88 us, 59 % of the copy rate (the same tokens
// in E4M3 137 us, 68 %, in bf16 182, all of it).
// Without the products the copies take 61 us (a tile's copies are small: codes by TMA, scales and exponents by cp.async);
// without the copies the products take 86, 45 of them to take codes apart.  That is 11 instructions for eight codes, and
// an AND-OR, a shift, a byte permutation and a packed multiply-add take two cycles each of a scheduler, the last not beside
// the others (ANDs and packed multiply-adds in turn: 2.1 cycles each with two warps, 1.8 with four; ANDs and integer
// multiply-adds 1.1).  So more warps do not help (twelve in place of eight, with fewer registers each: 119 us against 110
// at the time), nor does shifting by multiplication (the high half takes four cycles: 110 against 102).
#pragma once

#include "batches.cuh"
#include "kv_rows.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;      // compute
constexpr int kProducers = 2;  // start copies
constexpr int kQueryWarp = kWarps + kProducers;
constexpr int kQueryWarps = 2;  // the second also zeroes the rows of empty sequences
constexpr int kEndWarp = kWarps + 4;  // the first of those that end segments
constexpr int kEndThreads = 128;
constexpr int kThreads = kEndWarp * 32 + kEndThreads;
// Registers a thread of the four warpgroups (compute twice, producers, segment ends); the launch gives
// each 128, and the shares add up to that.
constexpr int kComputeRegs = 160, kProducerRegs = 80, kEndRegs = 112;
static_assert(2 * kComputeRegs + kProducerRegs + kEndRegs <= 4 * (65536 / kThreads), "registers");
constexpr size_t kSmemLimit = 227 * 1024;
constexpr int kMaxCtas = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMinExp = -100;  // least value exponent that enters m: keeps the sum inside fp32's range
static_assert(kMaxCtas <= kAttnTickets, "a counter a CTA");

template <RowKind kRows_, int kDim_, int kHeads_, bool kShort = false>
struct Shape {
  static constexpr RowKind kRows = kRows_;
  static constexpr bool kE4M3 = kRows == RowKind::kE4M3, kInt4 = kRows == RowKind::kInt4;
  using Args = std::conditional_t<kInt4, AttnScaledArgs, AttnArgs>;
  static constexpr int kDim = kDim_;      // head_dim rounded up to 64, 128 or 256 (copies fill with zeros)
  static constexpr int kHeads = kHeads_;  // query heads of a segment
  static constexpr int kRow = kE4M3 ? kDim : kInt4 ? kDim / 2 : kDim * 2;  // bytes
  static constexpr int kSpan = kRow < 128 ? kRow : 128;     // bytes of a row in one swizzled copy
  static constexpr int kSpans = kRow / kSpan;
  static constexpr int kSpanElems = kDim / kSpans;
  // 32 KB stages (16 KB for the narrowest rows); 16 or 32 tokens a warp, those of one product with the
  // values (INT4: 32 or 64)
  // INT4: stages of half the bytes up to 128 wide, but 256 tokens, as the producers' work a tile is most of a tile's time
  // with fewer (64 x 16k tokens, 8 heads a kv head: 90 us, with 128 tokens 105); 64 of them a warp where the registers
  // hold their scores.  With 128 tokens where segments are short, as more warps then share one (128
  // windows of 513: 23.3 us against 27.4; 177 sequences of up to 42: 19.4 against 25.8).
  static constexpr bool kWide = kInt4 && kRow <= 64 && !kShort;
  static constexpr int kTokens = kWide ? 256 : kRow <= 128 ? 128 : 128 * 128 / kRow;
  static constexpr int kPerWarp = kWide && kHeads == 8 ? 64 : kE4M3 || kInt4 ? 32 : 16;
  static constexpr int kGroupWarps = kTokens / kPerWarp;
  static constexpr int kGroups = kWarps / kGroupWarps;
  static constexpr int kTile = kTokens * kRow;
  static constexpr int kScales = kInt4 ? kTokens * (kDim / 16) : 0;  // room for the keys', or the values', scales
  // the keys' and the values' exponents, then their scales
  static constexpr int kExps = kE4M3 || kInt4 ? 2 * kTokens + 2 * kScales : 0;
  static constexpr int kStage = 2 * kTile;
  // the queries of kSlots segments as B operands: kQueryRegs registers a lane, and a factor a head
  static constexpr int kQueryRegs = kE4M3 ? kDim / 32 * (kHeads / 4) * 2 : kDim / 16 * (kHeads / 8) * 2;
  static constexpr int kQueries = kQueryRegs * 128 + kHeads * 4;
  static constexpr int kSlots = 4;
  // the join buffer: kPassDim elements of every warp's accumulators at a time, rows padded against
  // bank conflicts (two heads a lane group in the bf16 form, one in the E4M3 form)
  static constexpr int kPassDim = kDim < 1024 / kHeads ? kDim : 1024 / kHeads;
  static constexpr int kPasses = kDim / kPassDim;
  static constexpr int kJoinRow = kPassDim + (kE4M3 ? 8 : 4);
  static constexpr int kJoinWarp = kHeads * kJoinRow;        // floats
  static constexpr int kSlot = kHeads * (kDim + 2);          // floats of a partial result
  static constexpr int kMaxStages = 16;
  struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages], q_full[kSlots], q_empty[kSlots];
    uint64_t join_full[kGroups], join_empty[kGroups], merge_full;
    uint32_t valid[kMaxStages];  // a bit for each 16 tokens of the tile: copied
    int abort;
    int b0, off0, last, scan[kThreads / 32];
    float m[kWarps][kHeads], sum[kWarps][kHeads];
  };
  // layout: stages, exponents, queries, join buffer, control; 1 KB to align the stages
  static constexpr size_t kFixed = size_t(kSlots) * kQueries + size_t(kWarps) * kJoinWarp * 4 + sizeof(Control) + 1024;
  static constexpr int kRoom = int((kSmemLimit - kFixed) / (kStage + kExps));
  // a multiple of the groups: each has as many stages as the others
  static constexpr int kWanted = 192 * 1024 / kStage < kMaxStages ? 192 * 1024 / kStage : kMaxStages;
  static constexpr int kStages = (kRoom < kWanted ? kRoom : kWanted) / kGroups * kGroups;
  static constexpr size_t kExpsAt = size_t(kStages) * kStage;
  static constexpr size_t kQueriesAt = kExpsAt + size_t(kStages) * kExps;
  static constexpr size_t kJoinAt = kQueriesAt + size_t(kSlots) * kQueries;
  static constexpr size_t kControlAt = kJoinAt + size_t(kWarps) * kJoinWarp * 4;
  static constexpr size_t kSmem = kControlAt + sizeof(Control) + 1024;
  static_assert(kSmem <= kSmemLimit && kStages >= 4 && kStages <= kMaxStages, "shared memory");
  static_assert(kGroupWarps >= 1 && kWarps % kGroupWarps == 0, "groups");
  static_assert(kQueries % 16 == 0 && kJoinAt % 16 == 0 && kControlAt % 16 == 0, "alignment");
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
__device__ __forceinline__ void mma_bf16_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {  // exp2(-inf) = 0; relative error 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes (low half of `codes`) as fp32.
__device__ __forceinline__ float2 float2_of_codes(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes), __NV_E4M3)));
}
// Rows from `row` on (a box of a map made by cache_map), from element x on.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int x, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(row), "r"(0), "r"(smem_u32(bar))
      : "memory");
}
// mbar_wait, without its look at the clock where the phase is over already.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort) {
  return mbar_try_wait(bar, parity) || mbar_wait(bar, parity, abort);
}
// The same for what takes as long as a CTA's part of a segment does, which a call over the whole memory
// can stretch past mbar_wait's limit; a CTA that is stuck sets `abort` long before.
constexpr unsigned long long kPartLimitNs = 5ull * 1000 * 1000 * 1000;
__device__ __forceinline__ bool wait_part(uint64_t* bar, uint32_t parity, int* abort) {
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u) {
      if (*static_cast<volatile int*>(abort)) return false;
      if (global_timer_ns() - t0 > kPartLimitNs) {
        *static_cast<volatile int*>(abort) = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// `sum` times 2^d, d <= 0; returns 2^d.  In the E4M3 form 2^d may be too small for a float where the sum it
// scales is large: in two steps of 2^(d / 2).
template <typename S>
__device__ __forceinline__ float scale_sum(float& sum, float d) {
  if constexpr (S::kE4M3) {
    const float half = exp2_fast(0.5f * d);
    sum = sum * half * half;
    return half * half;
  } else {
    const float f = exp2_fast(d);
    sum *= f;
    return f;
  }
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
__device__ __forceinline__ void end_sync() { named_bar_sync(1, kEndThreads); }  // of the warps that end segments
__device__ __forceinline__ bool end_all(bool ok) {  // end_sync, and whether `ok` holds for all of them
  int all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(int(ok)), "n"(kEndThreads)
      : "memory");
  return all != 0;
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ----------------------------------------------------------------------- the split ----------

struct Span {  // the tokens of one sequence that are seen, and their tiles
  int first, end, tile0, tiles;
};

template <typename S>
__device__ __forceinline__ Span span_of_len(const AttnArgs& a, int len) {
  const int room = a.table.max_pages * a.cache.page;
  Span s;
  s.end = max(0, min(len, room));
  s.first = a.window > 0 ? max(0, s.end - a.window) : 0;
  s.tile0 = s.first / S::kTokens;
  s.tiles = (s.end + S::kTokens - 1) / S::kTokens - s.tile0;
  return s;
}

template <typename S>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  return span_of_len<S>(a, a.lens[b]);
}

// Walks a CTA's part of the line, segment by segment.  The length of the sequence to come is read one
// sequence ahead: where they are short, a trip to memory would be most of a segment's time.
template <typename S>
struct Walk {
  int b, seg, tile;  // sequence, segment in it, first tile (of the segment's) that is ours
  int take;          // how many tiles are ours
  int pos, hi;       // on the line (below 2^31 tiles)
  int len_to_come;   // of sequence b + 1
  Span span;

  __device__ __forceinline__ void start(const AttnArgs& a, int b0, int off0, int lo, int hi_) {
    pos = lo;
    hi = hi_;
    b = b0;
    if (pos >= hi) return;
    len_to_come = a.lens[min(b + 1, a.B - 1)];
    span = span_of<S>(a, b);
    seg = unsigned(off0) / unsigned(span.tiles);
    tile = off0 - seg * span.tiles;
    take = min(span.tiles - tile, hi - pos);
  }
  __device__ __forceinline__ bool done() const { return pos >= hi; }
  __device__ __forceinline__ void next(const AttnArgs& a, int segs) {
    pos += take;
    tile = 0;
    if (pos >= hi) return;
    if (++seg == segs) {
      seg = 0;
      do {
        span = span_of_len<S>(a, len_to_come);
        len_to_come = a.lens[min(++b + 1, a.B - 1)];
      } while (span.tiles == 0);  // pos < hi: a sequence with tiles follows
    }
    take = min(span.tiles, hi - pos);
  }
  __device__ __forceinline__ int kv(int head_blocks) const {  // the segment's kv head
    return head_blocks == 1 ? seg : unsigned(seg) / unsigned(head_blocks);
  }
  __device__ __forceinline__ bool whole() const { return take == span.tiles; }  // the segment is all ours
};

// The line cut into the CTAs' parts: the first `more` have one tile more than the others.
struct Parts {
  int each, more;
  __device__ __forceinline__ Parts(int total, int ctas) {
    each = ctas > 0 ? unsigned(total) / unsigned(ctas) : 0;
    more = total - each * ctas;
  }
  __device__ __forceinline__ int begin(int cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ int owner(int tile) const {
    const int wide = more * (each + 1);
    return tile < wide ? unsigned(tile) / unsigned(each + 1) : more + unsigned(tile - wide) / unsigned(each);
  }
};

// ------------------------------------------------------------------------ a warp ------------

// What a consumer warp needs to know of a tile.
struct TileView {
  uint32_t k, v;          // shared-memory addresses of the key and value tiles
  const uint8_t* exps;    // of the keys; the values' follow kTokens further
  uint32_t exps_at, scales_at;  // INT4: shared-memory addresses of them, and of the keys' scales; the values'
                                // scales follow kScales further
  uint32_t seen;          // a bit for each of the warp's tokens
  uint32_t seen_more;     // of the second 32
};

// Addresses for ldmatrix.  A tile lies in shared memory box by box (the tokens of one copy, a multiple
// of 16), a box span by span.  A 16-byte chunk i of row r of a span lies at chunk i ^ (r % 8) of the row
// (128-byte rows), or i ^ (r / 2 % 4) (64-byte rows).
template <typename S>
struct Rows {
  uint32_t at[S::kPerWarp / 16], flip, span;
  __device__ __forceinline__ Rows(int row, int odd_chunk, int box) {
#pragma unroll
    for (int i = 0; i < S::kPerWarp / 16; ++i) {
      const int r = row + i * 16;
      at[i] = uint32_t(r / box * box * S::kRow + r % box * S::kSpan);
    }
    flip = uint32_t((odd_chunk ^ (S::kSpan == 64 ? (row >> 1) & 3 : row & 7)) << 4);
    span = uint32_t(box * S::kSpan);
  }
  // chunk 2 i (lanes whose odd_chunk is 1: 2 i + 1) of the lane's row, `block` blocks of 16 rows down
  // (which leaves the swizzle as it is)
  __device__ __forceinline__ uint32_t operator()(uint32_t tile, int block, int i) const {
    constexpr int kPairs = S::kSpan / 32;
    return tile + at[block] + i / kPairs * span + (uint32_t((i % kPairs) << 5) ^ flip);
  }
};

// Zeros in the rows of a tile of values that a warp (rows row0 .. row0 + kPerWarp - 1) does not see: what
// lies there may be no number, and a weight of 0 would not make it vanish.  Lanes take rows, and chunks
// in an order of their own against bank conflicts.
template <typename S>
__device__ __forceinline__ void clear_rows(uint32_t tile, int row0, int box, uint32_t seen, int lane) {
  constexpr int kLanes = 32 / S::kPerWarp;  // of a row
  const int i = lane % S::kPerWarp, r = row0 + i;
  if (seen >> i & 1) return;
  const uint32_t at = tile + uint32_t(r / box * box * S::kRow + r % box * S::kSpan);
  constexpr int kChunks = S::kSpan / 16;  // of a span
#pragma unroll 4
  for (int c = lane / S::kPerWarp; c < S::kRow / 16; c += kLanes) {
    const uint32_t chunk = at + c / kChunks * (box * S::kSpan) + (((c ^ r) & (kChunks - 1)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(chunk), "r"(0) : "memory");
  }
}

// INT4: the values of rows row0 .. row0 + 31 of a tile that are not seen made zeros by their scales and exponents, a
// lane a row.
template <typename S>
__device__ __forceinline__ void clear_scales(uint8_t* exps, int pitch, int row0, uint32_t seen, int lane) {
  if (seen >> lane & 1) return;
  exps[S::kTokens + row0 + lane] = kInt4Zero;
  uint32_t* s = reinterpret_cast<uint32_t*>(exps + 2 * S::kTokens + S::kScales + (row0 + lane) * pitch);
  for (int w = 0; w < pitch / 4; ++w) s[w] = 0u;
}

// A bf16 cache's operands: rows as they lie.
template <typename S>
struct Bf16Operands {
  static constexpr int kKS = S::kDim / 16, kNB = S::kHeads / 8;
  Rows<S> k_rows, v_rows;

  __device__ __forceinline__ Bf16Operands(int row0, int lane, int box, int)
      : k_rows(row0 + (lane & 15), lane >> 4, box), v_rows(row0 + (lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1, box) {}

  // Register [ks][nb][i] of lane (g, t): head nb * 8 + g, elements 16 ks + 8 i + 2t and the next.
  static __device__ __forceinline__ void lay_out(uint8_t* queries, const __nv_bfloat16* q, int heads, int dim, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t r[kNB][kKS][2];
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(q + int64_t(nb * 8 + g) * dim) + t;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i)  // head_dim is a multiple of 16
          r[nb][ks][i] = nb * 8 + g < heads && ks * 16 < dim ? row[ks * 8 + i * 4] : 0u;
    }
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int ks = 0; ks < kKS; ks += 2)
        *reinterpret_cast<uint4*>(queries + ((nb * kKS + ks) / 2 * 32 + lane) * 16) =
            make_uint4(r[nb][ks][0], r[nb][ks][1], r[nb][ks + 1][0], r[nb][ks + 1][1]);
  }

  __device__ __forceinline__ void key(const TileView& tv, int mt, int ks, uint32_t (&r)[4]) {
    ldmatrix4(k_rows(tv.k, mt, ks), r);
  }
  __device__ __forceinline__ void value(const TileView& tv, int mt, int ks, uint32_t (&r)[4]) {
    ldmatrix4_trans(v_rows(tv.v, mt, ks), r);
  }
  // Elements of head h, `j0` products of 16 elements on, out of the accumulators of kPassDim / 16 of them.
  template <typename Acc>
  static __device__ __forceinline__ void put(float* out, const Acc& acc, int j0, int nb, int i, int lane) {
#pragma unroll
    for (int j = 0; j < S::kPassDim / 16; ++j) {
      out[j * 16 + (lane >> 2)] = acc[j0 + j][nb][i];
      out[j * 16 + 8 + (lane >> 2)] = acc[j0 + j][nb][2 + i];
    }
  }
};

// An INT4 cache's operands: bf16 numbers made of the codes, n s 2^e exactly, so that all that follows is as over a bf16
// cache of these values.
//
// Codes are taken apart as kv_rows.cuh has it: eight take 11 instructions, and their u and -192 u three.
//
// Keys.  The products' element axis may be in any order that queries share: lane (g, t) reads a quarter t of rows g
// and g + 8 in whole words, so that a word is two products' operands and a lane needs the scales of its own quarter only.
// Values.  ldmatrix with transpose moves 16-bit units: four elements of one token.  Lane (g, t) gets unit g of a 16-byte
// chunk for tokens 2t and 2t + 1: a pair of codes is one element of two tokens, as the A operand of values^T takes it;
// rows g and g + 8 of a product are two elements of a unit.
//
// Rows that a warp does not see have their values' scales and exponents set to what makes u = 0, whatever the codes are.
// An exponent byte of 255 makes u an infinity or a NaN, and the values inf - inf.
template <typename S>
struct Int4Operands {
  static constexpr int kKS = S::kDim / 16, kNB = S::kHeads / 8;
  static constexpr int kWords = S::kDim / 32;       // of a lane's quarter of a row, eight codes each
  static constexpr int kPitchWords = S::kDim / 64;  // of a row's scales
  uint32_t k_at, k_flip, v_at, v_flip;  // rows and swizzle of the lane's key words and ldmatrix rows
  uint32_t k_scale_at, v_scale_at;      // of the lane's first rows
  int pitch, g, t;
  uint32_t pick[2];                     // byte selectors for the scales of two tokens
  uint32_t word[2][kWords], unit[2][kWords / 2], minus[2][kWords / 2];  // key rows g and g + 8
  uint32_t chunk[4], v_scale[4][kPitchWords], v_exp[2];
  uint32_t mask, one;                   // constants that the compiler is to keep in registers

  // 16-byte chunk i of row r lies at chunk i ^ flip(r)
  static __device__ __forceinline__ uint32_t swizzle(int r) {
    return S::kRow == 32 ? (r >> 2) & 1 : S::kRow == 64 ? (r >> 1) & 3 : r & 7;
  }
  __device__ __forceinline__ Int4Operands(int row0, int lane, int, int dim) : g(lane >> 2), t(lane & 3) {
    k_at = uint32_t((row0 + g) * S::kRow);
    k_flip = swizzle(row0 + g);  // rows 8 further have the same
    const int v_row = row0 + (lane & 15);
    v_at = uint32_t(v_row * S::kRow);
    v_flip = swizzle(v_row) ^ (lane >> 4);
    pitch = scale_pitch(dim);
    mask = kept(0x00780078u);
    one = kept(0x43004300u);
    // a quarter past the row's end holds no codes that count (the queries there are 0): any scale will do
    const int col = t * (S::kDim / 64);
    k_scale_at = uint32_t(g * pitch + (col * 16 < dim ? col : 0));
    v_scale_at = uint32_t(S::kScales + 2 * t * pitch);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t k = 2 * i + (g >> 2);
      pick[i] = k | (8 + k) << 4 | (4 + k) << 8 | (12 + k) << 12;  // 8 +: the byte's sign, 0 in every scale
    }
  }

  // Register [ks][nb][i] of lane (g, t): head nb * 8 + g; word ks / 2 of the quarter, its elements 2 (ks % 2) + i and 4
  // further.
  static __device__ __forceinline__ void lay_out(uint8_t* queries, const __nv_bfloat16* q, int heads, int dim, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint4 u[kNB][kWords];
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const int d = t * (S::kDim / 4) + w * 8;
        u[nb][w] = nb * 8 + g < heads && d < dim
                       ? *reinterpret_cast<const uint4*>(q + int64_t(nb * 8 + g) * dim + d)
                       : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint4 x = u[nb][w];
        *reinterpret_cast<uint4*>(queries + ((nb * kKS + 2 * w) / 2 * 32 + lane) * 16) =
            make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                       __byte_perm(x.y, x.w, 0x7632));
      }
  }

  static __device__ __forceinline__ uint32_t kept(uint32_t x) {
    asm volatile("" : "+r"(x));
    return x;
  }
  static __device__ __forceinline__ uint32_t lds8(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
  }
  static __device__ __forceinline__ uint32_t lds16(uint32_t at) {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at) : "memory");
    return r;
  }
  static __device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
  }
  // __byte_perm, whose selectors know no signs
  static __device__ __forceinline__ uint32_t permute(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
  }
  __device__ __forceinline__ void key(const TileView& tv, int mt, int ks, uint32_t (&r)[4]) {
    if (ks == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = mt * 16 + h * 8;  // the swizzle is that of row g
        const uint32_t at = tv.k + k_at + uint32_t(row * S::kRow);
        if constexpr (S::kDim == 64) {
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                       : "=r"(word[h][0]), "=r"(word[h][1])
                       : "r"(at + (((t >> 1) ^ k_flip) << 4) + (t & 1) * 8)
                       : "memory");
        } else {
#pragma unroll
          for (int i = 0; i < kWords / 4; ++i)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(word[h][4 * i]), "=r"(word[h][4 * i + 1]), "=r"(word[h][4 * i + 2]), "=r"(word[h][4 * i + 3])
                         : "r"(at + (((t * (kWords / 4) + i) ^ k_flip) << 4))
                         : "memory");
        }
        const uint32_t s = tv.scales_at + k_scale_at + uint32_t(row * pitch);
        const uint32_t bytes = S::kDim == 64 ? lds8(s) : S::kDim == 128 ? lds16(s) : lds32(s);
        const uint32_t e = (lds8(tv.exps_at + row + g) - kInt4Zero) * 0x00800080u;
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) {
          unit[h][i] = __byte_perm(bytes, 0u, 0x4040 + i * 0x0101) * 16u + e;
          minus[h][i] = int4_minus_192(unit[h][i]);
        }
      }
    }
    const int w = ks / 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a, b;
      int4_pair(word[h][w], ks & 1, mask, one, a, b);
      r[h] = int4_fma(a, unit[h][w / 2], minus[h][w / 2]);
      r[2 + h] = int4_fma(b, unit[h][w / 2], minus[h][w / 2]);
    }
  }

  // Product md: chunk md / 2 of 32 elements, elements 2 (md % 2) and the next of each unit of four.
  __device__ __forceinline__ void value(const TileView& tv, int mt, int md, uint32_t (&r)[4]) {
    if (md == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
        const uint32_t s = tv.scales_at + v_scale_at + uint32_t((mt * 16 + (i & 1) + (i >> 1) * 8) * pitch);
        if constexpr (S::kDim == 128) {
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v_scale[i][0]), "=r"(v_scale[i][1]) : "r"(s) : "memory");
        } else {
#pragma unroll
          for (int w = 0; w < kPitchWords; ++w) v_scale[i][w] = lds32(s + 4 * w);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t e = lds16(tv.exps_at + S::kTokens + mt * 16 + 2 * t + i * 8);
        v_exp[i] = __byte_perm(e, 0u, 0x4140) * 128u - kInt4Zero * 0x00800080u;
      }
    }
    if (md % 4 == 0) ldmatrix4_trans(tv.v + v_at + uint32_t(mt * 16 * S::kRow) + (((md / 2) ^ v_flip) << 4), chunk);
    const int c = md / 2, cc = c & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // tokens 2t and 2t + 1, and 8 further
      const uint32_t u = permute(v_scale[2 * i][c / 2], v_scale[2 * i + 1][c / 2], pick[cc]) * 16u + v_exp[i];
      const uint32_t m = int4_minus_192(u);
      uint32_t a, b;
      int4_pair(chunk[2 * cc + i], md & 1, mask, one, a, b);
      r[2 * i] = int4_fma(a, u, m);
      r[2 * i + 1] = int4_fma(b, u, m);
    }
  }
  template <typename Acc>
  static __device__ __forceinline__ void put(float* out, const Acc& acc, int j0, int nb, int i, int lane) {
#pragma unroll
    for (int j = 0; j < S::kPassDim / 16; j += 2)
      *reinterpret_cast<float4*>(out + j * 16 + (lane >> 2) * 4) =
          make_float4(acc[j0 + j][nb][i], acc[j0 + j][nb][2 + i], acc[j0 + j + 1][nb][i], acc[j0 + j + 1][nb][2 + i]);
  }
};

// One warp's running result where the operands are bf16.  Scores: keys (16 tokens x 16 elements)
// times queries; the weights, rounded to bf16 (the type of the values: a product's operands have
// one), go through an 8 x 8 transpose to become the B operand of values^T times weights.  Lane
// (g, t) = (lane / 4, lane % 4) holds tokens g and g + 8 of a block, and heads 2t and 2t + 1 of a
// block of eight.
template <typename S>
struct WarpBf16 {
  using Operands = std::conditional_t<S::kInt4, Int4Operands<S>, Bf16Operands<S>>;
  static constexpr int kMT = S::kPerWarp / 16, kKS = S::kDim / 16, kNB = S::kHeads / 8;
  uint32_t q[kKS][kNB][2];
  float m[kNB][2], sum[kNB][2], acc[kKS][kNB][4];
  float factor;  // scores to base-2 exponents
  Operands operands;
  int g, t;

  __device__ __forceinline__ WarpBf16(int row0, int lane, int box, int dim)
      : operands(row0, lane, box, dim), g(lane >> 2), t(lane & 3) {}

  static __device__ __forceinline__ void lay_out(uint8_t* queries, const __nv_bfloat16* q, int heads, int dim,
                                                 float scale_log2e, int lane) {
    Operands::lay_out(queries, q, heads, dim, lane);
    if (lane < S::kHeads) reinterpret_cast<float*>(queries + S::kQueryRegs * 128)[lane] = scale_log2e;
  }

  __device__ __forceinline__ void begin(const uint8_t* queries, int lane) {
    factor = *reinterpret_cast<const float*>(queries + S::kQueryRegs * 128);
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      m[nb][0] = m[nb][1] = -INFINITY;
      sum[nb][0] = sum[nb][1] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[ks][nb][i] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kKS; ks += 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(queries + ((nb * kKS + ks) / 2 * 32 + lane) * 16);
        q[ks][nb][0] = u.x, q[ks][nb][1] = u.y, q[ks + 1][nb][0] = u.z, q[ks + 1][nb][1] = u.w;
      }
    }
  }

  __device__ __forceinline__ void tile(const TileView& tv) {
    const uint32_t seen = tv.seen >> g;
    float s[kMT][kNB][4];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      float s2[kNB][4];  // two chains of products
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][nb][i] = s2[nb][i] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        uint32_t r[4];
        operands.key(tv, mt, ks, r);
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) mma_bf16_16x8x16(ks & 1 ? s2[nb] : s[mt][nb], r, q[ks][nb][0], q[ks][nb][1]);
      }
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = (s[mt][nb][i] + s2[nb][i]) * factor;
          if constexpr (S::kInt4) s[mt][nb][i] = x;
          else s[mt][nb][i] = seen >> (mt * 16 + (i >> 1) * 8) & 1 ? x : -INFINITY;
        }
    }
    if constexpr (S::kInt4) {  // the masks are a part of the time here, and few tiles need them
      if ((S::kPerWarp == 64 ? tv.seen & tv.seen_more : tv.seen) != 0xffffffffu) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((mt < 2 ? seen : tv.seen_more >> g) >> (mt % 2 * 16 + (i >> 1) * 8) & 1)) s[mt][nb][i] = -INFINITY;
      }
    }
    float base[kNB][2], fix[kNB][2];
    bool moved = false;
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = fmaxf(s[0][nb][i], s[0][nb][2 + i]);
#pragma unroll
        for (int mt = 1; mt < kMT; ++mt) top = fmaxf(top, fmaxf(s[mt][nb][i], s[mt][nb][2 + i]));
        const float now = fmaxf(m[nb][i], max_over_rows(top));
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
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[ks][nb][i] *= fix[nb][i & 1];
      }
    }
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
          w[mt][nb][half] = transpose8x8(pack_bf16x2(p0, p1));
        }
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        uint32_t r[4];
        operands.value(tv, mt, ks, r);
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) mma_bf16_16x8x16(acc[ks][nb], r, w[mt][nb][0], w[mt][nb][1]);
      }
    }
  }

  // m and sum [kHeads], and elements [pass * kPassDim, ...) of the accumulators [kHeads][kJoinRow]
  __device__ __forceinline__ void publish_sums(float* m_out, float* sum_out) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float all = sum_over_rows(sum[nb][i]);
        if (g == 0) {
          m_out[nb * 8 + 2 * t + i] = m[nb][i];
          sum_out[nb * 8 + 2 * t + i] = all;
        }
      }
  }
  template <int kPass>
  __device__ __forceinline__ void publish(float* out, int heads) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = nb * 8 + 2 * t + i;
        if (h >= heads) continue;  // columns without a head
        Operands::put(out + h * S::kJoinRow, acc, kPass * (S::kPassDim / 16), nb, i, g * 4 + t);
      }
  }
};

// One warp's running result over an E4M3 cache.  The codes go into the products as they are
// (converting them to a wider type would cost more instructions than all the rest): E4M3 x E4M3
// products with fp32 sums.
//
// A query element x of 8 significant bits, scaled by a power of two to below 2^8, is split into two
// E4M3 numbers, hi = round(x) and lo = 32 (x - hi): both exact, unless x is below 2^-14 of its head's
// largest (then off by at most 2^-22 of that).  A weight w is split likewise, hi + lo / 32 of 256 w,
// which leaves the error of a bf16 rounding (2^-8).  A block of eight columns is four heads: column
// 2h holds the hi of head h, column 2h + 1 its lo, so lane (g, t) has both products of head t and
// adds them up.
//
// The weights are taken relative to the maximum over the warp's own 32 tokens, and the product is added
// to the accumulator by an fp32 factor: a long row of small weights keeps its precision beside a large
// one.  The split holds the 2^-8 down to 2^-15 of that maximum; where weights are smaller (and not 0),
// they take a product of their own, 2^15 times as large, and so on, down to 2^-75 of it.  (They matter
// where the large weights meet values of 0.)  So the time depends on how far apart the scores are.  With
// one product for all weights of a tile 64 sequences of up to 8k tokens, groups of 8, took 68.9 us; like
// this 71 at scores of a standard deviation of 1 nat, 79 at 1.7, 97 at 3, 122 at 5 and 156 at 9 (groups of
// 4: 61, 62, 68, 82 and 104).  The products are a loop, not copies: see above on the size of the code
// (52 mixed lengths of up to 499 tokens, 256 wide: 77 us against 68).
//
// The values' codes: a register of ldmatrix with transpose holds elements 2g and 2g + 1 of tokens 2t
// and 2t + 1; a byte permutation of it and the one of tokens 2t + 8 and 2t + 9 gives the four
// tokens of one element that the A operand takes.  The weights come out of the 8 x 8 transpose of
// (token g, token g + 8) pairs in that same order.
template <typename S>
struct WarpE4M3 {
  static constexpr int kKS = S::kDim / 32, kNB = S::kHeads / 4, kMD = S::kDim / 16;
  // of 256 times the weights: the least that the split holds, and the factor of the next product; how many
  // products leave weights to another
  static constexpr float kLeast = 1.0f / 128.0f, kLift = 32768.0f;
  static constexpr int kRounds = 4;
  // Factors are taken 2^24 times as large, as exp2 gives no numbers below 2^-126, and the largest of a tile
  // may be 2^-120 (values of 2^128); at the other end there is room (2^100).
  static constexpr float kAbove = 24.0f;
  static __device__ __forceinline__ bool below_least(float x) {  // and above 0 (no weight is negative)
    return __float_as_uint(x) - 1u < __float_as_uint(kLeast) - 1u;
  }
  static_assert(S::kPerWarp == 32, "the 32 tokens of one product with the values");
  uint32_t q[kKS][kNB][2];
  float m[kNB], sum[kNB], factor[kNB], acc[kMD][kNB][2];
  Rows<S> rows;
  int g, t;

  __device__ __forceinline__ WarpE4M3(int row0, int lane, int box, int)
      : rows(row0 + (lane & 15), lane >> 4, box), g(lane >> 2), t(lane & 3) {}

  // The hi (x) and lo (y) codes of four query elements.
  static __device__ __forceinline__ uint2 split4(uint2 u, float down) {
    const float x0 = __uint_as_float(u.x << 16) * down, x1 = __uint_as_float(u.x & 0xffff0000u) * down;
    const float x2 = __uint_as_float(u.y << 16) * down, x3 = __uint_as_float(u.y & 0xffff0000u) * down;
    const uint32_t h01 = e4m3_code2(x0, x1), h23 = e4m3_code2(x2, x3);
    const float2 f01 = float2_of_codes(h01), f23 = float2_of_codes(h23);
    const uint32_t l01 = e4m3_code2((x0 - f01.x) * 32.0f, (x1 - f01.y) * 32.0f);
    const uint32_t l23 = e4m3_code2((x2 - f23.x) * 32.0f, (x3 - f23.y) * 32.0f);
    return make_uint2(h01 | h23 << 16, l01 | l23 << 16);
  }

  // Register [ks][nb][i] of lane (g, t): column g of block nb (head nb * 4 + g / 2, its hi or lo),
  // elements 32 ks + 16 i + 4t and the three after.  The two lanes of a head split the elements of an i
  // each and exchange.
  static __device__ __forceinline__ void lay_out(uint8_t* queries, const __nv_bfloat16* q, int heads, int dim,
                                                 float scale_log2e, int lane) {
    const int g = lane >> 2, t = lane & 3, odd = g & 1;
#pragma unroll 1
    for (int nb = 0; nb < kNB; ++nb) {
      const int h = nb * 4 + (g >> 1);
      const uint2* row = reinterpret_cast<const uint2*>(q + int64_t(h) * dim) + t + odd * 4;
      uint2 u[kKS];
      float top = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks)
        u[ks] = h < heads && ks * 32 + odd * 16 < dim ? row[ks * 8] : make_uint2(0u, 0u);
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[ks].x << 16)), fabsf(__uint_as_float(u[ks].x & 0xffff0000u))));
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[ks].y << 16)), fabsf(__uint_as_float(u[ks].y & 0xffff0000u))));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // times 2^-e the largest is in [2^7, 2^8)
      const int e = min(120, max(-100, int(__float_as_uint(top) >> 23) - 127 - 7));
      const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        const uint2 mine = split4(u[ks], down);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? mine.x : mine.y, 4);
        *reinterpret_cast<uint2*>(queries + ((nb * kKS + ks) * 32 + lane) * 8) =
            odd ? make_uint2(other, mine.y) : make_uint2(mine.x, other);
      }
      // a query with an infinity or NaN has no finite scores
      const float lost = top < INFINITY ? 1.0f : __uint_as_float(0x7fc00000u);
      if (t == 0 && !odd)
        reinterpret_cast<float*>(queries + S::kQueryRegs * 128)[h] =
            scale_log2e * (__uint_as_float(uint32_t(127 + e) << 23) * lost);
    }
  }

  __device__ __forceinline__ void begin(const uint8_t* queries, int lane) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      m[nb] = -INFINITY;
      sum[nb] = 0.0f;
      factor[nb] = reinterpret_cast<const float*>(queries + S::kQueryRegs * 128)[nb * 4 + t];
#pragma unroll
      for (int md = 0; md < kMD; ++md) acc[md][nb][0] = acc[md][nb][1] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        const uint2 u = *reinterpret_cast<const uint2*>(queries + ((nb * kKS + ks) * 32 + lane) * 8);
        q[ks][nb][0] = u.x, q[ks][nb][1] = u.y;
      }
    }
  }

  __device__ __forceinline__ void tile(const TileView& tv) {
    const uint32_t seen_bits = tv.seen >> g;
    float s[2][kNB][2];  // tokens g and g + 8 of both blocks, head t of each column block
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float d[kNB][4];
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[nb][i] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        uint32_t r[4];
        ldmatrix4(rows(tv.k, mt, ks), r);
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) mma_e4m3_16x8x32(d[nb], r[0], r[1], r[2], r[3], q[ks][nb][0], q[ks][nb][1]);
      }
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        s[mt][nb][0] = fmaf(d[nb][1], 1.0f / 32.0f, d[nb][0]);
        s[mt][nb][1] = fmaf(d[nb][3], 1.0f / 32.0f, d[nb][2]);
      }
    }
    float unit[2][2];  // 2^c of the tokens' values
    float top[kNB];
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) top[nb] = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + g;
        const bool seen = seen_bits >> (mt * 16 + half * 8) & 1;
        const float k_unit = exp_value(tv.exps[r]);
        const uint32_t ve = tv.exps[S::kTokens + r];
        const float c = float(max(int(ve) - kExpBias, kMinExp));
        unit[mt][half] = seen ? exp_value(ve) : 0.0f;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
          float& x = s[mt][nb][half];
          x = seen ? x * (factor[nb] * k_unit) : -INFINITY;
          top[nb] = fmaxf(top[nb], x + c);
        }
      }
    float base[kNB], now[kNB];  // the maximum over these tokens, less kAbove, and over all so far
    bool moved = false;
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      const float here = max_over_rows(top[nb]);
      now[nb] = fmaxf(m[nb], here);
      moved |= now[nb] != m[nb];
      base[nb] = here == -INFINITY ? 0.0f : here - kAbove;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        const float fix = scale_sum<S>(sum[nb], now[nb] == -INFINITY ? 0.0f : m[nb] - now[nb]);
        m[nb] = now[nb];
#pragma unroll
        for (int md = 0; md < kMD; ++md) acc[md][nb][0] *= fix, acc[md][nb][1] *= fix;
      }
    }
    float into[kNB];  // of the product, in the accumulator: 2^-8 for the 256 times the weights
    bool small = false;  // weights that are too small for the split beside the largest
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      // the factors' 2^(base - m), in two halves as in scale_sum; at most 2^-kAbove, also where nothing is seen
      const float half_f = exp2_fast(fminf(0.5f * (base[nb] - m[nb]), -0.5f * kAbove));
      float all = 0.0f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float& x = s[mt][nb][half];
          x = exp2_fast(x - base[nb]);
          all += x;
          x *= unit[mt][half] * (256.0f * 0x1p-24f);  // 256 times the weight
          small |= below_least(x);
        }
      sum[nb] = fmaf(all * half_f, half_f, sum[nb]);
      into[nb] = half_f * (0x1p24f / 256.0f) * half_f;
    }
    bool rest = __any_sync(0xffffffffu, small);
#pragma unroll 1
    for (int round = 1;; ++round) {
      uint32_t w[kNB][2];
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          // what is too small waits for the next round
          const float w0 = rest && s[mt][nb][0] < kLeast ? 0.0f : s[mt][nb][0];
          const float w1 = rest && s[mt][nb][1] < kLeast ? 0.0f : s[mt][nb][1];
          const uint32_t hi = e4m3_code2(w0, w1);
          const float2 f2 = float2_of_codes(hi);
          const uint32_t lo = e4m3_code2((w0 - f2.x) * 32.0f, (w1 - f2.y) * 32.0f);
          w[nb][mt] = transpose8x8(hi | lo << 16);
        }
#pragma unroll
      for (int i = 0; i < kKS; ++i) {
        uint32_t r[2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          ldmatrix4_trans(rows(tv.v, mt, i), r[mt]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // element 2g of tokens 2t, 2t + 8, 2t + 1, 2t + 9 (row g of the operand), and 2g + 1 (row g + 8)
          const uint32_t a0 = __byte_perm(r[0][2 * h], r[0][2 * h + 1], 0x6240);
          const uint32_t a1 = __byte_perm(r[0][2 * h], r[0][2 * h + 1], 0x7351);
          const uint32_t a2 = __byte_perm(r[1][2 * h], r[1][2 * h + 1], 0x6240);
          const uint32_t a3 = __byte_perm(r[1][2 * h], r[1][2 * h + 1], 0x7351);
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_e4m3_16x8x32(d, a0, a1, a2, a3, w[nb][0], w[nb][1]);
            float(&o)[2] = acc[2 * i + h][nb];
            o[0] = fmaf(fmaf(d[1], 1.0f / 32.0f, d[0]), into[nb], o[0]);
            o[1] = fmaf(fmaf(d[3], 1.0f / 32.0f, d[2]), into[nb], o[1]);
          }
        }
      }
      if (!rest) break;
      small = false;
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        into[nb] *= 1.0f / kLift;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float& x = s[mt][nb][half];
            x = x < kLeast ? x * kLift : 0.0f;
            small |= below_least(x);
          }
      }
      rest = round < kRounds && __any_sync(0xffffffffu, small);
    }
  }

  __device__ __forceinline__ void publish_sums(float* m_out, float* sum_out) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      const float all = sum_over_rows(sum[nb]);
      if (g == 0) {
        m_out[nb * 4 + t] = m[nb];
        sum_out[nb * 4 + t] = all;
      }
    }
  }
  template <int kPass>
  __device__ __forceinline__ void publish(float* out, int heads) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      const int h = nb * 4 + t;
      if (h >= heads) continue;
#pragma unroll
      for (int j = 0; j < S::kPassDim / 16; ++j) {
        const float(&o)[2] = acc[kPass * (S::kPassDim / 16) + j][nb];
        *reinterpret_cast<float2*>(out + h * S::kJoinRow + j * 16 + 2 * g) = make_float2(o[0], o[1]);
      }
    }
  }
};

// ------------------------------------------------------------------------- kernel -----------

// A segment whose partial results (a slot each: kHeads maxima, kHeads sums, [kHeads][kDim] elements) are
// complete and left to this CTA to join: those of CTAs c0 .. c0 + n - 1.
struct Joint {
  int c0, n, heads;
  int64_t row;  // of the first head in the output
};

// Joins them, by the kEndThreads threads that end segments.  The slots are copied to `stage` (room for
// `stage_bytes`) by bulk copies, all at once or as many as fit, their start spread over the warps
// (starting one takes 100 to 200 cycles).  For 38 slots, loads to registers take several rounds to L2
// (4.8 us), and 16-byte cp.async copies 8 us.  Each warp arrives with the bytes of its own copies.
// `round` counts the uses of the barrier; `ok` is whether all went well so far for the thread, and
// without that nothing is written.
template <typename S>
__device__ __forceinline__ bool join_partials(const AttnArgs& a, const float* slots, const Joint& j, uint8_t* stage,
                                              int stage_bytes, int tid, uint64_t* bar, int& round, bool ok) {
  constexpr int kEach = (S::kHeads * S::kDim / 4 + kEndThreads - 1) / kEndThreads;  // items (4 elements) a thread
  const int row_items = a.cache.dim / 4, items = j.heads * row_items;
  const int bytes = (2 * S::kHeads + j.heads * S::kDim) * 4;
  const int batch = min(j.n, stage_bytes / bytes);
  float top[kEach], all[kEach], v[kEach][4];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    top[e] = -INFINITY;
    all[e] = v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0.0f;
  }
  constexpr int kEndWarps = kEndThreads / 32;
  auto start = [&](int i0, int n) {
    const int w = tid / 32;
    if (tid % 32 == 0) mbar_arrive_expect_tx(bar, (n - w + kEndWarps - 1) / kEndWarps * bytes);  // n - w >= -2
    __syncwarp();
    for (int k = w + kEndWarps * (tid % 32); k < n; k += kEndThreads) {
      const int i = i0 + k;
      bulk_g2s(stage + k * bytes, slots + (size_t(j.c0 + i) * 2 + (i == 0)) * S::kSlot, bytes, bar);
    }
    __syncwarp();
  };
  // not cut short by the CTA's `abort`: the copies are under way, and have to land before the CTA ends
  auto landed = [&] { return mbar_wait_copies(bar, round++ & 1); };
  auto use = [&](int, int n) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int item = tid + e * kEndThreads;
      if (item >= items) continue;
      const int h = item / row_items, d = (item - h * row_items) * 4;
      const float before = top[e];
      for (int k = 0; k < n; ++k) top[e] = fmaxf(top[e], *reinterpret_cast<const float*>(stage + k * bytes + h * 4));
      const float base = top[e] == -INFINITY ? 0.0f : top[e];
      const float fix = scale_sum<S>(all[e], before - base);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[e][x] *= fix;
#pragma unroll 2
      for (int k = 0; k < n; ++k) {
        const float* p = reinterpret_cast<const float*>(stage + k * bytes);
        float sum = p[S::kHeads + h];
        const float f = scale_sum<S>(sum, p[h] - base);
        const float4 x = *reinterpret_cast<const float4*>(p + 2 * S::kHeads + h * S::kDim + d);
        all[e] += sum;
        v[e][0] = fmaf(x.x, f, v[e][0]);
        v[e][1] = fmaf(x.y, f, v[e][1]);
        v[e][2] = fmaf(x.z, f, v[e][2]);
        v[e][3] = fmaf(x.w, f, v[e][3]);
      }
    }
  };
  ok = in_batches(j.n, batch, ok, end_all, start, landed, use);
  if (!ok) return false;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int item = tid + e * kEndThreads;
    if (item >= items) continue;
    const int h = item / row_items, d = (item - h * row_items) * 4;
    const float scale = all[e] == 0.0f ? 0.0f : 1.0f / all[e];
    *reinterpret_cast<uint2*>(a.out + (j.row + h) * a.cache.dim + d) =
        make_uint2(pack_bf16x2(v[e][0] * scale, v[e][1] * scale), pack_bf16x2(v[e][2] * scale, v[e][3] * scale));
    if (d == 0 && a.lse) a.lse[j.row + h] = all[e] == 0.0f ? -INFINITY : top[e] * kLn2 + logf(all[e]);
  }
  return true;
}

template <int... I, typename F>
__device__ __forceinline__ void for_constants(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_decode(const typename S::Args a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  int box, int copies, int page_boxes, uint32_t page_magic, int group, int head_blocks) {
  using Control = typename S::Control;
  using Compute = std::conditional_t<S::kE4M3, WarpE4M3<S>, WarpBf16<S>>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* exps = smem + S::kExpsAt;
  uint8_t* queries = smem + S::kQueriesAt;
  float* join = reinterpret_cast<float*>(smem + S::kJoinAt);
  Control* ctl = reinterpret_cast<Control*>(smem + S::kControlAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheDev& c = a.cache;
  const int segs = c.heads * head_blocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      // each producer warp, and the lanes of those that copy exponents (E4M3) or exponents and scales (INT4)
      mbar_init(&ctl->full[i], kProducers + (S::kE4M3 ? 32 : S::kInt4 ? kProducers * 32 : 0));
      mbar_init(&ctl->empty[i], S::kGroupWarps);
    }
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], kWarps);
    }
    for (int i = 0; i < S::kGroups; ++i) {
      mbar_init(&ctl->join_full[i], S::kGroupWarps);
      mbar_init(&ctl->join_empty[i], kEndThreads / 32);
    }
    mbar_init(&ctl->merge_full, kEndThreads / 32);
    ctl->abort = 0;
    mbar_fence_init();
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  // What a producer warp needs that no earlier kernel writes: lane's copy of every tile (one of keys or
  // values, one span or all, one box).
  const int me = warp - kWarps;
  const int boxes = S::kTokens / box;    // of a tile: a power of two up to 16
  const int box_shift = __ffs(2 * copies) - 1, row_shift = __ffs(box) - 1;
  const uint32_t job_bytes = uint32_t(box * S::kRow) >> (box_shift - 1);
  const int job = lane * kProducers + me;  // values after keys, span by span, box by box
  const bool has_job = job < boxes << box_shift;
  const int job_box = has_job ? job >> box_shift : 0, job_span = (job & (2 * copies - 1)) >> 1;
  const CUtensorMap* job_map = job & 1 ? &map_v : &map_k;
  const uint32_t job_at = smem_u32(smem) + (job & 1) * S::kTile + job_box * box * S::kRow + job_span * box * S::kSpan;
  // INT4: the boxes that the lane's pieces of the scales belong to
  constexpr int kScalePieces = S::kInt4 ? (S::kScales / 16 + 31) / 32 : 1;
  const int pitch = scale_pitch(c.dim);
  int scale_box[kScalePieces] = {};
  if constexpr (S::kInt4) {
    static_assert(kProducers == 2, "one for the keys' scales and one for the values'");
#pragma unroll
    for (int i = 0; i < kScalePieces; ++i) scale_box[i] = min((lane + i * 32) * 16 / (box * pitch), boxes - 1);
  }
  pdl_begin();

  // The line's length and the place where this CTA's part begins.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, int(threadIdx.x) * per), b_hi = min(a.B, b_lo + per);
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += span_of<S>(a, b).tiles * segs;
    if (blockIdx.x == 0 && a.lens[b] > a.table.max_pages * c.page) report_bad_page(a.table.status_flags);
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) ctl->scan[warp] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) upto += total;
    total += ctl->scan[w];
  }
  const int ctas = min(int(gridDim.x), total);
  const Parts line(total, ctas);
  const bool working = blockIdx.x < ctas;
  const int lo = working ? line.begin(blockIdx.x) : 0, hi = working ? line.begin(blockIdx.x + 1) : 0;
  if (lo < hi && lo >= upto - mine && lo < upto) {
    int at = upto - mine, b = b_lo;
    for (;; ++b) {
      const int n = span_of<S>(a, b).tiles * segs;
      if (lo < at + n) break;
      at += n;
    }
    ctl->b0 = b;
    ctl->off0 = lo - at;
  }
  __syncthreads();

  // Every warp walks the CTA's part by itself; `it` counts its tiles (the ring's position), `seg` its
  // segments.  Only the producers' and the query warps' walks end early, at a wait that ran out: the
  // others go on through the same barriers on whatever they find, and the status record says that it
  // is no result.
  Walk<S> walk;
  walk.start(a, ctl->b0, ctl->off0, lo, hi);
  int it = 0, seg = 0;

  if (warp >= kWarps && warp < kEndWarp) {
    fewer_registers<kProducerRegs>();
    if (warp < kQueryWarp) {
      // --------------------------------------------------------------- producers ------------
      bool ok = true;
      for (; ok && !walk.done(); walk.next(a, segs)) {
        const int kv = walk.kv(head_blocks);
        const int t_begin = walk.span.tile0 + walk.tile;
        const int32_t* pages = a.table.pages + int64_t(walk.b) * a.table.max_pages;
        // The pages of 32 boxes at a time, a lane each, and of the next 32 ahead of their use; with the
        // row in the page (the division by the page size is not for every tile).
        struct Boxes {
          int page, row;
        };
        auto look_up = [&](int rel) {
          const int i = t_begin * boxes + rel + lane, p = i << row_shift;
          const int slot = page_boxes == 1 ? i : __umulhi(i, page_magic);  // i / page_boxes
          const bool wanted = rel + lane < walk.take * boxes && p < walk.span.end && p + box > walk.span.first;
          return Boxes{wanted ? pages[slot] : -1, (i - slot * page_boxes) << row_shift};
        };
        Boxes cur = look_up(0), ahead = look_up(32);
        for (int n = 0; n < walk.take; ++n, ++it) {
          const int off = (n * boxes) & 31;
          if (n > 0 && off == 0) {
            cur = ahead;
            ahead = look_up(n * boxes + 32);
          }
          // lane i < boxes: box i of the tile, its page and the row of the cache where it begins
          const int p0 = (t_begin + n) * S::kTokens + lane * box;
          const bool wanted = lane < boxes && p0 < walk.span.end && p0 + box > walk.span.first;
          const int page = __shfl_sync(0xffffffffu, cur.page, (off + lane) & 31);
          const int in_page = __shfl_sync(0xffffffffu, cur.row, (off + lane) & 31);
          const bool good = wanted && page >= 0 && page < c.n_pages;
          if (wanted && !good) report_bad_page(a.table.status_flags);
          const int row = good ? (page * c.heads + kv) * c.page + in_page : 0;  // below 2^31
          const uint32_t copied = __ballot_sync(0xffffffffu, good);
          const int job_row = __shfl_sync(0xffffffffu, row, job_box);
          const bool mine_too = has_job && (copied >> job_box & 1);
          const uint32_t bits = __ballot_sync(0xffffffffu, lane < S::kTokens / 16 && (copied >> (lane * 16 >> row_shift) & 1));
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine_too)) * job_bytes;
          const int stage = it % S::kStages;
          ok = __all_sync(0xffffffffu, wait(&ctl->empty[stage], ((it / S::kStages) & 1) ^ 1, &ctl->abort));
          if (!ok) break;
          uint64_t* bar = &ctl->full[stage];
          if (lane == 0) {
            if (me == 0) ctl->valid[stage] = bits;
            mbar_arrive_expect_tx(bar, bytes);
          }
          __syncwarp();
          if (mine_too) tma_load_rows(job_at + stage * S::kStage, job_map, job_span * S::kSpanElems, job_row, bar);
          if constexpr (S::kE4M3) {
            if (me == kProducers - 1) {
              // the exponents of 16 tokens a lane (16 bytes: too little for a bulk copy to pay)
              constexpr int kPieces = S::kTokens / 16;
              const int r = lane % kPieces * 16, i = r >> row_shift, is_v = lane / kPieces;
              const int y = __shfl_sync(0xffffffffu, row, i) + (r & (box - 1));
              if (is_v < 2 && (copied >> i & 1))
                cp_async16(exps + stage * S::kExps + is_v * S::kTokens + r, (is_v ? c.v_exp : c.k_exp) + y);
              cp_async_arrive_noinc(bar);
            }
          }
          if constexpr (S::kInt4) {
            // the keys' by one warp, the values' by the other; a lane's pieces of 16 bytes lie in one box each
            uint8_t* to = exps + stage * S::kExps;
#pragma unroll
            for (int i = 0; i < kScalePieces; ++i) {
              const int y = __shfl_sync(0xffffffffu, row, scale_box[i]);
              const int at = (lane + i * 32) * 16;
              if (at < S::kTokens * pitch && (copied >> scale_box[i] & 1))
                cp_async16(to + 2 * S::kTokens + me * S::kScales + at,
                           (me ? a.v_scale : a.k_scale) + int64_t(y) * pitch + (at - scale_box[i] * box * pitch));
            }
            const int r = lane * 16 & (S::kTokens - 1), i = r >> row_shift;
            const int y = __shfl_sync(0xffffffffu, row, i) + (r & (box - 1));
            if (lane < S::kTokens / 16 && (copied >> i & 1))
              cp_async16(to + me * S::kTokens + r, (me ? c.v_exp : c.k_exp) + y);
            cp_async_arrive_noinc(bar);
          }
        }
      }
      if (lane == 0) {
        if (!ok) report_timeout_flag(a.table.status_flags, 40);
        // this CTA's copies must land before it ends, whatever became of those who wait for them
        const unsigned long long t0 = global_timer_ns();
        for (int i = max(0, it - S::kStages); i < it; ++i)
          while (!mbar_try_wait(&ctl->full[i % S::kStages], (i / S::kStages) & 1) &&
                 global_timer_ns() - t0 < kWaitLimitNs) {
          }
      }
    } else {
      if (warp == kQueryWarp + 1) {
        // ----------------------------------------- sequences without a token: zeros ---------
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
          if (span_of<S>(a, b).tiles != 0) continue;
          const int n = a.n_heads * c.dim / 8;
          uint4* out = reinterpret_cast<uint4*>(a.out + int64_t(b) * a.n_heads * c.dim);
          for (int i = lane; i < n; i += 32) out[i] = make_uint4(0, 0, 0, 0);
          if (a.lse)
            for (int h = lane; h < a.n_heads; h += 32) a.lse[int64_t(b) * a.n_heads + h] = -INFINITY;
        }
      }
      // ------------------------------- queries, the segments in turn by the two warps -------
      for (; !walk.done(); walk.next(a, segs), ++seg) {
        if (seg % kQueryWarps != warp - kQueryWarp) continue;
        const int kv = walk.kv(head_blocks), hb = walk.seg - kv * head_blocks, slot = seg % S::kSlots;
        if (!__all_sync(0xffffffffu, wait_part(&ctl->q_empty[slot], ((seg / S::kSlots) & 1) ^ 1, &ctl->abort))) {
          if (lane == 0) report_timeout_flag(a.table.status_flags, 41);
          break;
        }
        Compute::lay_out(queries + slot * S::kQueries,
                         a.q + walk.b * a.q_stride + int64_t(kv * group + hb * S::kHeads) * c.dim,
                         min(S::kHeads, group - hb * S::kHeads), c.dim, a.scale * kLog2e, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->q_full[slot]);
      }
    }
    return;
  }

  if (warp < kWarps) {
    // ------------------------------------------------------------------ compute -------------
    more_registers<kComputeRegs>();
    const int wg = warp / S::kGroupWarps, row0 = (warp % S::kGroupWarps) * S::kPerWarp;
    bool timed_out = false;
    int joins = 0;  // the group's passes through the join buffer so far
    Compute mine_w(row0, lane, box, c.dim);
    for (; !walk.done(); it += walk.take, walk.next(a, segs), ++seg) {
      const int hb = walk.seg - walk.kv(head_blocks) * head_blocks, slot = seg % S::kSlots;
      const int n0 = unsigned(wg - it) % S::kGroups;  // the group's first tile of the segment
      if (!wait(&ctl->q_full[slot], (seg / S::kSlots) & 1, &ctl->abort)) timed_out = true;
      // (under a condition, n0 < walk.take, more registers spill: 16 heads, 64 x 8k bf16 68.1 us against 66.5)
      mine_w.begin(queries + slot * S::kQueries, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_empty[slot]);
      if (n0 >= walk.take) continue;
      TileView tv;
      for (int n = n0; n < walk.take; n += S::kGroups) {
        const int stage = (it + n) % S::kStages;
        if (!wait(&ctl->full[stage], ((it + n) / S::kStages) & 1, &ctl->abort)) timed_out = true;
        tv.k = smem_u32(smem + size_t(stage) * S::kStage);
        tv.v = tv.k + S::kTile;
        tv.exps = exps + stage * S::kExps + row0;
        tv.exps_at = smem_u32(tv.exps);
        tv.scales_at = tv.exps_at - row0 + 2 * S::kTokens + row0 * pitch;
        // the warp's tokens of the tile that lie in what is seen
        const int pos0 = (walk.span.tile0 + walk.tile + n) * S::kTokens + row0;
        constexpr int kWord = S::kPerWarp < 32 ? S::kPerWarp : 32;
        constexpr uint32_t kAll = 0xffffffffu >> (32 - kWord);
        auto seen_of = [&](int at) {  // [from, to) of kWord tokens
          const int from = max(0, walk.span.first - pos0 - at), to = min(kWord, walk.span.end - pos0 - at);
          uint32_t bits = from < to ? kAll >> (kWord - to + from) << from : 0u;
          const uint32_t copied = ctl->valid[stage] >> ((row0 + at) / 16);
          if (!(copied & 1)) bits &= ~0xffffu;
          if (kWord == 32 && !(copied & 2)) bits &= 0xffffu;
          return bits;
        };
        tv.seen = seen_of(0);
        tv.seen_more = S::kPerWarp == 64 ? seen_of(32) : 0u;
        if ((tv.seen | tv.seen_more) != 0) {
          if (tv.seen != kAll || (S::kPerWarp == 64 && tv.seen_more != kAll)) {
            if constexpr (S::kInt4) {
              // (written by cp.async, like these stores: no other proxy)
              uint8_t* const e = exps + stage * S::kExps;
              clear_scales<S>(e, pitch, row0, tv.seen, lane);
              if constexpr (S::kPerWarp == 64) clear_scales<S>(e, pitch, row0 + 32, tv.seen_more, lane);
            } else {
              clear_rows<S>(tv.v, row0, box, tv.seen, lane);
              fence_proxy_async_smem();  // before the next copy into these rows
            }
            __syncwarp();
          }
          mine_w.tile(tv);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->empty[stage]);
      }
      const int heads = min(S::kHeads, group - hb * S::kHeads);
      for_constants(std::make_integer_sequence<int, S::kPasses>{}, [&](auto pass) {
        constexpr int kPass = decltype(pass)::value;
        if (kPass * S::kPassDim >= c.dim) return;
        if (!wait(&ctl->join_empty[wg], (joins & 1) ^ 1, &ctl->abort)) timed_out = true;
        if (kPass == 0) mine_w.publish_sums(ctl->m[warp], ctl->sum[warp]);
        mine_w.template publish<kPass>(join + warp * S::kJoinWarp, heads);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->join_full[wg]);
        ++joins;
      });
    }
    if (timed_out) report_timeout_flag(a.table.status_flags, 42);  // any lane: each waits for itself
    return;
  }

  // ---------------------------------------------------------------------- segment ends ------
  fewer_registers<kEndRegs>();
  const int tid = threadIdx.x - kEndWarp * 32;
  bool timed_out = false;
  int n_joints = 0;
  uint32_t phases = 0;  // a bit for each group: the parity of its next pass through the join buffer
  Joint joints[2] = {};
  for (; !walk.done(); it += walk.take, walk.next(a, segs)) {
    const int kv = walk.kv(head_blocks), hb = walk.seg - kv * head_blocks;
    const int heads = min(S::kHeads, group - hb * S::kHeads);
    const int64_t row = int64_t(walk.b) * a.n_heads + kv * group + hb * S::kHeads;  // of the first head in out
    const bool whole = walk.whole();  // finished here, or a partial result
    float* slots = reinterpret_cast<float*>(a.ws + kAttnPartialsAt);
    // slot 0: a segment that began before this CTA's part; slot 1: one that begins in it
    float* slot = slots + (size_t(blockIdx.x) * 2 + (walk.tile == 0)) * S::kSlot;

    // -------- the results of the warps that had a tile of it --------
    uint32_t groups = 0;
#pragma unroll
    for (int i = 0; i < S::kGroups; ++i) groups |= uint32_t(i < walk.take) << unsigned(it + i) % S::kGroups;
    for (int d0 = 0; d0 < c.dim; d0 += S::kPassDim, phases ^= groups) {
#pragma unroll
      for (int i = 0; i < S::kGroups; ++i)
        if ((groups >> i & 1) && !wait_part(&ctl->join_full[i], phases >> i & 1, &ctl->abort)) timed_out = true;
      constexpr int kVecs = S::kPassDim / 4;
      for (int item = tid; item < heads * kVecs; item += kEndThreads) {
        const int h = item / kVecs, d = (item % kVecs) * 4;
        float top = -INFINITY, all = 0.0f, v[4] = {};
        auto top_of = [&](int w) { top = fmaxf(top, ctl->m[w][h]); };
        auto add = [&](int w, float base) {
          float sum = ctl->sum[w][h];
          const float f = scale_sum<S>(sum, ctl->m[w][h] - base);
          const float4 x = *reinterpret_cast<const float4*>(join + w * S::kJoinWarp + h * S::kJoinRow + d);
          all += sum;
          v[0] = fmaf(x.x, f, v[0]);
          v[1] = fmaf(x.y, f, v[1]);
          v[2] = fmaf(x.z, f, v[2]);
          v[3] = fmaf(x.w, f, v[3]);
        };
        if (groups == (1u << S::kGroups) - 1) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top_of(w);
          const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) add(w, base);
        } else {
          for (uint32_t left = groups; left; left &= left - 1)
#pragma unroll
            for (int k = 0; k < S::kGroupWarps; ++k) top_of((__ffs(left) - 1) * S::kGroupWarps + k);
          const float base = top == -INFINITY ? 0.0f : top;
          for (uint32_t left = groups; left; left &= left - 1)
#pragma unroll
            for (int k = 0; k < S::kGroupWarps; ++k) add((__ffs(left) - 1) * S::kGroupWarps + k, base);
        }
        if (whole) {
          const float scale = all == 0.0f ? 0.0f : 1.0f / all;
          if (d0 + d < c.dim)
            *reinterpret_cast<uint2*>(a.out + (row + h) * c.dim + d0 + d) =
                make_uint2(pack_bf16x2(v[0] * scale, v[1] * scale), pack_bf16x2(v[2] * scale, v[3] * scale));
          if (d0 == 0 && d == 0 && a.lse) a.lse[row + h] = all == 0.0f ? -INFINITY : top * kLn2 + logf(all);
        } else {
          if (d0 + d < c.dim)
            __stcg(reinterpret_cast<float4*>(slot + 2 * S::kHeads + h * S::kDim + d0 + d),
                   make_float4(v[0], v[1], v[2], v[3]));
          if (d0 == 0 && d == 0) {
            __stcg(slot + h, top);
            __stcg(slot + S::kHeads + h, all);
          }
        }
      }
      __syncwarp();
      if (lane < S::kGroups && (groups >> lane & 1)) mbar_arrive(&ctl->join_empty[lane]);
    }
    if (whole) continue;

    // -------- the last of the segment's CTAs joins the partial results, at its own end --------
    // the CTAs whose parts hold the segment's first and last tile
    const int c0 = line.owner(walk.pos - walk.tile);
    const int n = line.owner(walk.pos - walk.tile + walk.span.tiles - 1) - c0 + 1;
    // the joint reads them by bulk copies
    asm volatile("fence.proxy.async.global;" ::: "memory");
    end_sync();
    if (tid == 0) {
      int* counter = reinterpret_cast<int*>(a.ws + kAttnTicketsAt) + c0;
      // releases the partial result (which the barrier put before this) and acquires the others'
      int before;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
      const bool last = before == n - 1;
      asm volatile("fence.proxy.async.global;" ::: "memory");
      if (last) *counter = 0;
      ctl->last = last;
    }
    end_sync();
    if (ctl->last) {
      joints[1] = Joint{c0, n, heads, row};
      if (n_joints++ == 0) joints[0] = joints[1];
    }
  }
  // The ring is free by now: every tile has been used, or a wait ran out, and nothing is joined.  (A part
  // has at most two segments that it shares.)
  bool ok = !timed_out;
  int round = 0;
#pragma unroll 1
  for (int i = 0; i < n_joints; ++i)
    ok = join_partials<S>(a, reinterpret_cast<const float*>(a.ws + kAttnPartialsAt), i == 0 ? joints[0] : joints[1], smem,
                          int(S::kExpsAt), tid, &ctl->merge_full, round, ok);
  if (timed_out || !ok) report_timeout_flag(a.table.status_flags, 43);  // any lane
}

// -------------------------------------------------------------------------- host ------------

// A map of the cache's rows, [n_pages * heads * page, dim], for boxes of `box` rows.  Where a row is a
// whole number of swizzled spans, a box holds all of them, span after span (`spans` of them, those past
// the row's end as zeros); else a box is one span wide (and what lies past the row's end is zeros).
bool cache_map(CUtensorMap* map, const void* base, const CacheDev& c, int box, int span, int spans) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t elem = c.rows == RowKind::kBf16 ? 2 : 1, row = row_bytes(c.rows, c.dim);
  const cuuint64_t dims[3] = {spans > 1 ? span / elem : row / elem,
                              cuuint64_t(c.n_pages) * c.heads * c.page, spans > 1 ? row / span : 1};
  const cuuint64_t strides[2] = {row, cuuint64_t(span)};
  const cuuint32_t boxes[3] = {cuuint32_t(span / elem), cuuint32_t(box), cuuint32_t(spans)};
  const cuuint32_t ones[3] = {1, 1, 1};
  return fn(map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            span == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
            : span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                         : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename S>
cudaError_t launch(const typename S::Args& a, cudaStream_t s) {
  const CacheDev& c = a.cache;
  static std::atomic<int> ready[kMaxDevices];
  cudaError_t attr = cudaSuccess;
  once_a_device(ready, current_device(), [&attr] {
    cudaFuncAttributes f;
    attr = cudaFuncGetAttributes(&f, k_attn_decode<S>);
    // the warpgroups divide up what the launch gets: with less than they ask for they would wait for ever
    if (attr == cudaSuccess && 4 * f.numRegs < 2 * kComputeRegs + kProducerRegs + kEndRegs)
      attr = cudaErrorInvalidConfiguration;
    if (attr == cudaSuccess)
      attr = cudaFuncSetAttribute(k_attn_decode<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::kSmem));
    return int(attr == cudaSuccess);
  });
  if (attr != cudaSuccess) return attr;
  const int ctas = std::min(sm_count(), kMaxCtas);
  if (ctas <= 0) return cudaErrorInvalidDevice;
  // tokens a copy: the largest power of two that divides a page, up to a tile
  const int box = std::min(S::kTokens, c.page & -c.page);
  const int spans = c.dim % S::kSpanElems == 0 ? S::kSpans : 1;  // of a row in one copy
  CUtensorMap mk, mv;
  if (!cache_map(&mk, c.k, c, box, S::kSpan, spans) || !cache_map(&mv, c.v, c, box, S::kSpan, spans))
    return cudaErrorInvalidValue;
  const int group = a.n_heads / c.heads, page_boxes = c.page / box;
  // i / page_boxes = the high half of i * page_magic, for i below 2^32 / page_boxes: positions below 2^28
  // make at most 2^24 boxes of 16, and a page at most 256
  const uint32_t page_magic = uint32_t(((uint64_t(1) << 32) + page_boxes - 1) / page_boxes);
  return launch_pdl(k_attn_decode<S>, dim3(ctas), dim3(kThreads), S::kSmem, s, a, mk, mv, box,
                    S::kSpans / spans, page_boxes, page_magic, group, (group + S::kHeads - 1) / S::kHeads);
}

}  // namespace
}  // namespace moe
