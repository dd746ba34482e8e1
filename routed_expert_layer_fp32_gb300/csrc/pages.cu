// The pages and places of new tokens: page_plan and page_release.
//
// Both are prefix sums over the sequences (tokens, then the pages of those whose tokens fit) followed by a pass over
// what they address (the new tokens, or the pages given back).  The sums are one CTA's work, a run of sequences a
// thread; the pass is the same CTA's where it is short, as in a decode step, else a second kernel's, a thread four
// tokens or a CTA a sequence.  What bounds the calls is the chain lengths -> sums -> table -> places: a step of 64
// sequences 3.3 us, 192 prompts with 342 thousand places 7.3 (4.9 MB: 0.7 at the copy rate), 64 of 256 sequences given
// back 4.7.  (Keeping the starts in shared memory for the search of a place's sequence changed nothing.)
//
// In place: n_free is read by every thread before the sums' barriers and written behind them; a length is read and
// written by one thread, which is done with it then.  A new page's entry is written by the thread of its first token, and the stack itself is not written by a
// plan, so the second kernel needs no order among its CTAs.
#include "decoder.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024;  // at most, of the CTA with the sums
constexpr int kShort = 4096;  // tokens or pages that the first CTA does itself

// Exclusive sum over the CTA; `part` holds a value a warp.  `all` receives the total.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T* part, T& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  __syncthreads();  // an earlier use of `part` is over
  if (lane == 31) part[warp] = upto;
  __syncthreads();
  T w = lane < int(blockDim.x >> 5) ? part[lane] : T(0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return upto - v + (warp > 0 ? before : T(0));
}

__device__ __forceinline__ int pages_of(int tokens, int page) { return int((unsigned(tokens) + page - 1) / unsigned(page)); }

// n_free as it counts.
__device__ __forceinline__ int free_count(const int32_t* n_free, int n_pages, int* status_flags) {
  const int n = *n_free;  // a plain load: it may be written at the end
  if ((n < 0 || n > n_pages) && threadIdx.x == 0) report_bad_page(status_flags);
  return min(max(n, 0), n_pages);
}

// ------------------------------------------------------------------------------- plan -------

// `first[b]`: where on the stack sequence b's first new page is; kRefused where its tokens have no place.
constexpr int kRefused = -1;

__device__ __forceinline__ int32_t* plan_first(const PlanArgs& a) { return reinterpret_cast<int32_t*>(a.ws + kPagesWordsAt); }

// Token t of the list: sequence b, its tokens from `start` on, the length it had before.
__device__ __forceinline__ void place_token(const PlanArgs& a, int t, int b, int start, int before, int first, int& pos,
                                            int& slot) {
  pos = slot = -1;
  if (first == kRefused) return;
  pos = before + (t - start);
  const int nth = unsigned(pos) / unsigned(a.page), row = pos - nth * a.page, held = pages_of(before, a.page);
  int page;
  if (nth < held) {
    page = a.table[int64_t(b) * a.max_pages + nth];
  } else {
    page = a.free_pages[first - (nth - held)];
    if (row == 0) a.table[int64_t(b) * a.max_pages + nth] = page;
  }
  if (page >= 0 && page < a.n_pages) slot = page * a.page + row;
  else report_bad_page(reinterpret_cast<int*>(a.ws));
}

// The last b in [lo, hi) with starts[b] <= t.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int lo, int hi, int t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <bool kAll>
__global__ void __launch_bounds__(kThreads) k_page_plan(PlanArgs a) {
  __shared__ int64_t part64[kThreads / 32];
  __shared__ int part[kThreads / 32];
  __shared__ int refused_any, given;
  pdl_begin();
  int* status = reinterpret_cast<int*>(a.ws);
  if (threadIdx.x == 0) refused_any = given = 0;
  const int threads = blockDim.x, per = (a.B + threads - 1) / threads;
  const int b0 = min(a.B, int(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  const int n_free = free_count(a.n_free, a.n_pages, status);
  const int room = a.max_pages * a.page;
  auto wanted = [&](int b) { return a.new_tokens ? max(a.new_tokens[b], 0) : 1; };
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += wanted(b);
  int64_t total;
  const int64_t at0 = block_exclusive(mine, part64, total);
  // pages, of those whose tokens fit the row of the table and the list: at most max_tokens of them in all
  auto needs = [&](int len, int n, int64_t end) {
    return n <= room - len && end <= a.max_tokens ? pages_of(len + n, a.page) - pages_of(len, a.page) : kRefused;
  };
  int need = 0;
  int64_t at = at0;
  for (int b = b0; b < b1; ++b) {
    const int n = wanted(b);
    at += n;
    need += max(needs(max(a.lens[b], 0), n, at), 0);
  }
  int need_all;
  int used = block_exclusive(need, part, need_all);
  int32_t* first = plan_first(a);
  bool refused = false;
  int got = 0;
  at = at0;
  for (int b = b0; b < b1; ++b) {
    const int n = wanted(b), len = max(a.lens[b], 0);
    const int pages = needs(len, n, at + n);
    const bool served = pages == 0 || (pages > 0 && used + pages <= n_free);
    a.starts[b] = int(min(at, int64_t(a.max_tokens)));
    first[b] = !served ? kRefused : pages > 0 ? n_free - 1 - used : 0;
    a.lens_out[b] = served ? len + n : len;
    refused |= !served && n > 0;
    got += served ? pages : 0;
    used += max(pages, 0);
    at += n;
  }
  if (refused) refused_any = 1;
  if (got) atomicAdd(&given, got);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.starts[a.B] = int(min(total, int64_t(a.max_tokens)));
    *a.n_free_out = n_free - given;
    if (refused_any) atomicOr(status, kFlagNoPages);
  }
  if constexpr (kAll) {
    __syncthreads();  // starts, first and lens_out of all threads
    for (int t = threadIdx.x; t < a.max_tokens; t += threads) {
      int b = -1, pos = -1, slot = -1;
      if (t < total) {
        b = sequence_of(a.starts, 0, a.B, t);
        const int start = a.starts[b], f = first[b];
        const int before = f == kRefused ? 0 : a.lens_out[b] - (a.starts[b + 1] - start);
        place_token(a, t, b, start, before, f, pos, slot);
      }
      a.seq[t] = b;
      a.pos[t] = pos;
      a.slot[t] = slot;
    }
  }
}

constexpr int kTokenThreads = 256, kTokensEach = 4;

__global__ void __launch_bounds__(kTokenThreads) k_page_tokens(PlanArgs a) {
  pdl_begin();
  const int t0 = (blockIdx.x * kTokenThreads + threadIdx.x) * kTokensEach;
  if (t0 >= a.max_tokens) return;
  const int32_t* first = plan_first(a);
  const int total = a.starts[a.B];
  int b = t0 < total ? sequence_of(a.starts, 0, a.B, t0) : 0;
  int start = 0, end = 0, before = 0, f = kRefused;
  bool fresh = true;
  int seq[kTokensEach], pos[kTokensEach], slot[kTokensEach];
#pragma unroll
  for (int i = 0; i < kTokensEach; ++i) {
    const int t = t0 + i;
    seq[i] = pos[i] = slot[i] = -1;
    if (t >= total) continue;
    if (fresh || t >= end) {  // the sequence of t: past those without tokens
      if (!fresh)
        while (a.starts[b + 1] <= t) ++b;
      fresh = false;
      start = a.starts[b], end = a.starts[b + 1], f = first[b];
      before = f == kRefused ? 0 : a.lens_out[b] - (end - start);
    }
    seq[i] = b;
    place_token(a, t, b, start, before, f, pos[i], slot[i]);
  }
  if (t0 + kTokensEach <= a.max_tokens) {
    *reinterpret_cast<int4*>(a.seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
    *reinterpret_cast<int4*>(a.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    *reinterpret_cast<int4*>(a.slot + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
  } else {
    for (int i = 0; t0 + i < a.max_tokens; ++i) a.seq[t0 + i] = seq[i], a.pos[t0 + i] = pos[i], a.slot[t0 + i] = slot[i];
  }
}

// ---------------------------------------------------------------------------- release -------

// Sequence b's pages, from place `at` of the stack on.  What is no page of the pool goes there as well, so that the stack has
// an entry for each that was taken (a plan gives no place in it), and is reported.
__device__ __forceinline__ void give_back(const ReleaseArgs& a, int b, int at, int n, int lane, int lanes) {
  for (int j = lane; j < n; j += lanes) {
    const int64_t to = int64_t(at) + j;
    const int page = a.table[int64_t(b) * a.max_pages + j];
    if (to < a.n_pages) a.free_pages[to] = page;
    if (page < 0 || page >= a.n_pages) report_bad_page(reinterpret_cast<int*>(a.ws));
  }
}

// Workspace words: where each sequence's pages begin on the stack, and the end.
template <bool kAll>
__global__ void __launch_bounds__(kThreads) k_page_release(ReleaseArgs a) {
  __shared__ int64_t part[kThreads / 32];
  pdl_begin();
  int* status = reinterpret_cast<int*>(a.ws);
  const int threads = blockDim.x, per = (a.B + threads - 1) / threads;
  const int b0 = min(a.B, int(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  const int n_free = free_count(a.n_free, a.n_pages, status);
  const int room = a.max_pages * a.page;
  auto held = [&](int b) { return a.ended[b] ? pages_of(min(max(a.lens[b], 0), room), a.page) : 0; };
  int64_t mine = 0, total;
  bool cut = false;
  for (int b = b0; b < b1; ++b) {
    mine += held(b);
    cut |= a.ended[b] && a.lens[b] > room;
  }
  // the places of all pages: those past the stack's end are one and the same, its end
  int64_t at = n_free + block_exclusive(mine, part, total);
  int32_t* places = reinterpret_cast<int32_t*>(a.ws + kPagesWordsAt);
  for (int b = b0; b < b1; ++b) {
    const int n = held(b), len = a.lens[b];
    places[b] = int(min(at, int64_t(a.n_pages)));
    at += n;
    a.lens_out[b] = a.ended[b] ? 0 : len;
  }
  if (cut) report_bad_page(status);
  if (threadIdx.x == 0) {
    const int64_t now = n_free + total;
    places[a.B] = *a.n_free_out = int(min(now, int64_t(a.n_pages)));
    if (now > a.n_pages) report_bad_page(status);
  }
  if constexpr (kAll) {
    __syncthreads();
    for (int b = threadIdx.x >> 5; b < a.B; b += threads / 32)
      give_back(a, b, places[b], places[b + 1] - places[b], threadIdx.x & 31, 32);
  }
}

__global__ void __launch_bounds__(128) k_page_give_back(ReleaseArgs a) {
  pdl_begin();
  const int32_t* places = reinterpret_cast<const int32_t*>(a.ws + kPagesWordsAt);
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    give_back(a, b, places[b], places[b + 1] - places[b], threadIdx.x, 128);
}

// Whole warps for as many sequences or tokens, up to kThreads: a small CTA starts and meets sooner (a step of 64: 3.6 -> 3.3
// us).
int threads_for(int64_t n) { return int(std::min<int64_t>(kThreads, std::max<int64_t>(1, (n + 31) / 32) * 32)); }

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
  if (a.max_tokens <= kShort)
    return launch_pdl(k_page_plan<true>, dim3(1), dim3(threads_for(std::max(a.B, a.max_tokens))), 0, s, a);
  const cudaError_t e = launch_pdl(k_page_plan<false>, dim3(1), dim3(threads_for(a.B)), 0, s, a);
  if (e != cudaSuccess) return e;
  const int each = kTokenThreads * kTokensEach;
  return launch_pdl(k_page_tokens, dim3((a.max_tokens + each - 1) / each), dim3(kTokenThreads), 0, s, a);
}

cudaError_t launch_page_release(const ReleaseArgs& a, cudaStream_t s) {
  if (int64_t(a.B) * a.max_pages <= kShort)
    return launch_pdl(k_page_release<true>, dim3(1), dim3(threads_for(int64_t(a.B) * a.max_pages)), 0, s, a);
  const cudaError_t e = launch_pdl(k_page_release<false>, dim3(1), dim3(threads_for(a.B)), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_page_give_back, dim3(std::min(a.B, 2048)), dim3(128), 0, s, a);
}

}  // namespace moe
