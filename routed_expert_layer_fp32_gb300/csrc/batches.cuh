// The order of steps in which a group of threads brings `n` slices into a buffer that holds `batch` of
// them, by asynchronous copies on one barrier, and uses them.  Apart from the kernel's own header so that
// the order can be run on the host, against a model of the barrier.
#pragma once

#ifdef __CUDACC__
#define MOE_STEPS __device__ __forceinline__
#else
#define MOE_STEPS inline
#endif

namespace moe {

// Every thread of the group calls it with the same n and batch, and whether all went well for it so far.
//   all_ok(ok)    joins the threads and tells each whether `ok` holds for all of them: nobody uses the
//                 buffer any more, and either all of them go on or none does
//   start(i0, m)  this thread's share of arrivals and copies for slices i0 .. i0 + m - 1
//   landed()      waits for the barrier's phase; false where it gave up
//   use(i0, m)    works on them
// A phase that somebody gave up on may not be over: an arrival for the next one would be one too many,
// and a copy could meet an earlier one in the buffer.  So nothing is started after that.  Returns this
// thread's ok.
template <typename AllOk, typename Start, typename Landed, typename Use>
MOE_STEPS bool in_batches(int n, int batch, bool ok, AllOk&& all_ok, Start&& start, Landed&& landed, Use&& use) {
  for (int i0 = 0; i0 < n; i0 += batch) {
    const int m = batch < n - i0 ? batch : n - i0;
    if (!all_ok(ok)) return false;
    start(i0, m);
    ok = landed();
    if (ok) use(i0, m);
  }
  return ok;
}

}  // namespace moe
