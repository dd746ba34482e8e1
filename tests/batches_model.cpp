// Runs in_batches (csrc/batches.cuh) on host threads, one a warp, against a model of an mbarrier and of
// asynchronous copies.  The model counts what the hardware leaves undefined: an arrival beyond the
// barrier's count, a copy into a slice that an earlier copy still fills, a use of a slice that has not
// landed.
//
//   batches_model n batch joints batch_given_up warps_that_give_up
// At that batch (counted over the joints; -1: none) the waits of the warps in the bit mask give up; its
// copies land only once one of the others waits for them.  Prints the violations, the batches that each
// warp used, and each warp's result.
#include <barrier>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <set>
#include <thread>
#include <vector>

#ifdef PLANTED  // goes on after a wait that gave up
namespace moe {
template <typename AllOk, typename Start, typename Landed, typename Use>
bool in_batches(int n, int batch, bool ok, AllOk&& all_ok, Start&& start, Landed&& landed, Use&& use) {
  for (int i0 = 0; i0 < n; i0 += batch) {
    const int m = batch < n - i0 ? batch : n - i0;
    all_ok(true);
    start(i0, m);
    ok = landed() && ok;
    use(i0, m);
  }
  return ok;
}
}  // namespace moe
#else
#include "../routed_expert_layer_fp32_gb300/csrc/batches.cuh"
#endif

namespace {

constexpr int kWarps = 4;
#ifdef PLANTED  // waits for what never comes
constexpr std::chrono::milliseconds kPatience{200};
#else
constexpr std::chrono::seconds kPatience{20};
#endif

struct Model {
  std::mutex m;
  std::condition_variable moved;
  std::barrier<> threads{kWarps};
  int given_up_at, who;  // the batch, the warps
  int votes_against = 0, violations = 0;
  int pending = kWarps, phase = 0;
  std::set<int> in_flight, landed;

  void settle() {  // with m held
    if (pending != 0 || !in_flight.empty()) return;
    pending = kWarps;
    ++phase;
    moved.notify_all();
  }
  void land() {  // with m held
    landed.insert(in_flight.begin(), in_flight.end());
    in_flight.clear();
    settle();
  }
};

struct Warp {
  Model& md;
  int w, round = 0, used = 0;

  bool all_ok(bool ok) {
    if (!ok) {
      std::lock_guard<std::mutex> l(md.m);
      ++md.votes_against;
    }
    md.threads.arrive_and_wait();
    const bool all = md.votes_against == 0;
    md.threads.arrive_and_wait();
    return all;
  }
  void start(int, int n) {
    std::lock_guard<std::mutex> l(md.m);
    if (md.pending == 0) ++md.violations;
    else --md.pending;
    for (int k = w; k < n; k += kWarps) {
      if (!md.in_flight.insert(k).second) ++md.violations;
      md.landed.erase(k);
    }
    if (round != md.given_up_at) md.land();
    md.moved.notify_all();
  }
  bool landed() {
    const int at = round++;
    std::unique_lock<std::mutex> l(md.m);
    if (at == md.given_up_at) {
      if (md.who >> w & 1) return false;
      md.moved.wait_for(l, kPatience, [&] { return md.pending == 0 || md.phase > at; });
      if (md.phase == at) md.land();
    }
    return md.moved.wait_for(l, kPatience, [&] { return md.phase > at; });
  }
  void use(int, int n) {
    std::lock_guard<std::mutex> l(md.m);
    for (int k = 0; k < n; ++k) md.violations += md.landed.count(k) == 0;
    ++used;
  }
};

}  // namespace

int main(int argc, char** argv) {
  if (argc != 6) return 2;
  const int n = atoi(argv[1]), batch = atoi(argv[2]), joints = atoi(argv[3]);
  Model md;
  md.given_up_at = atoi(argv[4]);
  md.who = atoi(argv[5]);
  std::vector<Warp> warps;
  for (int w = 0; w < kWarps; ++w) warps.push_back(Warp{md, w});
  int result[kWarps];
  std::vector<std::thread> run;
  for (int w = 0; w < kWarps; ++w)
    run.emplace_back([&, w] {
      bool ok = true;
      for (int j = 0; j < joints; ++j) ok = moe::in_batches(
            n, batch, ok, [&](bool mine) { return warps[w].all_ok(mine); }, [&](int i0, int m) { warps[w].start(i0, m); },
            [&] { return warps[w].landed(); }, [&](int i0, int m) { warps[w].use(i0, m); });
      result[w] = ok;
    });
  for (auto& t : run) t.join();
  printf("%d", md.violations);
  for (const auto& w : warps) printf(" %d", w.used);
  for (int r : result) printf(" %d", r);
  printf("\n");
}
