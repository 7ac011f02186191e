// A CTA's copies through csrc/copy_stages.h against a model of mbarriers (host only): every wait sees its own copy, and
// whoever gives up waits for exactly the copies that are under way.  Prints "ok", or what went wrong.
#include <cstdio>
#include <random>
#include <vector>

#include "../../linear_recurrent_sequence_causal_gb300/csrc/copy_stages.h"

namespace {

// A barrier in its phase 0, 1, ...: a wait for a parity sees whether the phase that is open has another one.
struct Bar {
  unsigned phase = 0;
  bool passes(unsigned parity) const { return (phase & 1) != parity; }
};

#define CHECK(x, what)                                                               \
  if (!(x)) {                                                                        \
    std::printf("S = %d, job %d, gives up at %d: %s\n", S, n, give_up, what);        \
    return false;                                                                    \
  }

// Jobs of which only some have copies; the copy of job `give_up` does not come in time.
template <int S>
bool run(std::mt19937& rng, int jobs, int give_up) {
  std::vector<bool> has(jobs + S, false);
  for (int i = 0; i < jobs; ++i) has[i] = rng() % 4 != 0;
  Bar bar[S];
  std::vector<int> coming;                         // jobs whose copy is under way
  const auto start = [&](int j) {
    if (j < jobs && has[j]) coming.push_back(j);
  };
  const auto land = [&](int j) {
    for (size_t i = 0; i < coming.size(); ++i)
      if (coming[i] == j) {
        coming.erase(coming.begin() + i);
        ++bar[j % S].phase;
        return true;
      }
    return false;
  };
  prism::CopyStages<S> stages;
  for (int j = 0; j < S; ++j) start(j);
  for (int n = 0; n < jobs; ++n) {
    if (has[n]) {
      if (n >= give_up) {
        std::vector<int> waited;
        bool early = false;
        stages.under_way(
            n, [&](int m) { return m < jobs && has[m]; },
            [&](int s, unsigned parity) {
              early |= bar[s].passes(parity);      // before its copy has landed
              int j = -1;
              for (int c : coming)
                if (c % S == s) j = c;
              if (j >= 0 && land(j) && bar[s].passes(parity)) waited.push_back(j);
              else waited.push_back(-1);
            });
        CHECK(!early, "a copy that is still under way counts as landed");
        CHECK(coming.empty(), "a copy outlives the CTA");
        for (int j : waited) CHECK(j >= 0, "a wait for a copy that nobody makes");
        return true;
      }
      CHECK(!bar[n % S].passes(stages.parity(n)), "a wait sees another job's copy");
      CHECK(land(n), "the copy was not made");
      CHECK(bar[n % S].passes(stages.parity(n)), "a copy that has landed is not seen");
      stages.taken(n);
    }
    start(n + S);
  }
  const int n = jobs;
  CHECK(coming.empty(), "a copy outlives the CTA");
  return true;
}

template <int S>
bool all() {
  std::mt19937 rng(S);
  for (int i = 0; i < 20000; ++i) {
    const int jobs = 1 + (int)(rng() % 12);
    if (!run<S>(rng, jobs, i % 2 ? (int)(rng() % jobs) : jobs)) return false;
  }
  return true;
}

}  // namespace

int main() {
  if (!all<1>() || !all<2>() || !all<3>() || !all<4>()) return 1;
  std::puts("ok");
  return 0;
}
