// The weight gradients' way through their grid (take_tiles_over), run on the host against a stand-in
// for the hardware that answers requests for unstarted clusters (the program makes no CUDA call).
// Exit status 0 = no tile is lost, whatever the order of grants and refusals.
#include <cstdio>
#include <deque>
#include <vector>

#include "grouped_wgrad.cuh"

using namespace moe;

int main() {
  int fails = 0;
  auto check = [&](bool ok, const char* what, unsigned pattern, int ahead) {
    if (!ok && fails++ < 10) std::printf("FAIL %s: pattern %x, ahead %d\n", what, pattern, ahead);
  };
  // bit i of `pattern`: whether the i-th request is granted; requests past 16 are refused
  for (int ahead = 1; ahead <= kGwSlots; ++ahead)
    for (unsigned pattern = 0; pattern < 1u << 16; ++pattern) {
      std::deque<int> answers;
      std::vector<int> granted, handed;
      int asked = 0, most = 0;
      bool observed = false, late = false;
      const bool ok = take_tiles_over(
          ahead,
          [&] {
            late |= observed;
            const bool grant = asked < 16 && (pattern >> asked & 1u);
            if (grant) granted.push_back(asked);
            answers.push_back(grant ? asked : -1);
            ++asked;
            most = (int)answers.size() > most ? (int)answers.size() : most;
            return true;
          },
          [&](int& tile) {
            if (answers.empty()) return false;   // a wait for an answer nobody asked for
            tile = answers.front();
            answers.pop_front();
            observed |= tile < 0;
            return true;
          },
          [&](int tile) {
            handed.push_back(tile);
            return true;
          });
      check(ok && answers.empty(), "every request is answered, and no more are waited for", pattern, ahead);
      check(!late, "no request after an observed refusal", pattern, ahead);
      check(most <= ahead, "requests open at once", pattern, ahead);
      check(!handed.empty() && handed.back() == -1, "-1 comes last", pattern, ahead);
      handed.pop_back();
      check(handed == granted, "every tile granted is handed on, in order, once", pattern, ahead);
    }
  // a wait that runs out ends the loop at once
  int calls = 0;
  check(!take_tiles_over(2, [&] { return ++calls < 2; }, [](int&) { return true; }, [](int) { return true; }) &&
            calls == 2, "a request that gives up", 0, 2);
  check(!take_tiles_over(2, [] { return true; }, [](int&) { return false; }, [](int) { return true; }),
        "an answer that gives up", 0, 2);
  check(!take_tiles_over(2, [] { return true; }, [](int& t) { t = 1; return true; }, [](int) { return false; }),
        "a reader that gives up", 0, 2);
  if (fails) return 1;
  std::printf("no tile is lost\n");
  return 0;
}
