"""The exchange of two warps that share rows, on the CPU: whichever wait runs out
in one warp or in both, neither stays behind at the barrier between them."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Two threads for two warps; waits fail from a given one on (once one has run out, all later ones of that warp give
# up), the barrier reports a partner that does not come within a second.
HARNESS = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>
#include "pair_loop.h"

struct Barrier {
  std::mutex m; std::condition_variable cv;
  int here = 0, phase = 0; bool all = true, last = true, stuck = false;
  bool meet(bool ok) {
    std::unique_lock<std::mutex> l(m);
    all = all && ok;
    const int p = phase;
    if (++here == 2) { last = all; all = true; here = 0; ++phase; cv.notify_all(); return last; }
    if (!cv.wait_for(l, std::chrono::seconds(1), [&] { return phase != p; })) { stuck = true; return false; }
    return last;
  }
};

int main() {
  const int n = 4, waits = 2 * n;                        // per tile one wait before the exchange and one after
  for (int a = 0; a <= waits; ++a)
    for (int b = 0; b <= waits; ++b) {
      Barrier bar;
      bool ret[2];
      auto warp = [&](int w, int first_bad) {
        int at = 0;
        auto wait = [&] { return at++ < first_bad; };
        auto before = [&](int, bool ok) { return ok && wait(); };
        auto meet = [&](int, bool ok) { return bar.meet(ok); };
        auto after = [&](int) { return wait(); };
        const int split = (a + b) % (n + 1);             // the tiles in two loops, one of them empty at times
        ret[w] = mbt::pair_tiles(0, split, true, before, meet, after);
        ret[w] = mbt::pair_tiles(split, n, ret[w], before, meet, after);
      };
      std::thread t0(warp, 0, a), t1(warp, 1, b);
      t0.join(); t1.join();
      const bool good = a == waits && b == waits;
      // a warp may come through if only the last wait of its partner ran out: nothing is exchanged after it
      const bool want0 = a == waits && b >= waits - 1, want1 = b == waits && a >= waits - 1;
      if (bar.stuck || ret[0] != want0 || ret[1] != want1 || (good && !(ret[0] && ret[1]))) {
        std::printf("waits %d, %d: stuck %d, %d %d\n", a, b, (int)bar.stuck, (int)ret[0], (int)ret[1]);
        return 1;
      }
    }
  return 0;
}
"""


@pytest.mark.parametrize("body,passes", [
    (None, True),
    # the check itself: a warp that leaves as soon as its own wait runs out strands its partner
    ("for (int j = from; j < to; ++j) { if (!before(j, true)) return false; if (!meet(j, true)) return false;"
     " if (!after(j)) return false; } return ok;", False)])
def test_neither_warp_is_left_at_the_barrier(tmp_path, body, passes):
    header = open(os.path.join(ROOT, "memory_bound_transformer_gb300", "csrc", "pair_loop.h")).read()
    if body:
        at, end = header.index("#pragma unroll 1"), header.index("  return ok;\n") + len("  return ok;\n")
        header = header[:at] + body + header[end:]
    (tmp_path / "pair_loop.h").write_text(header)
    (tmp_path / "t.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-w", "-o", str(tmp_path / "t"), str(tmp_path / "t.cpp")],
                   check=True, capture_output=True, timeout=120)
    assert (subprocess.run([str(tmp_path / "t")], timeout=120).returncode == 0) == passes
