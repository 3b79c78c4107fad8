"""The walks of warps that meet at named barriers: whichever of four warps gives
up, and wherever, all of them leave, having written the same.  Run on a barrier
that, like the hardware's, counts arrivals and waits without limit, for every
combination of places where the warps give up.  The walk by tiles is the d = 64
backward's own (csrc/fa_walk.h, compiled for the host); the walk by items has the steps of
its compute warps' loop.  A walk whose warps leave by themselves has to be found
hanging, and so has one whose warps arrive ahead for the barriers to come."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "exact_attention_98_gb300", "csrc")

PROGRAM = r"""
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>
#include "fa_walk.h"
using fa::Next;

constexpr int kWarps = 4;

// A named barrier of kWarps arrivals, and whether all that are left wait at it.
struct Barrier {
  std::mutex mu;
  std::condition_variable cv;
  int live = kWarps, arrived = 0, waiting = 0, round = 0;
  bool all = true, result = true, hung = false;
  void complete() {
    result = all;
    all = true;
    arrived = waiting = 0;
    ++round;
    cv.notify_all();
  }
  void check() {
    if (live > 0 && waiting == live) {
      hung = true;
      cv.notify_all();
    }
  }
  bool meet(bool ok) {
    std::unique_lock<std::mutex> l(mu);
    if (hung) return false;
    all = all && ok;
    if (++arrived == kWarps) {
      complete();
      return result;
    }
    ++waiting;
    const int mine = round;
    check();
    // (the next round cannot complete before this warp arrives again or has left: it then
    // does not look at the result)
    cv.wait(l, [&] { return round != mine || hung; });
    return round != mine && result;
  }
  void arrive() {
    std::lock_guard<std::mutex> l(mu);
    if (++arrived == kWarps) complete();
  }
  void leave() {
    std::lock_guard<std::mutex> l(mu);
    --live;
    check();
  }
};

// A warp's waits, counted; the one numbered `at` fails, and all behind it.
struct Waits {
  int at, n = 0;
  bool operator()() { return n++ < at; }
};

struct Items {
  std::vector<int> tiles;
  int next = 0, left = 0;
  Next look(Waits& waits) {
    if (!waits()) return Next::kGaveUp;
    if (next == static_cast<int>(tiles.size())) return Next::kEnd;
    left = tiles[next++];
    return Next::kItem;
  }
};

enum class Form { kItems, kTiles, kAlone, kAhead };
constexpr int kChunks = 4;

// What a warp writes: items, or tiles.
int warp(Form form, Barrier& bar, Items items, Waits waits) {
  int written = 0;
  if (form == Form::kItems) {
    Next next = items.look(waits);
    bool ok = bar.meet(next != Next::kGaveUp);
    while (ok && next == Next::kItem) {
      for (; ok && items.left > 0; --items.left) ok = waits();
      next = items.look(waits);
      if (next == Next::kGaveUp) ok = false;
      if (ok) ok = waits();  // (the products)
      if (!(ok = bar.meet(ok))) break;
      bar.meet(true);  // (the staged tile)
      ++written;
    }
  } else if (form == Form::kTiles) {
    fa::walk_tiles([&] { return items.look(waits); }, [&] { return waits(); }, [&](bool ok) { return bar.meet(ok); },
                   [&] {
                     for (int c = 1; c < kChunks; ++c) bar.meet(true);
                     ++written;
                   },
                   [&] { return --items.left > 0; });
  } else {  // each warp leaves by itself, for kAhead with arrivals for the tile's barriers
    while (items.look(waits) == Next::kItem) {
      bool ok = true;
      for (; ok && items.left > 0; --items.left) {
        if (!(ok = waits())) {
          for (int c = 0; form == Form::kAhead && c < kChunks; ++c) bar.arrive();
          break;
        }
        for (int c = 0; c < kChunks; ++c) bar.meet(true);
        ++written;
      }
      if (!ok) break;
    }
  }
  bar.leave();
  return written;
}

int main(int argc, char** argv) {
  const Form form = !strcmp(argv[1], "items") ? Form::kItems : !strcmp(argv[1], "tiles") ? Form::kTiles
                    : !strcmp(argv[1], "alone") ? Form::kAlone : Form::kAhead;
  Items items;
  int waits = 1;  // of a warp that goes through
  for (int i = 2; i < argc; ++i) {
    items.tiles.push_back(argv[i][0] - '0');
    waits += items.tiles.back() + 1 + (form == Form::kItems ? 1 : 0);
  }
  int runs = 1, hung = 0, apart = 0, whole = 0;
  for (int w = 0; w < kWarps; ++w) runs *= waits + 1;
  for (int r = 0; r < runs; ++r) {
    Barrier bar;
    std::thread threads[kWarps];
    int written[kWarps];
    for (int w = 0, x = r; w < kWarps; ++w, x /= waits + 1)
      threads[w] = std::thread([&, w, at = x % (waits + 1)] { written[w] = warp(form, bar, items, Waits{at}); });
    for (auto& t : threads) t.join();
    if (bar.hung) {
      ++hung;
      continue;
    }
    for (int w = 1; w < kWarps; ++w)
      if (written[w] != written[0]) {
        ++apart;
        break;
      }
    whole = written[0];  // (of the last run, in which none gives up)
  }
  printf("%d %d %d %d\n", runs, hung, apart, whole);
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    path = tmp_path_factory.mktemp("walk")
    (path / "walk.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O2", "-std=c++17", "-pthread", "-I", CSRC, str(path / "walk.cpp"), "-o", str(path / "walk")],
                   check=True)

    def run(form, items):
        r = subprocess.run([str(path / "walk"), form, *map(str, items)], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        return [int(x) for x in r.stdout.split()]

    return run


@pytest.mark.parametrize("form,items,whole", [("items", [], 0), ("items", [2], 1), ("items", [1, 0], 2),
                                              ("tiles", [], 0), ("tiles", [2], 2), ("tiles", [1, 2], 3)])
def test_all_leave_together(program, form, items, whole):
    runs, hung, apart, written = program(form, items)
    assert runs >= 16 and hung == 0 and apart == 0 and written == whole


@pytest.mark.parametrize("form", ["alone", "ahead"])
def test_finds_a_walk_that_hangs(program, form):
    runs, hung, _, written = program(form, [1, 2])
    assert written == 3 and 0 < hung < runs
