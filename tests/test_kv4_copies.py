"""Copies under way in the 4-bit cache's kernels when a wait runs out, on the CPU.

The bookkeeping that the kernels use (csrc/kv4_feed.cuh) is compiled for the
host and run against buffers that note what is in flight: no copy is started
into a buffer that another may still fill, and none is left behind at the end.
"""
import os
import subprocess

import pytest

import block_sparse_long_fwd_b200 as moba

CSRC = os.path.join(os.path.dirname(moba.__file__), "csrc")


def run(tmp_path, body):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include <initializer_list>\n#include "kv4_feed.cuh"\n'
                   "static int bad = 0;\n"
                   '#define CHECK(x) do { if (!(x)) { ++bad; std::printf("line %d: %s\\n", __LINE__, #x); } } while (0)\n'
                   + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)


ATTENTION = """
// The order of a warp in the attention kernel: `fails` is the wait (2 k: keys of tile k, 2 k + 1: its values) that runs
// out, its copy still under way.
int main() {
  for (int n = 1; n <= 6; ++n)
    for (int fails = 0; fails <= 2 * n; ++fails) {
      moba::Kv4Fetch f;
      f.left = n;
      int flying[2] = {-1, -1}, next = 0, started[2] = {0, 0};  // tile under way in the keys' and values' buffer
      auto start = [&](int buf, int tile) {
        CHECK(flying[buf] == -1);
        flying[buf] = tile;
        ++started[buf];
      };
      auto wait = [&](int buf, int tile, int at) {
        if (at == fails) return false;
        CHECK(flying[buf] == tile);
        flying[buf] = -1;
        return true;
      };
      next = 0, --f.left;
      start(0, 0);
      start(1, 0);
      for (int k = 0; k < n; ++k) {
        if (!f.dead && !wait(0, k, 2 * k)) f.gave_up(k);
        if (f.next_keys()) ++next, --f.left, start(0, next);
        if (!f.dead && !wait(1, k, 2 * k + 1)) f.gave_up(k);
        if (f.next_values()) start(1, next);
      }
      CHECK(f.dead == (fails < 2 * n));
      if (f.dead) {  // what the warp waits for before it leaves is all that is under way
        CHECK(flying[0] == -1 || flying[0] == f.last_keys(n));
        CHECK(flying[1] == -1 || flying[1] == f.last_values());
        CHECK(started[0] == f.last_keys(n) + 1 && started[1] == f.last_values() + 1);
      } else {
        CHECK(flying[0] == -1 && flying[1] == -1 && started[0] == n && started[1] == n);
      }
    }
  return bad != 0;
}
"""


def test_a_warp_that_gives_up_starts_no_copy_and_waits_for_those_under_way(tmp_path):
    r = run(tmp_path, ATTENTION)
    assert r.returncode == 0, r.stdout


FEED = """
// The loader starts its tiles; the products' warp then waits for them. `fails` is the wait that runs out, of those two
// roles' in the order in which they happen; the copy that was waited for lands only when the loader waits for it.
template <int BUFS>
struct Port {
  bool flag = false, flying[BUFS] = {};
  int waits = 0, fails = -1, taken[BUFS] = {}, sent[BUFS] = {};
  bool gone() { return flag || waits++ == fails ? (flag = true) : false; }
  bool empty(int x, uint32_t parity) {
    CHECK(parity == (uint32_t)((sent[x] & 1) ^ 1));
    if (taken[x] < sent[x]) take(x);  // the products come by when the loader has to wait for them
    return !gone();
  }
  void start(int x) {
    CHECK(!flying[x]);
    flying[x] = true;
    ++sent[x];
  }
  void take(int x) {
    if (gone()) return;
    flying[x] = false;
    ++taken[x];
  }
  void landed(int x, uint32_t parity) {
    CHECK(parity == (uint32_t)((sent[x] - 1) & 1));
    flying[x] = false;
  }
};

template <int BUFS>
void feed() {
  for (int tiles = 0; tiles <= 4; ++tiles)
    for (int fails = -1; fails <= 2 * BUFS * tiles; ++fails) {
      Port<BUFS> port;
      port.fails = fails;
      moba::Kv4Feeder<BUFS> f;
      bool going = true;
      for (int t = 0; going && t < tiles; ++t)
        for (int x = 0; going && x < BUFS; ++x) going = f.load(port, x);
      bool left[BUFS];
      const bool late = !port.flag;  // the other warps are still at work when the loader has nothing left to start
      f.finish(port);
      for (int x = 0; x < BUFS; ++x) left[x] = port.flying[x];
      if (late)
        for (int x = 0; x < BUFS; ++x)
          if (port.taken[x] < port.sent[x]) port.take(x);
      if (port.flag)  // given up: the block goes as it is
        for (int x = 0; x < BUFS; ++x) CHECK(!left[x]);
    }
}

int main() {
  feed<1>();
  feed<2>();
  return bad != 0;
}
"""


def test_no_query_tile_is_on_its_way_when_a_block_leaves(tmp_path):
    r = run(tmp_path, FEED)
    assert r.returncode == 0, r.stdout
