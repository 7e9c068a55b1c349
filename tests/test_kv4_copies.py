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
