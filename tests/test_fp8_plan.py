"""Host checks of how the E4M3 products cut their work (csrc/fp8_plan.h), compiled with g++ against the same header the
launches include: what a device cannot hold is never asked of it, a plan's tiles are as many as there may be, and
every thread plans with the same counts."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mixture_experts_layer_table_gb300", "csrc")

HARNESS = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <random>
#include <thread>
#include <vector>
#include "fp8_plan.h"
using namespace mok;

#define CHECK(x) do { if (!(x)) { std::printf("FAIL line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int plans() {
  const int64_t room = 6 * 32768;
  std::mt19937 rng(1);
  auto draw = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int split = 0;
  for (int i = 0; i < 20000; ++i) {
    const int E = draw(0, 2) ? 1 : draw(1, 64), MT = draw(1, 40), n_sm = draw(0, 3) ? 152 : draw(1, 152), nkb = draw(0, 70);
    const int64_t R = draw(1, draw(1, 5000)), groups = std::min<int64_t>(E, R), each = (R + groups - 1) / groups;
    const int counts[2] = {draw(0, 2) ? 36 : draw(0, 2), draw(0, 2) ? 15 : draw(0, 2)};
    const Fp8Plan p = f8_plan(E, MT, n_sm, nkb, groups, each, E == 1, counts, room);
    CHECK(p.nmax == 32 || p.nmax == 64 || p.nmax == 128 || p.nmax == 256);
    CHECK(p.splits == 1 || p.splits == 2 || p.splits == 4);
    if (p.splits > 1) {  // every tile has its cluster, and all of them fit
      ++split;
      CHECK(p.tiles <= counts[p.splits / 4]);
      CHECK(nkb >= 4 * p.splits);
      CHECK((p.splits - 1) * p.nmax * 512 <= room);
    }
    CHECK(p.tiles >= (E == 1 ? (R + p.nmax - 1) / p.nmax : (R + p.nmax - 1) / p.nmax + E) * MT);
    const int none[2] = {0, 0};
    CHECK(f8_plan(E, MT, n_sm, nkb, groups, each, E == 1, none, room).splits == 1);
  }
  CHECK(split > 100);
  return 0;
}

int counts() {
  enum Error { OK = 0, BAD = 7 };
  Fp8Clusters known;
  int c[2] = {-1, -1};
  CHECK(known.get<Error>(3, c, [](int (&n)[2]) { n[0] = 5; return BAD; }) == BAD);  // nothing is kept of a question that failed
  CHECK(known.get<Error>(3, c, [](int (&n)[2]) { n[0] = n[1] = 0; return OK; }) == OK);
  CHECK(c[0] == 0 && c[1] == 0);  // no cluster fits: 0, not 1
  std::atomic<int> asked{0}, wrong{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 32; ++i)
    threads.emplace_back([&, i] {
      int mine[2] = {0, 0};
      const int device = 10 + i % 2;
      const Error err = known.get<Error>(device, mine, [&](int (&n)[2]) {
        asked++;
        n[0] = 36;
        std::this_thread::sleep_for(std::chrono::milliseconds(20));
        n[1] = device;
        return OK;
      });
      if (err != OK || mine[0] != 36 || mine[1] != device) wrong++;
    });
  for (auto& t : threads) t.join();
  CHECK(asked == 2 && wrong == 0);
  return 0;
}

int main() { return plans() || counts(); }
"""


def test_plans_and_counts(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "plan.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "plan"
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
