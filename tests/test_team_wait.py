"""The waits that a team of threads shares, run by threads of the host: where the wait runs out for some threads
and not for others, all leave the loop at the same row and none is left at a barrier (CPU)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaled_precision_moe_gb300", "csrc")

PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>
#include "team_wait.cuh"

constexpr int N = 8;
// a barrier of N threads with the conjunction of what they bring; a thread left alone for 5 s ends the program
struct Barrier {
  std::mutex mu;
  std::condition_variable cv;
  int arrived = 0;
  long generation = 0;
  bool all = true, result = true;
  bool meet(bool v) {
    std::unique_lock<std::mutex> l(mu);
    const long mine = generation;
    all = all && v;
    if (++arrived == N) {
      result = all;
      all = true;
      arrived = 0;
      ++generation;
      cv.notify_all();
      return result;
    }
    if (!cv.wait_for(l, std::chrono::seconds(5), [&] { return generation != mine; })) {
      std::puts("left at a barrier");
      _Exit(3);
    }
    return result;
  }
} barrier;

struct Team {
  int id;
  bool first() const { return id == 0; }
  bool share(bool v) const { return barrier.meet(v); }
};

int main() {
  // each thread by its own clock would give up at another row; the first one's counts
  for (int limit = 0; limit < 6; ++limit) {
    std::vector<int> rows(N), ok(N);
    std::vector<std::thread> threads;
    for (int id = 0; id < N; ++id)
      threads.emplace_back([&, id] {
        auto wait = [&](int r) { return r < (limit + id % 3) * 4; };
        auto row = [&](int) {
          ++rows[id];
          barrier.meet(true);
        };
        ok[id] = mpm::rows_as_one(Team{id}, 0, 4, 16, wait, row);
        barrier.meet(true);                      // the barrier behind the loop
      });
    for (auto& t : threads) t.join();
    for (int id = 0; id < N; ++id)
      if (rows[id] != (limit < 4 ? limit : 4) || ok[id] != (limit >= 4)) {
        std::printf("limit %d, thread %d: %d rows, %d\n", limit, id, rows[id], ok[id]);
        return 1;
      }
  }
  std::puts("ok");
}
"""


def test_a_team_gives_up_as_a_whole(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src, exe = tmp_path / "team.cpp", tmp_path / "team"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-x", "c++", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_kernel_waits_for_other_blocks_as_teams_only():
    """Every wait for a count of another block is one thread's: in a role of one lane, or through the team."""
    with open(os.path.join(CSRC, "moe_few.cu")) as f:
        lines = [l.strip() for l in f if "wait_count(" in l and "MPM_DEV" not in l]
    teams = [l for l in lines if "auto there = " in l or "wait_as_one(" in l]
    lane = [l for l in lines if l not in teams]
    assert len(teams) == 2 and len(lane) == 2, lines       # the two of the rows' producer, which is one lane


def test_the_scoring_warps_give_up_as_a_whole():
    """A row's work has operations of a whole warp: whether it is begun, and whether its list may be worked on, is agreed."""
    with open(os.path.join(CSRC, "logprob.cu")) as f:
        source = f.read()
    next_row = source.split("auto next_row = [&]() {", 1)[1].split("};", 1)[0]
    assert "ok = warp_agrees(ok && mbar_wait(" in next_row and "return ok && row >= 0;" in next_row
    closing = source.split("// ---------------------------------------------------------------- closing", 1)[1]
    assert closing.index("ok = warp_agrees(ok && mbar_wait(smem_u32(&h.full)") < closing.index("if (listed > CAP && ok)")
