// Waits that a team of threads shares.  One thread waits and its verdict is
// everyone's, so that a wait that runs out takes the team out of its loop as a
// whole: threads that gave up each by its own clock would meet the others at
// different barriers, and those never end.  (Plain C++, so that the host can run it too.)
#pragma once

#ifdef __CUDACC__
#define MPM_TEAM __device__ __forceinline__
#else
#define MPM_TEAM inline
#endif

namespace mpm {

// team.first(): this thread is the one that waits.  team.share(v): the first thread's v, for all of the team, and what that
// thread has seen before it; the others pass true.
template <class Team, class Wait>
MPM_TEAM bool wait_as_one(const Team& team, Wait wait) {
  bool there = true;
  if (team.first()) there = wait();
  return team.share(there);
}

// row(r) for r = begin, begin + step, ... below end, each after wait(r); false where a wait ran out, for the whole team at
// the same r.
template <class Team, class Wait, class Row>
MPM_TEAM bool rows_as_one(const Team& team, int begin, int step, int end, Wait wait, Row row) {
  for (int r = begin; r < end; r += step) {
    if (!wait_as_one(team, [&]() { return wait(r); })) return false;
    row(r);
  }
  return true;
}

}  // namespace mpm
