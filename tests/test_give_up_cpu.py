"""The flags by which the warps of a group leave their loop together, on the
CPU: every interleaving of a few warps over a few tiles, each wait of each warp
free to give up."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "head_heterogeneous_block_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include "give_up.h"

constexpr int kWarps = 3, kTiles = 4;
struct OneFlag {                       // the same flag for every tile
  int flag;
  void clear() { flag = 0; }
  void raise(uint32_t) { flag = 1; }
  bool raised(uint32_t) const { return flag != 0; }
};
enum { kWait, kRaise, kArrive, kBlocked, kRead, kOut };
template <class Flags>
struct State {
  int step[kWarps], tile[kWarps], arrived;
  bool fail[kWarps];
  Flags flags;
  std::string key() const {
    std::string s;
    for (int w = 0; w < kWarps; ++w)
      s += char(step[w]), s += char(tile[w]), s += char(fail[w]);
    s += char(arrived);
    for (int t = 0; t < 2; ++t) s += char(flags.raised(t));
    return s;
  }
};
// returns the number of states in which some warps are out (or blocked) and no
// warp can go on
template <class Flags>
long explore(State<Flags> s, std::set<std::string>& seen) {
  if (!seen.insert(s.key()).second) return 0;
  long stuck = 0;
  bool moved = false, all_out = true;
  for (int w = 0; w < kWarps; ++w) {
    if (s.step[w] != kOut) all_out = false;
    if (s.step[w] == kOut || s.step[w] == kBlocked) continue;
    moved = true;
    State<Flags> n = s;
    switch (s.step[w]) {
      case kWait:                      // the tile's waits come through, or give up
        n.step[w] = kArrive;
        stuck += explore(n, seen);
        n.fail[w] = true;
        n.step[w] = kRaise;
        break;
      case kRaise:
        n.flags.raise(s.tile[w]);
        n.step[w] = kArrive;
        break;
      case kArrive:
        n.step[w] = kBlocked;
        if (++n.arrived == kWarps) {
          n.arrived = 0;
          for (int x = 0; x < kWarps; ++x)
            if (n.step[x] == kBlocked) n.step[x] = kRead;
        }
        break;
      case kRead:
        if (s.flags.raised(s.tile[w]) || s.tile[w] == kTiles - 1) {
          n.step[w] = kOut;
        } else {
          if (s.fail[w]) std::abort();  // a warp that gave up goes on
          ++n.tile[w];
          n.step[w] = kWait;
        }
        break;
    }
    stuck += explore(n, seen);
  }
  return stuck + (!moved && !all_out);
}
template <class Flags>
long run() {
  State<Flags> s;
  std::memset(static_cast<void*>(&s), 0, sizeof s);
  s.flags.clear();
  std::set<std::string> seen;
  const long stuck = explore(s, seen);
  std::printf("%zu states, %ld stuck\n", seen.size(), stuck);
  return stuck;
}
int main() {
  const long one = run<OneFlag>(), two = run<sa_dev::GiveUp>();
  return two ? 1 : one ? 0 : 2;        // one flag has to show that the search finds what it looks for
}
"""


def test_warps_leave_together(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "give_up.cpp", tmp_path / "give_up"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
