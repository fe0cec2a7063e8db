"""The kernels' schedules as far as they are arithmetic (csrc/schedule.h), run on the host."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conv2d_layer_gb300", "csrc")


def run(tmp_path, source):
    src, exe = tmp_path / "a.cpp", tmp_path / "a.out"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout


PLACES = """
#include <cstdio>
#include <vector>
#include "schedule.h"
using namespace c2d;
// A thread's loops over k-blocks kb0 .. kb1 - 1, one after the other round a ring of S stages, as the block-scaled products
// run them. Before k-block i is handled, those up to i - S are known to be done. Copies whose place a k-block still reads
// that is not known to be done; byStage: with a place for each stage.
int meets(int S, const std::vector<std::pair<int, int>>& loops, bool byStage) {
  ScalePlaces places = {static_cast<uint32_t>(S), 0};
  std::vector<int> reader(S, -1);  // a place's last k-block
  int i = 0, bad = 0;
  unsigned at = 0;
  for (auto [kb0, kb1] : loops)
    for (int kb = kb0; kb < kb1; ++kb, ++i) {
      if (scales_begin(kb, kb0)) {
        at = byStage ? i % S : places.next();
        if (at >= static_cast<unsigned>(S)) return -1;
        if (reader[at] >= 0 && reader[at] > i - S) ++bad;
      }
      reader[at] = i;
    }
  return bad;
}
int main() {
  for (int byStage = 0; byStage < 2; ++byStage) {
    long bad = 0;
    for (int S = 2; S <= 8; ++S)
      for (int first = 0; first < 8; ++first)
        for (int n = 1; n <= 40; ++n) {
          std::vector<std::pair<int, int>> loops;
          for (int u = 0; u < 9; ++u) loops.push_back({first, first + n});     // units of one length
          for (int u = 0; u < 9; ++u) loops.push_back({u, u + 1 + (n * u) % 7});  // shares that begin and end anywhere
          const int b = meets(S, loops, byStage);
          if (b < 0) return 1;
          bad += b;
        }
    std::printf("%ld\\n", bad);
  }
}
"""


def test_places_of_scales_are_read_no_more_when_they_are_written(tmp_path):
    in_turn, by_stage = map(int, run(tmp_path, PLACES).split())
    assert in_turn == 0
    assert by_stage > 0  # what the count is for: places that belong to the stages




BLOCKS = """
#include <algorithm>
#include <cstdio>
#include "schedule.h"
int main() {
  // what there was: never fewer than eight
  auto before = [](long most, long rows) { return most < rows ? std::max(8L, most / 8 * 8) : rows; };
  for (int old = 0; old < 2; ++old) {
    long many = 0, unlike = 0, idle = 0;
    for (long most = 1; most <= 320; ++most)
      for (long rows = 1; rows <= 700; ++rows) {
        const long b = old ? before(most, rows) : c2d::blocks_alike(most, rows);
        many += b > most || b > rows;
        unlike += b < rows && b % 8 != 0;
        idle += b == 0 && (most >= 8 || rows <= most);
      }
    std::printf("%ld %ld %ld\\n", many, unlike, idle);
  }
}
"""


def test_no_more_blocks_than_rows_or_than_the_workspace_has_room_for(tmp_path):
    here, before = run(tmp_path, BLOCKS).splitlines()
    assert here == "0 0 0"
    assert int(before.split()[0]) > 0  # what the count is for
