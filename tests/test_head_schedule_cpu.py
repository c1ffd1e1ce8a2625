"""The tile schedule of the head loss's products, compiled for the host from the kernel's source:
every tile is dealt exactly once, and the pairs' loads stay level."""

import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "matrix_optimizer_owner_gb300", "csrc", "head_loss.cu")

HARNESS = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
constexpr int kTile = 256, kBK = 64;
struct HeadArgs {
  const int32_t* nlive;
  int32_t dim, width, z_width, splits, want_dh, want_dw, group;
};
%s
template <int PHASE>
int check(const HeadArgs& p, int pairs) {
  std::map<std::tuple<int, int, int, int>, int> seen;
  std::vector<long> load(pairs, 0);
  long total = 0;
  // the deal counts a dH tile by its slice's whole length, though the last slice may be shorter
  const long slice = max(((p.width + 63) / 64 + p.splits - 1) / p.splits, 1);
  for (int q = 0; q < pairs; ++q) {
    TileList<PHASE> l(p, q, pairs);
    // what the MMA issuer counts is what the other roles walk
    std::vector<int> issued;
    for (int c = 0; c < TileList<PHASE>::kKinds; ++c)
      for (int i = 0; i < l.tiles_of(c); ++i) issued.push_back(l.blocks_of(p, c, i));
    size_t at = 0;
    for (TileWalk<PHASE> walk(p, l); walk.have; walk.next(p)) {
      const HeadTile& t = walk.t;
      if (at >= issued.size() || issued[at++] != t.nk) return 6;
      if (++seen[std::make_tuple(t.kind, t.tm, t.tn, t.split)] > 1) return 1;
      const long cost = t.kind == kDh ? slice : max(t.nk, 1);
      load[q] += cost;
      total += cost;
    }
    if (at != issued.size()) return 7;
  }
  const int live = *p.nlive, ntm = (live + 255) / 256, ntd = (p.dim + 255) / 256;
  const long nz = (long)ntm * ((p.z_width + 255) / 256);
  const long ndh = PHASE == kGrads && p.want_dh && p.width > 0 ? (long)ntm * ntd * p.splits : 0;
  const long ndw = PHASE == kGrads && p.want_dw ? (long)((p.width + 255) / 256) * ntd : 0;
  if ((long)seen.size() != nz + ndh + ndw) return 2;
  for (auto& e : seen) {
    const int kind = std::get<0>(e.first), tm = std::get<1>(e.first), tn = std::get<2>(e.first);
    const int rows = kind == kDw ? p.width : live, cols = kind == kZ ? p.z_width : p.dim;
    if (tm < 0 || tn < 0 || tm * 256 >= rows || tn * 256 >= cols) return 3;
    if (std::get<3>(e.first) >= (kind == kDh ? p.splits : 1)) return 4;
  }
  // no pair is above the mean by more than one of the longest tiles
  if (seen.empty()) return 0;
  long longest = 0;
  for (long x : load) longest = max(longest, x);
  const long kd = (p.dim + 63) / 64, kdw = (live + 63) / 64;
  const long kdh = ((p.width + 63) / 64 + p.splits - 1) / p.splits;
  const long most = max(nz ? kd : 0, max(ndw ? kdw : 0, ndh ? kdh : 0));
  return longest <= total / pairs + most + 1 ? 0 : 5;
}
int main() {
  unsigned seed = 7;
  auto rnd = [&](int lo, int hi) {
    seed = seed * 1664525u + 1013904223u;
    return lo + (int)((seed >> 8) %% (unsigned)(hi - lo + 1));
  };
  for (int it = 0; it < 3000; ++it) {
    int32_t live = rnd(0, 3) == 0 ? rnd(0, 300) : rnd(0, 9000);
    HeadArgs p{};
    p.nlive = &live;
    p.dim = rnd(1, 4500);
    p.width = rnd(0, 4) == 0 ? 0 : rnd(1, 12000);
    p.z_width = rnd(0, 4) == 0 ? 0 : rnd(1, 12000);
    p.splits = rnd(0, 2) ? 1 : rnd(1, 20);
    p.want_dh = rnd(0, 4) != 0;
    p.want_dw = rnd(0, 4) != 0;
    p.group = rnd(4, 64);
    const int pairs = rnd(0, 3) ? 76 : rnd(1, 90);
    const int a = check<kGrads>(p, pairs), b = check<kStats>(p, pairs);
    if (a || b) {
      std::printf("case %%d: %%d %%d (live %%d dim %%d width %%d z %%d splits %%d pairs %%d)\n", it, a, b,
                  live, p.dim, p.width, p.z_width, p.splits, pairs);
      return 1;
    }
  }
  std::puts("ok");
}
"""


def test_every_tile_is_dealt_once_and_level(tmp_path):
    with open(SRC, encoding="utf-8") as f:
        src = f.read()
    enums = "\n".join(re.findall(r"^enum \w+ : int \{[^}]*\};", src, flags=re.M))
    body = src[src.index("struct HeadTile {"):]
    body = body[:re.search(r"^};\n\n__device__", body, flags=re.M).start()] + "};\n"
    cc = tmp_path / "schedule.cpp"
    cc.write_text(HARNESS % (enums + "\n" + body))
    exe = str(tmp_path / "schedule")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-o", exe, str(cc)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
