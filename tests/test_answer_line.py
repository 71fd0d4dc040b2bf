"""The line of key tiles that the CTAs of the cached-keys kernel share
(csrc/line_walk.h), compiled for the host and checked without a GPU: for random
lengths the CTAs' pieces cover every key tile of every item once, a CTA leaves
at most one piece of an item begun by an earlier CTA (its first) and one that
goes on in the next (its last), the CTA named as an item's last is the one that
holds its last tile, and the parts differ by at most one unit."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_causal_attention_zigzag_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"

PROGRAM = r"""
#include <stdio.h>
#include <map>
#include <random>
#include <tuple>
#include <vector>
#include "line_walk.h"
using namespace cpattn;
using namespace cpattn::line;

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

template <bool kPaged>
int one(std::mt19937& rng) {
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  const int R = pick(1, 40), Hkv = pick(1, 9), grid = pick(1, 160);
  const int spans[] = {1, 9, 16, 32, 64, 128, 256}, span = spans[pick(0, 6)];
  const int most = pick(0, 3) == 0 ? 5000 : 200, new_most = pick(0, 2) == 0 ? 700 : 3;
  std::vector<int> ctx(R), cu(R + 1, 0), cu_k(R + 1, 0);
  for (int r = 0; r < R; ++r) {
    ctx[r] = pick(0, 4) == 0 ? 0 : pick(0, most);
    cu[r + 1] = cu[r] + (pick(0, 4) == 0 ? 0 : pick(0, new_most));
    cu_k[r + 1] = cu_k[r] + (pick(0, 4) == 0 ? 0 : pick(0, most));
  }
  unsigned long long word = 0;
  TreeArgs a = {};
  a.R = R;
  a.N = cu[R];
  a.Hkv = Hkv;
  a.cu = cu.data();
  a.ctx = ctx.data();
  a.width = 1000;
  a.cache.page_size = 16;
  a.tree = pick(0, 1) ? &word : nullptr;
  a.cu_k = cu_k.data();
  a.Nk = cu_k[R];
  a.causal = pick(0, 1);
  if (!kPaged) a.tree = nullptr;
  const bool chain = a.tree == nullptr;

  std::vector<Req> req(R);
  std::vector<long long> before(R + 1, 0);
  std::map<std::tuple<int, int, int>, int> tiles;  // of every item
  for (int r = 0; r < R; ++r) {
    load_req<kPaged>(a, r, req[r]);
    before[r + 1] = before[r] + head_cost(req[r], span, chain) * Hkv;
    for (int g = 0; g < Hkv; ++g)
      for (int m = 0; m < items_of(req[r], span); ++m)
        tiles[{r, g, m}] = tiles_of(req[r], span, chain, m);
  }
  const long long T = before[R], parts = (T + kMinPart - 1) / kMinPart;
  const int n = (int)(parts < grid ? parts : grid);
  Cuts cuts;
  cuts.init(T, n);
  std::map<std::tuple<int, int, int>, int> done, last_cta, named;
  long long small = T, large = 0;
  for (int c = 0; c < n; ++c) {
    const long long begin = cuts.begin(c), count = cuts.begin(c + 1) - begin;
    CHECK(count > 0);
    small = count < small ? count : small;
    large = count > large ? count : large;
    CHECK(cuts.of(begin) == c && cuts.of(begin + count - 1) == c);
    int r = 0;
    while (begin >= before[r + 1]) ++r;
    Walk<kPaged> w;
    w.init(a, span, r, req[r], begin - before[r], begin, count);
    bool first = true, open = false;
    while (w.next(a, span)) {
      const Piece& p = w.p;
      const std::tuple<int, int, int> item{p.r, p.g, p.m};
      CHECK(!open);  // a piece that goes on is the CTA's last
      CHECK(tiles.count(item) && p.tiles == tiles[item]);
      CHECK(p.t0 == done[item] && p.t1 > p.t0 && p.t1 <= p.tiles);
      CHECK(p.t0 == 0 || first);
      CHECK(p.x.q0 == req[p.r].q0 && p.x.n == req[p.r].n && p.x.total == req[p.r].total);
      if (p.t0 == 0) named[item] = cuts.of(p.item_at + kItemCost + p.tiles - 1);
      open = p.t1 < p.tiles;
      done[item] = p.t1;
      last_cta[item] = c;
      first = false;
    }
  }
  CHECK(n == 0 ? T == 0 : cuts.begin(n) == T);
  CHECK(large - small <= 1 || n == 0);
  for (auto& t : tiles) {
    CHECK(done[t.first] == t.second);
    CHECK(named[t.first] == last_cta[t.first]);
  }
  return 0;
}

int main() {
  std::mt19937 rng(7);
  for (int i = 0; i < 1500; ++i)
    if (one<true>(rng) || one<false>(rng)) return 1;
  printf("ok\n");
  return 0;
}
"""


def test_pieces_cover_every_key_tile_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "line.cpp", tmp_path / "line"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INCLUDE,
                    str(src), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
