"""The cached-weights kernel without a GPU: the line of products that its CTAs share
(csrc/weights_line.h, compiled for the host) and its mbarrier protocol under random
schedules.  For random lengths the CTAs' pieces cover every step of every item once,
an item's steps are the tiles of tokens that see any of its keys, the CTA named as an
item's last holds its last step, and rows are kept from piece to piece exactly where both
sides of the exchange expect it."""
import os
import random
import shutil
import subprocess

import pytest

from protocol_sims import weights_kernel

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_causal_attention_zigzag_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"

PROGRAM = r"""
#include <stdio.h>
#include <map>
#include <random>
#include <tuple>
#include <vector>
#include "weights_line.h"
using namespace cpattn;
using namespace cpattn::wline;

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int one(std::mt19937& rng) {
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  const int R = pick(1, 40), Hkv = pick(1, 9), grid = pick(1, 160);
  const int tpts[] = {1, 2, 9, 16, 18, 32, 42, 64, 128}, tpt = tpts[pick(0, 8)];
  const int most = pick(0, 3) == 0 ? 5000 : 300, new_most = pick(0, 2) == 0 ? 1500 : 3;
  std::vector<int> ctx(R), cu(R + 1, 0);
  for (int r = 0; r < R; ++r) {
    ctx[r] = pick(0, 4) == 0 ? 0 : pick(0, most);
    cu[r + 1] = cu[r] + (pick(0, 4) == 0 ? 0 : pick(0, new_most));
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
  a.tree = pick(0, 2) ? nullptr : &word;
  const bool chain = a.tree == nullptr, keep = pick(0, 1);
  std::vector<Req> req(R);
  std::vector<long long> before(R + 1, 0);
  std::map<std::tuple<int, int, int>, std::pair<int, int>> items;  // first tile and steps
  for (int r = 0; r < R; ++r) {
    load_req<true>(a, r, req[r]);
    const Req& x = req[r];
    long long sum = 0;
    for (int m = 0; x.n > 0 && m < items_of(x); ++m) {
      int first = -1;  // of the tiles whose last token sees the item's first key
      const int tiles = (x.n + tpt - 1) / tpt;
      for (int t = 0; t < tiles && first < 0; ++t) {
        const int last = t * tpt + tpt - 1;
        if (!chain || m * kPair <= x.ctx + last) first = t;
      }
      CHECK(first >= 0 && first == first_tile(x, tpt, chain, m * kPair));
      CHECK(sum == cost_upto(x, tpt, chain, m));
      sum += kItemCost + tiles - first;
      for (int g = 0; g < Hkv; ++g) items[{r, g, m}] = {first, tiles - first};
    }
    CHECK(sum == head_cost(x, tpt, chain));
    before[r + 1] = before[r] + sum * Hkv;
  }
  const long long T = before[R], parts = (T + kMinPart - 1) / kMinPart;
  const int n = (int)(parts < grid ? parts : grid);
  Cuts cuts;
  cuts.init(T, n);
  std::map<std::tuple<int, int, int>, int> done, last_cta, named;
  for (int c = 0; c < n; ++c) {
    const long long begin = cuts.begin(c), count = cuts.begin(c + 1) - begin;
    CHECK(count > 0 && cuts.of(begin) == c && cuts.of(begin + count - 1) == c);
    int r = 0;
    while (begin >= before[r + 1]) ++r;
    Walk w;
    w.init(a, tpt, r, req[r], begin - before[r], begin, count);
    bool first = true, open = false, kept = false;
    int pr = -1, pg = -1, pt = -1;
    while (w.next(a, tpt, keep)) {
      const Piece& p = w.p;
      const std::tuple<int, int, int> item{p.r, p.g, p.m};
      CHECK(!open);  // a piece that goes on is the CTA's last
      CHECK(items.count(item) && p.q0t == items[item].first && p.steps == items[item].second);
      CHECK(p.s0 == done[item] && p.s1 > p.s0 && p.s1 <= p.steps);
      CHECK(p.s0 == 0 || first);
      CHECK(p.x.q0 == req[p.r].q0 && p.x.n == req[p.r].n && p.x.total == req[p.r].total);
      // Rows that are kept are those of the piece's only tile.
      CHECK(p.fresh == !kept);
      if (kept) CHECK(p.r == pr && p.g == pg && p.q0t == pt && p.s1 - p.s0 == 1 && p.q0t == 0);
      kept = !p.last;
      CHECK(keep || !kept);
      if (kept) CHECK(w.more);
      pr = p.r, pg = p.g, pt = p.q0t + p.s1 - 1;
      for (int i = 0; i < 2; ++i) {
        const int b = p.begins(i, tpt, chain), k0 = p.m * kPair + i * kTcTile;
        CHECK(b >= p.s0 && b <= p.s1);
        for (int s = p.s0; s < p.s1; ++s) {
          const int last = (p.q0t + s) * tpt + tpt - 1;
          const bool needed = k0 < p.x.total && (!chain || k0 <= p.x.ctx + last);
          CHECK(needed == (s >= b));
        }
      }
      if (p.s0 == 0) named[item] = cuts.of(p.item_at + kItemCost + p.steps - 1);
      open = p.s1 < p.steps;
      done[item] = p.s1;
      last_cta[item] = c;
      first = false;
    }
  }
  CHECK(n == 0 ? T == 0 : cuts.begin(n) == T);
  for (auto& t : items) {
    CHECK(done[t.first] == t.second.second);
    CHECK(named[t.first] == last_cta[t.first]);
  }
  return 0;
}

int main() {
  std::mt19937 rng(7);
  for (int i = 0; i < 20000; ++i) {
    const int n = rng() % 30, m = 1 + rng() % 300, a = rng() % 600, b = rng() % 600;
    long long sum = 0;
    for (int k = 0; k < n; ++k) sum += (a * k + b) / m;
    if (sum != floor_sum(n, m, a, b)) return 2;
  }
  for (int i = 0; i < 1500; ++i)
    if (one(rng)) return 1;
  printf("ok\n");
  return 0;
}
"""


def test_pieces_cover_every_step_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "line.cpp", tmp_path / "line"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INCLUDE,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


PIECES = [(1, 0, 0, True), (1, 0, 0, False), (1, 0, 1, True), (2, 0, 0, False), (4, 0, 2, False), (5, 0, 5, False),
          (3, 0, 1, False), (2, 0, 2, False)]
RINGS = [dict(depth=1, rows=4), dict(rows=8), dict(depth=3, rows=1, deep=True), dict(depth=6, rows=1, deep=True)]


def draws(n, seed):
    rng = random.Random(seed)
    return [[rng.choice(PIECES) for _ in range(rng.randint(1, 9))] for _ in range(n)]


@pytest.mark.parametrize("ring", RINGS)
def test_protocol_holds_under_random_schedules(ring):
    for seed, work in enumerate(draws(1500, 5)):
        weights_kernel.run(work, seed, **ring)


@pytest.mark.parametrize("deep,mutation", [(False, m) for m in (1, 2, 3, 6, 7, 8, 9, 10, 11, 12, 13)] + [(True, m) for m in (1, 2, 3, 4, 5, 6, 7, 8, 9, 11)])
def test_planted_protocol_mistake_is_caught(deep, mutation):
    for seed, work in enumerate(draws(2000, 7)):
        try:
            weights_kernel.run(work, seed, mutation=mutation, depth=1 + seed % 2, deep=deep)
        except AssertionError:
            return
    pytest.fail(f"mutation {mutation} survived 2000 schedules")
