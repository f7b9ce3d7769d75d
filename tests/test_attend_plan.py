"""How the dense attention's work is cut (csrc/attend_plan.cuh), compiled and run on the host for
thousands of drawn batches: every key tile and every own page has exactly one owner, a share has
at most one item that began before it and one that goes on behind it (there is one slot for
each), the costs add up to the closed forms, and the joining kernel finds each item's first share.
No GPU is needed."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_block_sparse_vt_b200", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attend_plan.cuh"
using namespace vt;

static int ri(int lo, int hi) { return lo + rand() % (hi - lo + 1); }
#define CHECK(x) do { if (!(x)) { std::printf("seed %d: %s\n", seed, #x); return 1; } } while (0)

struct Item { Unit u; int t, tiles; int64_t pos, cost; };

int main() {
  for (int seed = 0; seed < 4000; ++seed) {
    srand(seed);
    const int G = ri(1, 8), tpt = kTile / G, heads = ri(1, 8), ctas = ri(1, 3) == 1 ? ri(1, 40) : 148;
    const bool causal = ri(0, 1);
    // row tiles: a line of items
    std::vector<Item> items;
    int64_t pos = 0;
    for (int b = ri(1, 20); b > 0; --b) {
      Unit u{};
      const int kind = ri(0, 3), ctx = ri(0, 2) ? ri(0, 9000) : 0, bad = ri(0, 9) == 0;
      u.n = kind == 0 ? 0 : kind == 1 ? ri(1, 5) : ri(1, kind == 2 ? 300 : 4000);
      u.step = causal && !bad;
      u.kv_len = bad ? 0 : ctx + u.n;
      u.vis0 = bad ? 0 : causal ? ctx + 1 : u.kv_len;
      int64_t head = 0;
      for (int t = 0; t < unit_items(u, tpt); ++t) {
        CHECK(cost_before(u, tpt, t) == head);
        head += item_cost(u, tpt, t);
      }
      CHECK(cost_before(u, tpt, unit_items(u, tpt)) == head);
      for (int h = 0; h < heads; ++h)
        for (int t = 0; t < unit_items(u, tpt); ++t) {
          items.push_back({u, t, (item_keys(u, tpt, t) + kKeys - 1) / kKeys, pos,
                           item_cost(u, tpt, t)});
          pos += items.back().cost;
        }
    }
    if (pos > 0) {
      const Line line = make_line(pos, ctas, kMinShare);
      CHECK(line.n >= 1 && line.n <= ctas);
      CHECK(share_begin(line, 0) == 0 && share_begin(line, line.n) == pos);
      std::vector<int> done(items.size(), 0), pieces(items.size(), 0);
      size_t first = 0;
      for (int c = 0; c < line.n; ++c) {
        const int64_t x0 = share_begin(line, c), x1 = share_begin(line, c + 1);
        CHECK(x0 < x1 && share_of(line, x0) == c && share_of(line, x1 - 1) == c);
        while (items[first].pos + items[first].cost <= x0) ++first;
        int continued = 0, open = 0;
        for (size_t i = first; i < items.size() && items[i].pos < x1; ++i) {
          const Item& it = items[i];
          const int w = item_weight(it.u, tpt, it.t);
          const int j0 = cut_tile(x0 - it.pos, it.cost, w, it.tiles);
          const int j1 = cut_tile(x1 - it.pos, it.cost, w, it.tiles);
          if (j0 < j1 || (it.tiles == 0 && it.pos >= x0)) {
            CHECK(j0 == done[i]);
            done[i] = j1;
            ++pieces[i];
            continued += j0 > 0;
            open += j0 == 0 && j1 < it.tiles;
            CHECK(share_of(line, it.pos) <= c);
          }
        }
        CHECK(continued <= 1 && open <= 1);
      }
      for (size_t i = 0; i < items.size(); ++i) {
        CHECK(done[i] == items[i].tiles);
        CHECK(items[i].tiles > 0 || pieces[i] == 1);
      }
    }
    // own pages: a line of (request, head) items, and the CTAs' split
    std::vector<Unit> own;
    int64_t pages = 0;
    for (int b = ri(1, 60); b > 0; --b) {
      Unit u{};
      u.kv_len = u.vis0 = ri(0, 4) ? ri(0, ri(0, 1) ? 60 : 3000) : 0;
      own.push_back(u);
      CHECK((own_cost(u) == 0) == (u.kv_len == 0));
      pages += heads * own_cost(u);
    }
    const int split = first_own(pos, pages, ctas);
    CHECK(split >= 0 && split <= ctas);
    CHECK((pages == 0) == (split == ctas) || ctas == 1 || pos == 0);
    CHECK(pos == 0 || pages == 0 || ctas == 1 || (split > 0 && split < ctas));
    if (pages > 0) {
      const Line line = make_line(pages, std::max(1, ctas - split) * kWarps, kMinPages);
      int64_t p = 0;
      std::vector<int> continued(line.n, 0);
      for (const Unit& u : own)
        for (int h = 0; h < heads; ++h) {
          int at = 0;
          for (int c = own_cost(u) ? share_of(line, p) : line.n;
               c < line.n && share_begin(line, c) < p + own_cost(u); ++c) {
            const int i0 = own_cut(share_begin(line, c) - p, own_pages(u));
            const int i1 = own_cut(share_begin(line, c + 1) - p, own_pages(u));
            if (i0 >= i1) continue;
            CHECK(i0 == at);
            at = i1;
            continued[c] += i0 > 0;
          }
          CHECK(at == own_pages(u));
          p += own_cost(u);
        }
      for (int c : continued) CHECK(c <= 1);
    }
  }
  std::printf("ok\n");
  return 0;
}
"""


def test_shares_of_drawn_batches():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "plan.cu"), os.path.join(d, "plan")
        with open(src, "w") as f:
            f.write(PROGRAM)
        subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                        "-I", CSRC, src, "-o", exe], check=True, capture_output=True)
        out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
