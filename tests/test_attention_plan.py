"""The block attention's division of work (csrc/attention_plan.h), on the CPU.

The header is plain integer arithmetic; a small program built from it walks the
parts of every CTA over random sets of items, and each token tile of each item
has to be taken exactly once, pieces have to follow the order that the joining
of partial results relies on, and the joining's own enumeration (first CTA,
then those that go on) has to name exactly the pieces that were taken."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "attention_plan.h"
using namespace dspark::plan;
struct Item { int64_t start; int tiles, w; };
#define CHECK(c) do { if (!(c)) { std::printf("failed: %s (case %d)\n", #c, which); return 1; } } while (0)
int main() {
    std::mt19937_64 g(1);
    auto pick = [&](int64_t lo, int64_t hi) { return (int64_t)(lo + g() % (uint64_t)(hi - lo + 1)); };
    for (int which = 0; which < 3000; ++which) {
        const int ctas = which % 3 == 0 ? 152 : (int)pick(1, 200), heads = (int)pick(1, 9);
        std::vector<Item> items;
        int64_t total = 0;
        const int lists = (int)pick(1, 40);
        for (int b = 0; b < lists; ++b) {
            const int rows = (int)pick(0, which % 5 == 0 ? 2000 : 300);
            const int tokens = (int)pick(0, which % 7 == 0 ? 200000 : 900), tiles = token_tiles(tokens);
            CHECK((int64_t)tiles * kTile >= tokens && (int64_t)(tiles - 1) * kTile < tokens);
            const int64_t per = head_units(rows, tiles);
            for (int h = 0; h < heads && per > 0; ++h) {
                int covered = 0;
                for (int rt = 0; rt < row_tiles(rows); ++rt) {
                    const int tr = tile_rows(rows, rt);
                    CHECK(tr >= 1 && tr <= kTileRows);
                    covered += tr;
                    const int64_t start = total + h * per + row_tile_start(rt, tiles);
                    items.push_back({start, tiles, weight(tr)});
                    CHECK(row_tile_of(start - total - h * per, rows, tiles) == rt);
                    CHECK(row_tile_of(start - total - h * per + (int64_t)tiles * weight(tr) - 1, rows, tiles) == rt);
                }
                CHECK(covered == rows);
            }
            total += per * heads;
        }
        int64_t at = 0;
        for (const Item &i : items) { CHECK(i.start == at); at += (int64_t)i.tiles * i.w; }
        CHECK(at == total);
        if (total == 0) continue;
        CHECK(cta_begin(0, total, ctas) == 0 && cta_begin(ctas, total, ctas) == total);
        std::vector<int> taken(items.size(), 0);
        std::vector<std::vector<int>> by(items.size());
        for (int c = 0; c < ctas; ++c) {
            const int64_t lo = cta_begin(c, total, ctas), hi = cta_begin(c + 1, total, ctas);
            int pieces = 0;
            for (size_t k = 0; k < items.size(); ++k) {
                const Item &i = items[k];
                const int64_t end = i.start + (int64_t)i.tiles * i.w;
                if (end <= lo || i.start >= hi) continue;
                const int64_t u = i.start > lo ? i.start : lo;      // the cursor
                const int t0 = first_tile(u, i.start, i.w, i.tiles), t1 = first_tile(hi, i.start, i.w, i.tiles);
                CHECK(t0 >= 0 && t0 <= t1 && t1 <= i.tiles);
                if (t0 == t1) continue;
                CHECK(t0 == taken[k]);               // in order, nothing twice, nothing left out
                CHECK(t0 == 0 || pieces == 0);       // only a CTA's first piece goes on with an item
                taken[k] = t1;
                by[k].push_back(c);
                ++pieces;
            }
        }
        for (size_t k = 0; k < items.size(); ++k) {
            const Item &i = items[k];
            CHECK(taken[k] == i.tiles);
            const int64_t end = i.start + (int64_t)i.tiles * i.w;
            std::vector<int> named;
            const int c0 = cta_of(i.start, total, ctas);
            CHECK(cta_begin(c0, total, ctas) <= i.start && i.start < cta_begin(c0 + 1, total, ctas));
            named.push_back(c0);
            for (int c = c0 + 1; c < ctas; ++c) {
                const int64_t from = cta_begin(c, total, ctas);
                if (from >= end) break;
                if (first_tile(from, i.start, i.w, i.tiles) < first_tile(cta_begin(c + 1, total, ctas), i.start, i.w, i.tiles))
                    named.push_back(c);
            }
            CHECK(named == by[k]);
            const bool alone = first_tile(cta_begin(c0 + 1, total, ctas), i.start, i.w, i.tiles) == i.tiles;
            CHECK(alone == (by[k].size() == 1));
        }
    }
    std::printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_every_tile_is_taken_once_and_named_by_the_join(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "speculative_decoding_draft_head_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", inc, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout
