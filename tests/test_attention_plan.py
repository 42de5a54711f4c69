"""The block attention's division of work (csrc/attention_plan.h), on the CPU.

The header is plain integer arithmetic; a small program built from it walks the
parts of every worker over random sets of items, and each token tile of each item
has to be taken exactly once, pieces have to follow the order that the joining
of partial results relies on, and the joining's own enumeration (first worker,
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
struct Item { int64_t start; int tiles, cls; };
#define CHECK(c) do { if (!(c)) { std::printf("failed: %s (case %d)\n", #c, which); return 1; } } while (0)
int main() {
    std::mt19937_64 g(1);
    auto pick = [&](int64_t lo, int64_t hi) { return (int64_t)(lo + g() % (uint64_t)(hi - lo + 1)); };
    for (int which = 0; which < 3000; ++which) {
        const int ctas = which % 3 == 0 ? 152 : (int)pick(1, 200), heads = (int)pick(1, 9), lists = (int)pick(1, 40);
        std::vector<int> rows(lists), tiles(lists);
        for (int b = 0; b < lists; ++b) {
            rows[b] = (int)pick(0, which % 5 == 0 ? 2000 : 300);
            const int tokens = (int)pick(0, which % 7 == 0 ? 200000 : 900);
            tiles[b] = token_tiles(tokens);
            CHECK((int64_t)tiles[b] * kTile >= tokens && (int64_t)(tiles[b] - 1) * kTile < tokens);
        }
        // the line: all pairs, then all singles
        std::vector<Item> items;
        int64_t at = 0, pairs = 0;
        for (int cls = 0; cls < 2; ++cls) {
            for (int b = 0; b < lists; ++b) {
                const int64_t per = head_units(cls, rows[b], tiles[b]);
                const int n = class_tiles(cls, rows[b]);
                for (int h = 0; h < heads && per > 0; ++h) {
                    for (int k = 0; k < n; ++k) {
                        const int rt = class_row_tile(cls, rows[b], k), tr = tile_rows(rows[b], rt);
                        CHECK(rt >= 0 && rt < row_tiles(rows[b]) && tr >= 1 && tr <= kTileRows && class_of(tr) == cls);
                        items.push_back({at + h * per + k * item_total(cls, tiles[b]), tiles[b], cls});
                    }
                }
                at += per * heads;
                CHECK(class_tiles(0, rows[b]) + class_tiles(1, rows[b]) == (rows[b] > 0 ? row_tiles(rows[b]) : 0));
            }
            if (cls == 0) pairs = at;
        }
        const int64_t total = at;
        int64_t to = 0;
        for (const Item &i : items) { CHECK(i.start == to); to += item_total(i.cls, i.tiles); }
        CHECK(to == total);
        if (total == 0) continue;
        CHECK(cta_begin(0, total, ctas) == 0 && cta_begin(ctas, total, ctas) == total);
        CHECK(single_begin(2 * ctas, pairs, total, ctas) == total);
        std::vector<int> taken(items.size(), 0);
        std::vector<std::vector<int>> by(items.size());
        for (int cls = 0; cls < 2; ++cls) {
            const int workers = cls == kPair ? ctas : 2 * ctas;
            for (int v = 0; v < workers; ++v) {
                int64_t lo = worker_begin(cls, v, pairs, total, ctas), hi = worker_begin(cls, v + 1, pairs, total, ctas);
                CHECK(lo <= hi);
                if (cls == kPair && hi > pairs) hi = pairs;
                int pieces = 0;
                for (size_t k = 0; k < items.size(); ++k) {
                    const Item &i = items[k];
                    if (i.cls != cls) continue;
                    const int64_t end = i.start + item_total(cls, i.tiles);
                    if (end <= lo || i.start >= hi) continue;
                    const int64_t u = i.start > lo ? i.start : lo;      // the cursor
                    const int t0 = first_tile(cls, u, i.start, i.tiles), t1 = first_tile(cls, hi, i.start, i.tiles);
                    CHECK(t0 >= 0 && t0 <= t1 && t1 <= i.tiles);
                    if (t0 == t1) continue;
                    CHECK(t0 == taken[k]);               // in order, nothing twice, nothing left out
                    CHECK(t0 == 0 || pieces == 0);       // only a worker's first piece goes on with an item
                    taken[k] = t1;
                    by[k].push_back(v);
                    ++pieces;
                }
            }
        }
        for (size_t k = 0; k < items.size(); ++k) {
            const Item &i = items[k];
            CHECK(taken[k] == i.tiles);
            const int64_t end = i.start + item_total(i.cls, i.tiles);
            std::vector<int> named;
            const int workers = i.cls == kPair ? ctas : 2 * ctas;
            const int v0 = worker_of(i.cls, i.start + item_units(i.cls), pairs, total, ctas);
            CHECK(v0 >= 0 && v0 < workers);
            named.push_back(v0);
            int64_t from = worker_begin(i.cls, v0 + 1, pairs, total, ctas);
            const bool alone = first_tile(i.cls, from, i.start, i.tiles) == i.tiles;
            for (int v = v0 + 1; v < workers && from < end; ++v) {
                const int64_t next = worker_begin(i.cls, v + 1, pairs, total, ctas);
                if (first_tile(i.cls, from, i.start, i.tiles) < first_tile(i.cls, next, i.start, i.tiles)) named.push_back(v);
                from = next;
            }
            CHECK(named == by[k]);
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
