"""Which of a ring's places a loader that gives up waits for (csrc/attention_plan.h),
on the CPU: every place whose copies it may have under way, and none that it has
not filled, whatever made it give up (also the wait for its next tile, before any
place is known)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_head_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <set>
#include "attention_plan.h"
using dspark::plan::Filled;
int main() {
    for (uint32_t ring = 1; ring <= 8; ++ring)
        for (uint32_t filled = 0; filled <= 40; ++filled) {
            Filled f = {0};
            for (uint32_t p = 0; p < filled; ++p) f.add(p);
            std::set<uint32_t> waited, want;
            for (uint32_t i = 0; i < f.held(ring); ++i) waited.insert(f.place(i));
            for (uint32_t p = filled > ring ? filled - ring : 0; p < filled; ++p) want.insert(p);
            if (waited != want) { std::printf("ring %u, %u filled\n", ring, filled); return 1; }
        }
    std::printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_the_last_filled_places_are_waited_for(tmp_path):
    src, exe = tmp_path / "drain.cpp", tmp_path / "drain"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout


def test_a_loader_waits_whatever_made_it_give_up():
    """The waits stand behind the loop over tiles, where every way out of it leads, not in one of its branches."""
    text = open(os.path.join(CSRC, "block_attention.cu")).read()
    role = text[text.index("loaders --"):text.index("tensor-core products --")]
    body, after = re.match(r"(.*?for_tiles\(.*?\n            \}\);)(.*)", role, re.S).groups()
    assert "kDrainLimit" not in body and re.search(r"if \(!ok\).*filled\.held.*kDrainLimit", after, re.S)
