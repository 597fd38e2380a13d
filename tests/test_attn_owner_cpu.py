"""The join of memq_attn_paged takes from the workspace where pieces and outputs lie; its check of those notes
(csrc/memq_attn_owner.cuh), run on the host over notes that something else wrote."""
import os
import re
import shutil
import subprocess

import pytest

from quantized_decode_memq_gb300.build import CSRC

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "memq_attn_owner.cuh"
using namespace memq;

static uint64_t state = 1;
static uint32_t next() { state = state * 6364136223846793005ull + 1442695040888963407ull; return state >> 33; }
static int any(int near) {  // about a border, or anything
    switch (next() % 4) {
        case 0: return static_cast<int>(next() << 1 ^ next());
        case 1: return next() % 2 ? 0x7fffffff - static_cast<int>(next() % 3) : -0x7fffffff - 1 + static_cast<int>(next() % 3);
        default: return static_cast<int>(next() % (near + 3)) - 1;
    }
}

int main() {
    long taken = 0, errors = 0;
    const int sizes[][5] = {{1, 1, 1, 8, 16}, {5, 2, 3, 16, 16}, {2, 3, 7, 1216, 16}, {7, 8, 8, 152, 256}, {40, 2, 1, 9, 128}};
    for (const auto &s : sizes) {
        const int n_tok = s[0], n_kv = s[1], group = s[2], runs = s[3], stride = s[4], nh = n_kv * group;
        for (int i = 0; i < 2000000; ++i) {
            AttnOwner o{any(n_tok), any(n_tok * group), any(runs), any(runs), any(n_kv), any(stride), {0, 0}};
            if (!attn_owner_ok(o, n_tok, n_kv, group, runs, stride)) continue;
            ++taken;
            // what the join reads and writes
            const int parts = (o.last < runs - 1 ? o.last : runs - 1) - o.first + 1;
            if (parts < 1 || o.first + parts > runs) ++errors;
            for (int r = 0; r < o.rows; r += o.rows > 1 ? o.rows - 1 : 1) {
                for (int k : {0, parts - 1}) {
                    const int64_t slot = static_cast<int64_t>(k == 0 ? 2 * o.first + 1 : 2 * (o.first + k)) * stride + r;
                    if (slot < 0 || slot >= static_cast<int64_t>(2) * runs * stride) ++errors;
                }
                const int64_t rr = static_cast<int64_t>(o.row0) + r, tok = rr / group;
                const int64_t at = (o.start + tok) * nh + static_cast<int64_t>(o.head) * group + (rr - tok * group);
                if (at < 0 || at >= static_cast<int64_t>(n_tok) * nh) ++errors;
            }
        }
        // every note of a call's own is taken
        for (int start = 0; start < n_tok; ++start)
            for (int t = 1; start + t <= n_tok; ++t)
                for (int row0 = 0; row0 < t * group; row0 += stride) {
                    const int left = t * group - row0;
                    AttnOwner o{start, row0, 0, runs - 1, n_kv - 1, left < stride ? left : stride, {0, 0}};
                    if (!attn_owner_ok(o, n_tok, n_kv, group, runs, stride)) ++errors;
                }
    }
    std::printf("%ld taken, %ld outside\n", taken, errors);
    return errors != 0 || taken < 1000;
}
"""


def test_notes_that_are_taken_stay_inside_the_arrays(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "owner.cpp", tmp_path / "owner"
    src.write_text(PROGRAM)
    subprocess.check_call([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[:2000]


def test_the_join_checks_a_note_before_it_uses_it():
    with open(os.path.join(CSRC, "memq_attn_paged.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("attn_join_kernel(const AttnArgs a"):text.index("using EncodeTiledFn")]
    check = body.index("attn_owner_ok(owner, a.n_tok, a.n_kv, a.group, runs, stride)")
    for use in ("owner.first", "owner.last", "owner.start", "owner.head", "owner.row0"):
        assert check < body.index(use)
