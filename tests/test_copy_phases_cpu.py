"""The bookkeeping by which the paged attention's copying warp awaits its copies in flight when it has to
stop early (csrc/memq_phases.cuh), run on the host against barriers that count their phases."""
import os
import shutil
import subprocess

import pytest

from quantized_decode_memq_gb300.build import CSRC

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "memq_phases.cuh"
using namespace memq;

struct Barrier { unsigned announced = 0; };  // phases announced; a phase is over when its copies are
static int errors = 0;
// A wait for `parity` returns once the phase that is under way has the other one.  All phases but the last
// announced are over here, so it outlasts the last one just when that one has this parity.
static void drained(const Barrier &b, unsigned uses, const char *what) {
    if (uses != b.announced) { ++errors; std::printf("%s: %u uses, %u announced\n", what, uses, b.announced); }
    if (uses && last_parity(uses) != ((b.announced - 1) & 1)) { ++errors; std::printf("%s: parity\n", what); }
}

int main() {
    for (unsigned slots = 1; slots <= 12; ++slots)
        for (unsigned pieces = 1; pieces <= 4 && pieces <= slots; pieces *= 2)
            for (int rope = 0; rope < 2; ++rope)
                for (unsigned stop = 0; stop < 90; ++stop) {  // the wait that expires
                    CopyPhases sent;
                    std::vector<Barrier> full(slots), scale(2);
                    Barrier ropes;
                    unsigned waits = 0;
                    for (bool dead = false; !dead;) {  // a tile, in the kernel's order
                        if ((dead = waits++ == stop)) break;
                        ++scale[sent.scales & 1].announced;
                        ++sent.scales;
                        if (rope) {
                            if ((dead = waits++ == stop)) break;
                            ++ropes.announced;
                            ++sent.ropes;
                        }
                        for (unsigned c = 0; c < pieces; ++c) {
                            if ((dead = waits++ == stop)) break;
                            if (sent.lap != full[sent.slot].announced) ++errors;
                            ++full[sent.slot].announced;
                            sent.piece_announced(slots);
                        }
                    }
                    for (unsigned s = 0; s < slots; ++s) drained(full[s], sent.pieces_in(s), "slot");
                    for (unsigned b = 0; b < 2; ++b) drained(scale[b], sent.scales_in(b), "scales");
                    drained(ropes, sent.ropes, "rope");
                }
    return errors != 0;
}
"""


def test_what_was_announced_is_what_is_awaited(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "phases.cpp", tmp_path / "phases"
    src.write_text(PROGRAM)
    subprocess.check_call([cxx, "-std=c++17", "-Wall", "-Werror", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[:2000]


def test_the_copying_warp_counts_where_it_announces():
    """Every announcement on a copy's barrier in the kernel is followed by its count, and an expired wait
    leaves the loops ahead of both."""
    with open(os.path.join(CSRC, "memq_mla_paged.cu")) as f:
        text = f.read()
    body = text[text.index("TMA producer"):text.index("tensor-core products")]
    for bar, count in (("scale_full", "++sent.scales"), ("rope_full", "++sent.ropes"), ("full[slot]", "sent.piece_announced")):
        at = body.index(f"mbar_arrive_expect_tx(&ctl->{bar}")
        assert body.rindex("if (wait.dead) break;", 0, at) < at < body.index(count)
        assert "wait(" not in body[at:body.index(count)]
    assert body.count("mbar_arrive_expect_tx") == 3
