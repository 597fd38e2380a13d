"""Order of cluster barriers and remote shared-memory accesses in the kernels' sources.

Another CTA's shared memory may be touched only once that CTA is known to run: a wait on a cluster
barrier has to stand before a kernel's first remote access, and one after its last (nobody leaves while
others still reach into it)."""
import os
import re

import pytest

from quantized_decode_memq_gb300.build import CSRC

WAIT = "barrier.cluster.wait"
REMOTE = re.compile(r"\b(?:ld|st|atom|red)\.[a-z.:]*shared::cluster")


def strip(text):
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


def functions(text):
    """(name, body) of the functions defined in a source, by their braces."""
    end = 0
    for m in re.finditer(r"(\w+)\s*\([^;{}]*\)\s*\{", text):
        if m.start() < end:  # a block inside the last one
            continue
        depth, i = 1, m.end()
        while depth and i < len(text):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        end = i
        yield m.group(1), text[m.end():i]


def check(text):
    """Kernels with remote accesses, each as (first wait, first access, last access, last wait)."""
    text = strip(text)
    bodies = list(functions(text))
    waits = [n for n, b in bodies if WAIT in b and len(b) < 400]
    remote = [n for n, b in bodies if REMOTE.search(b) and len(b) < 400]
    out = []
    for name, body in bodies:
        if name in waits or name in remote:
            continue
        at = lambda names: sorted(m.start() for n in names for m in re.finditer(rf"\b{n}\s*\(", body))
        w, r = at(waits), at(remote)
        if r:
            out.append((w[0] if w else None, r[0], r[-1], w[-1] if w else None))
    return out


@pytest.mark.parametrize("source,kernels", [("memq_add_producer.cu", 1), ("memq_mla.cu", 2)])
def test_a_cluster_barrier_on_either_side_of_remote_accesses(source, kernels):
    with open(os.path.join(CSRC, source)) as f:
        found = check(f.read())
    assert len(found) == kernels
    for first_wait, first, last, last_wait in found:
        assert first_wait is not None and first_wait < first, "remote access before any cluster barrier"
        assert last_wait > last, "no cluster barrier behind the last remote access"


def test_the_check_sees_a_missing_barrier():
    body = '''void put(int *p) { asm volatile("st.shared::cluster.u32 [%0], 0;" ::"r"(p)); }
    void meet() { asm volatile("barrier.cluster.arrive;\\n\\tbarrier.cluster.wait;"); }
    void kernel(int *p) { put(p); meet(); }
    void sound(int *p) { meet(); put(p); meet(); }'''
    (late, first, *_), (early, second, *_) = check(body)
    assert late > first and early < second
