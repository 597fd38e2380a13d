"""Cluster barriers between the sampler's accesses to shared memory that other CTAs touch, on every path.

All CTAs of a cluster run the same statements, each at its own pace.  Two accesses to one CTA's copy of a
field, of which one comes from another CTA and one writes, need a cluster barrier between them: an arrival
behind the first and, of the same phase, a wait ahead of the second.  Nobody may leave while an access of
another CTA to its memory may be under way, and none may be made once somebody can have left.

The source is parsed into statements (branches, loops, breaks, returns, the kernel's lambdas and helpers in
place of their calls) and walked with the set of accesses that no barrier has closed yet, loops until
nothing is added."""
import os
import re

import pytest

from quantized_decode_memq_gb300.build import CSRC

# Conditions that are the same in all CTAs of a cluster: formed from the row's settings, from the loops' own
# counters and from what all read between two barriers.  Barriers stand under no others.
UNIFORM = {
    "!(temperature > 0.f) || k == 1 || top_key <= kLeastKey", "k < a.vocab && each <= T / 2 && k <= kCap / 2",
    "n_all <= kCap", "k < a.vocab", "p < 1.f", "counting", "!sorted", "!sorted && !beyond", "beyond", "lo < hi",
    "from < to", "int level = 0; level < 2 && !sorted; ++level", "by_cta", "tabled", "BF16 && level == 0 && tabled",
}
INLINED = ("cluster_sum", "join_lists", "append", "bisect_k", "find_cut", "sort_list")
# Writes that never meet: places that an atomic gave out, one's own element, a value that one thread of the cluster has.
DISJOINT = {"list", "pair", "sums", "from_cta", "bounds", "step", "before", "cut", "partial"}


def strip(text):
    return re.sub(r"//[^\n]*", "", text)


def closing(s, i):
    """The index behind the bracket that closes the one at i."""
    pairs, depth = {"(": ")", "[": "]", "{": "}"}, 0
    a, b = s[i], pairs[s[i]]
    while True:
        depth += {a: 1, b: -1}.get(s[i], 0)
        i += 1
        if depth == 0:
            return i


def parse(s):
    """Statements of a text: ('if', cond, then, else), ('loop', cond, body), ('lambda', name, body), ('expr', text),
    ('return',), ('break',), ('continue',), ('block', statements)."""
    out, i = [], 0

    def one(i):
        m = re.compile(r"\s*(?:#[^\n]*\n\s*)*").match(s, i)
        i = m.end()
        if i >= len(s):
            return None, i
        if s[i] == "{":
            j = closing(s, i)
            return ("block", parse(s[i + 1:j - 1])), j
        m = re.compile(r"(if constexpr|if|for|while)\s*\(").match(s, i)
        if m:
            j = closing(s, m.end() - 1)
            cond = " ".join(s[m.end():j - 1].split())
            body, k = one(j)
            if m.group(1) in ("for", "while"):
                return ("loop", cond, body), k
            m = re.compile(r"\s*else\b").match(s, k)
            if m:
                other, k = one(m.end())
            else:
                other = ("block", [])
            return ("if", cond, body, other), k
        m = re.compile(r"const auto (\w+) = \[&\]\([^)]*\)(?: -> [\w ]+)?\s*\{").match(s, i)
        if m:
            j = closing(s, m.end() - 1)
            return ("lambda", m.group(1), parse(s[m.end():j - 1])), s.index(";", j) + 1
        j = i  # an expression: up to its semicolon, with whatever it holds in brackets
        while s[j] != ";":
            j = closing(s, j) if s[j] in "([{" else j + 1
        text = s[i:j].strip()
        for word in ("return", "break", "continue"):
            if re.match(rf"{word}\b", text):
                return (word, text), j + 1
        return ("expr", text), j + 1

    while True:
        node, i = one(i)
        if node is None:
            return out
        out.append(node)


def function(text, name):
    m = re.search(rf"\b{name}\([^;{{}}]*\)\s*\{{", text)
    return parse(text[m.end():closing(text, m.end() - 1) - 1])


ACCESS = re.compile(
    r"(?P<barrier>cluster_arrive_entry|cluster_wait_entry|cluster_arrive|cluster_wait|cluster_sync)\(\)"
    r"|(?P<call>" + "|".join(INLINED) + r")(?:<T>)?\((?P<args>[^()]*)"
    r"|in_cta\(&sh\.(?P<rfield>\w+)"                                               # another CTA's field
    r"|(?P<obj>first|other|in_cta\(&sh, (?P<who>\w+)\))->(?P<ofield>\w+)(?:\[[^\]]*\]|\.\w+)*(?P<oset>\s*=[^=])?"
    r"|\bsh\.(?P<field>\w+)")


class Walk:
    def __init__(self, text, by_cta):
        self.bodies = {n: function(text, n) for n in ("cluster_sum", "join_lists", "append", "sort_list")}
        self.env = {"by_cta": by_cta, "!by_cta": not by_cta}
        self.faults = set()
        self.conds = []       # the branches and loops around a statement
        self.loops = []       # states at the loops' breaks and continues
        self.other = None     # what `first` and `other` stand for
        self.inside = 0       # helpers and lambdas around a statement: a return leaves them alone
        self.returns = None   # states at their returns
        self.left_by = False  # the kernel was left under the conditions looked at
        self.atomic = False
        self.run(function(text, "sample_kernel"), (frozenset(), False, False))

    # A state: accesses not yet closed (kind, field, whose copies, armed by an arrival), whether all have begun, whether
    # somebody may have left.
    @staticmethod
    def join(a, b):
        if a is None or b is None:
            return b if a is None else a
        return a[0] | b[0], a[1] and b[1], a[2] or b[2]

    def fault(self, what):
        self.faults.add(what)

    def access(self, state, remote, field, write, to0=False):
        pending, begun, left = state
        how = "atomic" if self.atomic else "write" if write else "read"
        side_now = "remote" if remote else "local"
        not0 = not remote and "rank != 0" in self.conds
        if remote and not begun:
            self.fault(f"{field}: before all have begun")
        if remote and left:
            self.fault(f"{field}: somebody may have left")
        for (side, f, was), p0, pnot0, _ in pending:
            if f != field or side == side_now == "local" or was == how == "read":
                continue
            if was == how == "write" and field in DISJOINT:
                continue
            if was == "atomic" and how == "atomic":
                continue
            if (p0 and not0) or (pnot0 and to0):
                continue
            self.fault(f"{field}: {side} {was}, then {side_now} {how}")
        return pending | {((side_now, field, how), to0, not0, False)}, begun, left

    def expr(self, text, state):
        m = re.search(r"(first|other) = in_cta\(&sh, (\w+)\)", text)
        if m:
            self.other = m.group(2)
        for m in ACCESS.finditer(text):
            g = m.groupdict()
            self.atomic = text[:m.start()].endswith("atomicAdd(&")
            if g["barrier"]:
                state = self.barrier(state, g["barrier"])
            elif g["call"]:
                if g["call"] == "find_cut":
                    self.env["counting"] = "true_type" in text
                    self.env["!counting"] = not self.env["counting"]
                body = self.bodies.get(g["call"])
                if body is not None:
                    state = self.inline(body, state)
                if g["call"] == "find_cut":
                    del self.env["counting"], self.env["!counting"]
            elif g["rfield"]:
                state = self.access(state, True, g["rfield"], True)  # (only ever written through an address)
            elif g["obj"]:
                who = g["who"] or self.other
                state = self.access(state, True, g["ofield"], bool(g["oset"]) or self.atomic, who == "0")
            elif g["field"] != "table":
                tail = text[m.end():]
                sub = re.match(r"(?:\[[^\]]*\]|\.\w+)*\s*(=[^=]|\+=)", tail)
                state = self.access(state, False, g["field"], bool(sub) or self.atomic)
        return state

    def barrier(self, state, what):
        pending, begun, left = state
        if any(c not in UNIFORM and c != "loop" for c in self.conds):
            self.fault(f"{what} under a condition that CTAs may differ in: {self.conds}")
        if left:
            self.fault(f"{what}: somebody may have left")
        if what in ("cluster_arrive", "cluster_sync"):
            pending = frozenset((a, b, c, True) for a, b, c, _ in pending)
        if what in ("cluster_wait", "cluster_sync"):
            pending = frozenset(p for p in pending if not p[3])
        return pending, begun or what == "cluster_wait_entry", left

    def inline(self, body, state):
        saved, self.returns = self.returns, None
        self.inside += 1
        after = self.run(body, state)
        after = self.join(after, self.returns)
        self.inside -= 1
        self.returns = saved
        return after

    def run(self, body, state):
        for node in body:
            if state is None:
                break
            state = self.step(node, state)
        return state

    def step(self, node, state):
        kind = node[0]
        if kind == "block":
            return self.run(node[1], state)
        if kind == "lambda":
            self.bodies[node[1]] = node[2] if node[1] in INLINED else None
            # the others touch what their uses' places touch: taken where they stand
            return state if node[1] in INLINED else self.join(state, self.inline(node[2], state))
        if kind == "expr":
            return self.expr(node[1], state)
        if kind == "return":
            state = self.expr(node[1], state)
            if not self.inside:
                for (side, field, how), *_ in state[0]:
                    if side == "remote":
                        self.fault(f"{field}: a {how} of another CTA may be under way at a return")
                self.left_by = True
            else:
                self.returns = self.join(self.returns, state)
            return None
        if kind in ("break", "continue"):
            at = self.loops[-1]
            at[kind] = self.join(at[kind], state)
            return None
        if kind == "if":
            cond = node[1]
            state = self.expr(cond, state)
            if cond in self.env:
                return self.step(node[2] if self.env[cond] else node[3], state)
            self.conds.append(cond)
            gone, self.left_by = self.left_by, False
            a = self.step(node[2], state)
            b = self.step(node[3], state)
            self.conds.pop()
            out = self.join(a, b)
            if self.left_by and cond not in UNIFORM and out is not None:
                out = (out[0], out[1], True)
            self.left_by = gone or (self.left_by and cond not in UNIFORM)
            return out
        assert kind == "loop"
        cond = node[1]
        state = self.expr(cond, state)
        # loops without barriers may run a different number of turns
        self.conds.append(cond if cond in UNIFORM else "a loop")
        out = None
        while True:
            self.loops.append({"break": None, "continue": None})
            end = self.step(node[2], state)
            at = self.loops.pop()
            end = self.join(end, at["continue"])
            if end is not None:
                end = self.expr(cond, end)
            out = self.join(out, self.join(state, at["break"]))
            again = self.join(state, end)
            if again == state:
                break
            state = again
        self.conds.pop()
        return out


def faults(text):
    return set().union(*(Walk(text, by_cta).faults for by_cta in (False, True)))


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(CSRC, "memq_sample.cu")) as f:
        return strip(f.read())


def test_every_path_of_the_sampler_has_its_barriers(source):
    assert faults(source) == set()


def barriers(text):
    """(start, end) of every barrier statement of the kernel and the helpers that hold one."""
    lo = text.index("void cluster_sum(")
    return [(m.start(), m.end()) for m in re.finditer(r"\bcluster_(?:sync|wait)\(\);", text) if m.start() > lo]


def test_the_check_sees_each_missing_barrier(source):
    found = barriers(source)
    assert len(found) >= 12
    for lo, hi in found:
        cut = source[:lo] + ";" + source[hi:]
        assert faults(cut), source[max(0, lo - 120):hi]
    entry = source.replace("    cluster_wait_entry();", "")
    assert entry != source and faults(entry)
