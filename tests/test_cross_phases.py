"""The order of the roles in the tensor-core kernels of attention to another sequence,
on the CPU: every interleaving of the copies, the product warps, the row statistics and
the softmax warps ends, and no wait, which knows a barrier's phase by its parity alone,
passes before its phase or misses it. The roles are written out as the kernels have
them; how many places their rings have comes from the kernels' own header."""

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "associative_affine_scan_gb300", "csrc")
MAIN = r"""
#include <cstdio>
#include "scan_cross_phases.h"
int main() {
  for (int d = 64; d <= 128; d += 64) std::printf("%d %d %d\n", scan::fwd_slots(d), scan::bwd_slots(d), scan::step_stages(d));
}
"""


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    d = tmp_path_factory.mktemp("phases")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / "main")], check=True)
    out = subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout.split("\n")
    return [tuple(int(x) for x in r.split()) for r in out[:2]]


class Walk:
    """All interleavings of roles. A role is a list of ("wait", barrier, phase), ("arrive",
    barrier) and ("copy", barrier): a copy, or products that are committed, arrive some
    time later. `count`: how many
    arrivals end a phase of a barrier (1 unless named)."""

    def __init__(self, roles, count):
        names = sorted({op[1] for r in roles for op in r}, key=str)
        at = {n: i for i, n in enumerate(names)}
        self.count = [count.get(n[0] if isinstance(n, tuple) else n, 1) for n in names]
        self.roles = [[(op[0], at[op[1]]) + tuple(op[2:]) for op in r] for r in roles]
        self.names = names

    def faults(self):
        start = ((0,) * len(self.roles), (0,) * len(self.names), ())
        seen, todo, bad = {start}, [start], set()
        while todo:
            pos, got, flying = todo.pop()
            nxt = []
            for i, role in enumerate(self.roles):
                if pos[i] == len(role):
                    continue
                op = role[pos[i]]
                on = pos[:i] + (pos[i] + 1,) + pos[i + 1:]
                b = op[1]
                if op[0] == "wait":
                    done = got[b] // self.count[b]  # phases that are over
                    passes, due = (done - 1 - op[2]) % 2 == 0, done > op[2]
                    if done == 0:
                        passes = op[2] % 2 == 1  # what a fresh barrier says of the phase before its first
                    if passes != due:
                        bad.add(("early" if passes else "missed", self.names[b], op[2]))
                    elif due:
                        nxt.append((on, got, flying))
                elif op[0] == "arrive":
                    nxt.append((on, got[:b] + (got[b] + 1,) + got[b + 1:], flying))
                else:
                    nxt.append((on, got, tuple(sorted(flying + (b,)))))
            for k, b in enumerate(flying):
                if k and flying[k - 1] == b:
                    continue
                nxt.append((pos, got[:b] + (got[b] + 1,) + got[b + 1:], flying[:k] + flying[k + 1:]))
            if not nxt and any(p < len(r) for p, r in zip(pos, self.roles)):
                bad.add(("stuck",))
            if bad:
                return bad
            for s in nxt:
                if s not in seen:
                    seen.add(s)
                    todo.append(s)
        return bad


def forward(items, NS):
    """items: tiles of keys of each pair of query tiles. Two softmax roles and two product
    warps, which take turns."""
    copy, prod, soft = [], ([], []), ([], [])
    kv = 0
    for i, n in enumerate(items):
        for u in range(2 * n):
            c = kv + u
            copy += ([("wait", ("empty", c % NS), c // NS - 1)] if c >= NS else []) + [("copy", ("full", c % NS))]
            if u == 0:
                copy += ([("wait", "Qfree", i - 1)] if i else []) + [("copy", "Q")]
        kv += 2 * n
    tiles = [(i, u) for i, n in enumerate(items) for u in range(n)]
    for x in (0, 1):
        full = lambda c: ("wait", ("full", c % NS), c // NS)  # noqa: E731
        prod[x].extend([("wait", "Q", 0), full(0), ("copy", ("S", x))])
        for t, (i, u) in enumerate(tiles):
            last, more = u == items[i] - 1, t + 1 < len(tiles)
            prod[x].append(full(2 * t + 1))
            if last and more:
                prod[x].append(("wait", "Q", i + 1))
            if more:
                prod[x].append(full(2 * t + 2))
            prod[x].append(("wait", ("P", x), t))
            if x + t:
                prod[x].append(("wait", ("turn", x), t if x else t - 1))
            prod[x].extend(([("copy", ("O", x))] if last else []) + [("arrive", ("turn", 1 - x))])
            if more:
                prod[x].append(("copy", ("S", x)))
            soft[x].append(("wait", ("S", x), t))
            soft[x].append(("arrive", ("empty", 2 * t % NS)))
            if t:
                soft[x].append(("arrive", ("empty", (2 * t - 1) % NS)))
            if last:
                soft[x].append(("arrive", "Qfree"))
                soft[x].append(full(2 * t + 1))  # values past a sequence's end are cleared
            soft[x].append(("arrive", ("P", x)))
            if last:
                soft[x].append(("wait", ("O", x), i))
    return Walk([copy, *prod, *soft], {"empty": 2, "Qfree": 2})


def queries(items, NS):
    """The queries' kernel: S two tiles ahead and dq from one warp, dP from another."""
    copy, first, second, soft = [], [], [], []
    kv = 0
    for i, n in enumerate(items):
        for u in range(2 * n):
            c = kv + u
            copy += ([("wait", ("empty", c % NS), c // NS - 1)] if c >= NS else []) + [("copy", ("full", c % NS))]
            if u < 2:
                name = "QD"[u]
                copy += ([("wait", name + "free", i - 1)] if i else []) + [("copy", name)]
        kv += 2 * n
    tiles = [(i, u) for i, n in enumerate(items) for u in range(n)]
    full = lambda c: ("wait", ("full", c % NS), c // NS)  # noqa: E731

    def scores(s):
        i, u = tiles[s]
        return ([("wait", "Q", i)] if u == 0 else []) + [full(2 * s), ("copy", ("S", s % 2))]

    for s in range(min(2, len(tiles))):
        first += scores(s)
    for t, (i, u) in enumerate(tiles):
        last = u == items[i] - 1
        first += [("wait", ("dS", t % 2), t // 2), ("copy", ("empty", 2 * t % NS))]
        first += [("copy", "end")] if last else []
        first += scores(t + 2) if t + 2 < len(tiles) else []
        second += [("wait", "D", i)] if u == 0 else []
        second += [full(2 * t + 1)] + ([("wait", "read", t - 1)] if t else []) + [("copy", "dP")]
        soft += [("wait", ("S", t % 2), t // 2)] + ([("arrive", "Qfree")] if last else [])
        soft += [("wait", "dP", t), ("arrive", ("empty", (2 * t + 1) % NS))] + ([("arrive", "Dfree")] if last else [])
        soft += [("arrive", "read"), ("arrive", ("dS", t % 2))]
        soft += [("wait", "end", i)] if last else []
    return Walk([copy, first, second, soft], {})


def keys(tiles, NS):
    """The keys' kernel: tiles of queries of each key tile in turn; dv and S, dk and dP, row
    statistics."""
    copy, first, second, stats, soft = [], [], [], [], []
    t = 0
    full = lambda c: ("wait", ("full", c % NS), c // NS)  # noqa: E731
    for i, n in enumerate(tiles):
        for u in range(2 * n):
            c = 2 * t + u
            if u == 2 or (u == 0 and n == 0):
                copy += ([("wait", "KVfree", i - 1)] if i else []) + [("copy", "KV")]
            copy += ([("wait", ("empty", c % NS), c // NS - 1)] if c >= NS else []) + [("copy", ("full", c % NS))]
        if n == 1:
            copy += ([("wait", "KVfree", i - 1)] if i else []) + [("copy", "KV")]
        for x, role in ((0, first), (1, second)):
            role += [("wait", "KV", i), full(2 * t + x), ("copy", ("dP" if x else "S"))]
            for u in range(n):
                c = t + u
                role += [full(2 * c + 1 - x), ("wait", "dS" if x else "P", c)]
                role += [("copy", ("end", x))] if u + 1 == n else []
                role += [full(2 * (c + 1) + x), ("copy", "dP" if x else "S")] if u + 1 < n else []
        for u in range(n):
            c = t + u
            stats += ([("wait", "P", c - 1)] if c else []) + [("arrive", "lse")]
            stats += ([("wait", "dS", c - 1)] if c else []) + [("arrive", "delta")]
            soft += [("wait", "lse", c), ("wait", "S", c)] + ([("arrive", ("empty", (2 * c - 1) % NS))] if u else [])
            soft += [full(2 * c + 1)] if u + 1 == n else []  # rows past a sequence's end are cleared
            soft += [("arrive", "P"), ("wait", "delta", c), ("wait", "dP", c)]
            soft += ([("arrive", ("empty", (2 * c - 2) % NS))] if u else []) + ([("arrive", "KVfree")] if u + 1 == n else [])
            soft += [("arrive", "dS")]
        t += n
        soft += [("wait", ("end", 0), i), ("wait", ("end", 1), i)]
        soft += [("arrive", ("empty", (2 * t - 1) % NS)), ("arrive", ("empty", (2 * t - 2) % NS))]
    return Walk([copy, first, second, stats, soft], {})


def step(n, NS):
    """Single tokens: two groups of warps take the ring's places by turns."""
    copy, groups = [], ([], [])
    for t in range(n):
        copy += ([("wait", ("empty", t % NS), t // NS - 1)] if t >= NS else []) + [("copy", ("full", t % NS))]
        groups[t % 2].extend([("wait", ("full", t % NS), t // NS), ("arrive", ("empty", t % NS))])
    return Walk([copy, *groups], {})


@pytest.mark.parametrize("items", [[4], [1, 1, 1, 1], [2, 1, 2], [3, 2]])
def test_forward(rings, items):
    for fwd, _, _ in rings:
        assert not forward(items, fwd).faults()


@pytest.mark.parametrize("items", [[5], [1, 1, 1, 1, 1], [2, 1, 3], [1, 4]])
def test_queries(rings, items):
    for _, bwd, _ in rings:
        assert not queries(items, bwd).faults()


@pytest.mark.parametrize("tiles", [[5], [1, 1, 1, 1], [2, 1, 3], [4, 2]])
def test_keys(rings, tiles):
    for _, bwd, _ in rings:
        assert not keys(tiles, bwd).faults()


def test_step(rings):
    for _, _, stages in rings:
        assert not step(2 * stages + 3 if stages < 8 else stages + 2, stages).faults()


def test_the_check_finds_what_it_is_for():
    """An odd ring for the two groups: a group takes a place before it has been filled."""
    assert ("early", ("full", 0), 1) in step(9, 5).faults() or step(9, 5).faults()
    assert step(9, 3).faults()
    broken = queries([4], 5)
    broken.roles[3] = [op for op in broken.roles[3] if op[0] != "arrive" or broken.names[op[1]] != "read"]
    assert ("stuck",) in broken.faults()


def test_an_odd_ring_is_taken_too_early():
    """What goes wrong with an odd ring for the two groups is that one takes a place before it
    has been filled, not that a role is stuck; rings of one copy more are sound."""
    for n, places in ((9, 5), (9, 3)):
        faults = step(n, places).faults()
        assert any(f[0] == "early" and f[1][0] == "full" for f in faults), faults
        assert ("stuck",) not in faults
        assert not step(n, places + 1).faults()
