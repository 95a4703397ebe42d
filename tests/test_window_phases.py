"""The order of the roles in the queries' backward kernel of window attention, on
the CPU: every interleaving of the two product warps and the softmax warps, with
barriers whose waits know a phase by its parity alone, ends. Which barrier and
parity a tile has comes from the kernel's own header."""

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "associative_affine_scan_gb300", "csrc")
MAIN = r"""
#include <cstdio>
#include "scan_window_phases.h"
int main() {
  std::printf("%d\n", scan::kDsBarriers);
  for (int u = 0; u < 16; ++u) std::printf("%d %d\n", scan::ds_barrier(u), scan::ds_parity(u));
}
"""


@pytest.fixture(scope="module")
def phases(tmp_path_factory):
    d = tmp_path_factory.mktemp("phases")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / "main")], check=True)
    rows = subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout.split("\n")
    return int(rows[0]), [tuple(int(x) for x in r.split()) for r in rows[1:17]]


def stuck(n, count, at):
    """How many reachable states of a walk over n key tiles let no role go on."""
    def wait(kind, u):
        if kind == "dS":
            return ("wait", ("dS", at[u][0]), at[u][1])
        return ("wait", ("S", u & 1), (u >> 1) & 1) if kind == "S" else ("wait", ("dP", 0), u & 1)

    def done(kind, u):
        return ("arrive", ("dS", at[u][0]) if kind == "dS" else ("S", u & 1) if kind == "S" else ("dP", 0))

    first = [done("S", u) for u in range(min(n, 2))]  # issues S, two tiles ahead, and dq += dS k
    for u in range(n):
        first += [wait("dS", u)] + ([done("S", u + 2)] if u + 2 < n else [])
    second = []                                       # issues dP
    for u in range(n):
        second += ([wait("dS", u - 1)] if u else []) + [done("dP", u)]
    softmax = []
    for u in range(n):
        softmax += [wait("S", u), wait("dP", u), done("dS", u)]
    roles = [first, second, softmax, softmax]
    bars = [("S", 0), ("S", 1), ("dP", 0)] + [("dS", i) for i in range(count)]
    state = ((0,) * 4, ((0, 0),) * len(bars))
    seen, todo, dead = {state}, [state], 0
    while todo:
        at_op, held = todo.pop()
        moved = False
        for i, role in enumerate(roles):
            if at_op[i] == len(role):
                continue
            op, b = role[at_op[i]], bars.index(role[at_op[i]][1])
            phase, arrived = held[b]
            if op[0] == "wait":
                if phase == op[2]:
                    continue
                after = held
            else:
                full = arrived + 1 == (2 if op[1][0] == "dS" else 1)
                after = held[:b] + ((phase ^ 1, 0) if full else (phase, arrived + 1),) + held[b + 1:]
            moved = True
            new = (at_op[:i] + (at_op[i] + 1,) + at_op[i + 1:], after)
            if new not in seen:
                seen.add(new)
                todo.append(new)
        dead += not moved and any(at_op[i] < len(r) for i, r in enumerate(roles))
    return dead


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 13])
def test_every_order_of_the_roles_ends(phases, n):
    count, at = phases
    assert stuck(n, count, at) == 0


def test_one_barrier_would_not_do():
    """The same search finds the walk that stops when all tiles share a barrier."""
    assert stuck(3, 1, [(0, u & 1) for u in range(16)]) > 0
