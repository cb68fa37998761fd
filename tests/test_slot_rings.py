"""The operand ring of the chunk kernel for one query tile, as a model (no GPU).

The halves of a CTA take the even and the odd key tiles.  K_j and V_j pass through slots
2j and 2j + 1 (mod the number of slots), each with a "full" and a "free" barrier; a wait
goes by the parity of a barrier's phase.  The model runs the copies, both halves' MMA warps
and the MMAs' completions in every order that the barriers allow.  A state in which nobody
can go on is a wait that ends by its bound on the GPU, and a half that reads a slot which
holds another tile is a wrong result.
"""
import os
import subprocess

import pytest

import paged_kv_cache_338_b200.build as build


@pytest.fixture(scope="module")
def slot_halves(tmp_path_factory):
    """slot_halves() as the kernels see it, for one query tile, by the number of slots."""
    d = tmp_path_factory.mktemp("ring")
    src, exe = d / "ring.cpp", d / "ring"
    src.write_text('#include "prefill_scored.h"\n#include <cstdio>\nint main() {\n'
                   'for (int n = 1; n < 17; ++n) std::printf("%d %d\\n", ps::slot_halves(n, false),'
                   ' ps::slot_halves(n, true));\n}\n')
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-I",
                    os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out[1::2] == ["2"] * 16               # both halves read every tile of two
    return {n + 1: int(x) for n, x in enumerate(out[::2])}


def explore(slots, halves, tiles, looks=None):
    """All reachable states: the set of faults found ("stuck", "stale").  `halves` arrivals
    free a slot; a half looks at the other's tiles (and, where two arrivals free a slot,
    arrives) if `looks`, which goes with two arrivals."""
    looks = halves == 2 if looks is None else looks
    uses = 2 * tiles
    # A half's steps for the tiles in order, as (what, use): its own tile: wait for K, issue
    # S, wait for V, issue P.V; the other's: look at K, look at V.
    def program(x):
        steps = []
        for j in range(tiles):
            for u in (2 * j, 2 * j + 1):
                if j % 2 == x:
                    steps.append(("read", u))
                elif looks:
                    steps.append(("look", u))
        return steps
    prog = (program(0), program(1))

    # state: copies started, per slot (fills, frees arrived), per half its step and the
    # slots of the MMAs it has issued and that have not completed (they do in order)
    start = (0, tuple((0, 0) for _ in range(slots)), (0, 0), ((), ()))
    seen, todo, faults = {start}, [start], set()
    while todo:
        copied, ring, at, flying = todo.pop()
        nxt = []
        # copies: use u needs the slot's frees of phase u / slots - 1
        if copied < uses:
            s, ph = copied % slots, copied // slots
            fills, frees = ring[s]
            done = frees // halves               # phases of "free" completed
            if (done & 1) != ((ph & 1) ^ 1):     # parity wait; the first round passes at once
                r = list(ring)
                r[s] = (fills + 1, frees)
                nxt.append((copied + 1, tuple(r), at, flying))
        for x in (0, 1):
            if at[x] < len(prog[x]):
                what, u = prog[x][at[x]]
                s, ph = u % slots, u // slots
                fills, frees = ring[s]
                if (fills & 1) != (ph & 1):      # "full" of this parity is over
                    if fills != ph + 1 and (what == "read" or halves == 2):
                        faults.add("stale")      # the slot holds another tile by now (or not yet)
                    r, fl = list(ring), list(flying)
                    if what == "look":
                        r[s] = (fills, frees + halves - 1)
                    else:
                        fl[x] = fl[x] + (s,)
                    nxt.append((copied, tuple(r), at[:x] + (at[x] + 1,) + at[x + 1:], tuple(fl)))
            if flying[x]:                        # the oldest MMA completes: its commit arrives
                s = flying[x][0]
                r, fl = list(ring), list(flying)
                r[s] = (r[s][0], r[s][1] + 1)
                fl[x] = fl[x][1:]
                nxt.append((copied, tuple(r), at, tuple(fl)))
        finished = copied == uses and all(at[x] == len(prog[x]) for x in (0, 1)) and flying == ((), ())
        if not nxt and not finished:
            faults.add("stuck")
        for n in nxt:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return faults


def test_a_half_that_looks_without_a_part_in_freeing_gets_stuck():
    assert explore(3, halves=1, tiles=6, looks=True) == {"stuck"}


@pytest.mark.parametrize("slots", [3, 4, 5, 6, 8])
def test_no_order_of_the_halves_goes_wrong(slots, slot_halves):
    assert explore(slots, slot_halves[slots], 6) == set()
