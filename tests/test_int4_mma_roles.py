"""The roles of the 4-bit tensor-core kernel (copies, converting groups, MMAs)
walked on the CPU: every wait as the hardware does it, by the parity of a
barrier's phase, with random copy, conversion and MMA times.  The ring and
group numbers come from the kernel's own header, for every token tile.

A barrier knows only whether the phase of a given parity has ended, so a warp
that is two phases ahead of it is let through.  The walk keeps what each ring
slot and each converted block really holds, and reports every read of a block
that is not there and every overwriting of one that is still needed."""

import heapq
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "quantized_linear_gemm_b200", "csrc")
TILES = (16, 32, 64, 128, 256)


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """{tokens per tile: (ring slots, converting groups, converted blocks)} of int4_mma_shape.h."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("shape")
    src, exe = str(d / "shape.cpp"), str(d / "shape")
    with open(src, "w") as f:
        f.write('#include <cstdio>\n#include "int4_mma_shape.h"\n'
                'template <int NT> void show() { using S = lq::MmaShape<NT>;\n'
                '  std::printf("%d %d %d %d\\n", NT, S::kRing, S::kGroups, S::kA); }\nint main() {\n' +
                "".join(f"  show<{t}>();\n" for t in TILES) + "}\n")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", exe, src], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    return {r[0]: r[1:] for r in rows}


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passed(self, parity):
        """What try_wait.parity says: the phase in progress has the other parity."""
        return (self.done & 1) != parity


def walk(ring, groups, blocks_a, n, rng, slow):
    """One CTA over n blocks; returns what went wrong, as texts."""
    wrong = []
    full = [Barrier(1) for _ in range(ring)]
    empty = [Barrier(5) for _ in range(ring)]
    a_full = [Barrier(4) for _ in range(blocks_a)]
    a_empty = [Barrier(1) for _ in range(blocks_a)]
    holds = [None] * ring                     # the block whose copies have landed in a slot
    owes = [0] * ring                         # warps (and the MMAs) that still need the slot's block
    converted = [[None] * 4 for _ in range(blocks_a)]
    busy_a = [None] * blocks_a                # the block whose MMAs may be reading a converted block
    later = []                                # (time, order, effect)
    order = iter(range(1 << 30))

    def at(t, effect):
        heapq.heappush(later, (t, next(order), effect))

    now = [0.0]

    def loader():
        for j in range(n):
            s = j % ring
            yield lambda: empty[s].passed(((j // ring) & 1) ^ 1)
            if owes[s]:
                wrong.append(f"slot {s} overwritten by block {j} with {owes[s]} readers left")
            holds[s], owes[s] = None, 5

            def landed(s=s, j=j):
                holds[s] = j
                full[s].arrive()
            at(now[0] + rng.uniform(400, slow), landed)
            yield rng.uniform(5, 40)

    def converter(group, warp):
        for j in range(group, n, groups):
            s, b = j % ring, j % blocks_a
            yield lambda: full[s].passed((j // ring) & 1)
            if holds[s] != j:
                wrong.append(f"group {group} reads block {j} from slot {s}, which holds {holds[s]}")
            yield rng.uniform(20, 60)
            yield lambda: a_empty[b].passed(((j // blocks_a) & 1) ^ 1)
            if busy_a[b] is not None:
                wrong.append(f"converted block {b} overwritten by {j} under the MMAs of {busy_a[b]}")
            yield rng.uniform(100, 300)
            owes[s] -= 1
            empty[s].arrive()
            yield rng.uniform(5, 40)
            converted[b][warp] = j
            a_full[b].arrive()

    def mma():
        last = 0.0
        for j in range(n):
            s, b = j % ring, j % blocks_a
            yield lambda: a_full[b].passed((j // blocks_a) & 1)
            if any(c != j for c in converted[b]):
                wrong.append(f"MMAs of block {j} find {converted[b]} converted")
            if holds[s] != j:
                wrong.append(f"MMAs of block {j} find slot {s} holding {holds[s]}")
            busy_a[b] = j
            last = max(last, now[0]) + rng.uniform(60, 250)   # MMAs end in the order of their issue

            def ended(s=s, b=b):
                busy_a[b] = None
                a_empty[b].arrive()
                owes[s] -= 1
                empty[s].arrive()
            at(last, ended)
            yield rng.uniform(5, 30)

    roles = [loader(), mma()] + [converter(g, w) for g in range(groups) for w in range(4)]
    waiting = []

    def step(role):
        want = next(role, None)
        if want is None:
            return
        if callable(want):
            waiting.append((role, want))
        else:
            at(now[0] + want, role)

    for r in roles:
        step(r)
    while True:
        ready = [w for w in waiting if w[1]()]
        if ready:
            pick = rng.choice(ready)
            waiting.remove(pick)
            step(pick[0])
            continue
        if not later:
            break
        now[0], _, what = heapq.heappop(later)
        what() if callable(what) else step(what)
    if waiting:
        wrong.append(f"{len(waiting)} roles wait for ever")
    return wrong


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("slow", [500, 1200, 2500, 8000])
def test_no_block_is_read_before_it_arrives(shapes, tile, slow):
    ring, groups, blocks_a = shapes[tile]
    for seed in range(12):
        wrong = walk(ring, groups, blocks_a, 60, random.Random(seed), slow)
        assert not wrong, (tile, ring, groups, blocks_a, seed, wrong[:3])


@pytest.mark.parametrize("tile", TILES)
def test_phases_are_told_apart(shapes, tile):
    """The condition itself: the block that a wait must not be let through for has been seen to arrive."""
    ring, groups, blocks_a = shapes[tile]
    assert ring % groups == 0 or groups + blocks_a <= ring
    assert groups <= blocks_a and ring >= 2


@pytest.mark.parametrize("ring,groups,blocks_a", [(5, 2, 4), (3, 2, 2)])
def test_the_walk_finds_an_odd_ring(ring, groups, blocks_a):
    """Two groups that take turns at each slot of an odd ring: late copies are read before they land."""
    found = [walk(ring, groups, blocks_a, 60, random.Random(seed), 2500) for seed in range(12)]
    assert any("reads block" in w for f in found for w in f)
