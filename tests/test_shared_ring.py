"""The barriers of the wide attention kernel (k_shared_wide), replayed on the
host (no GPU) for the stage counts that its shared memory gives.

A wait on an mbarrier tells phases apart by one bit.  Waiting for phase k is
sound when phase k - 1 is complete before the wait begins (else the bit of
phase k - 2 lets it pass) and phase k + 1 cannot complete before the wait has
ended (else it never ends).  Here every role's instructions are written down in
order; what must happen before what follows from that order, from the barriers'
arrivals, from the tensor unit, which completes products in the order issued,
and from nothing else: a copy may land arbitrarily late.  Every wait of every
role is then checked against that order."""
import os
import shutil
import subprocess
from collections import defaultdict

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "bit_plane_kv_encode_gb300", "csrc")


class Protocol:
    """Events, each with those that come before it; an actor's events are in order."""

    def __init__(self):
        self.before = defaultdict(list)
        self.last = {}
        self.waits = []
        self.arrived = defaultdict(int)  # arrivals of an actor on a barrier so far
        self.products = None             # the tensor unit's last product

    def event(self, actor, *more):
        e = (actor, len(self.before))
        self.before[e] = [*more, *([self.last[actor]] if actor in self.last else [])]
        self.last[actor] = e
        return e

    def phase(self, bar, k):
        return ("phase", bar, k)

    def arrive(self, actor, bar, *more):
        k = self.arrived[actor, bar]
        self.arrived[actor, bar] += 1
        self.before[self.phase(bar, k)].append(self.event(actor, *more))

    def wait(self, actor, bar, k):
        if k < 0:
            return  # the phase before the first: passes at once
        begin = self.event(actor)
        self.before[self.phase(bar, k)]
        end = self.event(actor, self.phase(bar, k))
        self.waits.append((bar, k, begin, end))

    def product(self, actor):
        done = ("product", len(self.before))
        self.before[done] = [self.event(actor), *([self.products] if self.products else [])]
        self.products = done

    def commit(self, actor, bar):
        self.arrive(actor, bar, self.products)

    def faults(self):
        ids, order, past = {}, [], {}
        for root in list(self.before):  # depth first, without recursion
            stack = [(root, False)]
            while stack:
                e, done = stack.pop()
                if done:
                    if e not in past:
                        ids[e] = len(order)
                        order.append(e)
                        past[e] = 1 << ids[e]
                        for b in self.before[e]:
                            assert b in past, "events in a circle"
                            past[e] |= past[b]
                elif e not in past:
                    stack.append((e, True))
                    stack += [(b, False) for b in self.before.get(e, ())]

        def comes_before(a, b):
            return past[b] >> ids[a] & 1

        out = []
        for bar, k, begin, end in self.waits:
            if k > 0 and not comes_before(self.phase(bar, k - 1), begin):
                out.append(f"{begin[0]} may find {bar} before phase {k - 1}")
            later = self.phase(bar, k + 1)
            if later in past and not comes_before(end, later):
                out.append(f"{begin[0]} may find {bar} past phase {k + 1}")
        return out


def steps_of(seg, s):
    tiles, dual = seg[:2]
    return tiles if dual else (tiles + 1 - s) // 2


def tile_of(seg, s, j):
    return j if seg[1] else 2 * j + s


def replay(bits, n, segments):
    """The kernel's roles over segments (tiles, dual, copies, ragged): ragged when the last tile is not whole."""
    p = Protocol()
    fill = 0
    full = lambda use: (("full", use % n), use // n)  # noqa: E731

    for tiles, *_ in segments:  # loads
        for _ in range(2 * tiles):
            p.wait("load", ("empty", fill % n), fill // n - 1)
            landed = ("landed", fill)
            p.before[landed] = [p.event("load")]
            p.before[p.phase(*full(fill))].append(landed)
            fill += 1

    tile0, step = 0, [0, 0]
    for i_seg, seg in enumerate(segments):  # products
        tiles, dual = seg[:2]
        p.wait("mma", "q_full", i_seg)
        steps = 2 * tiles if dual else tiles
        tile = lambda i: tile0 + (i // 2 if dual else i)  # noqa: E731
        for i in range(steps + 1):
            if i < steps:
                s = i & 1
                if not dual or s == 0:
                    p.wait("mma", *full(2 * tile(i)))
                p.product("mma")
                p.commit("mma", ("s_full", s))
                if not dual or s:
                    p.commit("mma", ("empty", 2 * tile(i) % n))
                if i == steps - 1:
                    p.commit("mma", "q_empty")
            if i > 0:
                j, s = i - 1, (i - 1) & 1
                if not (dual and s):
                    p.wait("mma", *full(2 * tile(j) + 1))
                p.wait("mma", ("p_half", s), step[s])
                p.product("mma")
                p.wait("mma", ("p_ready", s), step[s])
                step[s] += 1
                p.product("mma")
                if not dual or s:
                    p.commit("mma", ("empty", (2 * tile(j) + 1) % n))
                if j + 2 >= steps:
                    p.commit("mma", ("o_done", s))
        tile0 += tiles

    for s in range(2) if bits == 8 else ():  # scales
        me, tile0, go, k = f"scales {s}", 0, 0, 0
        for seg in segments:
            if steps_of(seg, s):
                p.wait(me, ("sc_go", s), go)
                go += 1
            for j in range(steps_of(seg, s)):
                p.wait(me, ("sc_empty", s, k & 1), (k >> 1) - 1)
                p.wait(me, *full(2 * (tile0 + tile_of(seg, s, j)) + 1))
                p.arrive(me, ("sc_full", s, k & 1))
                k += 1
            tile0 += seg[0]

    for s in range(2):  # softmax
        for w in range(4):
            me, tile0, o_done, fin, k = f"softmax {s}.{w}", 0, 0, 0, 0

            def meet():
                nonlocal fin
                p.arrive(me, "fin")
                p.wait(me, "fin", fin)
                fin += 1

            for i_seg, seg in enumerate(segments):
                tiles, dual, copies, ragged = seg
                if i_seg:
                    p.wait(me, "q_empty", i_seg - 1)
                p.arrive(me, "q_full")
                p.wait(me, "q_full", i_seg)
                steps = steps_of(seg, s)
                if bits == 8 and steps:
                    p.arrive(me, ("sc_go", s))
                for j in range(steps):
                    t = tile_of(seg, s, j)
                    p.wait(me, ("s_full", s), k)
                    if bits == 8:
                        p.wait(me, ("sc_full", s, k & 1), k >> 1)
                    if ragged and t == tiles - 1 and (not dual or s == 0):
                        p.wait(me, *full(2 * (tile0 + t) + 1))
                    p.arrive(me, ("p_half", s))
                    p.arrive(me, ("p_ready", s))
                    if bits == 8:
                        p.arrive(me, ("sc_empty", s, k & 1))
                    k += 1
                if steps:
                    p.wait(me, ("o_done", s), o_done)
                    o_done += 1
                if not dual:
                    meet()
                if copies > 1:
                    meet()
                    if copies == 4:
                        meet()
                    meet()
                tile0 += tiles
    return p.faults()


@pytest.fixture(scope="module")
def stages(tmp_path_factory):
    nvcc = next((c for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path_factory.mktemp("ring") / "shared_ring_check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC,
                    os.path.join(HERE, "native", "shared_ring_check.cu"), "-o", exe],
                   check=True, capture_output=True, text=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    return {(int(b), bool(int(d))): int(n) for b, d, n in (x.split() for x in lines if x)}


# segments of a call of at most 128 query rows: (tiles, dual, copies, ragged)
FEW = [
    [(24, False, 1, True)], [(25, False, 2, False)], [(1, False, 4, True)] * 5,
    [(2, False, 1, True), (3, False, 4, True), (17, False, 2, True), (1, False, 1, False), (20, False, 1, False)],
    [(11, False, 4, False), (12, False, 4, True), (13, False, 1, True)],
]
# of more: units of more than 128 rows and others
MANY = FEW + [
    [(24, True, 1, True)], [(1, True, 1, True)] * 5, [(13, True, 1, False), (12, False, 2, True), (7, True, 1, True)],
    [(1, False, 1, True), (2, True, 1, False), (3, False, 4, False), (16, True, 1, True), (16, False, 1, True)],
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("many", [False, True])
def test_no_wait_rests_on_an_unknown_phase(stages, bits, many):
    for segments in MANY if many else FEW:
        assert replay(bits, stages[bits, many], segments) == []


@pytest.mark.parametrize("n,sound", [(7, False), (8, True), (9, True), (10, False), (11, True)])
def test_the_replay_tells_unsound_rings(n, sound):
    """With 10 stages V of tile t takes the place of V of tile t - 5, the other stream's, and with 7 that of K of tile
    t - 3: the scale warp that runs ahead knows of neither."""
    assert (replay(8, n, [(24, False, 1, False)]) == []) == sound
