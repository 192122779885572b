"""The rings of the tcgen05 kernel on 4-bit weights, on the CPU: stage counts from
the source, the order of waits and arrivals of its roles restated here.

An mbarrier wait names a parity, so a wait for phase p of a slot also passes while
phase p - 2 is the last one that completed.  A role that waits for some of a slot's
phases only (a set of decoding warps takes every SETS-th step) must therefore know
that the phase before the one that it waits for is complete.
"""
import random
import re
from pathlib import Path

import pytest

SOURCE = Path(__file__).resolve().parents[1] / "qwen3_transformer_forward_gb300" / "csrc" / "w4_gemm_tc.cu"


def constants(narrow):
    text = re.sub(r"//[^\n]*", "", SOURCE.read_text())
    tile = text[text.index("struct Tile {"):text.index("constexpr uint32_t kTmemCols")]

    def get(name):
        a, b, c = re.search(r"\b%s = (?:NARROW \? (\d+) : (\d+)|(\d+))" % name, tile).groups()
        return int(c if c is not None else a if narrow else b)
    return {n: get(n) for n in ("XS", "CS", "AS", "SETS")}


def walk(steps, shards, parts, part, tiles):
    """The steps of a pair that has `part` of `parts` of K in each of its tiles, as the copying warps count them:
    (place in the shard, end of the shard, number of its code stage); two steps a stage, the last of a shard may be alone."""
    stages = (steps + 1) // 2
    c0, c1 = shards * stages * part // parts, shards * stages * (part + 1) // parts
    out, number = [], 0
    for _ in range(tiles):
        for c in range(c0, c1):
            k = 2 * (c % stages)
            end = min(2 * ((c1 - 1) % stages) + 2, steps) if c // stages == (c1 - 1) // stages else steps
            out += [(i, end, number) for i in range(k, min(k + 2, end))]
            number += 1
    return out


def shapes():
    for steps in list(range(1, 14)) + [40]:
        for shards in (1, 2, 3, 5, 8):
            for parts in (1, 2, 3, 4):
                if parts > shards * ((steps + 1) // 2):
                    continue
                for part in range(parts):
                    one = len(walk(steps, shards, parts, part, 1))
                    yield steps, shards, parts, part, 1 if parts > 1 else -(-60 // one)   # parts: one tile each


@pytest.mark.parametrize("narrow", [False, True])
def test_no_set_waits_two_phases_ahead(narrow):
    """Before a set waits for the codes of step n, the copy before that one in the slot is known to have landed: the
    set took a step of it, or its last wait for a TMEM slot saw the MMAs of all steps up to n - SETS - AS, whose
    codes were decoded."""
    c = constants(narrow)
    for shape in shapes():
        w = walk(*shape)
        full = [set() for _ in range(c["SETS"])]     # stages that each set took a step of
        for n, (_, _, cs) in enumerate(w):
            own = full[n % c["SETS"]]
            seen = n - c["SETS"] - c["AS"]
            before = cs - c["CS"]
            assert before < 0 or before in own or (seen >= 0 and w[seen][2] >= before), (c, shape, n, cs)
            own.add(cs)


class Bar:
    """An mbarrier: phase parity and the arrivals that its phase still needs."""
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0, "more arrivals than a phase has"
        if self.left == 0:
            self.phase ^= 1
            self.left = self.count

    def passed(self, parity):
        return self.phase != parity


def simulate(narrow, shape, seed):
    """One pair of CTAs, its roles in a random order, copies landing in any order."""
    c = constants(narrow)
    XS, CS, AS, SETS = (c[n] for n in ("XS", "CS", "AS", "SETS"))
    rng = random.Random(seed)
    w = walk(*shape)
    ranks = (0, 1)
    xf, af = [Bar(2) for _ in range(XS)], [Bar(8) for _ in range(AS)]
    xe, cf, ce, ae = ([[Bar(n) for _ in range(s)] for _ in ranks] for s, n in ((XS, 1), (CS, 1), (CS, 8), (AS, 1)))
    codes = [[None] * CS for _ in ranks]      # the stage whose codes lie in a slot; None: on their way
    weights = [[None] * AS for _ in ranks]    # the step whose weights lie in a slot
    copies, mmas, state = [], [], {"done": False}

    def tokens(r):
        for n in range(len(w)):
            while not xe[r][n % XS].passed(((n // XS) & 1) ^ 1):
                yield False
            copies.append(lambda b=xf[n % XS]: b.arrive())
            yield True

    def code_copies(r):
        def land(cs):
            codes[r][cs % CS] = cs
            cf[r][cs % CS].arrive()
        for cs in range(w[-1][2] + 1):
            while not ce[r][cs % CS].passed(((cs // CS) & 1) ^ 1):
                yield False
            codes[r][cs % CS] = None
            copies.append(lambda cs=cs: land(cs))
            yield True

    def memory():
        while True:
            if copies:
                copies.pop(rng.randrange(len(copies)))()
            yield bool(copies)

    def decode(r, first):
        for n in range(first, len(w), SETS):
            k, end, cs = w[n]
            slot, a = cs % CS, n % AS
            while not cf[r][slot].passed((cs // CS) & 1):
                yield False
            assert codes[r][slot] == cs, "decodes other codes than its step's"
            yield True
            assert codes[r][slot] == cs, "codes overwritten while they are read"
            ce[r][slot].arrive(8 if k == end - 1 and k % 2 == 0 else 4)   # four warps, one arrival or two each
            while not ae[r][a].passed(((n // AS) & 1) ^ 1):
                yield False
            weights[r][a] = n
            yield True
            af[a].arrive(4)

    def issue():
        for n in range(len(w)):
            while not (xf[n % XS].passed((n // XS) & 1) and af[n % AS].passed((n // AS) & 1)):
                yield False
            mmas.append(n)
            yield True

    def tensor():
        for n in range(len(w)):
            while not mmas:
                yield False
            for _ in range(2):
                assert all(weights[r][n % AS] == n for r in ranks), "multiplies other weights than its step's"
                yield True
            mmas.pop(0)
            for r in ranks:
                ae[r][n % AS].arrive()
                xe[r][n % XS].arrive()
        state["done"] = True

    roles = [issue(), tensor(), memory()]
    for r in ranks:
        roles += [tokens(r), code_copies(r)] + [decode(r, s) for s in range(SETS)]
    speed = [rng.random() + 0.02 for _ in roles]
    idle = 0
    while not state["done"]:
        i = rng.choices(range(len(roles)), speed)[0]
        try:
            idle = 0 if next(roles[i]) else idle + 1
        except StopIteration:
            del roles[i], speed[i]
        assert idle < 20000, "no role can go on"


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("shape", [(1, 8, 1, 0, 4), (1, 5, 1, 0, 4), (1, 1, 1, 0, 20), (1, 7, 2, 1, 1), (2, 4, 1, 0, 4),
                                   (3, 3, 1, 0, 4), (3, 8, 3, 1, 1), (5, 2, 1, 0, 3), (7, 3, 1, 0, 2), (16, 2, 1, 0, 1)])
def test_pipeline_in_any_order(narrow, shape):
    for seed in range(40):
        simulate(narrow, shape, seed)
