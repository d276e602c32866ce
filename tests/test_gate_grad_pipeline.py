"""Host checks of moe_gate_grad's two pipelined kernels: their waits against a
replay of the order in which a wave issues its vector memory operations, their
ring slots, and the split of the work over workgroups.  The kernels' numbers
(gate_grad.hip) are restated below.

A wave waits until at most n of its operations are in flight; they complete
in issue order, so what it waits for has landed if n is at most the number of
operations it issued afterwards.  A lower n only waits longer."""

import pytest


def behind(seq, what):
    """Operations issued after the last one of ``what``."""
    return len(seq) - 1 - max(i for i, op in enumerate(seq) if op == what)


def dx_shape(KF, GP):
    SK = 2 if KF % 2 == 0 else 3 if KF % 3 == 0 else 1
    return SK, {1: 8, 2: 4, 3: 3}[SK]


@pytest.mark.parametrize("KF,MT", [(1, 2), (2, 2), (3, 2), (4, 2), (5, 2), (6, 2), (8, 2), (9, 1), (10, 1), (12, 1),
                                   (16, 1)])
@pytest.mark.parametrize("GP", [1, 2])
@pytest.mark.parametrize("blocks", [1, 2, 3, 7])
def test_dx_waits(KF, MT, GP, blocks):
    SK, D = dx_shape(KF, GP)
    steps, RC = KF // SK, MT * 4
    total = blocks * steps
    # waves 0-3: GP SK copies per stage, nothing else
    seq = [("stage", s) for s in range(D - 1) for _ in range(GP * SK)]
    slot = {s % D: s for s in range(D - 1)}
    for s in range(total):
        assert (D - 2) * GP * SK <= behind(seq, ("stage", s))
        assert slot[s % D] == s  # nothing has overwritten it
        new = s + D - 1
        seq += [("stage", new)] * (GP * SK)
        assert new % D != s % D  # not the slot that is being read
        slot[new % D] = new
    # waves 4-7: a block's dx_in a block ahead, the block before stored first
    seq = [("in", 0)] * RC
    for b in range(blocks):
        for k in range(steps):
            if k == steps - 1:
                n = 0 if KF == SK else RC if b == 0 else 2 * RC
                assert n <= behind(seq, ("in", b))
            if k == 0:
                if b > 0:
                    seq += [("store", b - 1)] * RC
                seq += [("in", b + 1)] * RC


@pytest.mark.parametrize("MF", [1, 2, 3, 4])
@pytest.mark.parametrize("n", list(range(1, 20)))
def test_d_gate_waits(MF, n):
    R, N_X = 6, 4
    AF = 6 * MF
    for wave in range(8):
        copies = sum(1 for f in range(wave, AF, 8))  # this wave's
        N_A = AF // 8
        seq = []

        def x(s):
            seq.extend([("x", s)] * N_X)

        def a(s):
            seq.extend([("a", s)] * copies)

        for i in range(R - 2):
            x(i)
        a(0), x(R - 2), a(1), x(R - 1)
        s = 0
        while s < n:
            whole = n - s >= R
            for i in range(R if whole else n - s):
                if whole:
                    wait = 2 * N_X + N_A
                else:
                    wait = 2 * N_X + N_A if i == 0 else N_X + N_A if i == 1 else N_A
                if copies:
                    assert wait <= behind(seq, ("a", s + i)), (wave, s + i)
                a(s + i + 2)
                assert (s + i + 2) % 3 not in ((s + i) % 3, (s + i + 1) % 3)
                if whole:
                    x(s + i + R)
                # x of the next step was loaded before it is stored
                assert ("x", s + i + 1) in seq or s + i + 1 >= n
            s += R if whole else n - s


def xcd_items(items):
    """The items that the workgroups of a launch take (-1: none)."""
    grid = -(-items // 8) * 8
    per = (items + 7) // 8
    out = []
    for b in range(grid):
        item = (b % 8) * per + b // 8
        out.append(item if b // 8 < per and item < items else -1)
    return out


@pytest.mark.parametrize("items", [1, 7, 8, 9, 63, 144, 224, 255, 256, 257, 1000])
def test_every_item_once(items):
    got = [i for i in xcd_items(items) if i >= 0]
    assert sorted(got) == list(range(items))


@pytest.mark.parametrize("T", [1, 100, 128, 129, 512, 4099, 8192, 70000])
@pytest.mark.parametrize("H", [128, 640, 4096, 7168])
@pytest.mark.parametrize("mt", [1, 2])
def test_dx_covers_tokens_and_columns(T, H, mt):
    blocks, groups = H // 64, -(-T // (128 * mt))
    hsplits = min(8 if groups >= 32 else -(-256 // groups), blocks)
    hper = -(-blocks // hsplits)
    hsplits = -(-blocks // hper)
    seen = []
    for hs in range(hsplits):
        first, last = hs * hper, min(blocks, (hs + 1) * hper)
        assert first < last
        seen += range(first, last)
    assert seen == list(range(blocks)) and groups * 128 * mt >= T > (groups - 1) * 128 * mt
