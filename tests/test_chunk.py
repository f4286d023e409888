"""CPU tests of the attention of new tokens: the workspace, every refusal, none of which reaches a kernel, and the
division of its work."""

import random

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd


def test_workspace():
    n = pd.pd_chunk_workspace_bytes
    assert n(0, 8, 2, 128) == 0 and n(4, 8, 3, 128) == 0 and n(4, 1, 2, 128) == 0 and n(4, 8, 2, 0) == 0 and n(4, 8, 2, 257) == 0
    # two slots for each CTA: a block of 256 rows, or of what the call has, of (m, l) and o
    for T, rows in ((1, 32), (9, 64), (64, 256), (100000, 256)):
        least = 2 * 152 * rows * (128 + 2) * 4
        assert least <= n(T, 32, 8, 128) <= least + 152 * 32 + 3 * 256
    assert n(1000, 16, 2, 256) == n(128, 16, 2, 256) < n(1000, 16, 2, 255) + 1


def _restated(starts, lens, Hq, Hkv, D, window):
    """Every (row of q, query head) and the key tiles that its item has to take, from the definition alone."""
    tile = 64 if D > 128 else 128
    need = {}
    for s, n in enumerate(lens):
        a, b = (s, s + 1) if starts is None else (starts[s], starts[s + 1])
        for t in range(a, b):
            p = n - (b - t)
            low = max(0, p + 1 - window) if window else 0
            need[t] = (s, set(range(low // tile, p // tile + 1)) if p >= 0 else set())
    return tile, need


def _check_walk(starts, lens, Hq, Hkv, D, window, ctas):
    segs, (units, C, block, tile, item_heads, box) = pd.pd_debug_chunk_walk(starts, lens, Hq, Hkv, D, window, ctas)
    restated, need = _restated(starts, lens, Hq, Hkv, D, window)
    G = Hq // Hkv
    assert tile == restated and block * item_heads <= (128 if D > 128 else 256) and block % box == 0 and box * item_heads <= max(32, item_heads)
    assert C <= ctas and (C == ctas or units <= 5 * ctas)
    items = {}
    for cta, seq, kvh, head, heads, row, rows, tile0, n, part, last in segs:
        assert head // G == kvh == (head + heads - 1) // G and heads <= item_heads and 0 < rows <= block and 0 <= cta <= last < C
        items.setdefault((head, row), []).append((cta, seq, heads, rows, tile0, n, part, last))
    taken = {}
    for (head, row), parts in items.items():
        ctas_of = [p[0] for p in parts]
        assert len({(p[1], p[2], p[3], p[7]) for p in parts}) == 1
        assert ctas_of == list(range(ctas_of[0], ctas_of[0] + len(parts))) 
        assert parts[0][6] == 2 or ctas_of[-1] == parts[0][7]  # what the fold goes by
        assert [p[6] for p in parts] == ([2] if len(parts) == 1 else [1] + [0] * (len(parts) - 1))
        at = parts[0][4]
        for p in parts:
            assert p[4] == at
            at += p[5]
            assert p[5] > 0 or (len(parts) == 1 and p[6] == 2)
        tiles = set(range(parts[0][4], at))
        _, seq, heads, rows = parts[0][:4]
        union = set()
        for t in range(row, row + rows):
            assert need[t][0] == seq
            union |= need[t][1]
            for h in range(head, head + heads):
                assert (t, h) not in taken
                taken[t, h] = True
        assert tiles == (set(range(min(union), max(union) + 1)) if union else set())
    assert len(taken) == len(need) * Hq
    # a CTA begins inside an item at most once and ends inside one at most once: its two slots
    for c in range(C):
        mine = [s for s in segs if s[0] == c]
        assert sum(s[9] == 0 for s in mine) <= 1 and sum(s[9] == 1 for s in mine) <= 1
    if C > 1:  # the shares: tiles and two units an item
        cost = [sum(s[8] for s in segs if s[0] == c) for c in range(C)]
        assert max(cost) <= units // C + 1


def test_walk_of_batches():
    for window in (0, 1, 70, 128, 1000):
        _check_walk(None, [0, 1, 16, 500, 4000, 0], 8, 2, 128, window, 152)
        _check_walk([0, 300], [300], 4, 1, 64, window, 152)
        _check_walk([3, 3, 260, 261, 261, 500], [9, 300, 1, 77, 2000], 8, 2, 128, window, 7)
        _check_walk([0, 40, 60], [10, 20], 8, 2, 256, window, 152)  # more new tokens than the sequence has
        _check_walk([0, 700], [701], 6, 2, 80, window, 152)
        _check_walk([0, 9, 12], [3000, 5], 300, 1, 64, window, 50)  # more query heads than an item's rows
        _check_walk([0, 9, 12], [3000, 5], 129, 1, 256, window, 1)
    segs, totals = pd.pd_debug_chunk_walk([0], [], 8, 2, 128)
    assert segs == [] and totals[:2] == (0, 0)


def test_walk_of_random_batches():
    rng = random.Random(5)
    for _ in range(300):
        S = rng.choice([1, 2, 3, 10])
        Hkv, G, D = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 100]), rng.choice([64, 128, 256])
        new = [rng.choice([0, 1, rng.randint(0, 9), rng.randint(0, 600)]) for _ in range(S)]
        lens = [max(0, n + rng.choice([0, rng.randint(0, 300), rng.randint(0, 5000), -rng.randint(0, 30)])) for n in new]
        starts = [rng.randint(0, 3)]
        for n in new:
            starts.append(starts[-1] + n)
        _check_walk(starts, lens, Hkv * G, Hkv, D, rng.choice([0, 0, rng.randint(1, 3000)]), rng.choice([1, 2, 13, 152]))


def test_walk_of_a_long_prompt():
    """Shares of hundreds of thousands of units, whose borders are found without a walk."""
    T = 131072
    segs, (units, C, block, tile, _, _) = pd.pd_debug_chunk_walk([0, T], [T + 70000], 64, 8, 128)
    assert units == 8 * sum(2 + -(-(70000 + t + block) // tile) for t in range(0, T, block)) and C == 152
    assert sum(s[8] for s in segs) == units - 2 * 8 * T // block
    shares = [sum(s[8] + 2 for s in segs if s[0] == c) for c in range(C)]
    assert max(shares) - min(shares) <= 5


def test_walk_refusals():
    for args in (([0, 5, 3], [9, 9], 8, 2, 128), ([0, 2], [-1], 8, 2, 128), ([0, 2], [9], 8, 3, 128), ([0, 2], [9], 8, 2, 12),
                 ([0, 2], [9], 8, 2, 128, -1), ([0, 2], [9], 8, 2, 128, 0, 0), ([0, 2], [9], 8, 2, 128, 0, 153)):
        with pytest.raises(pd.PdError):
            pd.pd_debug_chunk_walk(*args)
