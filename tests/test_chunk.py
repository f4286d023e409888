"""CPU tests of the attention of new tokens: the workspace, every refusal, none of which reaches a kernel, and the
division of its work."""

import math
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
    share = max(5, -(-units // ctas))
    assert C == -(-units // share) <= ctas
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
    cost = [sum(s[8] for s in segs if s[0] == c) for c in range(C)]  # tiles, beside two units an item
    assert all(c <= share for c in cost)


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
    shares = [sum(s[8] + 2 * (s[9] > 0) for s in segs if s[0] == c) for c in range(C)]
    assert max(shares) - min(shares[:-1]) <= 4 and shares[-1] <= max(shares)  # (two units of an item may be its neighbour's)


def test_walk_refusals():
    for args in (([0, 5, 3], [9, 9], 8, 2, 128), ([0, 2], [-1], 8, 2, 128), ([0, 2], [9], 8, 3, 128), ([0, 2], [9], 8, 2, 12),
                 ([0, 2], [9], 8, 2, 128, -1), ([0, 2], [9], 8, 2, 128, 0, 0), ([0, 2], [9], 8, 2, 128, 0, 153)):
        with pytest.raises(pd.PdError):
            pd.pd_debug_chunk_walk(*args)


def _chunk(**change):
    """pd_chunk_attn[_fp8] on addresses that are never followed: every call here is refused on the host."""
    a = dict(q=4096, q_tok=512, kc=65536, vc=131072, bt=1024, mb=4, cl=2048, ts=512, out=8192, lse=None, T=6, S=2, Hq=4, Hkv=1, D=128, bs=16,
             nb=8, scale=0.1, window=0, ws=1 << 20, ws_bytes=1 << 40, fp8=None)
    a.update(change)
    scales = [] if a["fp8"] is None else list(a["fp8"])
    fn = pd.lib().pd_chunk_attn if a["fp8"] is None else pd.lib().pd_chunk_attn_fp8
    return fn(a["q"], a["q_tok"], a["kc"], a["vc"], *scales, a["bt"], a["mb"], a["cl"], a["ts"], a["out"], a["lse"], a["T"], a["S"], a["Hq"],
              a["Hkv"], a["D"], a["bs"], a["nb"], a["scale"], a["window"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,code", [
    (dict(Hkv=0), pd.PD_ERR_INVALID), (dict(Hq=3, Hkv=2), pd.PD_ERR_INVALID), (dict(D=12), pd.PD_ERR_UNSUPPORTED),
    (dict(D=512), pd.PD_ERR_INVALID), (dict(bs=8), pd.PD_ERR_UNSUPPORTED), (dict(T=-1), pd.PD_ERR_INVALID), (dict(S=-1), pd.PD_ERR_INVALID),
    (dict(ts=None), pd.PD_ERR_INVALID), (dict(window=-1), pd.PD_ERR_INVALID), (dict(q=None), pd.PD_ERR_INVALID),
    (dict(kc=None), pd.PD_ERR_INVALID), (dict(vc=None), pd.PD_ERR_INVALID), (dict(bt=None), pd.PD_ERR_INVALID),
    (dict(cl=None), pd.PD_ERR_INVALID), (dict(out=None), pd.PD_ERR_INVALID), (dict(q=4104), pd.PD_ERR_INVALID),
    (dict(out=8200), pd.PD_ERR_INVALID), (dict(kc=65544), pd.PD_ERR_INVALID), (dict(vc=131080), pd.PD_ERR_INVALID),
    (dict(q_tok=504), pd.PD_ERR_INVALID), (dict(q_tok=516), pd.PD_ERR_INVALID), (dict(q_tok=-512), pd.PD_ERR_INVALID),
    (dict(mb=0), pd.PD_ERR_INVALID), (dict(nb=0), pd.PD_ERR_INVALID), (dict(mb=1 << 27), pd.PD_ERR_INVALID),
    (dict(T=2**31 - 100), pd.PD_ERR_INVALID), (dict(scale=math.nan), pd.PD_ERR_INVALID), (dict(scale=math.inf), pd.PD_ERR_INVALID),
    (dict(fp8=(math.nan, 1.0)), pd.PD_ERR_INVALID), (dict(fp8=(1.0, math.inf)), pd.PD_ERR_INVALID),
    (dict(fp8=(1.0, 1.0), D=24, q_tok=96), pd.PD_ERR_UNSUPPORTED)])
def test_chunk_refused(change, code):
    assert _chunk(**change) == code
    assert pd.last_error()


def test_chunk_of_nothing():
    assert _chunk(T=0) == pd.PD_OK and _chunk(S=0, T=0, ts=None) == pd.PD_OK and _chunk(S=0) == pd.PD_OK
    assert pd.last_error() == ""


def test_api_refuses_tensors():
    """Types, shapes and devices are refused before the library is called (the CPU stands in for the device here)."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(q=bf(6, 4, 64), k_cache=bf(4, 16, 1, 64), v_cache=bf(4, 16, 1, 64), block_table=i32(2, 2), context_lens=i32(2),
                token_starts=i32(3), out=None, lse=None, ws=None, dev=-1)
    api._check_chunk(**good)
    api._check_chunk(**{**good, "out": bf(6, 4, 64), "lse": torch.zeros(6, 4), "ws": torch.zeros(64, dtype=torch.uint8), "token_starts": None})
    for change in (dict(q=bf(6, 64)), dict(q=torch.zeros(6, 4, 64)), dict(q=bf(4, 6, 64).transpose(0, 1)), dict(k_cache=bf(4, 16, 1, 32)),
                   dict(v_cache=bf(5, 16, 1, 64)), dict(block_table=i32(3, 2)), dict(context_lens=i32(2).long()), dict(token_starts=i32(2)),
                   dict(out=bf(6, 4, 32)), dict(out=bf(6, 5, 64)[:, :4]), dict(lse=torch.zeros(6, 5)), dict(lse=torch.zeros(4, 6).T),
                   dict(lse=torch.zeros(6, 4).double()), dict(ws=torch.zeros(64, dtype=torch.uint8)[::2]), dict(dev=0)):
        with pytest.raises(ValueError):
            api._check_chunk(**{**good, **change})


def test_walk_of_a_long_prompt_behind_a_window():
    """2^27 tokens that see 128 keys each: 2^19 blocks of 256, of three tiles but for the first, although their keys before
    the window would make 2^39 units."""
    T, most = 2**27, 2**20
    segments, n, totals = (pd.ctypes.c_int32 * (11 * most))(), pd.ctypes.c_int(), (pd.ctypes.c_int64 * 6)()
    starts, lens = (pd.ctypes.c_int32 * 2)(0, T), (pd.ctypes.c_int32 * 1)(T)
    pd._check(pd.lib().pd_debug_chunk_walk(1, starts, lens, 1, 1, 64, 128, 152, segments, most, pd.ctypes.byref(n), totals))
    assert totals[2] == 256 and totals[3] == 128 and totals[0] == 5 * 2**19 - 1 and totals[1] == 152
    segs = torch.frombuffer(segments, dtype=torch.int32).view(-1, 11)[:n.value].long()
    rows, tile0, tiles = segs[:, 5], segs[:, 7], segs[:, 8]
    first, last = (rows - 127).clamp(min=0) // 128, (rows + 255) // 128
    assert int(tiles.sum()) == 3 * 2**19 - 1 and torch.equal(rows.unique(), torch.arange(0, T, 256))
    whole = segs[:, 9] == 2
    assert torch.equal(tile0[whole], first[whole]) and torch.equal(tiles[whole], (last - first + 1)[whole])
    begun = segs[:, 9] == 1  # a border's item: its first part, and the other ones behind it
    assert int((~whole).sum()) <= 2 * 151 and torch.equal(tile0[begun], first[begun])
