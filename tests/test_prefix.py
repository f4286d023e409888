"""CPU tests of decode attention behind shared prefixes: the workspace and every refusal, none of which reaches a kernel."""

import math
import random

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd


def test_workspace():
    n = pd.pd_prefix_workspace_bytes
    assert n(0, 1, 8, 2, 128, 1) == 0 and n(4, 0, 8, 2, 128, 1) == 0 and n(4, 1, 8, 3, 128, 1) == 0 and n(4, 1, 8, 2, 128, 0) == 0
    # the own partials; one slot for each CTA and each item: a block of 256 rows of (m, l) and o
    rows, items = 64 * 32 * 10, 8 * (1 + 64 * 4 // 256)
    least = rows * (128 + 2) * 4 + (items + 152) * 256 * (128 + 2) * 4
    assert least <= n(64, 1, 32, 8, 128, 10) <= least + 48 * 256 + 6 * 256
    assert n(64, 3, 32, 8, 128, 10) > n(64, 1, 32, 8, 128, 10)


def _walk(G, Hkv, groups, BR, tile, teams, whole):
    """The prefix pass's division of work, restated: every (group, KV head, item, CTA or both, tile) by the CTA that
    takes it, which has to be exactly one, and the slots the merge reads for it."""
    IR = 2 * BR

    def pair(rows):
        return rows > BR

    plan, W, first_item = [], 0, 0
    for seqs, tokens in groups:
        rows = seqs * G
        items, tiles = -(-rows // IR), -(-tokens // tile)
        head = (items - 1) * tiles + (tiles if pair(rows - (items - 1) * IR) else (tiles + 1) // 2)
        units = head * Hkv if items and tiles else 0
        plan.append((W, first_item, tiles, rows, items, head))
        W, first_item = W + units, first_item + (items * Hkv if units else 0)
    C, slots, used, run, base = min(W, teams), {}, {}, 0, [0]

    def places_of(rows, items, tiles, item):
        return tiles if item < items - 1 or pair(rows - (items - 1) * IR) else (tiles + 1) // 2

    def head_teams(tiles, rows, items, run):
        return sum(-(-places_of(rows, items, tiles, i) // run) for i in range(items)) if tiles else 0

    if whole and W:  # whole teams for every item, where they are enough
        for run in range(-(-W // C), 3 * W):
            if sum(Hkv * head_teams(t, r, i, run) for _, _, t, r, i, _ in plan) <= teams:
                break
        else:
            run = 0
    if run:
        ranges = []
        for first_unit, _, tiles, rows, items, head in plan:
            for kvh in range(Hkv if tiles else 0):
                for item in range(items):
                    n, u = places_of(rows, items, tiles, item), first_unit + kvh * head + item * tiles
                    parts = -(-n // run)
                    at = [u + n // parts * k + min(k, n % parts) for k in range(parts + 1)]
                    ranges += list(zip(at, at[1:]))
            base.append(len(ranges))
        C = len(ranges)
        assert C <= teams and all(a < b <= a + run for a, b in ranges)
    else:
        ranges = [(W * c // C, W * (c + 1) // C) for c in range(C)]
    for team, (begin, end) in enumerate(ranges):
        for rank in (0, 1):
            u = begin
            while u < end:
                gi = max(i for i, g in enumerate(plan) if g[0] <= u)
                first_unit, item0, tiles, rows, items, head = plan[gi]
                kvh, rem = divmod(u - first_unit, head)
                item = rem // tiles
                at, r = rem - item * tiles, min(IR, rows - item * IR)
                n = min(end - u, (tiles if pair(r) else (tiles + 1) // 2) - at)
                assert n >= 1 and kvh < Hkv and item < items  # the walk goes on, within the group
                half = (r + 1) // 2
                assert 0 < (r if not pair(r) else r - half if rank else half) <= BR  # rows one CTA can take
                slot = 2 * (item0 + kvh * items + item + team) + rank
                assert used.setdefault(slot, (gi, kvh, item, team, rank)) == (gi, kvh, item, team, rank)
                for t in range(at, at + n) if pair(r) else range(2 * at + rank, min(tiles, 2 * (at + n)), 2):
                    key = (gi, kvh, item, rank if pair(r) else None, t)
                    assert key not in slots
                    slots[key] = slot
                u += n
    assert not used or max(used) < 2 * (first_item + teams)
    for gi, (first_unit, item0, tiles, rows, items, head) in enumerate(plan):
        for kvh in range(Hkv if tiles else 0):
            for item in range(items):
                r = min(IR, rows - item * IR)
                places = tiles if pair(r) else (tiles + 1) // 2
                u = first_unit + kvh * head + item * tiles
                c0, c1 = ((u + 1) * C - 1) // W, ((u + places) * C - 1) // W  # the teams the merge reads
                if run:
                    c0 = base[gi] + kvh * head_teams(tiles, rows, items, run) + item * -(-tiles // run)
                    c1 = c0 + -(-places // run) - 1
                for rank in (0, 1) if pair(r) else (None,):
                    mine = {slots[gi, kvh, item, rank, t] for t in range(tiles)}
                    ranks = (0, 1) if rank is None else (rank,)
                    assert mine <= {2 * (item0 + kvh * items + item + c) + k for c in range(c0, c1 + 1) for k in ranks}
    return first_item


@pytest.mark.parametrize("BR,tile", [(256, 128), (128, 64)])
def test_work_division(BR, tile):
    rng = random.Random(7)
    for _ in range(300):
        G, Hkv = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 2, 8])
        groups = [(rng.choice([0, 1, 2, 5, 20, 32, 40, 64, 100]), rng.choice([0, 1, 17, 64, 100, 128, 129, 700, 3000]))
                  for _ in range(rng.randint(1, 5))]
        items = _walk(G, Hkv, groups, BR, tile, rng.choice([1, 3, 24, 76]), rng.random() < 0.6)
        assert items <= Hkv * (len(groups) + sum(n for n, _ in groups) * G // (2 * BR))  # what the workspace is sized for


def _call(**change):
    """pd_decode_attn_prefix on addresses that are never followed: every call here is refused on the host."""
    a = dict(q=4096, kc=8192, vc=16384, pt=1024, mpb=4, pl=2048, gs=512, G=2, bt=1024, mb=4, cl=2048, out=32768, S=3, Hq=8, Hkv=2,
             D=128, bs=16, nb=8, scale=0.1, N=2, ws=65536, bytes=1 << 40)
    a.update(change)
    return pd.lib().pd_decode_attn_prefix(*(a[k] for k in ("q", "kc", "vc", "pt", "mpb", "pl", "gs", "G", "bt", "mb", "cl", "out",
                                                           "S", "Hq", "Hkv", "D", "bs", "nb", "scale", "N", "ws", "bytes")), None)


@pytest.mark.parametrize("change,code", [
    (dict(Hkv=0), pd.PD_ERR_INVALID), (dict(Hq=9), pd.PD_ERR_INVALID), (dict(D=20), pd.PD_ERR_UNSUPPORTED),
    (dict(D=264), pd.PD_ERR_INVALID), (dict(bs=24), pd.PD_ERR_UNSUPPORTED), (dict(G=0), pd.PD_ERR_INVALID),
    (dict(G=257), pd.PD_ERR_INVALID), (dict(gs=None), pd.PD_ERR_INVALID), (dict(S=-1), pd.PD_ERR_INVALID),
    (dict(N=0), pd.PD_ERR_INVALID), (dict(N=17), pd.PD_ERR_INVALID), (dict(pt=None), pd.PD_ERR_INVALID),
    (dict(pl=None), pd.PD_ERR_INVALID), (dict(mpb=0), pd.PD_ERR_INVALID), (dict(mpb=1 << 27), pd.PD_ERR_INVALID),
    (dict(ws=None), pd.PD_ERR_WORKSPACE), (dict(bytes=1 << 10), pd.PD_ERR_WORKSPACE), (dict(ws=65544), pd.PD_ERR_INVALID),
    (dict(q=None), pd.PD_ERR_INVALID), (dict(kc=None), pd.PD_ERR_INVALID), (dict(cl=None), pd.PD_ERR_INVALID),
    (dict(out=None), pd.PD_ERR_INVALID), (dict(out=32776), pd.PD_ERR_INVALID), (dict(nb=0), pd.PD_ERR_INVALID),
    (dict(mb=0), pd.PD_ERR_INVALID), (dict(scale=math.nan), pd.PD_ERR_INVALID), (dict(S=1 << 29), pd.PD_ERR_INVALID)])
def test_refused(change, code):
    assert _call(**change) == code
    assert pd.last_error()


def test_empty_batch():
    assert _call(S=0, ws=None) == pd.PD_OK


def test_api_refuses_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(q=bf(3, 8, 64), k_cache=bf(4, 16, 2, 64), v_cache=bf(4, 16, 2, 64), prefix_table=i32(2, 2), prefix_lens=i32(2),
                group_starts=i32(3), block_table=i32(3, 2), context_lens=i32(3), inv_sqrt_d=0.1, num_splits=2)
    for change in (dict(), dict(q=bf(3, 8, 32)), dict(q=bf(3, 64)), dict(v_cache=bf(5, 16, 2, 64)), dict(k_cache=bf(4, 16, 64)),
                   dict(group_starts=i32(2)), dict(prefix_table=i32(3, 2)), dict(context_lens=i32(2)), dict(block_table=i32(2, 2)),
                   dict(prefix_lens=i32(2).long())):
        with pytest.raises(ValueError):
            api.decode_attn_prefix(**{**good, **change})


def test_api_refuses_workspaces():
    """A workspace that is not one buffer, or not on the device of the call (the CPU stands in for both sides here)."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    args = (bf(3, 8, 64), bf(4, 16, 2, 64), bf(4, 16, 2, 64), i32(2, 2), i32(2), i32(3), i32(3, 2), i32(3), None)
    api._check_prefix(*args, None, -1)
    api._check_prefix(*args, torch.zeros(64, dtype=torch.uint8), -1)
    with pytest.raises(ValueError, match="ws"):
        api._check_prefix(*args, torch.zeros(64, dtype=torch.uint8)[::2], -1)
    here = type("T", (), {"get_device": lambda self: 0, "is_contiguous": lambda self: True, "device": "cuda:0"})
    with pytest.raises(ValueError, match="ws"):
        api._check_prefix(*args, here(), -1)


def _check_walk(segments, parts, totals, starts, plens, G, Hkv, limit):
    """Every (group, KV head, row, tile) is one CTA's, no two runs share a slot, and the merge of a row reads the partials of
    exactly the runs that had it."""
    teams, _, BR, tile = totals
    slots = [s[9] for s in segments]
    assert len(set(slots)) == len(slots) and (not slots or max(slots) < limit)
    runs = {}
    for team, rank, g, kvh, row0, rows, tile0, stride, n, slot in segments:
        assert 0 <= team < teams and rank in (0, 1) and 0 < rows <= BR and n >= 0 and (stride, n > 0 or rank == 1) in ((1, True), (2, True))
        runs.setdefault((g, kvh), []).append((row0, rows, range(tile0, tile0 + n * stride, stride), slot))
    at = iter(parts)
    for g, plen in enumerate(plens):
        rows, tiles = (starts[g + 1] - starts[g]) * G, -(-plen // tile)
        for kvh in range(Hkv):
            mine = runs.pop((g, kvh), [])
            for x in range(rows):
                count, step, first = next(at)
                own = [r for r in mine if r[0] <= x < r[0] + r[1]]
                assert sorted(t for r in own for t in r[2]) == list(range(tiles))
                assert sorted(first + i * step * BR for i in range(count)) == sorted(r[3] * BR + x - r[0] for r in own)
            assert all(r[0] + r[1] <= rows for r in mine)
    assert not runs and next(at, None) is None


def _draw_walk(rng):
    G, Hkv, D = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 2, 8]), rng.choice([64, 128, 256])
    n = rng.choice([1, 1, 2, 5, 40])
    sizes = [rng.choice([0, 1, 2, 5, 20, 33, 40, 64][:8 if n < 40 else 4]) for _ in range(n)]
    plens = [rng.choice([0, 1, 17, 64, 100, 128, 129, 700, 3000, 200000]) for _ in range(n)]
    starts = [sum(sizes[:i]) for i in range(n + 1)]
    more = dict(fp8=rng.random() < 0.5, own_us=rng.choice([0.0, 30.0, 1e3, 1e5, 1e9]), max_teams=rng.choice([1, 3, 24, 76, 76]))
    return starts, plens, G, Hkv, D, more


def test_division_that_the_kernels_run():
    """pd_debug_prefix_walk runs the functions of the pass and the merge on the host."""
    kinds = set()
    for seed in range(8):
        rng = random.Random(seed)
        for _ in range(40):
            starts, plens, G, Hkv, D, more = _draw_walk(rng)
            segments, parts, totals = pd.pd_debug_prefix_walk(starts, plens, G * Hkv, Hkv, D, **more)
            assert totals[0] <= more["max_teams"]
            items = Hkv * (len(plens) + starts[-1] * G // (2 * totals[2]))  # what the workspace is sized for
            _check_walk(segments, parts, totals, starts, plens, G, Hkv, 2 * (items + 76))
            kinds |= {(len(plens) > 1, totals[1] > 0, s[7], s[8] == 0) for s in segments}
    # one line and whole teams, rows in halves and tiles in turn, places without a tile
    assert {(False, False, 1, False), (False, False, 2, False), (False, False, 2, True), (True, False, 1, False), (True, True, 1, False),
            (True, True, 2, False), (True, True, 2, True)} <= kinds


def test_division_check_sees_mistakes():
    """The check itself, on divisions with one mistake each."""
    starts, plens = [0, 70, 71], [900, 129]
    segments, parts, totals = pd.pd_debug_prefix_walk(starts, plens, 8, 2, 128)

    def check(s, p):
        _check_walk(s, p, totals, starts, plens, 4, 2, 2 * (2 * (2 + 71 * 4 // 512) + 76))

    check(segments, parts)
    for i in (0, len(segments) // 2, len(segments) - 1):
        for change in (None, (6, 1), (8, -1), (4, 1), (5, -1), (9, 1), (3, 1)):
            bad = list(segments)
            if change is None:
                del bad[i]
            else:
                row = list(bad[i])
                row[change[0]] += change[1]
                bad[i] = tuple(row)
            with pytest.raises((AssertionError, StopIteration)):
                check(bad, parts)
    for i in (0, len(parts) // 2, len(parts) - 1):
        for k, by in ((0, 1), (0, -1), (2, 1), (2, 256)):
            row = list(parts[i])
            row[k] += by
            with pytest.raises(AssertionError):
                check(segments, parts[:i] + [tuple(row)] + parts[i + 1:])


def test_walk_refusals():
    with pytest.raises(pd.PdError):
        pd.pd_debug_prefix_walk([0, 3], [-1], 4, 1, 64)
    with pytest.raises(pd.PdError):
        pd.pd_debug_prefix_walk([0, 3], [5], 4, 1, 64, max_teams=77)
    with pytest.raises(pd.PdError):
        pd.pd_debug_prefix_walk([0, 3], [5], 5, 2, 64)
    assert pd.pd_debug_prefix_walk([0, 3], [0], 4, 1, 64)[0] == []
