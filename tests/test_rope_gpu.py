"""GPU tests of the rotary positions and the append to the paged cache, against the definitions in 64 bits."""

import numpy as np
import pytest
import torch

import oracle
import rope_reference as R
from helpers import assert_within_tolerance
from paged_kv_decode_splitk_gb300 import api, pd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def make(D, rot, layout="half", **rule):
    names = dict(original="original_context")
    return (pd.Rope(D, rot, layout=layout, **{names.get(k, k): v for k, v in rule.items()}), *R.frequencies(rot, **rule))


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


def check(got, ref, size):
    err = np.abs(f64(got) - ref)
    bound = R.bf16_bound(ref, size)
    assert np.all(err <= bound), f"worst error / bound {np.max(err / bound)}"


# unit widths 8 (rot 128, 80), 4 (24), 2 (20), 1 (6); interleaved with a unit that ends in copied columns (20, 6)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 8, 2), (1, 40, 128, 128), (7, 3, 80, 80), (33, 5, 80, 24), (65, 4, 64, 20),
                                       (129, 2, 256, 6), (3, 17, 256, 64), (2049, 40, 128, 128), (5000, 19, 192, 96)])
def test_rope(T, H, D, rot, layout):
    rope, freq, c = make(D, rot, layout, base=10000.0)
    x = randn(T, H, D, seed=T)
    pos = np.random.default_rng(T).integers(0, 131072, T)
    ref, size = R.rotate(f64(x), pos, freq, c, layout)
    check(api.rope(rope, x, i32(pos)), ref, size)


@pytest.mark.parametrize("rule", [dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                  dict(scaling="banded", factor=8.0, original=8192),
                                  dict(scaling="yarn", factor=16.0, original=4096)], ids=lambda r: r["scaling"])
def test_rope_far_and_negative_positions(rule):
    """The angle is reduced exactly: up to the last int32 position, within the error of the reference's own
    frequencies (2^-52 relative, 2^31 radians at most: 2^-20) -- added to the bound."""
    rope, freq, c = make(128, 128, base=500000.0, **rule)
    pos = [0, 1, -1, 2**20, 10**6 + 7, 2**31 - 1, -(2**31), -77777, 123456789]
    x = randn(len(pos), 8, 128, seed=3)
    ref, size = R.rotate(f64(x), pos, freq, c, "half")
    err = np.abs(f64(api.rope(rope, x, i32(pos))) - ref)
    assert np.all(err <= R.bf16_bound(ref, size) + 2.0**-19 * size)


def test_rope_strided_in_place_inverse():
    rope, freq, c = make(128, 64, "half")
    row = randn(50, 12, 128, seed=4)
    pos = i32(np.arange(50) * 37)
    x = row[:, 2:9]  # heads 2..8 of a wider row
    ref, size = R.rotate(f64(x), pos.cpu().numpy(), freq, c, "half")
    out = torch.full((50, 20, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    api.rope(rope, x, pos, out=out[:, 5:12])
    check(out[:, 5:12], ref, size)
    assert torch.all(out[:, :5] == 7) and torch.all(out[:, 12:] == 7)
    by_head = x.transpose(0, 1).contiguous().transpose(0, 1)  # [T, H, D] stored head by head
    assert torch.equal(api.rope(rope, by_head, pos), out[:, 5:12])
    before = row.clone()
    got = api.rope(rope, x, pos, out=x)  # in place
    assert got.data_ptr() == x.data_ptr() and torch.equal(x, out[:, 5:12])
    assert torch.equal(row[:, :2], before[:, :2]) and torch.equal(row[:, 9:], before[:, 9:])
    # and back: two roundings to BF16 of values no larger than |a| + |b|
    back = f64(api.rope(rope, x, pos, inverse=True))
    one = f64(before[:, 2:9])
    _, s1 = R.rotate(one, pos.cpu().numpy(), freq, c, "half")
    assert np.all(np.abs(back - one)[..., :64] <= (2.0**-8 * 2 + 2.0**-8) * s1[..., :64] + 1e-30)
    assert np.array_equal(back[..., 64:], one[..., 64:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """inverse is the transposed map: against the formula in 64 bits, and <R(x + h e) - R(x - h e), g> / 2h (R is
    linear, so any step serves) in 64 bits for a few columns."""
    rope, freq, c = make(80, 40, layout, scaling="yarn", factor=8.0, original=2048)
    pos = np.arange(11) * 911
    x, g = randn(11, 3, 80, seed=5), randn(11, 3, 80, seed=6)
    got = api.rope(rope, g, i32(pos), inverse=True)
    ref, size = R.rotate(f64(g), pos, freq, c, layout, inverse=True)
    check(got, ref, size)
    for col in (0, 1, 19, 20, 39, 40, 79):
        e = np.zeros((11, 3, 80))
        e[..., col] = 0.5
        up, down = (R.rotate(f64(x) + s * e, pos, freq, c, layout)[0] for s in (1, -1))
        diff = ((up - down) * f64(g)).sum(-1)  # h = 1/2
        _, size = R.rotate(f64(g), pos, freq, c, layout)
        assert np.all(np.abs(f64(got)[..., col] - diff) <= R.bf16_bound(diff, size[..., col] + 1e-6))


def test_rope_copied_columns_keep_infinities():
    for layout in ("half", "interleaved"):
        rope, *_ = make(64, 20, layout)
        x = randn(4, 2, 64, seed=7)
        x[:, :, 20:] = float("inf")
        y = api.rope(rope, x, i32([5, 6, 7, 8]))
        assert torch.all(torch.isinf(y[..., 20:])) and torch.all(torch.isfinite(y[..., :20]))


def test_rope_nothing_streams_and_graphs():
    rope, freq, c = make(128, 128)
    assert api.rope(rope, randn(0, 4, 128), i32([])).shape == (0, 4, 128)
    x, pos = randn(300, 8, 128, seed=8), i32(np.arange(300))
    want = api.rope(rope, x, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.rope(rope, x, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out, g = torch.zeros_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rope(rope, x, pos, out=out)
    x2 = randn(300, 8, 128, seed=9)
    x.copy_(x2)
    g.replay()
    assert torch.equal(out, api.rope(rope, x2, pos))


def test_rope_handle_refusals():
    with pytest.raises(pd.PdError) as e:
        pd.pd_debug_fail_next_allocs(1)
        pd.Rope(64)
    assert e.value.code == pd.PD_ERR_ALLOC
    rope, *_ = make(64, 64)
    x, pos = randn(2, 2, 64), i32([0, 1])
    with pytest.raises(pd.PdError):  # in place with other strides
        pd._check(pd.lib().pd_rope_apply(rope.handle, x.data_ptr(), 128, 64, pos.data_ptr(), x.data_ptr(), 256, 64, 2, 2, 0, None))
    for strides in ((0, 64, 128, 64), (128, 60, 128, 64), (128, 64, -128, 64), (128, 64, 128, 12)):
        with pytest.raises(pd.PdError):
            pd._check(pd.lib().pd_rope_apply(rope.handle, x.data_ptr(), strides[0], strides[1], pos.data_ptr(),
                                             x.data_ptr() + 16, strides[2], strides[3], 2, 2, 0, None))
    with pytest.raises(pd.PdError):
        pd._check(pd.lib().pd_rope_apply(rope.handle, x.data_ptr() + 2, 128, 64, pos.data_ptr(), x.data_ptr(), 128, 64, 1, 1, 0, None))
    with pytest.raises(pd.PdError):
        pd._check(pd.lib().pd_rope_apply(rope.handle, x.data_ptr(), 128, 64, pos.data_ptr(), x.data_ptr(), 128, 64, 2, 2, 2, None))
    out = torch.empty(4096, dtype=torch.bfloat16, device=DEV)
    for T, H, token, head in ((2, 2, 64, 64), (3, 2, 128, 32), (3, 3, 192, 128), (2, 2, 8, 64), (3, 1, 32, 64)):  # overlapping rows
        with pytest.raises(pd.PdError, match="overlap"):
            pd._check(pd.lib().pd_rope_apply(rope.handle, out.data_ptr(), 192, 64, i32([0] * T).data_ptr(), out.data_ptr() + 2048,
                                             token, head, T, H, 0, None))
    for view in (torch.empty(2, 3, 64, dtype=torch.bfloat16, device=DEV).transpose(0, 1), torch.empty(2, 2, 96, dtype=torch.bfloat16,
                 device=DEV)[..., :64]):  # and rows that do not
        x = randn(*view.shape)
        pos = i32(range(len(x)))
        assert torch.equal(api.rope(rope, x, pos, out=view), api.rope(rope, x, pos))
    rope.close()
    with pytest.raises(ValueError, match="closed"):
        api.rope(rope, x, pos)


# ---- append ----------------------------------------------------------------------------------


class Append:
    """A cache, tables and new tokens: `new` per sequence, after `past` that are there already."""

    def __init__(self, new, past, Hq, Hkv, D, bs=16, fp8=False, lead=0, tail=0, seed=0, starts=True):
        rng = np.random.default_rng(seed)
        self.lens = [n + p for n, p in zip(new, past)]
        blocks = [-(-n // bs) for n in self.lens]
        pool, width = sum(blocks) + 3, max(1, max(blocks, default=1))
        ids = rng.permutation(pool)
        self.table = np.full((len(new), width), -5, dtype=np.int64)  # entries past a sequence's blocks are never read
        at = 0
        for s, n in enumerate(blocks):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.starts = [lead, *(lead + np.cumsum(new)).tolist()] if starts else list(range(len(new) + 1))
        self.T = lead + sum(new) + tail if starts else len(new)
        self.row = randn(self.T, Hq + 2 * Hkv, D, seed=seed)
        self.q, self.k, self.v = self.row[:, :Hq], self.row[:, Hq:Hq + Hkv], self.row[:, Hq + Hkv:]
        shape = (pool, bs, Hkv, D)
        if fp8:
            mk = lambda s: randn(*shape, seed=s).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        else:
            mk = lambda s: randn(*shape, seed=s)  # noqa: E731
        self.kc, self.vc = mk(seed + 1), mk(seed + 2)
        self.k_scale, self.v_scale = (0.011, 0.25) if fp8 else (1.0, 1.0)
        self.bs, self.fp8, self.has_starts = bs, fp8, starts

    def run(self, rope, q_out=None, **more):
        return api.append_kv(rope, self.q, self.k, self.v, self.kc, self.vc, i32(self.table), i32(self.lens),
                             token_starts=i32(self.starts) if self.has_starts else None, q_out=q_out, k_scale=self.k_scale,
                             v_scale=self.v_scale, **more)

    def tokens(self):
        if self.has_starts:
            return R.append_positions(self.starts, self.lens)
        return [(s, s, n - 1) for s, n in enumerate(self.lens) if n > 0]

    def check(self, freq, c, layout, q_out, before, skip=()):
        tok = [t for t in self.tokens() if t[0] not in skip]
        rows, pos = [t[0] for t in tok], [t[2] for t in tok]
        if freq is None:
            freq, c = np.zeros(0), 1.0
        if q_out is not None:
            ref, size = R.rotate(f64(self.q)[rows], pos, freq, c, layout)
            check(q_out[rows], ref, size)
        cells = [(int(self.table[s, p // self.bs]), p % self.bs) for _, s, p in tok]
        blk, off = [b for b, _ in cells], [o for _, o in cells]
        k, size = R.rotate(f64(self.k)[rows], pos, freq, c, layout)
        for cache, old, ref, sz, scale in ((self.kc, before[0], k, size, self.k_scale),
                                           (self.vc, before[1], f64(self.v)[rows], 0 * size, self.v_scale)):
            got = cache[blk, off]
            if self.fp8:
                code = np.clip(ref / np.float64(np.float32(scale)), -448, 448)
                err = np.abs(f64(got.view(torch.float8_e4m3fn)) - code)
                assert np.all(err <= R.e4m3_bound(code, sz, scale))
            else:
                check(got, ref, sz)
            rest = torch.ones(cache.shape[:2], dtype=torch.bool, device=DEV)
            rest[blk, off] = False
            assert torch.equal(cache[rest], old[rest])  # every other slot as it was


CASES = [  # new, past, Hq, Hkv, D, block size, rows before and after
    ([1], [0], 1, 1, 8, 16, 0, 0), ([1, 1, 1], [15, 16, 0], 4, 1, 64, 16, 0, 0), ([3, 0, 17, 1], [14, 9, 0, 300], 4, 2, 128, 16, 2, 3),
    ([0, 0, 5, 0], [0, 3, 0, 0], 8, 8, 80, 48, 1, 0), ([200, 1, 33], [7, 1000, 31], 6, 2, 256, 32, 0, 5),
    ([1] * 70 + [40] + [0] * 30, list(range(101)), 14, 2, 64, 16, 0, 1), ([1500, 700], [0, 13], 32, 8, 128, 16, 0, 0)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rot,layout", [(None, "half"), (0.5, "interleaved"), (6, "half")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[2]}-{c[3]}-{c[4]}")
def test_append(case, rot, layout, fp8):
    new, past, Hq, Hkv, D, bs, lead, tail = case
    if fp8 and D % 16:
        pytest.skip("E4M3 caches take head dims of 16")
    rot = D if rot is None else D // 2 if rot == 0.5 else rot
    rope, freq, c = make(D, rot, layout, scaling="linear", factor=2.0)
    a = Append(new, past, Hq, Hkv, D, bs, fp8, lead, tail, seed=len(new))
    before = a.kc.clone(), a.vc.clone()
    q_out = torch.full((a.T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    got = a.run(rope, q_out=q_out)
    assert got.data_ptr() == q_out.data_ptr()
    a.check(freq, c, layout, got, before)
    assert torch.all(got[:lead] == 9) and torch.all(got[a.T - tail:] == 9)  # rows of no sequence


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_append_single_tokens(fp8):
    """One token per sequence without token_starts; an empty sequence (a padded batch) has none."""
    lens = [1, 0, 16, 17, 500, 0]
    rope, freq, c = make(128, 128)
    a = Append([0] * 6, lens, 8, 2, 128, fp8=fp8, seed=3, starts=False)
    before = a.kc.clone(), a.vc.clone()
    q_out = torch.full((6, 8, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    a.check(freq, c, "half", a.run(rope, q_out=q_out), before)
    assert torch.all(q_out[[1, 5]] == 9)


def test_append_without_rotation_or_queries():
    a = Append([4, 1], [0, 20], 8, 2, 128, seed=4)
    before = a.kc.clone(), a.vc.clone()
    q = a.run(None)
    a.check(None, 1.0, "half", q, before)
    assert torch.equal(q, a.q)
    a.kc.copy_(before[0])
    a.q = None
    assert a.run(None) is None
    a.check(None, 1.0, "half", None, before)


def test_append_in_place_queries_and_streams():
    rope, freq, c = make(128, 128)
    a = Append([40, 9], [3, 0], 4, 2, 128, seed=5)
    before = a.kc.clone(), a.vc.clone()
    want = a.run(rope)
    k_want = a.kc.clone()
    a.q = a.q.contiguous()
    a.kc.copy_(before[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = a.run(rope, q_out=a.q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got.data_ptr() == a.q.data_ptr() and torch.equal(got, want) and torch.equal(a.kc, k_want)


def test_append_saturates():
    a = Append([3], [0], 1, 1, 64, fp8=True, seed=6)
    a.row[:] = 1e4
    before = a.kc.clone(), a.vc.clone()
    rope, freq, c = make(64, 32)
    a.check(freq, c, "half", a.run(rope), before)
    assert float(a.vc[int(a.table[0, 0]), 0].view(torch.float8_e4m3fn).float().max()) == 448


def test_append_flags():
    """Bad lengths and block ids are reported, their tokens left out, the others done."""
    rope, freq, c = make(64, 64)
    a = Append([2, 3, 1, 2], [0, 0, 40, 5], 2, 1, 64, seed=7)
    before = a.kc.clone(), a.vc.clone()
    a.lens[0] = 1                          # two new tokens of a sequence of one: the first has no place
    a.lens[2] = a.table.shape[1] * 16 + 1  # beyond the table
    q_out = torch.full((8, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    a.run(rope, q_out=q_out)
    assert pd.pd_device_status() == pd.PD_DEV_BAD_CONTEXT_LEN
    a.check(freq, c, "half", q_out, before, skip={0, 5})
    assert torch.all(q_out[[0, 5]] == 9)
    b = Append([2, 3], [0, 0], 2, 1, 64, seed=8)
    before = b.kc.clone(), b.vc.clone()
    keep = b.table.copy()
    for bad in (-1, b.kc.shape[0], 2**31 - 1):
        b.table[1, 0] = bad
        q = b.run(rope)
        assert pd.pd_device_status() == pd.PD_DEV_BAD_BLOCK_ID
    b.table = keep
    b.starts, b.lens, rows = [0, 2, 2], [2, 0], q.clone()  # what should be there: the first sequence alone
    b.check(freq, c, "half", rows, before)
    full = api.rope(rope, b.q, i32([0, 1, 0, 1, 2]))
    assert torch.equal(q, full)  # the queries are rotated all the same


def test_append_far_in_a_large_cache():
    """Element offsets past 2^32 (codes and BF16)."""
    rope, freq, c = make(256, 256)
    for fp8 in (True, False):
        nb = 2**32 // (16 * 8 * 256) + 40
        cache = torch.zeros((nb, 16, 8, 256), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
        k = randn(2, 8, 256, seed=9)
        table = i32([[nb - 1], [2]])
        api.append_kv(None, None, k, k, cache, cache, table, i32([16, 1]), k_scale=1.0, v_scale=1.0)
        for b, o, t in ((nb - 1, 15, 0), (2, 0, 1)):
            want = k[t].float().to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else k[t]
            assert torch.equal(cache[b, o], want)
        cache[nb - 1, 15] = 0
        cache[2, 0] = 0
        assert not bool(cache[::97].any()) and not bool(cache[-3:].any())
        del cache


def test_append_then_decode_in_one_graph():
    """A captured step: append with rotation, then the decode attention that reads it; replayed on new tokens."""
    Hq, Hkv, D, S = 8, 2, 128, 5
    rope, freq, c = make(D, D)
    lens = [1, 17, 300, 64, 1025]
    a = Append([0] * S, lens, Hq, Hkv, D, seed=10, starts=False)
    table, cl = i32(a.table), i32(lens)
    q_out = torch.empty((S, Hq, D), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q_out)
    ws = api.workspace(S, Hq, D, 4, DEV)

    def step():
        api.append_kv(rope, a.q, a.k, a.v, a.kc, a.vc, table, cl, q_out=q_out)
        api.decode_attn(q_out, a.kc, a.vc, table, cl, D**-0.5, 4, out=out, ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    a.row.copy_(randn(S, Hq + 2 * Hkv, D, seed=11))
    g.replay()
    torch.cuda.synchronize()
    ref, size = R.rotate(f64(a.q), [n - 1 for n in lens], freq, c, "half")
    check(q_out, ref, size)
    tab = np.maximum(a.table, 0).astype(np.int32)
    ref = oracle.decode_attn(api.bf16_bits(q_out), api.bf16_bits(a.kc), api.bf16_bits(a.vc), tab,
                             np.asarray(lens, dtype=np.int32), D**-0.5)
    assert_within_tolerance(f64(out), ref, "append then decode")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_by_autograd(layout):
    """A tensor that requires a gradient gets the transposed map's, here through a slice of a fused projection; the
    rotation is linear, so the gradient of the gradient is the rotation again."""
    rope, freq, c = make(80, 40, layout, scaling="yarn", factor=8.0, original=2048)
    pos = i32(np.arange(11) * 911)
    row, g = randn(11, 5, 80, seed=5).requires_grad_(), randn(11, 3, 80, seed=6)
    x = row[:, 1:4]
    y = api.rope(rope, x, pos)
    assert torch.equal(y, api.rope(rope, x.detach(), pos))
    want = api.rope(rope, g, pos, inverse=True)
    y.backward(g, retain_graph=True)
    assert torch.equal(row.grad[:, 1:4], want) and not row.grad[:, [0, 4]].any()
    ref, size = R.rotate(f64(g), np.arange(11) * 911, freq, c, layout, inverse=True)
    check(row.grad[:, 1:4], ref, size)
    # gradients that come broadcast, transposed, or 2 bytes off a 16-byte boundary
    ones = torch.ones_like(g)
    assert torch.equal(torch.autograd.grad(y.sum(), x, retain_graph=True)[0], api.rope(rope, ones, pos, inverse=True))
    odd = torch.empty(g.numel() + 1, dtype=g.dtype, device=DEV)[1:].view_as(g).copy_(g)
    turned = g.transpose(0, 2).contiguous().transpose(0, 2)
    for same in (odd, turned):
        assert torch.equal(torch.autograd.grad(y, x, same, retain_graph=True)[0], want)
    # the inverse's gradient, and the second
    assert torch.equal(torch.autograd.grad(api.rope(rope, x, pos, inverse=True), x, g)[0], api.rope(rope, g, pos))
    h = g.clone().requires_grad_()
    (back,) = torch.autograd.grad(y, x, h, create_graph=True)
    assert torch.equal(torch.autograd.grad(back, h, g)[0], api.rope(rope, g, pos))
    # by the difference quotient (R is linear: any step serves) of a sum in 64 bits, a column at a time
    for col in (0, 19, 20, 39, 79):
        e = np.zeros((11, 3, 80))
        e[..., col] = 0.5
        up, down = (R.rotate(f64(x) + s * e, np.arange(11) * 911, freq, c, layout)[0] for s in (1, -1))
        diff = ((up - down) * f64(g)).sum(-1)
        _, size = R.rotate(f64(g), np.arange(11) * 911, freq, c, layout)
        assert np.all(np.abs(f64(row.grad)[:, 1:4, col] - diff) <= R.bf16_bound(diff, size[..., col] + 1e-6))


def test_rope_gradient_streams_modes_and_graphs():
    rope, *_ = make(64, 64)
    x, g, pos = randn(40, 4, 64, seed=1).requires_grad_(), randn(40, 4, 64, seed=2), i32(range(40))
    want = api.rope(rope, x.detach(), pos), api.rope(rope, g, pos, inverse=True)
    with torch.no_grad():
        assert not api.rope(rope, x, pos).requires_grad
        out = torch.empty_like(g)
        assert api.rope(rope, x, pos, out=out) is out and torch.equal(out, want[0])
    with torch.inference_mode():
        assert torch.equal(api.rope(rope, x, pos), want[0])
    for bad in (torch.empty_like(g), x):
        with pytest.raises(ValueError, match="gradient"):
            api.rope(rope, x, pos, out=bad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = api.rope(rope, x, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0]) and torch.equal(torch.autograd.grad(y, x, g)[0], want[1])
    graph = torch.cuda.CUDAGraph()
    leaf, got = x.detach().clone().requires_grad_(), None
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y = api.rope(rope, leaf, pos)
        (got,) = torch.autograd.grad(y, leaf, g)
    for n in range(2):
        with torch.no_grad():
            leaf.copy_(randn(40, 4, 64, seed=7 + n))
            g.copy_(randn(40, 4, 64, seed=17 + n))
        graph.replay()
        assert torch.equal(y, api.rope(rope, leaf.detach(), pos)) and torch.equal(got, api.rope(rope, g, pos, inverse=True))
    pos2 = pos.clone()
    y = api.rope(rope, x, pos2)
    pos2.add_(1)
    with pytest.raises(RuntimeError, match="modified"):  # the positions the gradient needs are gone
        torch.autograd.grad(y, x, g)


@pytest.mark.parametrize("scales", [(0.011, 0.0125), (3.0, 0.75), (0.3, 1e-3), (2.0**-9, 7.0)])
def test_append_fp8_codes(scales):
    """The codes of copied rows, bit for bit: x times the FP32 reciprocal of the scale, in FP32, to the nearest E4M3 value."""
    a = Append([40, 1, 17], [3, 200, 0], 4, 2, 64, fp8=True, seed=21)
    a.k_scale, a.v_scale = scales
    a.run(None)
    rows, cells = zip(*((r, (int(a.table[s, p // a.bs]), p % a.bs)) for r, s, p in a.tokens()))
    at = tuple(torch.tensor(c, device=DEV) for c in zip(*cells))
    for cache, x, scale in ((a.kc, a.k, a.k_scale), (a.vc, a.v, a.v_scale)):
        reciprocal = float(np.float32(1) / np.float32(scale))
        want = (x[list(rows)].float() * reciprocal).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(cache[at], want)
