"""GPU tests of the head norms with the rotation, their gradients and their append, against the definitions in 64 bits."""

import gc
import weakref

import numpy as np
import pytest
import torch

import rope_reference as R
from paged_kv_decode_splitk_gb300 import api, pd
from test_rope_gpu import CASES, Append, f64, i32, make, randn

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


def normed(x, w, offset, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w + offset)


def value(x, w, offset, eps, pos, freq, c, layout):
    """The definition, and what an FP32 error is relative to in each column: the rotated pair's sizes, or the value."""
    y = normed(x, w, offset, eps)
    if freq is None:
        return y, np.abs(y)
    ref, size = R.rotate(y, pos, freq, c, layout)
    return ref, size + np.abs(ref)


# BF16 rounds by at most half a step, 2^-8 of the value.  FP32 before it: a sum of at most 256 squares in chains of 8 and
# by halves (13 additions, 2^-24 each, halved by the root), its reciprocal root (2 ulp: 2^-22), three products, and the
# rotation's 2^-20 of the pair's sizes (rope_reference): below 2^-19 of the sizes together.
def bound(ref, size):
    return 2.0**-8 * np.abs(ref) + 2.0**-19 * size + 2.0**-133


def check(got, ref, lim):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= lim), f"worst error / bound {np.max(err / lim)}"


def gradients(x, w, offset, eps, pos, freq, c, layout, g):
    """(dx, its bound, dw, its bound) from the formula.

    FP32 errors: u = R^T g as a rotation (2^-20 of the pair's sizes, 2^-24 each for products), 1/rms 2^-21, the row sums
    2^-20 of the sums of sizes: below 2^-18 of what the terms' sizes add up to.  dw sums a lane's rows, a block's lines, the
    blocks, in chains shorter than 128: 2^-17 of the sum of sizes beside each term's 2^-19."""
    D = x.shape[-1]
    ww = np.ones(D) if w is None else w + offset
    u, size = (g, np.abs(g)) if freq is None else R.rotate(g, pos, freq, c, layout, inverse=True)
    size = size + np.abs(u)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx = r * (u * ww - x * r * r * (x * u * ww).sum(-1, keepdims=True) / D)
    big = r * np.abs(ww) * size + np.abs(x) * r**3 * (np.abs(x * ww) * size).sum(-1, keepdims=True) / D
    dw = (u * x * r).reshape(-1, D).sum(0)
    dw_big = (size * np.abs(x * r)).reshape(-1, D).sum(0)
    return dx, 2.0**-8 * np.abs(dx) + 2.0**-18 * big + 2.0**-133, dw, 2.0**-8 * np.abs(dw) + (2.0**-17 + 2.0**-19) * dw_big + 2.0**-133


def weight(D, offset, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(D, generator=g) * 0.5 + 1 - offset).to(torch.bfloat16).to(DEV)


# lanes of 8, 16 and 32 with columns left over (80, 8, 192); pairs 8 columns apart at a time (rot a multiple of 16), anywhere
# (rot 20, 6, 2), units that end in copied columns; one row, tokens that end inside a block, several heads a lane
SHAPES = [(1, 1, 8, 2), (1, 40, 128, 128), (7, 3, 80, 80), (33, 5, 80, 24), (65, 4, 64, 20), (129, 2, 256, 6), (3, 17, 256, 64), (2049, 40, 128, 128),
          (900, 19, 192, 96), (4000, 7, 64, 64)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", SHAPES)
def test_norm_rope(T, H, D, rot, layout):
    rope, freq, c = make(D, rot, layout, base=10000.0, scaling="yarn", factor=8.0, original=2048)
    offset = float(T % 2)
    x, w = randn(T, H, D, seed=T, scale=3.0), weight(D, offset)
    pos = np.random.default_rng(T).integers(-10, 131072, T)
    got = api.norm_rope(rope, x, w, i32(pos), weight_offset=offset)
    ref, size = value(f64(x), f64(w), offset, 1e-6, pos, freq, c, layout)
    check(got, ref, bound(ref, size))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", SHAPES)
def test_norm_rope_backward(T, H, D, rot, layout):
    rope, freq, c = make(D, rot, layout, base=10000.0, scaling="yarn", factor=8.0, original=2048)
    offset = float(T % 2)
    x, w, g = randn(T, H, D, seed=T, scale=3.0), weight(D, offset), randn(T, H, D, seed=T + 1)
    pos = np.random.default_rng(T).integers(0, 131072, T)
    dx, dw = api.norm_rope_backward(rope, x, w, i32(pos), g, weight_offset=offset)
    rx, bx, rw, bw = gradients(f64(x), f64(w), offset, 1e-6, pos, freq, c, layout, f64(g))
    check(dx, rx, bx)
    check(dw, rw, bw)
    again = api.norm_rope_backward(rope, x, w, i32(pos), g, weight_offset=offset)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # the order of the sums is fixed


# So many rows that blocks walk them: tokens whose turns pass the room for them (248 columns), one head (more tokens a block
# than are held at a time), pairs anywhere, tokens that the blocks do not divide.
@pytest.mark.parametrize("T,H,D,rot,layout", [(20011, 8, 256, 248, "half"), (160001, 1, 256, 20, "half"), (50003, 13, 64, 62, "half"),
                                              (20011, 16, 128, 128, "half"), (9001, 40, 128, 64, "interleaved")])
def test_norm_of_many_rows(T, H, D, rot, layout):
    rope, freq, c = make(D, rot, layout)
    x, w, g = randn(T, H, D, seed=T, scale=3.0), weight(D, 0.0), randn(T, H, D, seed=T + 1)
    pos = np.random.default_rng(T).integers(0, 131072, T)
    got = api.norm_rope(rope, x, w, i32(pos))
    dx, dw = api.norm_rope_backward(rope, x, w, i32(pos), g)
    torch.cuda.synchronize()
    ref, size = value(f64(x), f64(w), 0.0, 1e-6, pos, freq, c, layout)
    check(got, ref, bound(ref, size))
    rx, bx, rw, bw = gradients(f64(x), f64(w), 0.0, 1e-6, pos, freq, c, layout, f64(g))
    check(dx, rx, bx)
    check(dw, rw, bw)


def test_norm_gradient_by_differences():
    """<y(x + h e) - y(x - h e), g> / 2h in 64 bits: off by h^2 / 6 of the third derivative, here below 1e-7 of the sizes."""
    rope, freq, c = make(80, 40, "half")
    pos = np.arange(11) * 911
    x, w, g = randn(11, 3, 80, seed=5), weight(80, 0.0), randn(11, 3, 80, seed=6)
    dx, dw = api.norm_rope_backward(rope, x, w, i32(pos), g)
    _, bx, _, bw = gradients(f64(x), f64(w), 0.0, 1e-6, pos, freq, c, "half", f64(g))
    f = lambda a, b: (value(a, b, 0.0, 1e-6, pos, freq, c, "half")[0] * f64(g))  # noqa: E731
    h = 1e-4
    for col in (0, 1, 19, 20, 39, 40, 79):
        e = np.zeros(80)
        e[col] = h
        diff = (f(f64(x) + e, f64(w)) - f(f64(x) - e, f64(w))).sum(-1) / (2 * h)
        assert np.all(np.abs(f64(dx)[..., col] - diff) <= bx[..., col] + 1e-6)
        diff = (f(f64(x), f64(w) + e) - f(f64(x), f64(w) - e)).sum() / (2 * h)
        assert abs(f64(dw)[col] - diff) <= bw[col] + 1e-5


def test_norm_without_rotation_or_weight():
    for D in (64, 200):
        x, w, g = randn(31, 6, D, seed=D), weight(D, 1.0), randn(31, 6, D, seed=1)
        for wt, offset in ((w, 1.0), (None, 1.0)):
            got = api.norm_rope(None, x, wt, None, weight_offset=offset)
            ref, size = value(f64(x), None if wt is None else f64(wt), offset, 1e-6, None, None, 1, None)
            check(got, ref, bound(ref, size))
            dx, dw = api.norm_rope_backward(None, x, wt, None, g, weight_offset=offset)
            rx, bx, rw, bw = gradients(f64(x), None if wt is None else f64(wt), offset, 1e-6, None, None, 1, None, f64(g))
            check(dx, rx, bx)
            assert dw is None if wt is None else check(dw, rw, bw) is None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_rows_of_nothing_and_small_ones(layout):
    """Rows of zeros stay zeros, rows far below eps are scaled by 1 / sqrt(eps) alone, an eps of 0 divides by the row's own."""
    rope, freq, c = make(64, 32, layout)
    x, pos = randn(5, 2, 64, seed=2), np.arange(5)
    x[1] = 0
    x[2] *= 2.0**-40
    x[3, :, 32:] = float("inf")  # (copied columns: the row's mean square is infinite, so it is 0 over it, and NaN where inf / inf)
    got = api.norm_rope(rope, x, None, i32(pos))
    ok = [0, 1, 2, 4]
    ref, size = value(f64(x)[ok], None, 0, 1e-6, pos[ok], freq, c, layout)
    check(got[ok], ref, bound(ref, size))
    assert not got[1].any() and not got[3, :, :32].any() and torch.isnan(got[3, :, 32:]).all()
    x = randn(5, 2, 64, seed=2, scale=2.0**-20)
    ref, size = value(f64(x), None, 0, 0.0, pos, freq, c, layout)
    check(api.norm_rope(rope, x, None, i32(pos), eps=0.0), ref, bound(ref, size))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_strided_and_in_place(layout):
    rope, freq, c = make(128, 64, layout)
    row, w, pos = randn(50, 12, 128, seed=4), weight(128, 0.0), i32(np.arange(50) * 37)
    x = row[:, 2:9]  # heads 2..8 of a wider row
    want = api.norm_rope(rope, x.contiguous(), w, pos)
    out = torch.full((50, 20, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    api.norm_rope(rope, x, w, pos, out=out[:, 5:12])
    assert torch.equal(out[:, 5:12], want) and torch.all(out[:, :5] == 7) and torch.all(out[:, 12:] == 7)
    by_head = x.transpose(0, 1).contiguous().transpose(0, 1)  # [T, H, D] stored head by head
    assert torch.equal(api.norm_rope(rope, by_head, w, pos), want)
    g = randn(50, 7, 128, seed=5)
    dx, dw = api.norm_rope_backward(rope, x.contiguous(), w, pos, g)
    other = api.norm_rope_backward(rope, by_head, w, pos, g.transpose(0, 1).contiguous().transpose(0, 1))
    assert torch.equal(other[0], dx) and torch.equal(other[1], dw)
    before = row.clone()
    assert api.norm_rope(rope, x, w, pos, out=x).data_ptr() == x.data_ptr() and torch.equal(x, want)
    assert torch.equal(row[:, :2], before[:, :2]) and torch.equal(row[:, 9:], before[:, 9:])
    pd.pd_norm_rope_backward(rope, before[:, 2:9], w, pos, g, g, None, None)  # over the gradient itself
    assert torch.equal(g, dx)


@pytest.mark.parametrize("quick", [True, False], ids=["module", "binding"])
def test_norm_autograd(quick, monkeypatch):
    """Through a slice of a fused projection; gradients that come broadcast, transposed or at an odd place; of the weight
    alone; and what cannot be had.  (Through the CPython module's node, and through the ctypes binding.)"""
    if not quick:
        monkeypatch.setattr(pd, "_quick", pd._Declined())
    rope, freq, c = make(80, 40, "half", scaling="yarn", factor=8.0, original=2048)
    pos = i32(np.arange(11) * 911)
    row, w, g = randn(11, 5, 80, seed=5).requires_grad_(), weight(80, 0.0).requires_grad_(), randn(11, 3, 80, seed=6)
    x = row[:, 1:4]
    y = api.norm_rope(rope, x, w, pos)
    assert torch.equal(y, api.norm_rope(rope, x.detach(), w.detach(), pos))
    want = api.norm_rope_backward(rope, x.detach(), w.detach(), pos, g)
    y.backward(g, retain_graph=True)
    assert torch.equal(row.grad[:, 1:4], want[0]) and not row.grad[:, [0, 4]].any() and torch.equal(w.grad, want[1])
    ones = torch.ones_like(g)
    assert torch.equal(torch.autograd.grad(y.sum(), x, retain_graph=True)[0], api.norm_rope_backward(rope, x.detach(), w.detach(), pos, ones)[0])
    odd = torch.empty(g.numel() + 1, dtype=g.dtype, device=DEV)[1:].view_as(g).copy_(g)
    turned = g.transpose(0, 2).contiguous().transpose(0, 2)
    for same in (odd, turned):
        got = torch.autograd.grad(y, (x, w), same, retain_graph=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    (dw,) = torch.autograd.grad(api.norm_rope(rope, x.detach(), w, pos), w, g)
    assert torch.equal(dw, want[1])
    (dx,) = torch.autograd.grad(api.norm_rope(rope, x, w.detach(), pos), x, g)
    assert torch.equal(dx, want[0])
    (dx,) = torch.autograd.grad(api.norm_rope(None, x, None, None), x, g)
    assert torch.equal(dx, api.norm_rope_backward(None, x.detach(), None, None, g)[0])
    with torch.no_grad():
        assert not api.norm_rope(rope, x, w, pos).requires_grad
    h = g.clone().requires_grad_()
    (back,) = torch.autograd.grad(y, x, h, create_graph=True)
    with pytest.raises(RuntimeError):  # no second gradient
        torch.autograd.grad(back.float().sum(), h)
    y = api.norm_rope(rope, x, w, pos)
    kept = weakref.ref(rope)
    del rope  # (the gradient keeps the rotation)
    gc.collect()
    assert kept() is not None and torch.equal(torch.autograd.grad(y, x, g, retain_graph=True)[0], want[0])
    pos.add_(1)
    with pytest.raises(RuntimeError, match="modified"):  # the positions the gradient needs are gone
        torch.autograd.grad(y, x, g)
    del y
    gc.collect()
    assert kept() is None
    y = api.norm_rope(None, x, w, None)
    with torch.no_grad():
        w.mul_(2)
    with pytest.raises(RuntimeError, match="modified"):
        torch.autograd.grad(y, x, g)
    both = torch.randn(11, 3, 80, device=DEV, dtype=torch.bfloat16).requires_grad_()
    y = api.norm_rope(None, both, None, None)
    torch.autograd.grad(y, both, g)
    with pytest.raises(RuntimeError):  # its tensors were given back
        torch.autograd.grad(y, both, g)


def test_norm_nothing_streams_and_graphs():
    rope, *_ = make(64, 64)
    w, none = weight(64, 0.0), randn(0, 4, 64)
    assert api.norm_rope(rope, none, w, i32([])).shape == (0, 4, 64)
    dx, dw = api.norm_rope_backward(rope, none, w, i32([]), none)
    assert dx.shape == (0, 4, 64) and not dw.any()
    x, g, pos = randn(300, 4, 64, seed=1), randn(300, 4, 64, seed=2), i32(range(300))
    want = api.norm_rope(rope, x, w, pos), *api.norm_rope_backward(rope, x, w, pos, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.norm_rope(rope, x, w, pos, stream=side), *api.norm_rope_backward(rope, x, w, pos, g, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    leaf, leaf_w = x.clone().requires_grad_(), w.clone().requires_grad_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y = api.norm_rope(rope, leaf, leaf_w, pos)
        dx, dw = torch.autograd.grad(y, (leaf, leaf_w), g)
    for n in range(2):
        with torch.no_grad():
            leaf.copy_(randn(300, 4, 64, seed=7 + n))
            leaf_w.copy_(weight(64, 0.0, seed=n))
            g.copy_(randn(300, 4, 64, seed=17 + n))
        graph.replay()
        x, w = leaf.detach(), leaf_w.detach()
        want = api.norm_rope_backward(rope, x, w, pos, g)
        assert torch.equal(y, api.norm_rope(rope, x, w, pos)) and torch.equal(dx, want[0]) and torch.equal(dw, want[1])


# ---- append ----------------------------------------------------------------------------------


class NormedAppend(Append):
    def __init__(self, *args, offset=0.0, **more):
        super().__init__(*args, **more)
        D = self.row.shape[2]
        self.offset, self.qw, self.kw = offset, weight(D, offset, 1), weight(D, offset, 2)

    def run(self, rope, q_out=None, **more):
        return api.append_kv_normed(rope, self.q, self.k, self.v, self.qw, self.kw, self.kc, self.vc, i32(self.table), i32(self.lens),
                                    token_starts=i32(self.starts) if self.has_starts else None, q_out=q_out, weight_offset=self.offset,
                                    k_scale=self.k_scale, v_scale=self.v_scale, **more)

    def check(self, freq, c, layout, q_out, before):
        tok = self.tokens()
        rows, pos = [t[0] for t in tok], [t[2] for t in tok]
        one = lambda w: None if w is None else f64(w)  # noqa: E731
        if q_out is not None:
            ref, size = value(f64(self.q)[rows], one(self.qw), self.offset, 1e-6, pos, freq, c, layout)
            check(q_out[rows], ref, bound(ref, size))
        blk, off = [int(self.table[s, p // self.bs]) for _, s, p in tok], [p % self.bs for _, _, p in tok]
        k, size = value(f64(self.k)[rows], one(self.kw), self.offset, 1e-6, pos, freq, c, layout)
        for cache, old, ref, sz, scale in ((self.kc, before[0], k, size, self.k_scale),
                                           (self.vc, before[1], f64(self.v)[rows], None, self.v_scale)):
            got = cache[blk, off]
            if self.fp8:
                code = np.clip(ref / np.float64(np.float32(scale)), -448, 448)
                err = np.abs(f64(got.view(torch.float8_e4m3fn)) - code)
                assert np.all(err <= R.e4m3_bound(code, 0 * ref if sz is None else 2 * sz, scale))
            elif sz is None:
                assert np.array_equal(f64(got), ref)
            else:
                check(got, ref, bound(ref, sz))
            rest = torch.ones(cache.shape[:2], dtype=torch.bool, device=DEV)
            rest[blk, off] = False
            assert torch.equal(cache[rest], old[rest])  # every other slot as it was


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rot,layout", [(None, "half"), (0.5, "interleaved"), (6, "half"), (0, None)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[2]}-{c[3]}-{c[4]}")
def test_append_normed(case, rot, layout, fp8):
    new, past, Hq, Hkv, D, bs, lead, tail = case
    if fp8 and D % 16:
        pytest.skip("E4M3 caches take head dims of 16")
    if rot == 0:
        rope, freq, c = None, None, 1.0
    else:
        rope, freq, c = make(D, D if rot is None else D // 2 if rot == 0.5 else rot, layout, scaling="linear", factor=2.0)
    a = NormedAppend(new, past, Hq, Hkv, D, bs, fp8, lead, tail, seed=len(new), offset=float(len(new) % 2))
    before = a.kc.clone(), a.vc.clone()
    q_out = torch.full((a.T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    got = a.run(rope, q_out=q_out)
    assert got.data_ptr() == q_out.data_ptr()
    a.check(freq, c, layout, got, before)
    assert torch.all(got[:lead] == 9) and torch.all(got[a.T - tail:] == 9)  # rows of no sequence


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,rot,layout", [(8, 4, 256, 248, "half"), (32, 4, 128, 128, "half"), (30, 3, 128, 64, "interleaved")])
def test_append_normed_of_many_rows(Hq, Hkv, D, rot, layout, fp8):
    rope, freq, c = make(D, rot, layout)
    a = NormedAppend([6000, 1, 0, 4005], [0, 5, 9, 13], Hq, Hkv, D, 16, fp8, 3, 2, seed=D)
    before = a.kc.clone(), a.vc.clone()
    q_out = torch.full((a.T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    a.check(freq, c, layout, a.run(rope, q_out=q_out), before)
    assert torch.all(q_out[:3] == 9) and torch.all(q_out[-2:] == 9)


def test_append_normed_single_tokens_streams_and_bits():
    """One token a sequence, an empty one among them; another stream, in place, and norm_rope's own bits."""
    rope, freq, c = make(128, 128)
    a = NormedAppend([0] * 6, [1, 0, 16, 17, 500, 0], 8, 2, 128, seed=3, starts=False)
    before = a.kc.clone(), a.vc.clone()
    q_out = torch.full((6, 8, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    a.check(freq, c, "half", a.run(rope, q_out=q_out), before)
    assert torch.all(q_out[[1, 5]] == 9)
    pos = i32([max(0, n - 1) for n in a.lens])
    live = [0, 2, 3, 4]
    assert torch.equal(q_out[live], api.norm_rope(rope, a.q, a.qw, pos)[live])
    k = api.norm_rope(rope, a.k, a.kw, pos)
    for s in live:
        p = a.lens[s] - 1
        assert torch.equal(a.kc[int(a.table[s, p // 16]), p % 16], k[s])
    a.q = a.q.contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = a.run(rope, q_out=a.q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got.data_ptr() == a.q.data_ptr() and torch.equal(got[live], q_out[live])


def test_append_normed_without_queries_or_weights():
    rope, freq, c = make(64, 64)
    a = NormedAppend([40, 3], [0, 20], 8, 2, 64, seed=4)
    before = a.kc.clone(), a.vc.clone()
    a.q, a.kw, a.qw = None, None, None
    assert a.run(rope) is None
    a.check(freq, c, "half", None, before)


def test_append_normed_flags():
    """Bad lengths and block ids are reported, their tokens left out, the others done."""
    rope, freq, c = make(64, 64)
    a = NormedAppend([2, 3, 1, 2], [0, 0, 40, 5], 2, 1, 64, seed=7)
    good, before = a.run(rope), (a.kc.clone(), a.vc.clone())
    lens = list(a.lens)
    a.lens[0], a.lens[2] = 1, a.table.shape[1] * 16 + 1
    q_out = torch.full((8, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    a.run(rope, q_out=q_out)
    assert pd.pd_device_status() == pd.PD_DEV_BAD_CONTEXT_LEN
    assert torch.all(q_out[[0, 5]] == 9) and torch.equal(q_out[[2, 3, 4, 6, 7]], good[[2, 3, 4, 6, 7]])
    a.lens = lens
    a.run(rope)
    keep = a.table.copy()
    for bad in (-1, a.kc.shape[0], 2**31 - 1):
        a.table[1, 0] = bad
        assert torch.equal(a.run(rope), good)  # the queries are made all the same
        assert pd.pd_device_status() == pd.PD_DEV_BAD_BLOCK_ID
    a.table = keep
    assert torch.equal(a.kc, before[0]) and torch.equal(a.vc, before[1])


def test_quick_calls_take_what_fits_and_leave_the_rest():
    quick = pd.quick()
    rope, *_ = make(64, 64)
    far = torch.cuda.current_stream().cuda_stream
    x, w, pos = randn(2, 8, 64, seed=1), weight(64, 0.0), i32([5, 9])
    good = [rope.handle, 64, x, w, pos, None, 1e-6, 0.0]
    assert torch.equal(quick.norm_rope(*good), api.norm_rope(rope, x, w, pos, stream=far))
    assert torch.equal(quick.norm_rope(0, 0, x, None, None, None, 1e-6, 0.0), api.norm_rope(None, x, None, None, stream=far))
    for i, bad in ((0, 0), (1, 128), (2, x.float()), (2, x[0]), (3, w[:32]), (3, w.float()), (4, None), (4, pos[:1]), (4, pos.long()), (5, x[:1]),
                   (6, -1.0), (6, "a"), (7, None)):
        assert quick.norm_rope(*good[:i], bad, *good[i + 1:]) is NotImplemented, (i, bad)
    a = NormedAppend([2, 3], [0, 7], 8, 2, 64, seed=4)
    want, k = a.run(rope, stream=far), a.kc.clone()
    good = [rope.handle, 64, a.q, a.k, a.v, a.qw, a.kw, a.kc, a.vc, i32(a.table), i32(a.lens), i32(a.starts), None, 1e-6, 0.0, 1.0, 1.0]
    assert torch.equal(quick.append_kv_normed(*good), want) and torch.equal(a.kc, k)
    for i, bad in ((1, 128), (2, None), (2, a.q[:1]), (3, a.k[:, :1]), (5, a.kw[:8]), (6, a.kw.double()), (7, a.kc[1:]), (9, good[9][:1]),
                   (11, good[11][:2]), (11, None), (12, x), (13, -1.0), (15, "a")):
        assert quick.append_kv_normed(*good[:i], bad, *good[i + 1:]) is NotImplemented, (i, bad)
