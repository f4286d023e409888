"""GPU tests of norm_rope between autograd's other parts: closed rotations, the caller's hooks on saved tensors, checkpoints,
second and forward-mode gradients.  Each through the CPython module's node and through the ctypes binding."""

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwd
from torch.autograd.graph import saved_tensors_hooks
from torch.utils.checkpoint import checkpoint

from paged_kv_decode_splitk_gb300 import api, pd
from test_norm_gpu import weight
from test_rope_gpu import i32, make, randn

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T, H, D = 11, 3, 80


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


@pytest.fixture(params=["module", "binding"], autouse=True)
def way(request, monkeypatch):
    if request.param == "binding":
        monkeypatch.setattr(pd, "_quick", pd._Declined())


class Call:
    def __init__(self):
        self.rope = make(D, 40)[0]
        self.pos = i32(np.arange(T) * 911)
        self.x, self.w, self.g = randn(T, H, D, seed=5).requires_grad_(), weight(D, 0.0).requires_grad_(), randn(T, H, D, seed=6)

    def __call__(self, **more):
        return api.norm_rope(self.rope, self.x, self.w, self.pos, **more)

    def want(self):
        return api.norm_rope_backward(self.rope, self.x.detach(), self.w.detach(), self.pos, self.g)


def test_closed_rotation():
    """A rotation that is closed is refused on the host, by the call and by the gradient of an earlier one."""
    c = Call()
    y = c()
    c.rope.close()
    with pytest.raises(ValueError, match="closed"):
        torch.autograd.grad(y, (c.x, c.w), c.g)
    with pytest.raises(ValueError, match="closed"):
        c()


def test_hooks_that_give_back_another_layout():
    """The same values in other places: laid out anew."""
    c = Call()
    want = c.want()

    def turned(t):
        return t.transpose(0, -1).contiguous().transpose(0, -1) if t.dim() > 1 else torch.stack([t, t], 1)[:, 0]

    def odd(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view_as(t).copy_(t)

    def broadcast(t):
        return t.mean(0, keepdim=True).expand_as(t) if t.dim() == 3 else t

    for unpack in (turned, odd):
        with saved_tensors_hooks(lambda t: t.detach(), unpack):
            y = c()
        assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, (c.x, c.w), c.g), want))
    with saved_tensors_hooks(lambda t: t.detach(), broadcast):
        y = c()
    got = torch.autograd.grad(y, (c.x, c.w), c.g)
    want = api.norm_rope_backward(c.rope, broadcast(c.x.detach()).contiguous(), c.w.detach(), c.pos, c.g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.autograd.graph.save_on_cpu():
        y = c()
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, (c.x, c.w), c.g), c.want()))


@pytest.mark.parametrize("which", ["x", "weight", "positions"])
def test_hooks_that_give_back_something_else(which):
    """Another type, shape or device: refused on the host."""
    c = Call()
    mine = {"x": c.x, "weight": c.w, "positions": c.pos}[which].shape
    for change in (lambda t: t.double(), lambda t: t[:1], lambda t: t[None], lambda t: t[0], lambda t: t.cpu(),
                   lambda t: torch.cat([t, t], -1)):
        with saved_tensors_hooks(lambda t: t.detach(), lambda t: change(t) if t.shape == mine else t):
            y = c()
        with pytest.raises(ValueError):
            torch.autograd.grad(y, (c.x, c.w), c.g)


def projection(x, m, rope, w, pos):
    return api.norm_rope(rope, (x @ m).view(len(x), H, D), w, pos)


def test_checkpointed():
    """A projection with its norm, whose recomputation torch ends from inside the norm's last saved tensor."""
    c = Call()
    x, m = randn(T, 64, seed=1).requires_grad_(), randn(64, H * D, seed=2, scale=0.1).requires_grad_()
    want = torch.autograd.grad(projection(x, m, c.rope, c.w, c.pos), (x, m, c.w), c.g)
    for _ in range(2):
        y = checkpoint(projection, x, m, c.rope, c.w, c.pos, use_reentrant=False)
        got = torch.autograd.grad(y, (x, m, c.w), c.g)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_errors_of_hooks_pass():
    c = Call()

    class Full(Exception):
        pass

    packed = []

    def pack(t):
        packed.append(t)
        raise Full("no room")

    with saved_tensors_hooks(pack, lambda t: t), pytest.raises(Full):
        c()
    assert len(packed) == 1
    with saved_tensors_hooks(lambda t: t.detach(), lambda t: pack(t)):
        y = c()
    with pytest.raises(Full):
        torch.autograd.grad(y, c.x, c.g)


def test_no_second_gradient():
    """A gradient made with create_graph carries an error, whatever it came from, instead of no history."""
    c = Call()
    for grad in (c.g, c.g.clone().requires_grad_()):
        y = c()
        dx, dw = torch.autograd.grad(y, (c.x, c.w), grad, create_graph=True)
        assert dx.requires_grad and dw.requires_grad and all(torch.equal(a, b) for a, b in zip((dx, dw), c.want()))
        for more in (dx, dw):
            with pytest.raises(RuntimeError, match="no second gradient"):  # not the first one alone
                ((y.float() ** 2).sum() + more.float().pow(2).sum()).backward(retain_graph=True)
    y = api.norm_rope(None, c.x, None, None)
    (dx,) = torch.autograd.grad(y, c.x, c.g, create_graph=True)
    assert torch.equal(dx, api.norm_rope_backward(None, c.x.detach(), None, None, c.g)[0])
    with pytest.raises(RuntimeError, match="no second gradient"):
        dx.float().sum().backward()
    got = torch.autograd.grad(c(), (c.x, c.w), c.g)
    assert not any(t.requires_grad for t in got)


@pytest.mark.parametrize("leaf", [True, False])
def test_forward_mode_is_refused(leaf):
    """A tangent, which neither call carries on, is not lost in silence."""
    c = Call()
    x, w = (t.detach().clone().requires_grad_(leaf) for t in (c.x, c.w))
    with fwd.dual_level():
        for a, b in ((fwd.make_dual(x, torch.ones_like(x)), c.w.detach()), (c.x.detach(), fwd.make_dual(w, torch.ones_like(w)))):
            for out in (None,) if leaf else (None, torch.empty_like(x)):
                with pytest.raises(RuntimeError, match="forward"):
                    api.norm_rope(c.rope, a, b, c.pos, out=out)
        with pytest.raises(RuntimeError, match="forward"):
            api.rope(c.rope, fwd.make_dual(x, torch.ones_like(x)), c.pos)
        assert torch.equal(api.norm_rope(c.rope, x.detach(), w.detach(), c.pos), c().detach())  # (no tangent, nothing to lose)
    assert torch.equal(api.norm_rope(c.rope, x, w, c.pos), c().detach())


def test_gradients_of_tangents_are_refused():
    """Forward mode over a backward pass: what comes back to the call has a tangent, and its answer would not."""
    c = Call()
    y = c()
    z = api.rope(c.rope, c.x, c.pos)
    with fwd.dual_level():
        g = fwd.make_dual(c.g, torch.ones_like(c.g))
        for out in (y, z):
            with pytest.raises(RuntimeError, match="forward"):
                torch.autograd.grad(out, c.x, g, retain_graph=True)
    assert torch.equal(torch.autograd.grad(y, c.x, c.g)[0], c.want()[0])
