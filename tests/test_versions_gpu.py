"""GPU tests that torch learns of what the library writes: a tensor that is saved for a gradient and then overwritten by a
call is refused by the gradient.  Each call through the CPython module and through the ctypes binding."""

import numpy as np
import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd
from test_norm_gpu import weight
from test_rope_gpu import i32, make, randn

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T, HQ, HKV, D = 6, 4, 2, 64


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


@pytest.fixture(params=["module", "binding"], autouse=True)
def way(request, monkeypatch):
    if request.param == "binding":
        monkeypatch.setattr(pd, "_quick", pd._Declined())


class Tensors:
    def __init__(self, fp8=False):
        self.rope = make(D, D)[0]
        self.x, self.w, self.pos = randn(T, HQ, D, seed=1), weight(D, 0.0), i32(np.arange(T))
        self.k, self.v = randn(T, HKV, D, seed=2), randn(T, HKV, D, seed=3)
        self.kc, self.vc = randn(T, 16, HKV, D, seed=4), randn(T, 16, HKV, D, seed=5)
        if fp8:
            self.kc, self.vc = (c.to(torch.float8_e4m3fn).view(torch.uint8).clone() for c in (self.kc, self.vc))
        self.table, self.lens = i32([[i] for i in range(T)]), i32([1 + i for i in range(T)])
        self.out, self.lse = torch.empty_like(self.x), torch.empty(T, HQ, device=DEV)
        self.ws = torch.empty(max(pd.pd_workspace_bytes(T, HQ, D, 2), pd.pd_prefix_workspace_bytes(T, 1, HQ, HKV, D, 1),
                                  pd.pd_chunk_workspace_bytes(T, HQ, HKV, D)), dtype=torch.uint8, device=DEV)

    def prefixed(self, **more):
        return api.decode_attn_prefix(self.x, self.kc, self.vc, i32([[0, 1]]), i32([20]), None, self.table, self.lens, 0.1, 1, **more)


CALLS = {  # what is called, and what it writes of the caller's
    "rope": (lambda t, s: api.rope(t.rope, t.x, t.pos, out=t.out, stream=s), ["out"]),
    "norm_rope": (lambda t, s: api.norm_rope(t.rope, t.x, t.w, t.pos, out=t.out, stream=s), ["out"]),
    "append_kv": (lambda t, s: api.append_kv(t.rope, t.x, t.k, t.v, t.kc, t.vc, t.table, t.lens, q_out=t.out, stream=s), ["out", "kc", "vc"]),
    "append_kv_normed": (lambda t, s: api.append_kv_normed(t.rope, t.x, t.k, t.v, t.w, t.w, t.kc, t.vc, t.table, t.lens, q_out=t.out, stream=s),
                         ["out", "kc", "vc"]),
    "append_kv_normed of keys": (lambda t, s: api.append_kv_normed(t.rope, None, t.k, t.v, None, t.w, t.kc, t.vc, t.table, t.lens, stream=s),
                                 ["kc", "vc"]),
    "chunk_attn": (lambda t, s: api.chunk_attn(t.x, t.kc, t.vc, t.table, t.lens, 0.1, out=t.out, lse=t.lse, ws=t.ws, stream=s), ["out", "lse", "ws"]),
    "decode_attn": (lambda t, s: api.decode_attn(t.x, t.kc, t.vc, t.table, t.lens, 0.1, 2, out=t.out, ws=t.ws, stream=s), ["out", "ws"]),
    "decode_attn_prefix": (lambda t, s: t.prefixed(out=t.out, ws=t.ws, stream=s), ["out", "ws"]),
}


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_have_a_new_version(name, fp8, stream):
    call, written = CALLS[name]
    t = Tensors(fp8)
    mine = {n: v for n, v in vars(t).items() if torch.is_tensor(v)}
    before = {n: v._version for n, v in mine.items()}
    call(t, torch.cuda.current_stream() if stream else None)
    assert {n for n, v in mine.items() if v._version != before[n]} == set(written)


def test_a_saved_tensor_that_a_call_overwrites():
    t = Tensors()
    w = t.w.clone().requires_grad_()
    for write in (lambda x: api.norm_rope(t.rope, x, t.w, t.pos, out=x), lambda x: api.rope(t.rope, x, t.pos, out=x),
                  lambda x: api.append_kv_normed(t.rope, x, t.k, t.v, t.w, t.w, t.kc, t.vc, t.table, t.lens, q_out=x),
                  lambda x: pd.pd_norm_rope_backward(t.rope, x, t.w, t.pos, x, x, None, None)):
        x = t.x.clone()
        y = api.norm_rope(t.rope, x, w, t.pos)
        write(x)
        with pytest.raises(RuntimeError, match="modified"):
            torch.autograd.grad(y, w, t.x)
    positions = t.pos.clone()
    y = api.norm_rope(t.rope, t.x, w, positions)
    api.rope(t.rope, t.x, positions, out=t.out)  # (what is only read keeps its version)
    torch.autograd.grad(y, w, t.x)


@pytest.mark.parametrize("name", CALLS)
def test_inference_tensors_are_written(name):
    """They have no version to raise, inside their mode and outside of it."""
    call, written = CALLS[name]
    want = Tensors()
    call(want, None)
    with torch.inference_mode():
        t, inside = Tensors(), Tensors()
        call(inside, None)
    call(t, None)
    for n in set(written) - {"ws"}:
        assert torch.equal(getattr(t, n), getattr(want, n)) and torch.equal(getattr(inside, n), getattr(want, n))
