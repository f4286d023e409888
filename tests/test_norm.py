"""CPU tests of the head norms with the rotation: every refusal, none of which reaches a kernel."""

import math

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd


def _apply(**change):
    """pd_norm_rope_apply on addresses that are never followed."""
    a = dict(rope=None, x=4096, xt=256, xh=128, w=1024, eps=1e-6, offset=0.0, pos=None, out=8192, ot=256, oh=128, T=3, H=2, D=128)
    a.update(change)
    return pd.lib().pd_norm_rope_apply(a["rope"], a["x"], a["xt"], a["xh"], a["w"], a["eps"], a["offset"], a["pos"], a["out"], a["ot"], a["oh"],
                                       a["T"], a["H"], a["D"], None)


def _backward(**change):
    a = dict(rope=None, x=4096, xt=256, xh=128, w=1024, eps=1e-6, offset=0.0, pos=None, g=16384, gt=256, gh=128, dx=8192, dt=256, dh=128, dw=2048,
             T=3, H=2, D=128, ws=1 << 20, ws_bytes=1 << 30)
    a.update(change)
    return pd.lib().pd_norm_rope_backward(a["rope"], a["x"], a["xt"], a["xh"], a["w"], a["eps"], a["offset"], a["pos"], a["g"], a["gt"], a["gh"],
                                          a["dx"], a["dt"], a["dh"], a["dw"], a["T"], a["H"], a["D"], a["ws"], a["ws_bytes"], None)


COMMON = [(dict(T=-1), pd.PD_ERR_INVALID), (dict(H=-1), pd.PD_ERR_INVALID), (dict(D=12), pd.PD_ERR_UNSUPPORTED),
          (dict(D=264), pd.PD_ERR_UNSUPPORTED), (dict(D=0), pd.PD_ERR_UNSUPPORTED), (dict(eps=-1e-9), pd.PD_ERR_INVALID),
          (dict(eps=math.nan), pd.PD_ERR_INVALID), (dict(offset=math.inf), pd.PD_ERR_INVALID), (dict(w=1026), pd.PD_ERR_INVALID),
          (dict(x=None), pd.PD_ERR_INVALID), (dict(x=4104), pd.PD_ERR_INVALID), (dict(xt=0), pd.PD_ERR_INVALID),
          (dict(xh=132), pd.PD_ERR_INVALID), (dict(xh=-128), pd.PD_ERR_INVALID)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(out=None), pd.PD_ERR_INVALID), (dict(out=8200), pd.PD_ERR_INVALID), (dict(ot=248), pd.PD_ERR_INVALID),  # rows that overlap
    (dict(ot=128, oh=128), pd.PD_ERR_INVALID), (dict(oh=64), pd.PD_ERR_INVALID), (dict(out=4096, xt=512), pd.PD_ERR_INVALID),
    (dict(T=2**31 - 1, H=4, ot=512), pd.PD_ERR_INVALID)])
def test_norm_refused(change, code):
    assert _apply(**change) == code
    assert pd.last_error()


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(g=None), pd.PD_ERR_INVALID), (dict(dx=None), pd.PD_ERR_INVALID), (dict(g=16392), pd.PD_ERR_INVALID),
    (dict(dx=8200), pd.PD_ERR_INVALID), (dict(dt=128), pd.PD_ERR_INVALID), (dict(gh=60), pd.PD_ERR_INVALID), (dict(w=None), pd.PD_ERR_INVALID),
    (dict(ws=None), pd.PD_ERR_WORKSPACE), (dict(ws_bytes=100), pd.PD_ERR_WORKSPACE), (dict(ws=(1 << 20) + 8), pd.PD_ERR_INVALID)])
def test_norm_backward_refused(change, code):
    assert _backward(**change) == code
    assert pd.last_error()


def test_norm_of_nothing():
    assert _apply(T=0) == pd.PD_OK and _apply(H=0) == pd.PD_OK and _backward(T=0, dw=None) == pd.PD_OK
    n = pd.pd_norm_rope_workspace_bytes
    assert n(0) == 0 and n(257) == 0 and n(8) == n(64) and n(128) == 2 * n(64) and n(256) == 2 * n(128)


def _append(**change):
    """pd_append_kv_normed[_fp8]: the append's own refusals, and the norm's."""
    a = dict(rope=None, q=4096, q_tok=512, k=8192, k_tok=128, v=16384, v_tok=128, qw=512, kw=768, eps=1e-6, offset=0.0, q_out=32768, kc=65536,
             vc=131072, bt=1024, mb=4, cl=2048, ts=None, T=2, S=2, Hq=4, Hkv=1, D=128, bs=16, nb=8, fp8=None)
    a.update(change)
    scales = [] if a["fp8"] is None else list(a["fp8"])
    fn = pd.lib().pd_append_kv_normed if a["fp8"] is None else pd.lib().pd_append_kv_normed_fp8
    return fn(a["rope"], a["q"], a["q_tok"], a["k"], a["k_tok"], a["v"], a["v_tok"], a["qw"], a["kw"], a["eps"], a["offset"], a["q_out"], a["kc"],
              a["vc"], *scales, a["bt"], a["mb"], a["cl"], a["ts"], a["T"], a["S"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["nb"], None)


@pytest.mark.parametrize("change,code", [
    (dict(eps=-1.0), pd.PD_ERR_INVALID), (dict(eps=math.inf), pd.PD_ERR_INVALID), (dict(offset=math.nan), pd.PD_ERR_INVALID),
    (dict(qw=520), pd.PD_ERR_INVALID), (dict(kw=770), pd.PD_ERR_INVALID), (dict(Hq=3, Hkv=2), pd.PD_ERR_INVALID),
    (dict(D=12), pd.PD_ERR_UNSUPPORTED), (dict(bs=8), pd.PD_ERR_UNSUPPORTED), (dict(T=3), pd.PD_ERR_INVALID), (dict(k=None), pd.PD_ERR_INVALID),
    (dict(q_out=None), pd.PD_ERR_INVALID), (dict(k_tok=132), pd.PD_ERR_INVALID), (dict(q_out=4096, q_tok=520), pd.PD_ERR_INVALID),
    (dict(mb=1 << 28), pd.PD_ERR_INVALID), (dict(fp8=(0.0, 1.0)), pd.PD_ERR_INVALID),
    (dict(fp8=(1.0, 1.0), D=24, q_tok=96, k_tok=24, v_tok=24), pd.PD_ERR_UNSUPPORTED)])
def test_append_normed_refused(change, code):
    assert _append(**change) == code
    assert pd.last_error()


def test_append_normed_of_nothing():
    assert _append(T=0, S=0) == pd.PD_OK and _append(T=0, ts=512) == pd.PD_OK


def test_api_refuses_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rotation = type("Rotation", (), {"head_dim": 64, "handle": 1})
    api._check_norm(rotation, bf(3, 2, 64), bf(64), i32(3), -1)
    api._check_norm(None, bf(3, 2, 80), None, None, -1)
    for args in ((rotation, bf(3, 2, 32), bf(32), i32(3)), (rotation, bf(3, 2, 64), bf(32), i32(3)), (rotation, bf(3, 2, 64), bf(64), None),
                 (rotation, bf(3, 2, 64), bf(64), i32(2)), (rotation, bf(3, 2, 64), bf(64).float(), i32(3)), (None, bf(3, 64), None, None),
                 (rotation, bf(3, 2, 64), bf(128)[::2], i32(3)), (None, bf(3, 2, 64), None, i32(3)), (None, torch.zeros(3, 2, 64), None, None),
                 (None, bf(3, 64, 2).transpose(1, 2), None, None)):
        with pytest.raises(ValueError):
            api._check_norm(*args, -1)
    for leaf in (bf(3, 2, 64).requires_grad_(), bf(64).requires_grad_()):
        x, w = (leaf, bf(64)) if leaf.dim() == 3 else (bf(3, 2, 64), leaf)
        with pytest.raises(ValueError, match="gradient"):
            api.norm_rope(rotation, x, w, i32(3), out=bf(3, 2, 64))
