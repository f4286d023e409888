"""CPU tests of the rotary positions and the append: the frequency rules against their definitions, and every
refusal, none of which reaches a kernel."""

import ctypes
import math

import numpy as np
import pytest
import torch

import rope_reference as R
from paged_kv_decode_splitk_gb300 import api, pd

RULES = [dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
         dict(scaling="banded", factor=8.0, original=8192), dict(scaling="yarn", factor=16.0, original=4096),
         dict(scaling="yarn", factor=1.0, original=4096), dict(scaling="yarn", factor=4.0, original=2048, low=2.0, high=16.0),
         dict(scaling="banded", factor=3.0, original=100, low=0.5, high=1.5)]


@pytest.mark.parametrize("rule", RULES, ids=lambda r: "-".join(map(str, r.values())))
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (20, 10000.0), (4, 10000.0), (256, 1e6)])
def test_frequencies(rule, rot, base):
    want, factor = R.frequencies(rot, base, **rule)
    names = dict(original="original_context", low="low_turns", high="high_turns")
    got, c = pd.pd_rope_frequencies(pd.rope_desc(256, rot, base=base, **{names.get(k, k): v for k, v in rule.items()}))
    # pow, log and a few products in 64 bits, each within 2^-52
    np.testing.assert_allclose(got, want, rtol=2.0**-46)
    assert c == pytest.approx(factor, rel=2.0**-50)


def test_table_rule_and_factor():
    f = [0.5, -0.25, 0.0, 7.0]
    got, c = pd.pd_rope_frequencies(pd.rope_desc(64, 8, frequencies=f, attention_factor=1.5))
    assert got == f and c == 1.5


@pytest.mark.parametrize("change,code", [
    (dict(head_dim=12), pd.PD_ERR_UNSUPPORTED), (dict(head_dim=264), pd.PD_ERR_UNSUPPORTED),
    (dict(head_dim=0), pd.PD_ERR_UNSUPPORTED), (dict(rot_dim=0), pd.PD_ERR_INVALID), (dict(rot_dim=7), pd.PD_ERR_INVALID),
    (dict(rot_dim=66), pd.PD_ERR_INVALID), (dict(layout=2), pd.PD_ERR_INVALID), (dict(scaling=9), pd.PD_ERR_INVALID),
    (dict(base=1.0), pd.PD_ERR_INVALID), (dict(base=math.nan), pd.PD_ERR_INVALID),
    (dict(scaling="linear", factor=0.0), pd.PD_ERR_INVALID), (dict(scaling="linear", factor=math.inf), pd.PD_ERR_INVALID),
    (dict(scaling="ntk", rot_dim=2, factor=2.0), pd.PD_ERR_INVALID), (dict(scaling="yarn", factor=2.0), pd.PD_ERR_INVALID),
    (dict(scaling="banded", factor=2.0, original_context=64, low_turns=4.0, high_turns=4.0), pd.PD_ERR_INVALID),
    (dict(attention_factor=-1.0), pd.PD_ERR_INVALID), (dict(scaling="table"), pd.PD_ERR_INVALID),
    (dict(rot_dim=4, frequencies=[1.0, math.inf]), pd.PD_ERR_INVALID)])
def test_description_refused(change, code):
    args = {**dict(head_dim=64, rot_dim=64), **change}
    with pytest.raises(pd.PdError) as e:
        pd.pd_rope_frequencies(pd.rope_desc(**args))
    assert e.value.code == code
    with pytest.raises(pd.PdError) as e:  # the same check stands before anything is allocated
        pd.pd_rope_create(pd.rope_desc(**args))
    assert e.value.code == code


def test_description_names():
    with pytest.raises(ValueError, match="layout"):
        pd.rope_desc(64, layout="halves")
    with pytest.raises(ValueError, match="scaling"):
        pd.rope_desc(64, scaling="linearly")
    with pytest.raises(ValueError, match="frequencies"):
        pd.rope_desc(64, 8, frequencies=[1.0])
    with pytest.raises(pd.PdError):
        pd._check(pd.lib().pd_rope_create(None, ctypes.byref(ctypes.c_void_p())))


def _append(**change):
    """pd_append_kv[_fp8] on addresses that are never followed: every call here is refused on the host."""
    a = dict(rope=None, q=4096, q_tok=512, k=8192, k_tok=128, v=16384, v_tok=128, q_out=32768, kc=65536, vc=131072, bt=1024,
             mb=4, cl=2048, ts=None, T=2, S=2, Hq=4, Hkv=1, D=128, bs=16, nb=8, fp8=None)
    a.update(change)
    scales = [] if a["fp8"] is None else list(a["fp8"])
    fn = pd.lib().pd_append_kv if a["fp8"] is None else pd.lib().pd_append_kv_fp8
    return fn(a["rope"], a["q"], a["q_tok"], a["k"], a["k_tok"], a["v"], a["v_tok"], a["q_out"], a["kc"], a["vc"], *scales,
              a["bt"], a["mb"], a["cl"], a["ts"], a["T"], a["S"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["nb"], None)


@pytest.mark.parametrize("change,code", [
    (dict(Hkv=0), pd.PD_ERR_INVALID), (dict(Hq=3, Hkv=2), pd.PD_ERR_INVALID), (dict(D=12), pd.PD_ERR_UNSUPPORTED),
    (dict(D=512), pd.PD_ERR_INVALID), (dict(bs=8), pd.PD_ERR_UNSUPPORTED), (dict(T=-1), pd.PD_ERR_INVALID),
    (dict(S=-1, T=-1), pd.PD_ERR_INVALID), (dict(T=3), pd.PD_ERR_INVALID), (dict(k=None), pd.PD_ERR_INVALID),
    (dict(v=None), pd.PD_ERR_INVALID), (dict(q_out=None), pd.PD_ERR_INVALID), (dict(kc=None), pd.PD_ERR_INVALID),
    (dict(bt=None), pd.PD_ERR_INVALID), (dict(cl=None), pd.PD_ERR_INVALID), (dict(k=8200), pd.PD_ERR_INVALID),
    (dict(q_out=32776), pd.PD_ERR_INVALID), (dict(vc=131080), pd.PD_ERR_INVALID), (dict(q_tok=504), pd.PD_ERR_INVALID),
    (dict(k_tok=132), pd.PD_ERR_INVALID), (dict(v_tok=0), pd.PD_ERR_INVALID), (dict(k_tok=-128), pd.PD_ERR_INVALID),
    (dict(q_out=4096, q_tok=520), pd.PD_ERR_INVALID), (dict(mb=0), pd.PD_ERR_INVALID), (dict(nb=0), pd.PD_ERR_INVALID),
    (dict(mb=1 << 28), pd.PD_ERR_INVALID), (dict(fp8=(0.0, 1.0)), pd.PD_ERR_INVALID),
    (dict(fp8=(1.0, -1.0)), pd.PD_ERR_INVALID), (dict(fp8=(math.nan, 1.0)), pd.PD_ERR_INVALID),
    (dict(fp8=(1.0, math.inf)), pd.PD_ERR_INVALID),
    (dict(fp8=(1.0, 1.0), D=24, q_tok=96, k_tok=24, v_tok=24), pd.PD_ERR_UNSUPPORTED)])
def test_append_refused(change, code):
    assert _append(**change) == code
    assert pd.last_error()


def test_append_of_nothing():
    assert _append(T=0, S=0) == pd.PD_OK
    assert _append(T=0, S=2, ts=512) == pd.PD_OK
    assert pd.last_error() == ""


def test_apply_null_handle():
    assert pd.lib().pd_rope_apply(None, 16, 8, 8, 16, 16, 8, 8, 1, 1, 0, None) == pd.PD_ERR_INVALID


def test_api_refuses_tensors():
    """Types, shapes and devices are refused before the library is called (all tensors here are on the CPU)."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731

    class Fake:
        head_dim, handle = 64, 0

    for x, pos in ((torch.zeros(2, 4, 64), i32(2)), (bf(2, 4, 32), i32(2)), (bf(2, 4, 64), i32(2)), (bf(2, 64), i32(2)),
                   (bf(2, 64, 64).transpose(1, 2), i32(2))):
        with pytest.raises(ValueError):
            api.rope(Fake, x, pos)
    good = dict(q=bf(2, 4, 64), k=bf(2, 1, 64), v=bf(2, 1, 64), k_cache=bf(4, 16, 1, 64), v_cache=bf(4, 16, 1, 64),
                block_table=i32(2, 2), context_lens=i32(2))
    for change in (dict(), dict(k=bf(2, 64)), dict(v=bf(2, 2, 64)), dict(q=bf(3, 4, 64)), dict(v_cache=bf(5, 16, 1, 64)),
                   dict(k_cache=bf(4, 16, 2, 64)), dict(block_table=i32(3, 2)), dict(context_lens=i32(2).long()),
                   dict(token_starts=i32(2)), dict(q=None, q_out=bf(2, 4, 64))):
        with pytest.raises(ValueError):
            api.append_kv(None, **{**good, **change})


def test_rope_given_outputs_take_no_gradient():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, requires_grad=True)
    rotation = type("Rotation", (), {"head_dim": 64, "handle": 1})
    with pytest.raises(ValueError, match="gradient"):
        api.rope(rotation, x, torch.zeros(2, dtype=torch.int32), out=torch.empty_like(x))
