"""CPU tests of decode attention behind shared prefixes: the workspace and every refusal, none of which reaches a kernel."""

import math

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd


def test_workspace():
    n = pd.pd_prefix_workspace_bytes
    assert n(0, 1, 8, 2, 128, 1) == 0 and n(4, 0, 8, 2, 128, 1) == 0 and n(4, 1, 8, 3, 128, 1) == 0 and n(4, 1, 8, 2, 128, 0) == 0
    # the own partials; one slot for each CTA and each item: a block of 256 rows of (m, l) and o
    rows, items = 64 * 32 * 10, 8 * (1 + 64 * 4 // 256)
    least = rows * (128 + 2) * 4 + (items + 152) * 256 * (128 + 2) * 4
    assert least <= n(64, 1, 32, 8, 128, 10) <= least + 32 * 256 + 6 * 256
    assert n(64, 3, 32, 8, 128, 10) > n(64, 1, 32, 8, 128, 10)


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
