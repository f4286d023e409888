"""GPU tests of batches of new tokens in which one item's data could meet another's, against the definition in 64 bits."""

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd
from test_chunk_gpu import DEV, Chunks, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_empty_sequences_between_others(D, fp8):
    """Sequences of two key tiles whose queries differ by 2^12 in turn, one or two empty ones between them: over FP8 a row
    goes by the scale of its own queries, in whichever of its two places."""
    for empty in (1, 2):
        past = ([199] + [-1] * empty) * 500
        b = Chunks([1] * len(past), past, 4, 1, D, fp8=fp8, single=True, seed=empty)
        b.q[::2 * (empty + 1)] *= 2.0**6
        b.q[empty + 1::2 * (empty + 1)] *= 2.0**-6
        got, lse = b.run(return_lse=True)
        b.check(got, f"{empty} empty", lse)


def test_a_long_prompt_behind_a_window():
    """2^20 tokens of 32 heads over 8, whose table would make more than 2^30 units and whose window makes few.

    Weights and the output are rounded to BF16 (2^-8 each); a score's FP32 sum of 8 products, the exponential and the sum of
    100 weights are off by less than 2^-16 of weights and sums for scores below 2^6."""
    T, window, Hq, Hkv, D, blocks = 2**20, 100, 32, 8, 8, 64
    q, kc, vc = randn(T, Hq, D, seed=1), randn(blocks, 16, Hkv, D, seed=2), randn(blocks, 16, Hkv, D, seed=3)
    table = (torch.arange(T // 16, device=DEV, dtype=torch.int32) * 37 % blocks)[None].contiguous()
    got, lse = api.chunk_attn(q, kc, vc, table, i32([T]), D**-0.5, token_starts=i32([0, T]), window=window, return_lse=True)
    for p in (0, 5, 98, 99, 100, 127, 128, 1023, 2**19 + 3, 2**20 - 64, 2**20 - 1):
        j = torch.arange(max(0, p + 1 - window), p + 1, device=DEV)
        at = table[0, j // 16].long(), j % 16
        k, v = (c[at].double().permute(1, 0, 2) for c in (kc, vc))
        z = (q[p].double().view(Hkv, Hq // Hkv, D) @ k.transpose(1, 2)) * D**-0.5
        w = torch.softmax(z, -1)
        ref, size = (w @ v).view(Hq, D), (w @ v.abs()).view(Hq, D)
        assert float(z.abs().max()) < 2**6
        assert bool(((got[p].double() - ref).abs() <= 2.0**-8 * (size + ref.abs()) + 2.0**-14 * size + 2.0**-100).all()), p
        assert bool(((lse[p].double() - torch.logsumexp(z, -1).view(Hq)).abs() <= 2.0**-14).all()), p
