"""GPU tests of batches of new tokens in which one item's data could meet another's, against the definition in 64 bits."""

import pytest
import torch

from paged_kv_decode_splitk_gb300 import pd
from test_chunk_gpu import Chunks

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_empty_sequences_between_others(D, fp8):
    """Sequences of two key tiles whose queries differ by 2^12 in turn, one, two or no empty ones between them: over FP8 a row
    goes by the scale of its own queries, in whichever of its two places."""
    for empty in (0, 1, 2):
        past = ([199] + [-1] * empty) * 900
        b = Chunks([1] * len(past), past, 4, 1, D, fp8=fp8, single=True, seed=empty)
        b.q[::2 * (empty + 1)] *= 2.0**6
        b.q[empty + 1::2 * (empty + 1)] *= 2.0**-6
        got, lse = b.run(return_lse=True)
        b.check(got, f"{empty} empty", lse)
