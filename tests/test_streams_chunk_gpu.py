"""Attention of new tokens, norms and their append on another stream than the current one: as tests/test_streams_gpu.py has it
of the other calls, what they allocate belongs to that stream's order."""

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd
from test_streams_gpu import DEV, HKV, HQ, SLEEP, Calls, D, S, i32, randn

pytestmark = pytest.mark.gpu

NAMES = ["chunk", "chunk_lse", "norm", "norm_gradients", "append_normed"]


class More(Calls):
    def __init__(self):
        super().__init__()
        self.weight, self.grad = torch.ones(D, dtype=torch.bfloat16, device=DEV), randn(S, HQ, D, seed=5)
        self.starts = i32([0, 1000, S])  # 1000 and 280 new tokens of two sequences
        self.two, self.after = torch.randint(S, (2, 80), device=DEV).to(torch.int32), i32([1000, 1280])

    def chunk(self, **more):
        return api.chunk_attn(self.q, self.kc, self.vc, self.two, self.after, D**-0.5, token_starts=self.starts, **more)

    def chunk_lse(self, **more):
        return self.chunk(return_lse=True, **more)

    def norm(self, **more):
        return api.norm_rope(self.rotation, self.q, self.weight, self.positions, **more)

    def norm_gradients(self, **more):
        return api.norm_rope_backward(self.rotation, self.q, self.weight, self.positions, self.grad, **more)

    def append_normed(self, **more):
        return api.append_kv_normed(self.rotation, self.q, self.kv, self.kv, self.weight, self.weight, self.kc, self.vc, self.table, self.lens,
                                    **more)


def several(x):
    return x if isinstance(x, tuple) else (x,)


@pytest.mark.parametrize("by", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_results_on_another_stream(name, by):
    """Work of the current stream on memory that is free again, still to come when the other stream's kernels run."""
    call = getattr(More(), name)
    current = torch.cuda.current_stream()
    want = several(call(stream=current))
    side = torch.cuda.Stream()
    given = side if by == "stream" else side.cuda_stream
    call(stream=given)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(SLEEP)
    for t in old:
        t.fill_(float("nan"))
    del old, t
    got = several(call(stream=given))
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["chunk", "norm_gradients"])
def test_workspace_on_another_stream(name):
    """A call's workspace is not handed out again before its kernels are done."""
    call = getattr(More(), name)
    current, side = torch.cuda.current_stream(), torch.cuda.Stream()
    want = several(call(stream=current))
    n = pd.pd_chunk_workspace_bytes(S, HQ, HKV, D) if name == "chunk" else pd.pd_norm_rope_workspace_bytes(D)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = several(call(stream=side))
    other = torch.full((n,), 7, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(got, want))
    assert bool((other == 7).all())


@pytest.mark.parametrize("name", NAMES)
def test_forked_stream_in_a_graph(name):
    """A captured step that forks to another stream and joins again, results allocated on the way."""
    calls, side = More(), torch.cuda.Stream()
    call = getattr(calls, name)
    want = several(call(stream=torch.cuda.current_stream()))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [several(call(stream=side)), several(call(stream=side.cuda_stream))]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in (*got[0], *got[1]):
            t.zero_()
        graph.replay()
        assert all(bool((a == b).all()) for g in got for a, b in zip(g, want))
