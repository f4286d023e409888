"""Calls on another stream than the current one: the tensors they allocate belong to that stream's order, so memory that
the current stream still has to write, or may take again, is not theirs."""

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
S, HQ, HKV, D = 1280, 32, 8, 128  # q and out of 10.5 MB: blocks of their own in the allocator
SLEEP = 200_000_000  # cycles: a tenth of a second


def randn(*shape, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Calls:
    """The library's calls that allocate what they return."""

    def __init__(self):
        self.rotation = pd.Rope(D)
        self.q, self.kv = randn(S, HQ, D, seed=1), randn(S, HKV, D, seed=2)
        self.positions = torch.arange(S, dtype=torch.int32, device=DEV)
        self.kc, self.vc = randn(S + 8, 16, HKV, D, seed=3), randn(S + 8, 16, HKV, D, seed=4)
        self.table = torch.arange(S, dtype=torch.int32, device=DEV).view(S, 1)
        self.lens = i32([1 + i % 16 for i in range(S)])
        self.far = torch.randint(S, (S, 20), device=DEV).to(torch.int32)  # 320 tokens: two splits, with partials
        self.long = self.lens + 300
        self.prefix, self.span = i32([list(range(S, S + 8))]), i32([100])
        torch.cuda._sleep(10)  # (everything the tests use is loaded before they start)
        self.q.clone().fill_(0).zero_()
        torch.full((16,), 7, dtype=torch.uint8, device=DEV)

    def rope(self, **more):
        return api.rope(self.rotation, self.q, self.positions, **more)

    def append(self, **more):
        return api.append_kv(None, self.q, self.kv, self.kv, self.kc, self.vc, self.table, self.lens, **more)

    def decode(self, **more):
        return api.decode_attn(self.q, self.kc, self.vc, self.far, self.long, D**-0.5, 2, **more)

    def prefixed(self, **more):
        return api.decode_attn_prefix(self.q, self.kc, self.vc, self.prefix, self.span, None, self.far, self.long, D**-0.5, 2,
                                      **more)


@pytest.mark.parametrize("by", ["stream", "handle"])
@pytest.mark.parametrize("name", ["rope", "append", "decode", "prefixed"])
def test_results_on_another_stream(name, by):
    """Work of the current stream on memory that is free again, still to come when the other stream's kernels run."""
    call = getattr(Calls(), name)
    want = call()
    side = torch.cuda.Stream()
    given = side if by == "stream" else side.cuda_stream
    call(stream=given)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.empty_like(want)
    torch.cuda._sleep(SLEEP)
    old.fill_(float("nan"))
    del old
    got = call(stream=given)
    side.synchronize()
    torch.cuda.synchronize()
    assert bool((got == want).all())


@pytest.mark.parametrize("name", ["decode", "prefixed"])
def test_workspace_on_another_stream(name):
    """A call's workspace is not handed out again before its kernels are done."""
    call = getattr(Calls(), name)
    want, out = call(), torch.empty((S, HQ, D), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    n = (pd.pd_workspace_bytes(S, HQ, D, 2) if name == "decode" else pd.pd_prefix_workspace_bytes(S, 1, HQ, HKV, D, 2))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    call(stream=side, out=out)
    other = torch.full((n,), 7, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert bool((out == want).all())
    assert bool((other == 7).all())


def test_results_are_kept_for_the_current_stream():
    """A result that the current stream still reads when it is let go is not overwritten by the other stream's next call."""
    calls, side = Calls(), torch.cuda.Stream()
    want = calls.rope()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = calls.rope(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    kept = got.clone()
    del got
    for _ in range(2):
        api.rope(calls.rotation, calls.q, calls.positions + 1, stream=side).zero_()
    torch.cuda.synchronize()
    assert bool((kept == want).all())


@pytest.mark.parametrize("name", ["rope", "append", "decode", "prefixed"])
def test_forked_stream_in_a_graph(name):
    """A captured step that forks to another stream and joins again, results allocated on the way."""
    calls, side = Calls(), torch.cuda.Stream()
    call = getattr(calls, name)
    want = call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [call(stream=side), call(stream=side.cuda_stream)]
        torch.cuda.current_stream().wait_stream(side)
        twice = got[0] + got[1]
    for _ in range(2):
        for t in (*got, twice):
            t.zero_()
        graph.replay()
        assert all(bool((t == want).all()) for t in got) and bool((twice == want + want).all())
