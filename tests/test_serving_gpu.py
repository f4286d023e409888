"""A layer's serving steps as a user runs them: prompts in chunks, then single tokens, with the head norms, the rotation,
the append and the attention over one paged cache, eagerly and from one captured graph, against the layer in 64 bits."""

import numpy as np
import pytest
import torch

import rope_reference as R
from paged_kv_decode_splitk_gb300 import api, pd
from test_norm_gpu import normed, weight
from test_rope_gpu import f64, i32, make, randn

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HQ, HKV, D, BS = 8, 2, 64, 16


class Layer:
    """Sequences whose tokens' q, k, v are drawn once; the cache holds what the steps have appended."""

    def __init__(self, totals, fp8, window, seed=0):
        self.totals, self.fp8, self.window = totals, fp8, window
        self.rope, self.freq, self.c = make(D, D, "half", base=10000.0)
        self.qw, self.kw = weight(D, 0.0, 1), weight(D, 0.0, 2)
        self.qkv = [randn(n, HQ + 2 * HKV, D, seed=seed + s) for s, n in enumerate(totals)]
        need = [-(-n // BS) for n in totals]
        ids = np.random.default_rng(seed).permutation(sum(need) + 1)
        self.table = np.zeros((len(totals), max(need)), dtype=np.int64)
        for s, n in enumerate(need):
            self.table[s, :n] = ids[sum(need[:s]):sum(need[:s]) + n]
        kind = torch.uint8 if fp8 else torch.bfloat16
        self.kc, self.vc = (torch.full((sum(need) + 1, BS, HKV, D), 0x7F if fp8 else float("nan"), dtype=kind, device=DEV) for _ in range(2))
        self.scales = dict(k_scale=2.0**-5, v_scale=2.0**-5) if fp8 else {}

    def batch(self, new, lens):
        """The rows of a step whose sequences get `new` tokens behind lens."""
        return torch.cat([x[n:n + m] for x, n, m in zip(self.qkv, lens, new)])

    def step(self, rows, lens_after, starts, **more):
        q, k, v = rows.split([HQ, HKV, HKV], 1)
        q = api.append_kv_normed(self.rope, q, k, v, self.qw, self.kw, self.kc, self.vc, i32(self.table) if isinstance(lens_after, list) else
                                 self.table_gpu, lens_after if not isinstance(lens_after, list) else i32(lens_after),
                                 token_starts=starts if not isinstance(starts, list) else i32(starts), **self.scales)
        return api.chunk_attn(q, self.kc, self.vc, i32(self.table) if isinstance(lens_after, list) else self.table_gpu,
                              lens_after if not isinstance(lens_after, list) else i32(lens_after), D**-0.5,
                              token_starts=starts if not isinstance(starts, list) else i32(starts), window=self.window, **self.scales, **more)

    def value(self, s, n):
        """The layer's output for the first n tokens of sequence s, and its error bound, in 64 bits.

        q and k are off by their rounding, 2^-8 each relative (k to E4M3: 2^-4, or half the smallest step): a score
        moves by at most (their sum) times sum |q k| scale, which the weights take twice; v is exact (E4M3: 2^-4 and half a
        smallest step), weights round by 2^-8 and the output by 2^-8."""
        x = f64(self.qkv[s][:n])
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        pos = np.arange(n)
        q = R.rotate(normed(q, f64(self.qw), 0.0, 1e-6), pos, self.freq, self.c, "half")[0]
        k = R.rotate(normed(k, f64(self.kw), 0.0, 1e-6), pos, self.freq, self.c, "half")[0]
        step = (2.0**-4, 2.0**-10 * 2.0**-5) if self.fp8 else (2.0**-8, 0.0)
        out, lim = np.zeros((n, HQ, D)), np.zeros((n, HQ, D))
        far = pos[:, None] - pos[None]
        seen = (far >= 0) & (far < (self.window or n))
        for h in range(HQ):
            kk, vv = k[:, h // (HQ // HKV)], v[:, h // (HQ // HKV)]
            z = np.where(seen, q[:, h] @ kk.T * D**-0.5, -np.inf)
            w = np.exp(z - z.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            off = (np.abs(q[:, h]) @ (np.abs(kk) * (2.0**-8 + step[0]) + step[1]).T * D**-0.5 * 1.01).max(-1, keepdims=True)
            out[:, h] = w @ vv
            lim[:, h] = (np.expm1(2 * off) + 2.0**-7) * (w @ np.abs(vv)) + w @ (np.abs(vv) * (step[0] if self.fp8 else 0) + step[1]) + 2.0**-8 * np.abs(w @ vv)
        return out, lim


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_prompts_in_chunks_and_tokens(fp8, window):
    """Chunks of prompts beside single tokens of other sequences, step by step; every output against the layer."""
    layer = Layer([150, 90, 33, 70], fp8, window, seed=1)
    plan = [[100, 0, 33, 1], [0, 64, 0, 1], [50, 1, 0, 1], [0, 25, 0, 67]]
    lens, got = [0, 0, 0, 0], [[], [], [], []]
    for new in plan:
        starts = [0, *np.cumsum(new).tolist()]
        after = [n + m for n, m in zip(lens, new)]
        out = layer.step(layer.batch(new, lens), after, starts)
        for s in range(4):
            got[s].append(out[starts[s]:starts[s + 1]])
        lens = after
    for s in range(4):
        ref, lim = layer.value(s, lens[s])
        err = np.abs(f64(torch.cat(got[s])) - ref)
        assert np.all(err <= lim), f"sequence {s}: worst error / bound {np.max(err / lim)}"


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_tokens_from_one_graph(fp8):
    """Decode steps replayed from one captured graph that counts the lengths itself, behind eager prompts."""
    layer = Layer([60, 41, 17], fp8, 0, seed=2)
    lens = [50, 31, 7]
    layer.step(layer.batch(lens, [0, 0, 0]), lens, [0, 50, 81, 88])
    layer.table_gpu, own = i32(layer.table), i32(lens)
    rows = torch.zeros(3, HQ + 2 * HKV, D, dtype=torch.bfloat16, device=DEV)
    ws = api.chunk_workspace(3, HQ, HKV, D, DEV)

    def step():
        own.add_(1)
        return layer.step(rows, own, None, ws=ws)

    kept = layer.kc.clone(), layer.vc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # (everything is loaded before the capture)
    torch.cuda.synchronize()
    own.copy_(i32(lens))
    layer.kc.copy_(kept[0])
    layer.vc.copy_(kept[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for n in range(10):
        rows.copy_(layer.batch([1, 1, 1], [m + n for m in lens]))
        graph.replay()
        for s in range(3):
            ref, lim = layer.value(s, lens[s] + n + 1)
            assert np.all(np.abs(f64(out[s]) - ref[-1]) <= lim[-1]), f"step {n}, sequence {s}"
    assert own.tolist() == [m + 10 for m in lens] and pd.pd_device_status() == 0
