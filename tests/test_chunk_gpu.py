"""GPU tests of the attention of new tokens over the paged cache, against the definition in 64 bits."""

import numpy as np
import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, pd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def no_flags():
    yield
    assert pd.pd_device_status() == 0


class Chunks:
    """new: new tokens of each sequence, behind `past` that are there; lead and tail: rows of no sequence.  Every cache slot
    that no new token sees holds NaN, table entries of blocks that none does are bad, and rows of no sequence are NaN."""

    def __init__(self, new, past, Hq, Hkv, D, bs=16, fp8=False, window=0, lead=0, tail=0, seed=0, q_scale=1.0, single=False, poison=True,
                 stride=0):
        rng = np.random.default_rng(seed)
        self.new, self.past, self.lens = list(new), list(past), [n + p for n, p in zip(new, past)]
        self.bs, self.fp8, self.window, self.single = bs, fp8, window, single
        self.starts = list(range(len(new) + 1)) if single else [lead, *(lead + np.cumsum(new)).tolist()]
        T = len(new) if single else lead + sum(new) + tail
        need = [-(-n // bs) for n in self.lens]
        pool = sum(need) + 2
        ids, at = rng.permutation(pool), 0
        self.rows = []
        for n in need:
            self.rows.append(ids[at:at + n].tolist())
            at += n
        self.table = np.full((len(new), max(1, max(need, default=1))), -7)
        dead = torch.ones((pool, bs), dtype=torch.bool, device=DEV)
        for s, (row, n) in enumerate(zip(self.rows, self.lens)):
            low = max(0, self.past[s] + 1 - window) if window else 0
            for j, b in enumerate(row):
                if (j + 1) * bs > low and self.new[s]:
                    self.table[s, j] = b
                    dead[b, max(0, low - j * bs): min(bs, n - j * bs)] = False
        self.wide = randn(T, Hq + stride, D, seed=seed + 1, scale=q_scale)
        self.q = self.wide[:, :Hq]
        if poison and not single:
            self.q[:lead] = float("nan")
            self.q[lead + sum(new):] = float("nan")
        self.kc, self.vc = randn(pool, bs, Hkv, D, seed=seed + 2), randn(pool, bs, Hkv, D, seed=seed + 3)
        if poison and not fp8:
            self.kc[dead] = float("nan")
            self.vc[dead] = float("nan")
        self.k_scale, self.v_scale = 1.0, 1.0
        if fp8:
            self.kc, self.vc = ((c * 2).to(torch.float8_e4m3fn).view(torch.uint8) for c in (self.kc, self.vc))
            self.k_scale, self.v_scale = 0.5, 0.25
            if poison:
                self.kc[dead] = 0x7F
                self.vc[dead] = 0x7F
        self.scale = D**-0.5

    def run(self, **more):
        more = {"token_starts": None if self.single else i32(self.starts), **more}
        return api.chunk_attn(self.q, self.kc, self.vc, i32(self.table), i32(self.lens), self.scale, window=self.window,
                              k_scale=self.k_scale, v_scale=self.v_scale, **more)

    def tokens(self, cache, s, a, b, scale):
        j = torch.arange(a, b, device=DEV)
        x = cache[torch.tensor(self.table[s], device=DEV)[j // self.bs], j % self.bs]
        return (x.double() if not self.fp8 else x.view(torch.float8_e4m3fn).double() * scale).permute(1, 0, 2)

    def reference(self):
        """(out, its error bound, lse, its error bound) in 64 bits; rows of no sequence 0.

        With weights w (sum 1) and A = sum w |v|: the weights are rounded to BF16 (half a step, 2^-8 of each; over an FP8
        cache to f16, 2^-11, those below 2^-13 of the largest by 2^-24 of it, times the sum of |v|).  A score's FP32 sum of D
        products is off by at most (D + 8) 2^-24 of sum |q k| scale; the factor log2 e, the exponential (2^-21) and the
        sum of a row's weights (one of 64 chained additions in a tile, and one for each tile: 2^-24 each) come on the
        weights and on their sum.  The output rounds to BF16 (2^-8), lse to FP32 with its reference, logarithm and ln 2
        (2^-22 of |lse| and of the largest |score|, and 2^-22)."""
        T, Hq, D = self.q.shape
        Hkv = self.kc.shape[2]
        G = Hq // Hkv
        out, bound = (torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV) for _ in range(2))
        lse, lse_bound = (torch.zeros((T, Hq), dtype=torch.float64, device=DEV) for _ in range(2))
        for s, m in enumerate(self.lens):
            a, b = self.starts[s], self.starts[s + 1]
            for t0 in range(a, b, 256):
                t1 = min(b, t0 + 256)
                pos = torch.arange(m - b + t0, m - b + t1, device=DEV)
                low = max(0, int(pos[0]) + 1 - self.window) if self.window else 0
                end = max(low, int(pos[-1]) + 1)
                if end == 0:
                    lse[t0:t1] = -float("inf")
                    continue
                k, v = self.tokens(self.kc, s, low, end, self.k_scale), self.tokens(self.vc, s, low, end, self.v_scale)
                far = pos[:, None] - torch.arange(low, end, device=DEV)[None]
                seen = (far >= 0) & (far < (self.window or end + 1))
                q = self.q[t0:t1].double().view(t1 - t0, Hkv, G, D).permute(1, 2, 0, 3)
                z = (q @ k[:, None].transpose(2, 3)) * self.scale
                size = ((q.abs() @ k[:, None].abs().transpose(2, 3)) * abs(self.scale)).masked_fill(~seen, 0).amax(-1, keepdim=True)
                z = z.masked_fill(~seen, -float("inf"))
                w = torch.softmax(z, -1).nan_to_num(0)
                ref, size_v = w @ v[:, None], w @ v[:, None].abs()
                off = (D + 8) * 2.0**-24 * size + 2.0**-21 + (64 + (end - low) / 64) * 2.0**-24
                e = (2.0**-11 if self.fp8 else 2.0**-8) * size_v + 2 * off * size_v + 2.0**-8 * ref.abs() + 2.0**-100
                if self.fp8:
                    e = e + 2.0**-24 * w.amax(-1, keepdim=True) * (seen.double() @ v[:, None].abs())
                L = torch.logsumexp(z, -1)
                out[t0:t1], bound[t0:t1] = (x.permute(2, 0, 1, 3).reshape(t1 - t0, Hq, D) for x in (ref, 1.02 * e))
                lse[t0:t1] = L.permute(2, 0, 1).reshape(t1 - t0, Hq)
                le = off[..., 0] + 2.0**-22 * (1 + L.abs().nan_to_num(0, 0, 0) + size[..., 0])
                lse_bound[t0:t1] = le.permute(2, 0, 1).reshape(t1 - t0, Hq)
        return out, bound, lse, lse_bound

    def check(self, got, what="", lse=None):
        ref, bound, ref_lse, lse_bound = self.reference()
        rows = slice(self.starts[0], self.starts[-1])
        ref, bound, got = ref[rows], bound[rows], got[rows]
        assert bool(torch.isfinite(got).all()), f"{what}: not finite"
        err = (got.double() - ref).abs()
        bad = err > bound
        assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} over the bound, first at "
                                     f"{bad.nonzero()[0].tolist()}, worst error / bound {float((err / bound).max())}")
        if lse is not None:
            ref, bound, got = ref_lse[rows], lse_bound[rows], lse[rows]
            none = torch.isinf(ref)
            assert torch.equal(torch.isinf(got) & (got < 0), none)
            err = torch.where(none, 0, got.double() - ref).abs()
            assert bool((err <= bound).all()), f"{what}: lse off by {float((err / bound).max())} of the bound"


SHAPES = {  # new, past, Hq, Hkv, D, block size, rows before and after
    "one token": ([1], [0], 1, 1, 64, 16, 0, 0),
    "single tokens": ([1] * 9, [0, 14, 15, 16, 127, 128, 900, 2000, 3], 8, 2, 128, 16, 0, 0),
    "drafts": ([5, 0, 3, 9, 1], [300, 7, 0, 1000, 50], 8, 2, 128, 16, 2, 3),
    "prompt": ([300], [0], 4, 1, 128, 16, 0, 0),
    "prompt, narrow": ([700], [0], 4, 2, 64, 16, 0, 0),
    "prompt, wide": ([500], [0], 8, 2, 256, 16, 0, 0),
    "chunk": ([130], [1000], 8, 2, 128, 16, 1, 0),
    "chunk, narrow": ([130], [1111], 8, 2, 64, 16, 0, 1),
    "chunk, wide": ([77], [900], 8, 2, 256, 16, 0, 0),
    "as many heads": ([513, 100], [0, 65], 4, 4, 128, 16, 0, 0),
    "groups of 3": ([200, 31], [40, 3], 6, 2, 128, 16, 0, 0),
    "groups of 5": ([200, 31], [40, 3], 10, 2, 64, 16, 0, 0),
    "groups of 7": ([129, 31], [40, 300], 7, 1, 128, 16, 0, 0),
    "groups of 7, wide": ([129, 31], [40, 300], 7, 1, 256, 16, 0, 0),
    "groups of 16": ([64, 17], [40, 500], 32, 2, 128, 16, 0, 0),
    "group of 100": ([20, 1], [40, 500], 100, 1, 64, 16, 0, 0),
    "group of 300": ([9, 1], [140, 500], 300, 1, 64, 16, 0, 0),
    "group of 130, wide": ([9, 1], [140, 500], 130, 1, 256, 16, 0, 0),
    "head dim 80": ([150, 20], [33, 0], 4, 2, 80, 16, 0, 0),
    "head dim 8": ([150, 20], [33, 0], 4, 2, 8, 16, 0, 0),
    "head dim 192": ([150, 20], [33, 0], 4, 2, 192, 16, 0, 0),
    "block 48": ([150, 20], [333, 0], 4, 2, 128, 48, 0, 0),
    "block 256": ([150, 20, 1], [333, 0, 511], 4, 2, 128, 256, 0, 0),
    "mixed": ([1, 700, 1, 40, 0, 1, 256, 1], [2000, 0, 5, 80, 10, 700, 256, 1300], 8, 2, 128, 16, 3, 5),
    "many": ([(7 * i) % 60 for i in range(70)], [(37 * i) % 300 for i in range(70)], 4, 2, 64, 16, 1, 1),
    "a thousand": ([1] * 1000, [(37 * i) % 300 for i in range(1000)], 2, 1, 64, 16, 0, 0),
}


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", SHAPES)
def test_chunk(name, fp8, window):
    new, past, Hq, Hkv, D, bs, lead, tail = SHAPES[name]
    if fp8 and D % 16:
        pytest.skip("E4M3 caches take head dims of 16")
    b = Chunks(new, past, Hq, Hkv, D, bs, fp8, window, lead, tail, seed=len(name))
    out = torch.full((len(b.q), Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(b.q), Hq), 9.0, device=DEV)
    got, l = b.run(out=out, lse=lse)
    assert got.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
    b.check(out, name, lse)
    for x in (out, lse):
        assert torch.all(x[:lead] == 9) and torch.all(x[len(b.q) - tail:] == 9)  # rows of no sequence


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 128, 129, 500, 5000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_windows(window, D):
    """Windows from a token to more than there are; in between, rows of an item whose first tiles hold none of their keys."""
    b = Chunks([300, 1, 70], [900, 700, 3], 4, 1, D, window=window, seed=window)
    got, lse = b.run(return_lse=True)
    b.check(got, f"window {window}", lse)
    b = Chunks([520], [130], 2, 2, D, window=window, fp8=True, seed=window)  # two streams of one head
    got, lse = b.run(return_lse=True)
    b.check(got, f"window {window} over FP8", lse)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_chunk_long(fp8):
    b = Chunks([2100, 1], [9000, 20000], 8, 2, 128, fp8=fp8, seed=5)
    got, lse = b.run(return_lse=True)
    b.check(got, "long", lse)


def test_chunk_single_tokens_agree_with_decode():
    """Without token_starts one token each; an empty sequence's row is 0 with a sum of nothing.  pd_decode_attn computes the
    same, so the two are within both bounds (decode keeps 16 bits of a weight)."""
    b = Chunks([1] * 7, [0, 15, 16, 500, -1, 3000, 128], 8, 2, 128, seed=3, single=True)
    got, lse = b.run(return_lse=True)
    b.check(got, "single", lse)
    assert not got[4].any() and torch.all(lse[4] == -float("inf"))
    whole = api.decode_attn(b.q, b.kc, b.vc, i32(b.table), i32(b.lens), b.scale, 4)
    assert bool(((got.double() - whole.double()).abs() <= 2 * b.reference()[1]).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("S,longest,Hq,Hkv,D", [(1, 500, 32, 8, 128), (1, 9000, 4, 1, 64), (5, 1500, 8, 2, 256), (16, 1024, 16, 16, 64),
                                                (200, 700, 8, 8, 128), (30, 900, 16, 2, 128), (30, 900, 32, 2, 64), (300, 40, 6, 2, 80),
                                                (9, 300, 34, 2, 128)])
def test_chunk_single_tokens_alone(S, longest, Hq, Hkv, D, fp8):
    """Without lse and window, contiguous and not: whichever kernel takes them."""
    past = np.random.default_rng(S).integers(0, longest, S)
    past[0] = longest - 1
    a = Chunks([1] * S, past.tolist(), Hq, Hkv, D, fp8=fp8, single=True, seed=S)
    a.check(a.run(), "contiguous")
    b = Chunks([1] * S, past.tolist(), Hq, Hkv, D, fp8=fp8, single=True, seed=S, stride=1)
    b.check(b.run(), "strided")
    b.q = b.q.contiguous()
    for scale in (-0.1, 0.0):
        b.scale = scale
        b.check(b.run(), "scale")
    if fp8:
        b.scale, b.k_scale = 0.1, -0.25
        b.check(b.run(), "scale of the keys")


def test_chunk_is_the_prompt_in_pieces():
    """A prompt at once, and in chunks of odd lengths over the same cache: the same tokens, so within both bounds."""
    b = Chunks([900], [0], 8, 2, 128, seed=4)
    whole, bound = b.run(), b.reference()[1]
    at = 0
    for n in (1, 130, 17, 400, 352):
        part = api.chunk_attn(b.q[at:at + n], b.kc, b.vc, i32(b.table), i32([at + n]), b.scale, token_starts=i32([0, n]))
        assert bool(((part.double() - whole[at:at + n].double()).abs() <= 2 * bound[at:at + n]).all())
        at += n


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_rising_scores(D):
    """Keys that meet the query ever better, so that the reference moves at almost every tile, and large scores."""
    for new in (3, 200):
        b = Chunks([new], [2000], 4, 1, D, seed=2, q_scale=3.0, poison=False)
        flat = b.kc[b.rows[0]].flatten(0, 1)
        flat *= torch.linspace(0.1, 4.0, len(flat), device=DEV).to(torch.bfloat16)[:, None, None]
        b.kc[b.rows[0]] = flat.view(-1, 16, 1, D)
        got, lse = b.run(return_lse=True)
        b.check(got, f"rising, {new} tokens", lse)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1.0])
def test_chunk_any_scale(scale, fp8):
    b = Chunks([5, 200], [300, 450], 8, 2, 128, fp8=fp8, seed=3)
    b.q[1] = 0
    b.scale = scale
    got, lse = b.run(return_lse=True)
    b.check(got, f"scale {scale}", lse)


@pytest.mark.parametrize("size", [2.0**-20, 2.0**20])
def test_chunk_fp8_query_sizes(size):
    """Queries far below and above f16's range over an FP8 cache: the scores stay ordinary through the scale."""
    b = Chunks([3, 90], [500, 70], 8, 2, 128, fp8=True, seed=12, q_scale=size)
    b.scale /= size
    b.q[:, 0] = 0
    b.check(b.run(), f"q of {size}")


def test_chunk_strided_queries():
    """q as a slice of a fused projection, and a view with one token's rows."""
    b = Chunks([40, 7], [100, 0], 8, 2, 128, seed=6, stride=5)
    assert b.q.stride(0) == 13 * 128
    got = b.run()
    b.check(got, "strided")
    b.q = b.q.contiguous()
    assert torch.equal(b.run(), got)


def test_chunk_more_new_tokens_than_the_sequence_has():
    b = Chunks([40, 20], [0, 30], 8, 2, 128, seed=7)
    b.lens[0] = 25  # its first fifteen rows see nothing
    got, lse = b.run(return_lse=True)
    assert pd.pd_device_status() == pd.PD_DEV_BAD_CONTEXT_LEN
    b.check(got, "short", lse)
    assert not got[:15].any() and torch.all(lse[:15] == -float("inf"))


def test_chunk_flags():
    b = Chunks([30, 20, 9], [200, 300, 0], 8, 2, 128, seed=9, poison=False)
    good, bound = b.run(), b.reference()[1]
    table = b.table.copy()
    for bad in (-1, b.kc.shape[0], 2**31 - 1, -(2**31)):
        b.table[0, 4] = bad
        got = b.run()
        assert pd.pd_device_status() == pd.PD_DEV_BAD_BLOCK_ID
        assert torch.equal(got[30:], good[30:])
    b.table = table
    keep = b.kc.clone(), b.vc.clone()  # zeros were read there
    b.kc[int(table[0, 4])] = 0
    b.vc[int(table[0, 4])] = 0
    b.check(got, "a block of zeros")
    b.kc, b.vc = keep
    most = b.table.shape[1] * 16
    for s, n in ((0, -3), (1, most + 1)):
        lens = list(b.lens)
        b.lens[s] = n
        b.run()
        assert pd.pd_device_status() == pd.PD_DEV_BAD_CONTEXT_LEN
        b.lens = lens
    for starts, rows in (([-1, 30, 50, 59], (30, 59)), ([0, 30, 50, 60], (0, 50)), ([0, 30, 20, 29], (0, 30))):
        out = torch.full_like(good, 5.0)
        b.run(out=out, token_starts=i32(starts))
        assert pd.pd_device_status() & pd.PD_DEV_BAD_GROUPS
        if starts[2] == 50:  # the other sequences' rows are theirs (cut elsewhere, so each within its bound), the rest as it was
            assert bool(((out.double() - good.double()).abs() <= 2 * bound)[slice(*rows)].all())
            assert torch.all(out[: rows[0]] == 5) and torch.all(out[rows[1]:] == 5)
    assert torch.equal(b.run(), good)


def test_chunk_sequences_that_overlap():
    """2000 sequences in turn of all 256000 rows and of -256000: more units than 32 bits hold.  Nothing is done."""
    S, T, bs, width = 2001, 256000, 256, 4096
    q = torch.zeros(T, 1, 64, dtype=torch.bfloat16, device=DEV)
    kc = torch.zeros(1, bs, 1, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(S, width, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 5.0)
    starts = i32([T * (s % 2) for s in range(S + 1)])
    api.chunk_attn(q, kc, kc.clone(), table, i32([width * bs] * S), 0.1, token_starts=starts, out=out)
    assert pd.pd_device_status() == pd.PD_DEV_BAD_GROUPS
    assert torch.all(out == 5)


def test_chunk_streams_graph_and_workspaces():
    a, b = (Chunks([300, 1, 30], [500, 900, 0], 8, 2, 128, seed=s) for s in (6, 7))
    want = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [x.run(stream=s) for _ in range(4) for x, s in ((a, s1), (b, s2))]
    for s in (s1, s2):
        torch.cuda.current_stream().wait_stream(s)
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2])
    # one captured step on a workspace that an eager call shares
    ws = api.chunk_workspace(331, 8, 2, 128, DEV)
    out = torch.empty_like(a.q)
    lens, starts, table = i32(a.lens), i32(a.starts), i32(a.table)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.chunk_attn(a.q, a.kc, a.vc, table, lens, a.scale, token_starts=starts, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(b.run(ws=ws), want[1])
        assert torch.equal(out, want[0])
    # replayed on other lengths and another division of the rows
    a.starts, a.new, a.lens = [0, 100, 331, 331], [100, 231, 0], [600, 901, 30]
    lens.copy_(i32(a.lens))
    starts.copy_(i32(a.starts))
    g.replay()
    a.check(out, "replayed")


def test_chunk_same_bits_again():
    b = Chunks([64, 3, 1000, 1], [3000, 700, 129, 5000], 32, 8, 128, seed=8)
    first = b.run()
    b.check(first)
    for _ in range(5):
        assert torch.equal(b.run(), first)


def test_chunk_far_in_a_large_cache():
    """Element offsets past 2^32 in the sequences' blocks."""
    nb = 2**32 // (16 * 8 * 256) + 40
    kc = torch.zeros((nb, 16, 8, 256), dtype=torch.bfloat16, device=DEV)
    small = Chunks([70, 1], [5, 300], 16, 8, 256, seed=10, poison=False)
    n = small.kc.shape[0]
    vc = kc.clone()
    kc[nb - n:], vc[nb - n:] = small.kc, small.vc
    assert torch.equal(api.chunk_attn(small.q, kc, vc, i32(small.table + nb - n), i32(small.lens), small.scale, token_starts=i32(small.starts)),
                       small.run())


def test_chunk_nothing():
    b = Chunks([2], [50], 4, 2, 64, seed=11)
    out = api.chunk_attn(b.q[:0], b.kc, b.vc, i32(b.table), i32([0]), b.scale, token_starts=i32([0, 0]),
                         ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert out.shape == (0, 4, 64)
    out = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)  # rows, none of which is a sequence's
    api.chunk_attn(randn(5, 4, 64), b.kc, b.vc, i32(b.table), i32([52]), b.scale, token_starts=i32([2, 2]), out=out)
    assert torch.all(out == 3)


def test_quick_calls_take_what_fits_and_leave_the_rest():
    quick = pd.quick()
    b = Chunks([5, 2], [40, 3], 8, 2, 64, seed=3)
    far = torch.cuda.current_stream().cuda_stream
    lse = torch.empty(7, 8, device=DEV)
    args = [b.q, b.kc, b.vc, i32(b.table), i32(b.lens), i32(b.starts), b.scale, 0, None, None, None, 1.0, 1.0]
    want, want_lse = b.run(stream=far, return_lse=True)
    assert torch.equal(quick.chunk_attn(*args), want)
    assert torch.equal(quick.chunk_attn(*args[:9], lse, *args[10:]), want) and torch.equal(lse, want_lse)
    for i, bad in ((0, b.q.float()), (0, b.q[0]), (0, b.q.transpose(0, 1)), (1, b.kc[1:]), (2, b.vc.cpu()), (3, args[3][:1]), (4, args[4].long()),
                   (5, args[5][:1]), (5, None), (6, "a"), (7, -1), (7, 2**31), (8, want[:1]), (9, lse[:1]), (9, want_lse.double()), (10, want),
                   (10, torch.empty(16, dtype=torch.uint8, device=DEV)), (11, None)):
        assert quick.chunk_attn(*args[:i], bad, *args[i + 1:]) is NotImplemented, (i, bad)
    assert quick.chunk_attn(*args[:-1]) is NotImplemented


@pytest.mark.parametrize("lse", [False, True])
def test_chunk_of_70000_sequences(lse):
    """One token each, behind none or one: its own value, or between the two."""
    S = 70000
    q, kc, vc = randn(S, 1, 64, seed=1), randn(S // 8, 16, 1, 64, seed=2), randn(S // 8, 16, 1, 64, seed=3)
    table = (torch.arange(S, device=DEV, dtype=torch.int32) // 8)[:, None].contiguous()
    lens = (torch.arange(S, device=DEV, dtype=torch.int32) % 3)
    got = api.chunk_attn(q, kc, vc, table, lens, 0.125, return_lse=lse)
    out = got[0] if lse else got
    k, v = kc[table[:, 0].long(), :2, 0].double(), vc[table[:, 0].long(), :2, 0].double()
    z = (q.double() @ k.transpose(1, 2))[:, 0] * 0.125
    z[lens == 1, 1] = -float("inf")
    w = torch.softmax(z, -1) * (lens > 0)[:, None]
    ref, size = (w[:, :, None] * v).sum(1), (w[:, :, None] * v.abs()).sum(1)
    # weights and the output rounded to BF16 (2^-8 each), scores off by 72 additions of products (2^-24 each) of at most 2^8
    assert bool(((out[:, 0].double() - ref).abs() <= 2.0**-8 * (size + ref.abs()) + 2.0**-9 * size + 2.0**-100).all())
    assert not bool(out[lens == 0].any())


def test_chunk_windows_past_31_bits():
    a = Chunks([40], [300], 4, 2, 64, window=0)
    want = a.run()
    for window in (2**31 - 1, 2**31, 2**32 + 5, 2**40):
        a.window = window
        assert torch.equal(a.run(), want)
    for window in (-1, -(2**32) + 5):
        a.window = window
        with pytest.raises(pd.PdError):
            a.run()
