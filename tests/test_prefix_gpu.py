"""GPU tests of decode attention behind shared prefixes, against the definition in 64 bits."""

import math

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


class Batch:
    """sizes: sequences of each group (lead and tail: of none); every cache slot of no live token holds NaN."""

    def __init__(self, sizes, plens, lens, Hq, Hkv, D, bs=16, fp8=False, lead=0, tail=0, seed=0, q_scale=1.0, poison=True):
        rng = np.random.default_rng(seed)
        S = lead + sum(sizes) + tail
        assert len(lens) == S and len(plens) == len(sizes)
        self.plens, self.lens, self.D, self.bs, self.fp8 = list(plens), list(lens), D, bs, fp8
        self.starts = [lead, *(lead + np.cumsum(sizes)).tolist()]
        need = [-(-n // bs) for n in self.plens + self.lens]
        pool = sum(need) + 2
        ids, at = rng.permutation(pool), 0
        self.rows = []
        for n in need:
            self.rows.append(ids[at:at + n].tolist())
            at += n
        G = len(sizes)
        self.ptable = self.padded(self.rows[:G])
        self.table = self.padded(self.rows[G:])
        self.q = randn(S, Hq, D, seed=seed + 1, scale=q_scale)
        self.kc, self.vc = randn(pool, bs, Hkv, D, seed=seed + 2), randn(pool, bs, Hkv, D, seed=seed + 3)
        if poison:
            dead = torch.ones((pool, bs), dtype=torch.bool, device=DEV)
            for row, n in zip(self.rows, self.plens + self.lens):
                for j, b in enumerate(row):
                    dead[b, : min(bs, n - j * bs)] = False
            if not fp8:
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

    @staticmethod
    def padded(rows):
        w = max(1, max(len(r) for r in rows))
        return np.array([r + [-7] * (w - len(r)) for r in rows])  # entries past a length are never read

    def run(self, splits=3, **more):
        more = {"group_starts": i32(self.starts), **more}
        return api.decode_attn_prefix(self.q, self.kc, self.vc, i32(self.ptable), i32(self.plens), more.pop("group_starts"),
                                      i32(self.table), i32(self.lens), self.scale, splits, k_scale=self.k_scale,
                                      v_scale=self.v_scale, **more)

    def value(self, cache, scale):
        return cache.double() if not self.fp8 else cache.view(torch.float8_e4m3fn).double() * scale

    def tokens(self, cache, row, n, scale):
        if n == 0:
            return torch.zeros((0, *cache.shape[2:]), dtype=torch.float64, device=DEV)
        return self.value(cache[torch.tensor(row[: -(-n // self.bs)], device=DEV)], scale).flatten(0, 1)[:n]

    def reference(self):
        """(out, the error bound), both [S, Hq, D] in 64 bits.

        With weights w (sum 1) and A = sum w |v|: the prefix's weights are rounded to 8 bits (BF16: half a step, 2^-8;
        f16: 2^-11), own weights to 16 (2^-16); a score's FP32 sum of D products is off by at most (D + 8) 2^-24 of
        sum |q k| scale, and by its factor of log2 e and the exponential's 2^-21 beside it, on the weight and on their
        sum; the output rounds to BF16 (2^-8)."""
        S, Hq, D = self.q.shape
        Hkv = self.kc.shape[2]
        out = torch.zeros((S, Hq, D), dtype=torch.float64, device=DEV)
        bound = torch.zeros_like(out)
        G = len(self.plens)
        pre = [tuple(self.tokens(c, self.rows[g], self.plens[g], s) for c, s in ((self.kc, self.k_scale), (self.vc, self.v_scale)))
               for g in range(G)]
        none = tuple(x[:0] for x in pre[0])
        for s in range(S):
            g = next((g for g in range(G) if self.starts[g] <= s < self.starts[g + 1]), None)
            pk, pv = none if g is None else pre[g]
            k = torch.cat([pk, self.tokens(self.kc, self.rows[G + s], self.lens[s], self.k_scale)])
            v = torch.cat([pv, self.tokens(self.vc, self.rows[G + s], self.lens[s], self.v_scale)])
            if not len(k):
                continue
            q = self.q[s].double().view(Hkv, Hq // Hkv, D)
            k, v = k.permute(1, 0, 2), v.permute(1, 0, 2)
            w = torch.softmax(q @ k.transpose(1, 2) * self.scale, -1)
            size = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(self.scale)
            ref = w @ v
            n = len(pk)
            a_pre = w[..., :n] @ v[:, :n].abs()
            a_all = w @ v.abs()
            weight = 2.0 * ((D + 8) * 2.0**-24 * size + 2.0**-21) + 2.0**-16
            out[s] = ref.reshape(Hq, D)
            bound[s] = (1.02 * ((2.0**-11 if self.fp8 else 2.0**-8) * a_pre + weight * a_all) + 2.0**-8 * ref.abs()
                        + 2.0**-100).reshape(Hq, D)
        return out, bound

    def check(self, got, what=""):
        ref, bound = self.reference()
        err = (got.double() - ref).abs()
        assert bool(torch.isfinite(got).all()), f"{what}: not finite"
        bad = err > bound
        assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} over the bound, first at "
                                     f"{bad.nonzero()[0].tolist()}, worst error / bound {float((err / bound).max())}")


SHAPES = {  # sizes, prefix lengths, own lengths, Hq, Hkv, D, block size, sequences before and after
    "one token": ([1], [1], [0], 1, 1, 64, 16, 0, 0),
    "one tile": ([2], [100], [0, 5], 4, 1, 64, 16, 0, 0),
    "tile less one": ([3], [127], [1, 0, 40], 8, 2, 128, 16, 0, 0),
    "tile": ([3], [128], [1, 0, 40], 8, 2, 128, 16, 0, 0),
    "tile and one": ([3], [129], [1, 0, 40], 8, 2, 128, 16, 0, 0),
    "three tiles": ([5], [384], [16] * 5, 4, 4, 128, 16, 0, 0),
    "129 rows": ([43], [300], [3] * 43, 3, 1, 128, 16, 0, 0),
    "blocks of rows": ([40], [333], list(range(40)), 16, 2, 128, 16, 0, 0),
    "blocks of rows, one tile": ([40], [90], [0] * 40, 16, 2, 64, 16, 0, 0),
    "long": ([6], [5003], [100, 0, 17, 513, 1, 0], 8, 2, 128, 16, 0, 0),
    "wide": ([6], [1000], [100, 0, 17, 513, 1, 0], 16, 2, 256, 16, 0, 0),
    "wide, one tile": ([2], [64], [0, 3], 8, 1, 256, 16, 0, 0),
    "wide, blocks of rows": ([40], [200], [2] * 40, 16, 2, 256, 16, 0, 0),
    "narrow": ([4], [700], [0, 9, 70, 300], 4, 2, 64, 16, 0, 0),
    "head dim 80": ([4], [260], [0, 9, 70, 300], 14, 2, 80, 16, 0, 0),
    "head dim 8": ([4], [260], [0, 9, 70, 300], 4, 2, 8, 16, 0, 0),
    "head dim 136": ([4], [260], [0, 9, 70, 300], 4, 2, 136, 16, 0, 0),
    "block 48": ([4], [1000], [0, 9, 70, 300], 4, 2, 128, 48, 0, 0),
    "block 256": ([4], [1000], [0, 9, 70, 300], 4, 2, 64, 256, 0, 0),
    "groups": ([0, 3, 0, 5, 1], [10, 0, 50, 700, 2000], [5] * 11, 8, 2, 128, 16, 1, 1),
    "no prefix": ([2, 2], [0, 0], [0, 7, 1, 300], 8, 2, 128, 16, 0, 0),
    "nothing": ([2], [0], [0, 0], 8, 2, 128, 16, 0, 0),
    "uneven groups": ([70, 1, 30], [500, 3000, 17], [4] * 101, 8, 1, 128, 16, 0, 0),
    "group of 16": ([20], [400], [30] * 20, 32, 2, 64, 16, 0, 0),
    "many groups": ([2] * 70, [(37 * i) % 300 for i in range(70)], [3] * 140, 4, 2, 64, 16, 0, 0),
    "heads": ([9], [600], [20] * 9, 32, 32, 128, 16, 0, 0),
    # items of one or two tiles that end inside a cache block, one after another, their rows in halves
    "short halves": ([33] * 8, [1, 127, 90, 17, 130, 3, 65, 255], [1] * 264, 64, 8, 80, 80, 0, 0),
    "short halves, narrow": ([33] * 8, [1, 127, 90, 17, 130, 3, 65, 255], [1] * 264, 64, 8, 64, 16, 0, 0),
    "short halves, wide": ([17] * 8, [1, 63, 45, 17, 66, 3, 65, 127], [1] * 136, 64, 8, 256, 32, 0, 0),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", SHAPES)
def test_prefix(name, fp8):
    sizes, plens, lens, Hq, Hkv, D, bs, lead, tail = SHAPES[name]
    if fp8 and D % 16:
        pytest.skip("E4M3 caches take head dims of 16")
    b = Batch(sizes, plens, lens, Hq, Hkv, D, bs, fp8, lead=lead, tail=tail, seed=len(name))
    b.check(b.run(), name)


@pytest.mark.parametrize("size", [2.0**-20, 1.0, 2.0**20])
def test_prefix_fp8_query_sizes(size):
    """Queries far below and above f16's range over an FP8 cache: the scores stay ordinary through the scale."""
    for rows in (3, 50):
        b = Batch([rows], [500], [9] * rows, 8, 2, 128, fp8=True, seed=12, q_scale=size)
        b.scale /= size
        b.q[:, 0] = 0
        b.check(b.run(), f"q of {size}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_rising_scores(D):
    """Keys that meet the query ever better, so that the reference moves at almost every tile, and large scores."""
    for rows in (4, 50):
        b = Batch([rows], [2000], [33] * rows, 4, 1, D, seed=2, q_scale=3.0, poison=False)
        flat = torch.cat([b.kc[r] for r in b.rows[0]]).clone()
        flat *= torch.linspace(0.1, 4.0, len(flat), device=DEV).to(torch.bfloat16)[:, None, None]
        for j, r in enumerate(b.rows[0]):
            b.kc[r] = flat[j * 16:(j + 1) * 16]
        b.check(b.run(), f"rising, {rows} sequences")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1.0])
def test_prefix_any_scale(scale, fp8):
    b = Batch([5, 40], [300, 450], [20] * 45, 8, 2, 128, fp8=fp8, seed=3)
    b.q[1] = 0
    b.scale = scale
    b.check(b.run(), f"scale {scale}")


def test_prefix_whole_batch_and_splits():
    b = Batch([7], [900], [0, 1, 255, 256, 257, 900, 3000], 8, 2, 128, seed=4)
    for splits in (1, 2, 16):
        b.check(b.run(splits), f"{splits} splits")
        assert torch.equal(b.run(splits, group_starts=None), b.run(splits))  # one group by default, the same bits again


def test_prefix_agrees_with_whole_tables():
    """pd_decode_attn over tables that begin with the prefix's blocks: the same tokens, so within both bounds."""
    b = Batch([5], [640], [1, 30, 64, 500, 7], 8, 2, 128, seed=5)
    n = 640 // 16
    table = np.concatenate([np.repeat(b.ptable[:, :n], 5, 0), b.table], 1)
    whole = api.decode_attn(b.q, b.kc, b.vc, i32(table), i32([640 + x for x in b.lens]), b.scale, 4)
    _, bound = b.reference()
    assert bool(((b.run().double() - whole.double()).abs() <= 2 * bound).all())


def test_prefix_streams_graph_and_workspaces():
    a, b = (Batch([30], [1500], list(range(30)), 8, 2, 128, seed=s) for s in (6, 7))
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
    ws = api.prefix_workspace(30, 1, 8, 2, 128, 3, DEV)
    out = torch.empty_like(a.q)
    args = (a.kc, a.vc, i32(a.ptable), i32(a.plens), i32(a.starts), i32(a.table))
    lens = i32(a.lens)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.decode_attn_prefix(a.q, *args, lens, a.scale, 3, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(b.run(ws=ws), want[1])
        assert torch.equal(out, want[0])
    a.lens = [0] * 30
    lens.zero_()
    g.replay()
    a.check(out, "replayed on other lengths")


def test_prefix_same_bits_again():
    b = Batch([64, 3, 20], [3000, 700, 129], [9] * 87, 32, 8, 128, seed=8)
    first = b.run()
    b.check(first)
    for _ in range(5):
        assert torch.equal(b.run(), first)


def test_prefix_flags():
    b = Batch([3, 2], [200, 300], [5] * 5, 8, 2, 128, seed=9, poison=False)
    good = b.run()
    table = b.ptable.copy()
    for bad in (-1, b.kc.shape[0], 2**31 - 1, -(2**31)):
        b.ptable[0, 4] = bad
        b.run()
        assert pd.pd_device_status() == pd.PD_DEV_BAD_BLOCK_ID
    # zeros were read there: 16 keys and values of the first prefix
    got = b.run()
    assert pd.pd_device_status() == pd.PD_DEV_BAD_BLOCK_ID
    b.ptable = table
    keep = b.kc.clone(), b.vc.clone()
    b.kc[int(table[0, 4])] = 0
    b.vc[int(table[0, 4])] = 0
    b.check(got, "a block of zeros")
    b.kc, b.vc = keep
    most = b.ptable.shape[1] * 16
    for g, n in ((0, -3), (1, most + 1)):
        plens = list(b.plens)
        b.plens[g] = n
        got = b.run()
        assert pd.pd_device_status() & pd.PD_DEV_BAD_CONTEXT_LEN
        b.plens = plens
    for starts in ([-1, 3, 5], [0, 4, 3], [0, 3, 6], [5, 0, 5]):
        got = b.run(group_starts=i32(starts))
        assert pd.pd_device_status() == pd.PD_DEV_BAD_GROUPS
        plens, b.plens = b.plens, [0, 0]
        rows, b.rows = b.rows, [[], []] + b.rows[2:]
        b.check(got, "own tokens alone")
        b.plens, b.rows = plens, rows
    assert torch.equal(b.run(), good)


def test_prefix_far_in_a_large_cache():
    """Element offsets past 2^32 in the prefix's blocks and the sequences' own."""
    nb = 2**32 // (16 * 8 * 256) + 40
    kc = torch.zeros((nb, 16, 8, 256), dtype=torch.bfloat16, device=DEV)
    small = Batch([3], [70], [5, 0, 20], 16, 8, 256, seed=10, poison=False)
    n = small.kc.shape[0]
    vc = kc.clone()
    kc[nb - n:], vc[nb - n:] = small.kc, small.vc
    args = (i32(small.ptable + nb - n), i32(small.plens), None, i32(small.table + nb - n), i32(small.lens), small.scale, 2)
    assert torch.equal(api.decode_attn_prefix(small.q, kc, vc, *args), small.run(2))


def test_prefix_empty_batch():
    b = Batch([2], [50], [1, 1], 4, 2, 64, seed=11)
    out = api.decode_attn_prefix(b.q[:0], b.kc, b.vc, i32(b.ptable), i32(b.plens), None, i32(b.table)[:0], i32(b.lens)[:0],
                                 b.scale, 2, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("plens", [[128, 64], [130, 77]], ids=["whole blocks", "ragged"])
def test_steps_of_a_batch_in_one_graph(plens, fp8):
    """Steps of a served batch: the new tokens rotated and appended behind each sequence's own, then the attention over
    the group's prefix and those, all in one captured graph that counts the lengths itself.  Where a prefix ends with a
    block, the append takes tables that begin with its blocks; else the tokens are rotated first, by their positions."""
    steps, Hq, Hkv, D = 3, 8, 2, 64
    lens = [0, 15, 16, 31, 5, 200, 47]
    whole = plens[0] % 16 == 0
    b = Batch([3, 2], plens, [n + steps for n in lens], Hq, Hkv, D, fp8=fp8, lead=1, tail=1, seed=9)
    S = len(lens)
    rope = pd.Rope(D, base=500000.0, layout="interleaved")
    groups = [next((g for g in range(2) if b.starts[g] <= s < b.starts[g + 1]), None) for s in range(S)]
    spans = i32([0 if g is None else plens[g] for g in groups])
    tables = i32(b.padded([([] if g is None else b.rows[g]) + b.rows[2 + s] for s, g in enumerate(groups)]))
    own, qkv = i32(lens), torch.empty(S, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    ptable, plens, starts, table = i32(b.ptable), i32(b.plens), i32(b.starts), i32(b.table)
    ws = api.prefix_workspace(S, 2, Hq, Hkv, D, 4, DEV)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)

    def step():
        own.add_(1)
        kr = api.rope(rope, k, own + spans - 1)
        if whole:
            qr = api.append_kv(rope, q, k, v, b.kc, b.vc, tables, own + spans, k_scale=b.k_scale, v_scale=b.v_scale)
        else:
            qr = api.rope(rope, q, own + spans - 1)
            api.append_kv(None, None, kr, v, b.kc, b.vc, table, own, k_scale=b.k_scale, v_scale=b.v_scale)
        return qr, kr, api.decode_attn_prefix(qr, b.kc, b.vc, ptable, plens, starts, table, own, b.scale, 4, ws=ws, k_scale=b.k_scale,
                                              v_scale=b.v_scale)

    kept = b.kc.clone(), b.vc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qkv.zero_()
    with torch.cuda.stream(side):
        step()  # (everything is loaded before the capture)
    torch.cuda.synchronize()
    own.copy_(i32(lens))
    b.kc.copy_(kept[0])
    b.vc.copy_(kept[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qr, kr, out = step()
    for n in range(1, steps + 1):
        qkv.copy_(randn(S, Hq + 2 * Hkv, D, seed=20 + n))
        graph.replay()
        torch.cuda.synchronize()
        assert own.tolist() == [m + n for m in lens] and torch.equal(qr, api.rope(rope, q, own + spans - 1))
        for s in range(S):
            i = lens[s] + n - 1
            block, slot = b.rows[2 + s][i // 16], i % 16
            if fp8:
                # (the fused append rounds once: off by half a step of E4M3, 2^-4, or of its subnormals, from the rotation,
                # and that from the rounded one by half a step of BF16)
                got, want = b.value(b.kc[block, slot], b.k_scale), kr[s].double()
                assert torch.all((got - want).abs() <= want.abs() * (2.0**-4 * (1 + 2.0**-8) + 2.0**-8) + 0.5 * 2.0**-10)
                assert torch.equal(b.vc[block, slot], (v[s].float() * 4).to(torch.float8_e4m3fn).view(torch.uint8))
            else:
                assert torch.equal(b.kc[block, slot], kr[s]) and torch.equal(b.vc[block, slot], v[s])
        b.q, b.lens = qr, [m + n for m in lens]
        ref, bound = b.reference()
        assert torch.all((out.double() - ref).abs() <= bound)


def test_quick_calls_take_what_fits_and_leave_the_rest():
    """The CPython module answers calls that are as it needs them, with the bits of the other way, and declines others."""
    quick = pd.quick()
    b = Batch([2], [40], [3, 17], 8, 2, 64, seed=3)
    rope = pd.Rope(64)
    x, pos = randn(2, 8, 64, seed=1), i32([5, 9])
    far = torch.cuda.current_stream().cuda_stream
    assert torch.equal(quick.rope(rope.handle, 64, x, pos, None, False), api.rope(rope, x, pos, stream=far))
    for bad in ((x.float(), pos, None, 0), (x, pos.long(), None, 0), (x, pos[:1], None, 0), (x, pos.cpu(), None, 0), (x[0], pos, None, 0),
                (x, pos, x[:1], 0), (x, pos, None, 2), (x.cpu(), pos, None, 0), ("x", pos, None, 0), (x, None, None, 0),
                (x.transpose(1, 2), pos, None, 0)):
        assert quick.rope(rope.handle, 64, *bad) is NotImplemented
    assert quick.rope(rope.handle, 128, x, pos, None, 0) is NotImplemented
    args = [b.q, b.kc, b.vc, i32(b.ptable), i32(b.plens), i32(b.starts), i32(b.table), i32(b.lens), b.scale, 2, None, None, 1.0, 1.0]
    out = quick.decode_attn_prefix(*args)
    assert torch.equal(out, b.run(splits=2, stream=far))
    for i, bad in ((0, b.q.float()), (0, b.q[:1]), (1, b.kc[1:]), (1, b.kc.transpose(0, 1)), (2, b.vc.cpu()), (3, args[3][:, ::2]), (4, args[4].long()),
                   (5, args[5][:1]), (6, args[6][0]), (7, None), (8, "a"), (9, 0), (9, 5000), (10, out[:1]), (11, out), (12, None)):
        assert quick.decode_attn_prefix(*args[:i], bad, *args[i + 1:]) is NotImplemented, (i, bad)
    assert quick.decode_attn_prefix(*args[:-1]) is NotImplemented
    k, v = randn(2, 2, 64, seed=2), randn(2, 2, 64, seed=4)
    more = [rope.handle, 64, x, k, v, b.kc, b.vc, i32(b.table), i32(b.lens), None, None, 1.0, 1.0]
    assert torch.equal(quick.append_kv(*more), api.rope(rope, x, i32([2, 16])))
    for i, bad in ((1, 128), (2, None), (2, x[:1]), (3, k[:, :1]), (4, v.float()), (5, b.vc[1:]), (7, more[7][:1]), (8, more[8].cpu()), (9, pos), (10, x[:1]),
                   (11, "a")):
        assert quick.append_kv(*more[:i], bad, *more[i + 1:]) is NotImplemented, (i, bad)


def test_workspaces_elsewhere_are_refused():
    b = Batch([2], [40], [3, 17], 8, 2, 64, seed=3)
    n = api.prefix_workspace(2, 1, 8, 2, 64, 3, DEV).numel()
    far = torch.cuda.current_stream().cuda_stream
    for stream in (None, far):
        for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
            with pytest.raises(ValueError, match="ws"):
                b.run(ws=ws, stream=stream)
        b.check(b.run(ws=torch.empty(n // 4 + 1, dtype=torch.float32, device=DEV), stream=stream))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_padded_batch_over_recycled_memory(D, fp8):
    """Sequences of length 0 pad the batch: the append gives their rows nothing, so a q_out that it makes holds there what
    its memory held, NaN here.  No other row's attention, behind a prefix or not, takes a bit of it."""
    Hq, Hkv = 8, 2
    for sizes in ([7], [70], [3, 4]):
        S = sum(sizes)
        lens = [0 if s % 3 == 1 else 1 + 40 * s % 290 for s in range(S)]
        b = Batch(sizes, [333, 50][:len(sizes)], lens, Hq, Hkv, D, fp8=fp8, seed=13)
        k, v = randn(S, Hkv, D, seed=3), randn(S, Hkv, D, seed=4)
        table, own = i32(np.maximum(b.table, 0)), i32(lens)
        args = (b.q, k, v, b.kc, b.vc, table, own)
        more = dict(k_scale=b.k_scale, v_scale=b.v_scale)
        zeroed = api.append_kv(None, *args, q_out=torch.zeros_like(b.q), **more)
        pad = [s for s in range(S) if not lens[s]]
        live = [s for s in range(S) if lens[s]]
        assert not zeroed[pad].any() and torch.equal(zeroed[live], b.q[live])
        for stream in (None, torch.cuda.current_stream()):
            old = [torch.full_like(b.q, float("nan")) for _ in range(64)]
            del old
            q = api.append_kv(None, *args, stream=stream, **more)
            assert torch.equal(q[live], b.q[live])
            q[pad] = float("nan")  # (whatever memory it was)
            for call in (lambda q: api.decode_attn_prefix(q, b.kc, b.vc, i32(b.ptable), i32(b.plens), i32(b.starts), table, own, b.scale, 3,
                                                          **more),
                         lambda q: api.decode_attn(q, b.kc, b.vc, table, own, b.scale, 2, **more)):
                assert torch.equal(call(q)[live], call(zeroed)[live])


def test_prefix_fp8_small_weights():
    """f16 weights below 2^-14 are off by up to half of 2^-24, against a reference m that a raise leaves up to 1 above the
    largest score: up to 2^-24 of the largest weight.  One key in tile 1 lifts m from 0 to 16 and scores 15.0625; the one
    key whose value is not 0 scores -7.4140625, 1.501 units of 2^-24 below 2^16, which round to 2.  (Scores in powers of
    two, and exact: keys of two terms.)"""
    b = Batch([40], [8192], [0] * 40, 8, 1, 64, fp8=True, seed=1, poison=False)
    b.k_scale = b.v_scale = 1.0
    b.scale = math.log(2)
    b.q.zero_()
    b.q[:, :, :2] = 1
    k, v = torch.zeros(8192, 64, device=DEV), torch.zeros(8192, 64, device=DEV)
    k[128:, 0] = -16
    k[130, 0], k[130, 1] = 15, 0.0625
    k[200, 0], k[200, 1] = -7.5, 0.0859375
    v[200] = 448
    for cache, x in ((b.kc, k), (b.vc, v)):
        codes = x.to(torch.float8_e4m3fn)
        assert torch.equal(codes.float(), x)
        cache[torch.tensor(b.rows[0], device=DEV)] = codes.view(torch.uint8).view(-1, 16, 1, 64)
    got = b.run(splits=1).double()
    w = torch.exp2(k[:, :2].double().sum(1))
    ref = float(w[200] / w.sum() * 448)
    assert bool(torch.isfinite(got).all())
    # (and the output's rounding, 2^-8 of up to 2 / 1.5 of ref, beside which the FP32 sums are nothing)
    assert float((got - ref).abs().max()) <= 2.0**-24 * float(w.max() / w.sum()) * 448 + 2.0**-8 * 1.5 * ref  # found: 2^-24.06 of the largest
