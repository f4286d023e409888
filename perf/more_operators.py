"""Prompt and training operators around the paged cache, as they are measured.

Three operators that stand beside the decode step, the rotation and the append:

* chunk:  attention of new tokens (prompt chunks, drafts, single tokens) over a paged K/V cache that holds them already;
* norm:   each head's RMS norm with the position rotation in the same pass, forward alone or with its gradients;
* append: the same norm and rotation of queries and keys on their way into the paged cache.

`run` computes them in plain torch operations where `own` is false, and with the library's calls where it is true.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 16  # tokens of a cache block
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------


def listed():
    return [
        # the smallest call: one short prompt, a single KV head
        dict(name="chunk_small", op="chunk", seqs=1, new_min=100, new_max=100, past_min=0, past_max=0, q_heads=4, kv_heads=1,
             head_dim=64, cache="bf16", window=0, lse=False),
        # a step of single tokens that also wants the logarithms of the sums
        dict(name="chunk_tokens", op="chunk", seqs=64, new_min=1, new_max=1, past_min=200, past_max=4096, q_heads=32, kv_heads=8,
             head_dim=128, cache="bf16", window=0, lse=True),
        # drafts of five tokens checked at once, wide heads
        dict(name="chunk_drafts", op="chunk", seqs=48, new_min=5, new_max=5, past_min=507, past_max=4091, q_heads=16, kv_heads=2,
             head_dim=256, cache="bf16", window=0, lse=False),
        # one long prompt
        dict(name="chunk_prompt", op="chunk", seqs=1, new_min=8192, new_max=8192, past_min=0, past_max=0, q_heads=32, kv_heads=8,
             head_dim=128, cache="bf16", window=0, lse=False),
        # a mixed step: prompts of up to 2731 tokens beside single tokens
        dict(name="chunk_mixed", op="chunk", seqs=24, new_min=1, new_max=2731, past_min=0, past_max=2048, q_heads=32, kv_heads=8,
             head_dim=128, cache="bf16", window=0, lse=False),
        # the last chunk of a document: 2048 tokens over 32768
        dict(name="chunk_document", op="chunk", seqs=1, new_min=2048, new_max=2048, past_min=32768, past_max=32768, q_heads=32,
             kv_heads=8, head_dim=128, cache="bf16", window=0, lse=False),
        # prompt chunks of odd lengths over an FP8 cache
        dict(name="chunk_fp8", op="chunk", seqs=15, new_min=33, new_max=1025, past_min=0, past_max=4097, q_heads=32, kv_heads=8,
             head_dim=128, cache="e4m3", window=0, lse=False),
        # a layer with a sliding window, as many KV heads as query heads
        dict(name="chunk_window", op="chunk", seqs=3, new_min=1500, new_max=4001, past_min=0, past_max=9000, q_heads=16, kv_heads=16,
             head_dim=64, cache="bf16", window=1024, lse=False),
        # one decode step of 64 sequences: the queries of a layer that reads another layer's cache
        dict(name="norm_decode", op="norm", tokens=64, heads=32, row_heads=48, head_dim=128, rot=128, layout="half", scaling="none",
             base=10000.0, factor=1.0, original=32768, max_pos=32768, offset=0.0, train=False),
        # a training step's query heads, forward and backward
        dict(name="norm_train", op="norm", tokens=16384, heads=32, row_heads=32, head_dim=128, rot=128, layout="half", scaling="none",
             base=500000.0, factor=1.0, original=8192, max_pos=8192, offset=0.0, train=True),
        # one decode step of a large batch into an FP8 cache
        dict(name="append_norm_decode", op="append", seqs=256, new_min=1, new_max=1, past_min=0, past_max=2048, q_heads=32, kv_heads=8,
             head_dim=128, rot=128, layout="half", scaling="banded", base=500000.0, factor=8.0, original=8192, offset=0.0, cache="e4m3"),
        # prompt chunks of wide heads, a quarter of each turned by neighbouring pairs, weights kept as their distance from one
        dict(name="append_norm_prompts", op="append", seqs=24, new_min=1, new_max=2731, past_min=0, past_max=2048, q_heads=16, kv_heads=2,
             head_dim=256, rot=64, layout="interleaved", scaling="yarn", base=10000.0, factor=16.0, original=4096, offset=1.0,
             cache="bf16"),
    ]


def _log_int(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def _draw_rotation(rng, head_dim):
    rot = head_dim if rng.random() < 0.5 else 2 * rng.randint(2, head_dim // 2)
    scaling = rng.choice(["none", "linear", "ntk", "banded", "yarn"])
    return dict(rot=rot, layout=rng.choice(["half", "interleaved"]), scaling=scaling, base=rng.choice([10000.0, 500000.0]),
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 16.0]), original=rng.choice([4096, 8192]),
                offset=rng.choice([0.0, 1.0]))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "norm", "append"])
    if op == "norm":
        D = rng.choice([64, 80, 128, 192, 256])
        heads = rng.randint(1, 40)
        most = 16384 * 32 * 128 // (heads * D)
        return dict(op=op, tokens=_log_int(rng, 1, min(32768, most)), heads=heads, row_heads=heads + rng.choice([0, 1, 8]), head_dim=D,
                    max_pos=rng.choice([4096, 32768, 131072]), train=rng.random() < 0.6, **_draw_rotation(rng, D))
    Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 80, 128, 256])
    while Hkv * (G + 2) * D > 48 * 128:
        G = max(1, G // 2)
        Hkv = max(1, Hkv // 2)
    cache = rng.choice(["bf16", "e4m3"])
    if op == "append":
        one = rng.random() < 0.4
        return dict(op=op, seqs=_log_int(rng, 1, 256) if one else _log_int(rng, 1, 24), new_min=1, new_max=1 if one else _log_int(rng, 2, 2700),
                    past_min=0, past_max=_log_int(rng, 1, 2048), q_heads=Hkv * G, kv_heads=Hkv, head_dim=D, cache=cache,
                    **_draw_rotation(rng, D))
    kind = rng.choice(["tokens", "drafts", "chunks", "prompts"])
    seqs = {"tokens": 64, "drafts": 48, "chunks": 24, "prompts": 4}[kind]
    seqs = _log_int(rng, 1, seqs)
    low, high = {"tokens": (1, 1), "drafts": (2, 9), "chunks": (17, 1024), "prompts": (513, 8192)}[kind]
    new = _log_int(rng, low, max(low, high // (1 if kind != "prompts" else seqs)))
    past = _log_int(rng, 1, {"tokens": 8192, "drafts": 8192, "chunks": 16384 // seqs, "prompts": 2048}[kind])
    return dict(op=op, seqs=seqs, new_min=new if seqs == 1 else rng.randint(1, new), new_max=new, past_min=past if seqs == 1 else
                rng.randint(0, past), past_max=past, q_heads=Hkv * G, kv_heads=Hkv, head_dim=D, cache=cache,
                window=_log_int(rng, 33, 4096) if rng.random() < 0.3 else 0, lse=rng.random() < 0.3)


def _spread(low, high, n):
    """n whole numbers evenly from low to high, the same for every seed."""
    return [low + (high - low) * i // max(1, n - 1) for i in range(n)]


def _lens(case):
    """(new tokens, tokens with them) of each sequence."""
    new = _spread(case["new_min"], case["new_max"], case["seqs"])
    past = _spread(case["past_min"], case["past_max"], case["seqs"])[::-1]
    return new, [n + p for n, p in zip(new, past)]


def work(case):
    D = case["head_dim"]
    if case["op"] == "norm":
        n = case["tokens"] * case["heads"] * D
        if case["train"]:  # x, the gradient, y and x's gradient
            return {"bytes": 8 * n + 4 * case["tokens"] + 4 * D, "flops": 16 * n + 12 * case["tokens"] * case["heads"] * case["rot"] / 2}
        return {"bytes": 4 * n + 4 * case["tokens"] + 2 * D, "flops": 4 * n + 6 * case["tokens"] * case["heads"] * case["rot"] / 2}
    Hq, Hkv = case["q_heads"], case["kv_heads"]
    elem = 1 if case["cache"] == "e4m3" else 2
    new, lens = _lens(case)
    t = sum(new)
    if case["op"] == "append":
        return {"bytes": t * D * (2 * (Hq + 2 * Hkv) + 2 * Hq + 2 * elem * Hkv) + 12 * case["seqs"] + 4 * D,
                "flops": t * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    pairs, live = 0, 0
    for n, m in zip(new, lens):
        w = case["window"] or m
        live += m - max(0, m - n + 1 - w)
        whole = min(n, max(0, w - (m - n) - 1))  # tokens that see less than the window
        pairs += sum(range(m - n + 1, m - n + 1 + whole)) + (n - whole) * w if case["window"] else n * (m - n) + n * (n + 1) // 2
    return {"bytes": 2 * elem * Hkv * D * live + 4 * t * Hq * D + (4 * t * Hq if case["lse"] else 0) + live // 4 + 8 * case["seqs"],
            "flops": 4 * Hq * D * pairs}


# ---- inputs ----------------------------------------------------------------------------------


def _frequencies(case):
    """Angle per position of each pair (float64) and the factor on cosine and sine."""
    rot, base, s, orig = case["rot"], case["base"], case["factor"], case["original"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk":
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "banded":  # by wavelengths within the original context: 1 and 4 of them bound the band
        turns = orig * f / (2 * math.pi)
        smooth = ((turns - 1) / 3).clamp(0, 1)
        return f * ((1 - smooth) / s + smooth), 1.0
    if case["scaling"] == "yarn":  # a ramp over the pair index between 32 turns and 1 turn within the original context
        at = [rot * math.log(orig / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (ramp / s + 1 - ramp), 0.1 * math.log(s) + 1
    return f, 1.0


def _rope_handle(case):
    from paged_kv_decode_splitk_gb300 import pd

    return pd.Rope(case["head_dim"], case["rot"], layout=case["layout"], base=case["base"], scaling=case["scaling"],
                   factor=case["factor"], original_context=case["original"])


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _weight(case, g):
    """A norm's learned weight, near one; where it is kept as its distance from one, near zero."""
    w = torch.randn(case["head_dim"], generator=g, device="cuda") * 0.2 + (1.0 - case["offset"])
    return w.to(torch.bfloat16)


def _cache(blocks, case, g):
    """A pool of cache blocks, every slot filled: BF16, or E4M3 codes (bytes)."""
    x = _normal((blocks, BLOCK, case["kv_heads"], case["head_dim"]), g)
    return x if case["cache"] == "bf16" else (x * 2).to(torch.float8_e4m3fn).view(torch.uint8)


def _tables(counts, g):
    """Block ids of rows of the given block counts, from one shuffled pool a quarter larger than needed."""
    total, width = sum(counts), max(1, max(counts))
    pool = total + total // 4 + 1
    ids = torch.randperm(pool, generator=g, device="cuda")[:total].to(torch.int32)
    n = torch.tensor(counts, device="cuda")
    start = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    live = j[None, :] < n[:, None]
    table = torch.zeros((len(counts), width), dtype=torch.int32, device="cuda")
    table[live] = ids[(start[:, None] + j[None, :])[live]]
    return table, pool


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    D = case["head_dim"]
    st = {"case": case}
    if case["op"] != "chunk":
        st["freq"], st["factor"] = _frequencies(case)
        if own:
            st["rope"] = _rope_handle(case)
    if case["op"] == "norm":
        row = _normal((case["tokens"], case["row_heads"], D), g)  # the projection's output: q, k (and v) side by side
        st["x"] = row[:, : case["heads"]]
        st["w"] = _weight(case, g)
        st["positions"] = torch.randint(0, case["max_pos"], (case["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        if case["train"]:
            st["grad"] = _normal((case["tokens"], case["heads"], D), g)
            st["x"].requires_grad_(True)
            st["w"].requires_grad_(True)
        return st
    Hq, Hkv = case["q_heads"], case["kv_heads"]
    st["k_scale"], st["v_scale"] = (1.0, 1.0) if case["cache"] == "bf16" else (0.011, 0.0125)
    new, lens = _lens(case)
    order = list(range(case["seqs"]))
    random.Random(seed).shuffle(order)
    new, lens = [new[i] for i in order], [lens[i] for i in order]
    st["new"], st["host_lens"], tokens = new, lens, sum(new)
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    table, pool = _tables([-(-n // BLOCK) for n in lens], g)
    st.update(table=table, lens=_ints(lens), starts=_ints(starts), tokens=tokens, single=case["new_max"] == 1)
    st["k_cache"], st["v_cache"] = _cache(pool, case, g), _cache(pool, case, g)
    if case["op"] == "append":
        qkv = _normal((tokens, Hq + 2 * Hkv, D), g)
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq : Hq + Hkv], v=qkv[:, Hq + Hkv :], q_weight=_weight(case, g), k_weight=_weight(case, g))
        return st
    if case["cache"] == "e4m3":
        st["k_scale"], st["v_scale"] = 0.5, 0.25
    st.update(q=_normal((tokens, Hq, D), g), scale=1 / math.sqrt(D))
    if own:
        from paged_kv_decode_splitk_gb300 import api

        st["ws"] = api.chunk_workspace(tokens, Hq, Hkv, D, "cuda")  # kept from call to call
    return st


# ---- the plain forms -------------------------------------------------------------------------


def _turned(x, cos, sin, layout):
    """x [T, H, D] in 32 bits with its first 2 * cos.shape[1] columns rotated by the angles of cos, sin [T, R]."""
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if layout == "half":
        a, b = x[..., :half], x[..., half : 2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half :]], -1)


def _angles(st, positions):
    angle = positions.double()[:, None] * st["freq"][None, :]
    return (angle.cos() * st["factor"]).float(), (angle.sin() * st["factor"]).float()


def _normed(x, w, offset):
    """(x in 32 bits over its root mean square, one over that, the whole weight)."""
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r, w.float() + offset


def _plain_norm(st):
    case = st["case"]
    x, w = st["x"].detach(), st["w"].detach()
    cos, sin = _angles(st, st["positions"])
    xn, r, ww = _normed(x, w, case["offset"])
    y = _turned(xn * ww, cos, sin, case["layout"]).to(torch.bfloat16)
    if not case["train"]:
        return y
    g = _turned(st["grad"].float(), cos, -sin, case["layout"])
    gx = g * ww
    dx = (gx - xn * (gx * xn).mean(-1, keepdim=True)) * r
    dw = (g * xn).sum(0).sum(0)
    return {"y": y, "dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


def _plain_append(st):
    case = st["case"]
    new = st["starts"][1:] - st["starts"][:-1]
    seq = torch.repeat_interleave(torch.arange(new.shape[0], device="cuda"), new, output_size=st["tokens"])
    pos = torch.arange(st["tokens"], device="cuda") - st["starts"][1:][seq] + st["lens"][seq]
    cos, sin = _angles(st, pos)
    blk, off = st["table"][seq, pos // BLOCK].long(), pos % BLOCK

    def both(x, w):
        xn, _, ww = _normed(x, w, case["offset"])
        return _turned(xn * ww, cos, sin, case["layout"])

    q = both(st["q"], st["q_weight"]).to(torch.bfloat16)
    for cache, x, scale in ((st["k_cache"], both(st["k"], st["k_weight"]), st["k_scale"]), (st["v_cache"], st["v"].float(), st["v_scale"])):
        if cache.dtype == torch.uint8:
            x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[blk, off] = x.to(cache.dtype)
    return q


def _plain_chunk(st):
    case = st["case"]
    T, Hq, D = st["q"].shape
    Hkv = case["kv_heads"]
    G = Hq // Hkv
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    at = 0
    for s, (n, m) in enumerate(zip(st["new"], st["host_lens"])):
        low = max(0, m - n + 1 - case["window"]) // BLOCK if case["window"] else 0
        ids = st["table"][s, low : -(-m // BLOCK)].long()
        low *= BLOCK
        k, v = ((c[ids] if c.dtype != torch.uint8 else c[ids].view(torch.float8_e4m3fn)).float().flatten(0, 1)[: m - low] * x
                for c, x in ((st["k_cache"], st["k_scale"]), (st["v_cache"], st["v_scale"])))
        q = st["q"][at : at + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
        scores = (q @ k.permute(1, 2, 0)[:, None]).mul_(st["scale"])
        pos, key = torch.arange(m - n, m, device="cuda")[:, None], torch.arange(low, m, device="cuda")[None, :]
        dead = key > pos
        if case["window"]:
            dead |= key <= pos - case["window"]
        scores.masked_fill_(dead, float("-inf"))
        top = scores.amax(-1, keepdim=True)
        scores.sub_(top).exp_()
        total = scores.sum(-1, keepdim=True)
        o = (scores @ v.permute(1, 0, 2)[:, None]) / total
        out[at : at + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(torch.bfloat16)
        lse[at : at + n] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(n, Hq)
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def run(st):
    case = st["case"]
    if own:
        from paged_kv_decode_splitk_gb300 import api
    if case["op"] == "norm":
        if not own:
            return _plain_norm(st)
        y = api.norm_rope(st["rope"], st["x"], st["w"], st["positions"], eps=EPS, weight_offset=case["offset"])
        if not case["train"]:
            return y
        dx, dw = torch.autograd.grad(y, (st["x"], st["w"]), st["grad"])
        return {"y": y.detach(), "dx": dx, "dw": dw}
    if case["op"] == "append":
        if own:
            q = api.append_kv_normed(st["rope"], st["q"], st["k"], st["v"], st["q_weight"], st["k_weight"], st["k_cache"], st["v_cache"],
                                     st["table"], st["lens"], token_starts=None if st["single"] else st["starts"], eps=EPS,
                                     weight_offset=case["offset"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        else:
            q = _plain_append(st)
        kind = torch.float8_e4m3fn if case["cache"] == "e4m3" else torch.bfloat16
        return {"q": q, "k_cache": st["k_cache"].view(kind), "v_cache": st["v_cache"].view(kind)}
    if not own:
        return _plain_chunk(st)
    got = api.chunk_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["scale"],
                         token_starts=None if st["single"] else st["starts"], window=case["window"], return_lse=case["lse"], ws=st["ws"],
                         k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"out": got[0], "lse": got[1]} if case["lse"] else {"out": got}


# ---- the definition in 64 bits ---------------------------------------------------------------


def _exact_table(case):
    """Angles per position and the factor on cosine and sine, pair by pair."""
    rot, s, orig, out = case["rot"], case["factor"], case["original"], []
    base = case["base"] * (s ** (rot / (rot - 2)) if case["scaling"] == "ntk" else 1.0)
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(base))
        if case["scaling"] == "linear":
            f /= s
        elif case["scaling"] == "banded":
            wavelength = 2 * math.pi / f
            if wavelength > orig:
                f /= s
            elif wavelength > orig / 4.0:
                t = (orig / wavelength - 1.0) / 3.0
                f = (1.0 - t) * f / s + t * f
        elif case["scaling"] == "yarn":
            low = max(0, math.floor(rot * math.log(orig / (64 * math.pi)) / (2 * math.log(base))))
            high = min(rot - 1, math.ceil(rot * math.log(orig / (2 * math.pi)) / (2 * math.log(base))))
            t = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = f * (1.0 - t) + f / s * t
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda"), (1.0 + 0.1 * math.log(s) if case["scaling"] == "yarn" else 1.0)


def _exact_rotated(case, x, positions):
    """x [T, H, D] in 64 bits, each pair a complex number times its turn."""
    freq, factor = _exact_table(case)
    turn = torch.polar(torch.full_like(freq, factor)[None, :].expand(len(positions), -1).contiguous(),
                       positions.to(torch.float64)[:, None] * freq[None, :])[:, None, :]
    rot = case["rot"]
    half = rot // 2
    if case["layout"] == "half":
        z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)
    z = torch.view_as_complex(x[..., :rot].contiguous().unflatten(-1, (half, 2))) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)


def _exact_norm(case, x, w):
    return x / torch.sqrt(EPS + (x * x).sum(-1, keepdim=True) / case["head_dim"]) * (w + case["offset"])


def _exact_e4m3(x):
    """x rounded to the nearest E4M3 value (ties to even), saturating."""
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0**-6))[1].double() - 4)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(case, st):
    at, seq = [], []
    for i, (n, m) in enumerate(zip(st["new"], st["host_lens"])):
        at += range(m - n, m)
        seq += [i] * n
    at, seq = torch.tensor(at, device="cuda"), torch.tensor(seq, device="cuda")
    where = st["table"].long()[seq, torch.div(at, BLOCK, rounding_mode="floor")] * BLOCK + at % BLOCK
    fp8 = case["cache"] == "e4m3"
    q, k = (_exact_rotated(case, _exact_norm(case, st[x].double(), st[w].double()), at) for x, w in (("q", "q_weight"), ("k", "k_weight")))
    out = {"q": q}
    for name, x, scale in (("k_cache", k, st["k_scale"]), ("v_cache", st["v"].double(), st["v_scale"])):
        c = st[name].view(torch.float8_e4m3fn) if fp8 else st[name]
        c = c.double().flatten(0, 1)
        c[where] = _exact_e4m3(x / scale) if fp8 else x
        out[name] = c.view(st[name].shape)
    return out


def _exact_chunk(case, st):
    """Every head and every 512 tokens by themselves, each with the keys that any of them sees."""
    T, Hq, D = st["q"].shape
    G = Hq // case["kv_heads"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")

    def rows(name, s, a, b, head, scale):
        j = torch.arange(a, b, device="cuda")
        x = st[name][st["table"][s].long()[j // BLOCK], j % BLOCK, head]
        return (x if x.dtype != torch.uint8 else x.view(torch.float8_e4m3fn)).double() * scale

    first = 0
    for s, (n, m) in enumerate(zip(st["new"], st["host_lens"])):
        for t0 in range(0, n, 512):
            t1 = min(n, t0 + 512)
            pos = torch.arange(m - n + t0, m - n + t1, device="cuda")
            a, b = (max(0, m - n + t0 + 1 - case["window"]) if case["window"] else 0), m - n + t1
            far = pos[:, None] - torch.arange(a, b, device="cuda")[None, :]
            seen = (far >= 0) & (far < (case["window"] or b + 1))
            for head in range(case["kv_heads"]):
                k, v = rows("k_cache", s, a, b, head, st["k_scale"]), rows("v_cache", s, a, b, head, st["v_scale"])
                q = st["q"][first + t0 : first + t1, head * G : (head + 1) * G].double().transpose(0, 1)
                z = torch.where(seen, q @ k.T / math.sqrt(D), -math.inf)
                out[first + t0 : first + t1, head * G : (head + 1) * G] = (torch.softmax(z, -1) @ v).transpose(0, 1)
                lse[first + t0 : first + t1, head * G : (head + 1) * G] = torch.logsumexp(z, -1).T
        first += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "chunk":
        return _exact_chunk(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    x, w = (st[n].detach().double().requires_grad_(case["train"]) for n in ("x", "w"))
    y = _exact_rotated(case, _exact_norm(case, x, w), st["positions"])
    if not case["train"]:
        return y
    dx, dw = torch.autograd.grad(y, (x, w), st["grad"].double())
    return {"y": y.detach(), "dx": dx, "dw": dw}
