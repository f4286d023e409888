"""The operators around the paged decode step, as they are measured.

Three operators of one serving path over the paged K/V cache:

* rope:   rotary positions on the heads of a token batch (q and k of a fused projection);
* append: new tokens' keys (rotated) and values into the paged cache, the queries rotated on the way;
* prefix: decode attention of a batch whose sequences share long prefixes, each prefix read once for all.

`run` computes them in plain torch operations where `own` is false, and with the library's calls where it is true.
"""

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------------------


def listed():
    return [
        # one decode step of 64 sequences: the rotated heads of a layer that reads another layer's cache
        dict(name="rope_decode", op="rope", tokens=64, heads=40, row_heads=48, head_dim=128, rot=128, layout="half",
             scaling="none", base=10000.0, factor=1.0, original=32768, max_pos=32768),
        # a long prompt batch, full rotation, contexts stretched by wavelength bands
        dict(name="rope_prompt", op="rope", tokens=32768, heads=40, row_heads=48, head_dim=128, rot=128, layout="half",
             scaling="banded", base=500000.0, factor=8.0, original=8192, max_pos=131072),
        # a prompt chunk of odd length, a quarter of each wide head rotated, interleaved pairs, stretched sixteen times
        dict(name="rope_partial", op="rope", tokens=8191, heads=18, row_heads=20, head_dim=256, rot=64, layout="interleaved",
             scaling="yarn", base=10000.0, factor=16.0, original=4096, max_pos=65536),
        # one decode step of 64 sequences into a BF16 cache
        dict(name="append_decode", op="append", seqs=64, new_min=1, new_max=1, past_max=2048, q_heads=32, kv_heads=8,
             head_dim=128, rot=128, layout="half", scaling="none", base=10000.0, factor=1.0, original=32768, cache="bf16"),
        # one decode step of a large batch into an FP8 cache
        dict(name="append_decode_fp8", op="append", seqs=256, new_min=1, new_max=1, past_max=2048, q_heads=32, kv_heads=8,
             head_dim=128, rot=128, layout="half", scaling="banded", base=500000.0, factor=8.0, original=8192, cache="e4m3"),
        # a mixed step: prompts of up to 2731 tokens beside single decode tokens
        dict(name="append_prompts", op="append", seqs=24, new_min=1, new_max=2731, past_max=2048, q_heads=32, kv_heads=8,
             head_dim=128, rot=128, layout="half", scaling="linear", base=10000.0, factor=4.0, original=32768, cache="bf16"),
        # prompt chunks into an FP8 cache of wide heads, partly rotated
        dict(name="append_chunks_fp8", op="append", seqs=15, new_min=33, new_max=1025, past_max=4097, q_heads=16, kv_heads=2,
             head_dim=256, rot=64, layout="interleaved", scaling="yarn", base=10000.0, factor=16.0, original=4096, cache="e4m3"),
        # the smallest decode step: four sequences behind a short system prompt
        dict(name="prefix_small", op="prefix", groups=1, seqs=4, prefix_min=500, prefix_max=500, own_min=0, own_max=90, q_heads=4,
             kv_heads=1, head_dim=64, cache="bf16"),
        # an ordinary batch behind one system prompt
        dict(name="prefix_batch", op="prefix", groups=1, seqs=64, prefix_min=8192, prefix_max=8192, own_min=1, own_max=1024,
             q_heads=32, kv_heads=8, head_dim=128, cache="bf16"),
        # several prompts of odd lengths, each shared by some sequences, wide heads
        dict(name="prefix_groups", op="prefix", groups=6, seqs=48, prefix_min=1001, prefix_max=6007, own_min=0, own_max=700,
             q_heads=16, kv_heads=2, head_dim=256, cache="bf16"),
        # a large batch over one long document
        dict(name="prefix_document", op="prefix", groups=1, seqs=256, prefix_min=32768, prefix_max=32768, own_min=0, own_max=512,
             q_heads=32, kv_heads=8, head_dim=128, cache="bf16"),
        # a document in an FP8 cache, longer answers
        dict(name="prefix_document_fp8", op="prefix", groups=1, seqs=32, prefix_min=16385, prefix_max=16385, own_min=0,
             own_max=2000, q_heads=32, kv_heads=8, head_dim=128, cache="e4m3"),
    ]


def _log_int(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def _draw_rotation(rng, head_dim):
    rot = head_dim if rng.random() < 0.5 else 2 * rng.randint(2, head_dim // 2)
    scaling = rng.choice(["none", "linear", "ntk", "banded", "yarn"])
    return dict(rot=rot, layout=rng.choice(["half", "interleaved"]), scaling=scaling, base=rng.choice([10000.0, 500000.0]),
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 16.0]), original=rng.choice([4096, 8192]))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix"])
    if op == "rope":
        D = rng.choice([64, 80, 128, 192, 256])
        heads = rng.randint(1, 40)
        most = 32768 * 40 * 128 // (heads * D)
        return dict(op=op, tokens=_log_int(rng, 1, min(65536, most)), heads=heads, row_heads=heads + rng.choice([0, 1, 8]),
                    head_dim=D, max_pos=rng.choice([4096, 32768, 131072, 1000000]), **_draw_rotation(rng, D))
    Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([64, 80, 128, 256])
    while Hkv * (G + 2) * D > 48 * 128:
        G = max(1, G // 2)
        Hkv = max(1, Hkv // 2)
    cache = rng.choice(["bf16", "e4m3"])
    if op == "append":
        one = rng.random() < 0.4
        seqs = _log_int(rng, 1, 256) if one else _log_int(rng, 1, 24)
        return dict(op=op, seqs=seqs, new_min=1, new_max=1 if one else _log_int(rng, 2, 2700), past_max=_log_int(rng, 1, 2048),
                    q_heads=Hkv * G, kv_heads=Hkv, head_dim=D, cache=cache, **_draw_rotation(rng, D))
    groups = rng.choice([1, 1, 2, 3, 7])
    seqs = groups * _log_int(rng, 1, 256 // groups)
    high = _log_int(rng, 33, 32768 // groups)
    low = high if groups == 1 else rng.randint(1, high)
    own_max = _log_int(rng, 1, max(2, min(4096, 256 * 512 // seqs)))
    return dict(op=op, groups=groups, seqs=seqs, prefix_min=low, prefix_max=high, own_min=rng.choice([0, 1]), own_max=own_max,
                q_heads=Hkv * G, kv_heads=Hkv, head_dim=D, cache=cache)


def _spread(low, high, n):
    """n whole numbers evenly from low to high, the same for every seed."""
    return [low + (high - low) * i // max(1, n - 1) for i in range(n)]


def _append_lens(case):
    """(new tokens, tokens after the append) of each sequence."""
    new = _spread(case["new_min"], case["new_max"], case["seqs"])
    past = _spread(0, case["past_max"], case["seqs"])[::-1]
    return new, [n + p for n, p in zip(new, past)]


def _prefix_lens(case):
    """(prefix lengths, sequences of each group, own lengths)."""
    groups, seqs = case["groups"], case["seqs"]
    sizes = [seqs // groups] * groups
    for i in range(0, groups - 1, 2):  # uneven groups: one gives what the next takes
        move = sizes[i] // 3
        sizes[i], sizes[i + 1] = sizes[i] - move, sizes[i + 1] + move
    return _spread(case["prefix_min"], case["prefix_max"], groups), sizes, _spread(case["own_min"], case["own_max"], seqs)


def work(case):
    D = case["head_dim"]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * D
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 6 * case["tokens"] * case["heads"] * case["rot"] / 2}
    Hq, Hkv = case["q_heads"], case["kv_heads"]
    elem = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        t = sum(_append_lens(case)[0])
        return {"bytes": t * D * (2 * (Hq + 2 * Hkv) + 2 * Hq + 2 * elem * Hkv) + 12 * case["seqs"],
                "flops": 6 * t * (Hq + Hkv) * case["rot"] / 2}
    plens, sizes, lens = _prefix_lens(case)
    pairs = sum(p * n for p, n in zip(plens, sizes)) + sum(lens)
    return {"bytes": 2 * elem * Hkv * D * (sum(plens) + sum(lens)) + 4 * case["seqs"] * Hq * D + (sum(plens) + sum(lens)) // 4,
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


def _cache(blocks, case, g):
    """A pool of 16-token cache blocks, every slot filled: BF16, or E4M3 codes (bytes)."""
    x = _normal((blocks, 16, case["kv_heads"], case["head_dim"]), g)
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
    if case["op"] != "prefix":
        st["freq"], st["factor"] = _frequencies(case)
        if own:
            st["rope"] = _rope_handle(case)
    if case["op"] == "rope":
        row = _normal((case["tokens"], case["row_heads"], D), g)  # the projection's output: q, k (and v) side by side
        st["x"] = row[:, : case["heads"]]
        st["positions"] = torch.randint(0, case["max_pos"], (case["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        return st
    Hq, Hkv = case["q_heads"], case["kv_heads"]
    st["k_scale"], st["v_scale"] = (1.0, 1.0) if case["cache"] == "bf16" else (0.011, 0.0125)
    order = np.random.default_rng(seed).permutation(case["seqs"])
    if case["op"] == "append":
        new, lens = ([v[i] for i in order] for v in _append_lens(case))
        table, pool = _tables([-(-n // 16) for n in lens], g)
        qkv = _normal((sum(new), Hq + 2 * Hkv, D), g)
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq : Hq + Hkv], v=qkv[:, Hq + Hkv :], table=table, lens=_ints(lens),
                  starts=_ints([0, *np.cumsum(new).tolist()]), tokens=sum(new), decode=case["new_max"] == 1)
        st["k_cache"], st["v_cache"] = _cache(pool, case, g), _cache(pool, case, g)
        return st
    plens, sizes, lens = _prefix_lens(case)
    lens = [lens[i] for i in order]
    every, pool = _tables([-(-n // 16) for n in plens + lens], g)
    n = len(plens)
    st.update(q=_normal((case["seqs"], Hq, D), g), k_cache=_cache(pool, case, g), v_cache=_cache(pool, case, g),
              prefix_table=every[:n, : max(1, -(-max(plens) // 16))].contiguous(), prefix_lens=_ints(plens),
              group_starts=_ints([0, *np.cumsum(sizes).tolist()]),
              table=every[n:, : max(1, -(-max(lens) // 16))].contiguous(), lens=_ints(lens), scale=1 / math.sqrt(D))
    if case["cache"] == "e4m3":
        st["k_scale"], st["v_scale"] = 0.5, 0.25
    # split count by the Auto rule; which rows of q each group has, padded to the largest group
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    st["splits"] = max(1, min(16, -(-2 * sms // Hq)))
    most = max(sizes)
    st["members"] = torch.tensor([[sum(sizes[:i]) + min(j, sizes[i] - 1) for j in range(most)] for i in range(n)], device="cuda")
    st["gid"] = torch.tensor([i for i in range(n) for _ in range(sizes[i])], device="cuda")
    st["slot"] = torch.tensor([j for i in range(n) for j in range(sizes[i])], device="cuda")
    return st


# ---- the plain forms -------------------------------------------------------------------------


def _rotate(x, cos, sin, layout):
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


def _plain_append(st):
    new = st["starts"][1:] - st["starts"][:-1]
    seq = torch.repeat_interleave(torch.arange(new.shape[0], device="cuda"), new, output_size=st["tokens"])
    pos = torch.arange(st["tokens"], device="cuda") - st["starts"][1:][seq] + st["lens"][seq]
    cos, sin = _angles(st, pos)
    layout = st["case"]["layout"]
    blk, off = st["table"][seq, pos // 16].long(), pos % 16
    q = _rotate(st["q"].float(), cos, sin, layout).to(torch.bfloat16)
    for cache, x, scale in ((st["k_cache"], _rotate(st["k"].float(), cos, sin, layout), st["k_scale"]),
                            (st["v_cache"], st["v"].float(), st["v_scale"])):
        if cache.dtype == torch.uint8:
            x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[blk, off] = x.to(cache.dtype)
    return q


def _gathered(cache, table, scale):
    """The rows a block table names, in 32 bits: [rows, heads, tokens, head dim]."""
    x = cache[table.long()]
    x = x.float() if x.dtype != torch.uint8 else x.view(torch.float8_e4m3fn).float() * scale
    return x.flatten(1, 2).transpose(1, 2)


def _scores(q, k, lens, scale):
    """q [rows, heads, n, D] against k [rows, heads, tokens, D]; tokens past each row's length are -inf."""
    s = (q @ k.transpose(-1, -2)).mul_(scale)
    dead = torch.arange(k.shape[2], device="cuda")[None, :] >= lens[:, None]
    return s.masked_fill_(dead[:, None, None, :], float("-inf"))


def _plain_prefix(st):
    S, Hq, D = st["q"].shape
    Hkv = st["k_cache"].shape[2]
    q = st["q"].float().view(S, Hkv, Hq // Hkv, D)
    NG, most = st["members"].shape
    qg = q[st["members"]].permute(0, 2, 1, 3, 4).reshape(NG, Hkv, -1, D)
    sp = _scores(qg, _gathered(st["k_cache"], st["prefix_table"], st["k_scale"]), st["prefix_lens"], st["scale"])
    so = _scores(q, _gathered(st["k_cache"], st["table"], st["k_scale"]), st["lens"], st["scale"])

    def of_sequences(x):  # [NG, Hkv, most * G, ...] -> [S, Hkv, G, ...]
        x = x.view(NG, Hkv, most, Hq // Hkv, -1).transpose(1, 2)
        return x[st["gid"], st["slot"]]

    mp = sp.amax(-1, keepdim=True)
    mp = torch.where(mp == float("-inf"), torch.zeros_like(mp), mp)
    mo = so.amax(-1, keepdim=True)
    mo = torch.where(mo == float("-inf"), torch.zeros_like(mo), mo)
    ep, eo = sp.sub_(mp).exp_(), so.sub_(mo).exp_()
    lp, lo = of_sequences(ep.sum(-1, keepdim=True)), eo.sum(-1, keepdim=True)
    op = of_sequences(ep @ _gathered(st["v_cache"], st["prefix_table"], st["v_scale"]))
    oo = eo @ _gathered(st["v_cache"], st["table"], st["v_scale"])
    mp = of_sequences(mp)
    m = torch.maximum(mp, mo)
    ap, ao = (mp - m).exp(), (mo - m).exp()
    l = lp * ap + lo * ao
    out = torch.where(l > 0, (op * ap + oo * ao) / l, torch.zeros_like(op))
    return out.view(S, Hq, D).to(torch.bfloat16)


def run(st):
    op = st["case"]["op"]
    if own:
        from paged_kv_decode_splitk_gb300 import api
    if op == "rope":
        if own:
            return api.rope(st["rope"], st["x"], st["positions"])
        cos, sin = _angles(st, st["positions"])
        return _rotate(st["x"].float(), cos, sin, st["case"]["layout"]).to(torch.bfloat16)
    if op == "append":
        if own:
            q = api.append_kv(st["rope"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                              token_starts=None if st["decode"] else st["starts"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        else:
            q = _plain_append(st)
        kind = torch.float8_e4m3fn if st["case"]["cache"] == "e4m3" else torch.bfloat16
        return {"q": q, "k_cache": st["k_cache"].view(kind), "v_cache": st["v_cache"].view(kind)}
    if own:
        return api.decode_attn_prefix(st["q"], st["k_cache"], st["v_cache"], st["prefix_table"], st["prefix_lens"],
                                      st["group_starts"], st["table"], st["lens"], st["scale"], st["splits"],
                                      k_scale=st["k_scale"], v_scale=st["v_scale"])
    return _plain_prefix(st)


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
    freq, factor = _exact_table(case)
    turn = torch.polar(torch.full_like(freq, factor)[None, :].expand(len(positions), -1).contiguous(),
                       positions.to(torch.float64)[:, None] * freq[None, :])[:, None, :]
    y, rot = x.to(torch.float64), case["rot"]
    half = rot // 2
    one, two = (slice(0, half), slice(half, rot)) if case["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """x rounded to the nearest E4M3 value (ties to even), saturating."""
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0**-6))[1].double() - 4)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(case, st):
    lens, starts, at, seq = st["lens"].tolist(), st["starts"].tolist(), [], []
    for i, n in enumerate(lens):
        new = starts[i + 1] - starts[i]
        at += range(n - new, n)
        seq += [i] * new
    at, seq = torch.tensor(at, device="cuda"), torch.tensor(seq, device="cuda")
    where = st["table"].long()[seq, torch.div(at, 16, rounding_mode="floor")] * 16 + at % 16
    fp8 = case["cache"] == "e4m3"
    out = {"q": _exact_rotated(case, st["q"], at)}
    for name, x, scale in (("k_cache", _exact_rotated(case, st["k"], at), st["k_scale"]), ("v_cache", st["v"].double(), st["v_scale"])):
        c = st[name].view(torch.float8_e4m3fn) if fp8 else st[name]
        c = c.double().flatten(0, 1)
        c[where] = _exact_e4m3(x / scale) if fp8 else x
        out[name] = c.view(st[name].shape)
    return out


def _exact_prefix(st):
    S, Hq, D = st["q"].shape
    Hkv = st["k_cache"].shape[2]
    G = Hq // Hkv
    out = torch.zeros((S, Hq, D), dtype=torch.float64, device="cuda")

    def rows(name, table, n, scale):
        x = st[name][table[: -(-n // 16)].long()].flatten(0, 1)[:n]
        x = x.double() if x.dtype != torch.uint8 else x.view(torch.float8_e4m3fn).double() * scale
        return x.permute(1, 0, 2)

    starts = st["group_starts"].tolist()
    for gi, n in enumerate(st["prefix_lens"].tolist()):
        pk, pv = (rows(c, st["prefix_table"][gi], n, st[s]) for c, s in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
        for s in range(starts[gi], starts[gi + 1]):
            m = int(st["lens"][s])
            k = torch.cat([pk, rows("k_cache", st["table"][s], m, st["k_scale"])], 1) if m else pk
            v = torch.cat([pv, rows("v_cache", st["table"][s], m, st["v_scale"])], 1) if m else pv
            if k.shape[1]:
                w = torch.softmax(st["q"][s].double().view(Hkv, G, D) @ k.transpose(1, 2) / math.sqrt(D), -1)
                out[s] = (w @ v).reshape(Hq, D)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotated(case, st["x"], st["positions"])
    return _exact_append(case, st) if case["op"] == "append" else _exact_prefix(st)
