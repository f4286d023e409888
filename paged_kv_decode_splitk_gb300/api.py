"""Torch-level helpers over the C ABI: device placement of host inputs and
one-call wrappers that allocate outputs and the split-K workspace.

Plumbing only: every computation is a libpd kernel launched through `pd`.
"""

from __future__ import annotations

import numpy as np
import torch
from torch.autograd.forward_ad import unpack_dual

from . import pd


def bf16_tensor(bits: np.ndarray, device) -> torch.Tensor:
    """A torch BF16 tensor holding the given BF16 bit patterns (uint16)."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.view(torch.bfloat16).to(device)


def i32_tensor(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    """BF16 bit patterns (uint16) of a torch BF16 tensor, on the host."""
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def bf16_to_f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


class PagedInputs:
    """Device copies of a workloads.PagedWorkload."""

    def __init__(self, w, device="cuda"):
        self.w = w
        self.device = torch.device(device)
        self.q = bf16_tensor(w.q, self.device)
        if getattr(w, "kv_dtype", "bf16") == "e4m3":   # FP8 E4M3 codes, one byte each
            self.k = torch.from_numpy(np.ascontiguousarray(w.k_cache, dtype=np.uint8)).to(self.device)
            self.v = torch.from_numpy(np.ascontiguousarray(w.v_cache, dtype=np.uint8)).to(self.device)
        else:
            self.k = bf16_tensor(w.k_cache, self.device)
            self.v = bf16_tensor(w.v_cache, self.device)
        self.block_table = i32_tensor(w.block_table, self.device)
        self.context_lens = i32_tensor(w.context_lens, self.device)

    def splits(self, policy: str | None = None, pin: int | None = None, sm_count: int | None = None,
               max_decode_seqs: int | None = None) -> int:
        w = self.w
        return pd.pd_num_splits(policy or w.policy, w.pin if pin is None else pin,
                                w.sm_count if sm_count is None else sm_count, w.num_q_heads,
                                w.num_seqs, w.max_decode_seqs if max_decode_seqs is None
                                else max_decode_seqs)


def _fresh(shape, dtype, device, stream):
    """An uninitialised tensor that a launch on `stream` (a torch stream or a handle; None: the current one) writes.  It is
    allocated in that stream's order, since what the current stream has freed it may still have to write; and it is not
    reused before what the current stream does with it until it is freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream, device=device)
    if s.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(s):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def workspace(num_seqs: int, num_q_heads: int, head_dim: int, num_splits: int, device, stream=None) -> torch.Tensor | None:
    """The split-K workspace of a call (None where it needs none); stream: of a call on another stream than the current one."""
    n = pd.pd_workspace_bytes(num_seqs, num_q_heads, head_dim, num_splits)
    if num_splits <= 1 or n == 0:
        return None
    return _fresh(n, torch.uint8, device, stream)


def decode_attn(q, k_cache, v_cache, block_table, context_lens, inv_sqrt_d: float, num_splits: int,
                gqa_pack: int = 0, out=None, ws=None, stream=None, k_scale: float = 1.0,
                v_scale: float = 1.0):
    """Paged-decode attention; returns out [S, Hq, D] BF16 (or None when the packed
    pass does not apply to the shape, mirroring PD_NOT_APPLICABLE).  uint8 caches
    are FP8 E4M3 codes with per-tensor scales k_scale / v_scale."""
    S, Hq, D = q.shape
    if out is None:
        out = _fresh((S, Hq, D), torch.bfloat16, q.device, stream)
    if ws is None and num_splits > 1:
        ws = workspace(S, Hq, D, num_splits, q.device, stream)
    if k_cache.dtype == torch.uint8:
        rc = pd.pd_decode_attn_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, out,
                                   inv_sqrt_d, num_splits, ws, gqa_pack, stream)
    else:
        rc = pd.pd_decode_attn(q, k_cache, v_cache, block_table, context_lens, out, inv_sqrt_d,
                               num_splits, ws, gqa_pack, stream)
    if rc == pd.PD_NOT_APPLICABLE:
        return None
    return out


def run_paged(inp: PagedInputs, num_splits: int | None = None, gqa_pack: bool | None = None, out=None,
              ws=None, stream=None):
    w = inp.w
    n = inp.splits() if num_splits is None else num_splits
    pack = w.gqa_pack if gqa_pack is None else gqa_pack
    return decode_attn(inp.q, inp.k, inp.v, inp.block_table, inp.context_lens, w.inv_sqrt_d, n,
                       pack, out, ws, stream, getattr(w, "k_scale", 1.0), getattr(w, "v_scale", 1.0))


# The calls of a decode step launch in a few microseconds, so they first try the
# library's CPython module, which takes arguments that are just as they should be
# (pd_binding.cpp); only what it declines is checked here, one by one, for the message,
# and goes through the ctypes binding.
_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8


def _refuse(name: str, t, kind: str, shape, device: int):
    want = f"{name}: {kind} [{', '.join('any' if n is None else str(n) for n in shape)}] on the current device"
    if t.get_device() != device:
        raise ValueError(f"{want} (cuda:{device}) is wanted, it is on {t.device}")
    raise ValueError(f"{want} is wanted, not {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def _rows(name: str, t, tokens, heads, head_dim: int, device: int, side_by_side: bool) -> None:
    """t is BF16 [tokens, heads, head_dim] (None: any) on the device, its rows contiguous; side_by_side: the
    heads of a token too."""
    if t.dtype is _BF16 and t.dim() == 3 and t.get_device() == device:
        n, h, d = t.shape
        st = t.stride()
        if (d == head_dim and st[2] == 1 and (tokens is None or n == tokens) and (heads is None or h == heads)
                and (not side_by_side or st[1] == d or h == 1)):
            return
    _refuse(name, t, "BF16 with contiguous rows" + (" and a token's heads side by side" if side_by_side else ""),
            (tokens, heads, head_dim), device)


def _indices(name: str, t, shape, device: int) -> None:
    """t is contiguous int32 of the shape (None: any size) on the device."""
    if t.dtype is _I32 and t.dim() == len(shape) and t.is_contiguous() and t.get_device() == device:
        if all([w is None or h == w for h, w in zip(t.shape, shape)]):
            return
    _refuse(name, t, "contiguous int32", shape, device)


def _caches(k_cache, v_cache, num_kv_heads: int, head_dim: int, device: int) -> None:
    kind = k_cache.dtype
    if k_cache.dim() == 4 and (kind is _BF16 or kind is _U8):
        shape = k_cache.shape
        if (shape[2] == num_kv_heads and shape[3] == head_dim and v_cache.shape == shape and v_cache.dtype is kind
                and k_cache.is_contiguous() and v_cache.is_contiguous() and k_cache.get_device() == device
                and v_cache.get_device() == device):
            return
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if (c.dtype not in (_BF16, _U8) or c.dim() != 4 or c.shape[2:] != (num_kv_heads, head_dim)
                or not c.is_contiguous() or c.get_device() != device):
            _refuse(name, c, "contiguous BF16, or uint8 for E4M3 codes,", (None, None, num_kv_heads, head_dim), device)
    raise ValueError(f"k_cache and v_cache have one type and one shape, not {kind} {tuple(k_cache.shape)} and "
                     f"{v_cache.dtype} {tuple(v_cache.shape)}")


def _check_rope(rotation, x, positions, out, dev: int) -> None:
    _rows("x", x, None, None, rotation.head_dim, dev, False)
    T, H, D = x.shape
    _indices("positions", positions, (T,), dev)
    if out is not None:
        _rows("out", out, T, H, D, dev, False)


def _laid_out(grad):
    """grad (or what a hook on saved tensors gave back) [T, H, D], its rows laid out anew where it comes broadcast, transposed
    or at an odd place."""
    if grad.dim() != 3:
        return grad
    if grad.data_ptr() % 16 or grad.stride(2) != 1 or any(n > 1 and (s <= 0 or s % 8) for n, s in zip(grad.shape[:2], grad.stride())):
        return grad.clone(memory_format=torch.contiguous_format)
    return grad


def _in_order(t):
    """t (or None) contiguous, at a place that a row may have."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _no_tangent(what: str, *tensors) -> None:
    """Refuses forward-mode tangents, which no call here carries on."""
    if any([t is not None and unpack_dual(t).tangent is not None for t in tensors]):
        raise RuntimeError(f"{what} has no forward-mode derivative")


class _Rotation(torch.autograd.Function):
    """rope where x requires a gradient, which is the transposed map's value."""

    @staticmethod
    def forward(ctx, x, rotation, positions, inverse, stream):
        ctx.rotation, ctx.inverse = rotation, inverse
        ctx.save_for_backward(positions)
        return rope(rotation, x, positions, inverse=inverse, stream=stream)

    @staticmethod
    def backward(ctx, grad):
        (positions,) = ctx.saved_tensors
        return rope(ctx.rotation, _laid_out(grad), positions, inverse=not ctx.inverse), None, None, None, None


def rope(rotation: pd.Rope, x, positions, out=None, inverse: bool = False, stream=None):
    """Rotary positions: x [T, H, D] BF16 (strided in tokens and heads, e.g. the q and k heads of a fused
    projection) rotated by positions [T] int32; returns out [T, H, D] (contiguous unless given; x itself
    rotates in place).  inverse applies the transposed map, the rotation back with the same factor, which takes
    gradients of out to gradients of x; where x requires a gradient, autograd calls it (out cannot be given then; a
    backward pass is captured into a graph, as torch wants it, while no eager graph of the same leaves lives)."""
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out: no gradient can pass through a tensor that is given; call under torch.no_grad() or let rope make it")
        _no_tangent("rope", x)
        return _Rotation.apply(x, rotation, positions, inverse, stream)
    if stream is None:
        done = pd.quick().rope(pd._handle(rotation), rotation.head_dim, x, positions, out, inverse)
        if done is not NotImplemented:
            return done
    _no_tangent("rope", x)
    _check_rope(rotation, x, positions, out, pd.current_device())
    if out is None:
        out = _fresh(x.shape, _BF16, x.device, stream)
    pd.pd_rope_apply(rotation, x, positions, out, inverse, stream)
    return out


def _check_append(q, k, v, k_cache, v_cache, block_table, context_lens, token_starts, q_out, dev: int) -> None:
    if k.dim() != 3:
        _refuse("k", k, "BF16", (None, None, None), dev)
    T, Hkv, D = k.shape
    _rows("k", k, T, Hkv, D, dev, True)
    _rows("v", v, T, Hkv, D, dev, True)
    _caches(k_cache, v_cache, Hkv, D, dev)
    _indices("context_lens", context_lens, (None,), dev)
    S = context_lens.shape[0]
    _indices("block_table", block_table, (S, None), dev)
    if token_starts is not None:
        _indices("token_starts", token_starts, (S + 1,), dev)
    if q is not None:
        _rows("q", q, T, None, D, dev, True)
        if q_out is not None:
            _rows("q_out", q_out, T, q.shape[1], D, dev, True)
            if not q_out.is_contiguous():
                raise ValueError("q_out has to be contiguous")
    elif q_out is not None:
        raise ValueError("q_out without q")


def append_kv(rotation, q, k, v, k_cache, v_cache, block_table, context_lens, token_starts=None, q_out=None,
              k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Append new tokens to the paged cache: k [T, Hkv, D] rotated (rotation: a pd.Rope, or None for none) and
    v as they are, at the last positions of context_lens [S] (lengths after the append); q [T, Hq, D] (or
    None) rotated on the way and returned as q_out [T, Hq, D].  token_starts [S + 1] says which rows each
    sequence has; None: one each.  uint8 caches hold E4M3 codes of x * (1 / k_scale) and x * (1 / v_scale).  Rows of no
    sequence, a sequence of length 0 and a token without a place get nothing: a q_out that is given keeps what it
    holds there, one made here holds anything (NaN among it), which reaches no other row of the attention; give a
    zeroed q_out where such rows are read.  A serving call: no gradient passes through it."""
    if stream is None and q is not None:
        done = pd.quick().append_kv(pd._handle(rotation) or 0, 0 if rotation is None else rotation.head_dim, q, k, v, k_cache,
                                    v_cache, block_table, context_lens, token_starts, q_out, k_scale, v_scale)
        if done is not NotImplemented:
            return done
    _check_append(q, k, v, k_cache, v_cache, block_table, context_lens, token_starts, q_out, pd.current_device())
    if q is not None and q_out is None:
        q_out = _fresh(q.shape, _BF16, q.device, stream)
    if k_cache.dtype is _U8:
        pd.pd_append_kv_fp8(rotation, q, k, v, q_out, k_cache, v_cache, k_scale, v_scale, block_table, context_lens,
                            token_starts, stream)
    else:
        pd.pd_append_kv(rotation, q, k, v, q_out, k_cache, v_cache, block_table, context_lens, token_starts, stream)
    return q_out


def _weight(name: str, t, head_dim: int, device: int) -> None:
    if t is not None and not (t.dtype is _BF16 and t.shape == (head_dim,) and t.is_contiguous() and t.get_device() == device):
        _refuse(name, t, "contiguous BF16", (head_dim,), device)


def _check_norm(rotation, x, weight, positions, dev: int) -> None:
    _rows("x", x, None, None, rotation.head_dim if rotation is not None else (x.shape[-1] if x.dim() == 3 else None), dev, False)
    _weight("weight", weight, x.shape[2], dev)
    if rotation is not None:
        if positions is None:
            raise ValueError("positions: a rotation wants them")
        _indices("positions", positions, (x.shape[0],), dev)
    elif positions is not None:
        raise ValueError("positions without a rotation")


class _Last(torch.autograd.Function):
    """A gradient of norm_rope, which has none itself: an error where one is asked for."""

    @staticmethod
    def forward(ctx, t):
        return t.view_as(t)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("norm_rope has no second gradient")


class _NormRotation(torch.autograd.Function):
    """norm_rope where x or weight requires a gradient."""

    @staticmethod
    def forward(ctx, x, weight, rotation, positions, eps, weight_offset, stream):
        ctx.rotation, ctx.eps, ctx.offset = rotation, eps, weight_offset
        ctx.save_for_backward(x, weight, positions)
        return norm_rope(rotation, x, weight, positions, eps, weight_offset, stream=stream)

    @staticmethod
    def backward(ctx, grad):
        _no_tangent("norm_rope's gradient", grad)
        x, weight, positions = ctx.saved_tensors  # (which the caller's hooks may give back in another layout)
        with torch.no_grad():
            dx, dw = norm_rope_backward(ctx.rotation, _laid_out(x), _in_order(weight), _in_order(positions), _laid_out(grad), ctx.eps,
                                        ctx.offset, weight_grad=ctx.needs_input_grad[1])
        if torch.is_grad_enabled():
            dx, dw = (None if t is None else _Last.apply(t.requires_grad_()) for t in (dx, dw))
        return dx if ctx.needs_input_grad[0] else None, dw, None, None, None, None, None


def norm_rope(rotation, x, weight, positions, eps: float = 1e-6, weight_offset: float = 0.0, out=None, stream=None):
    """The RMS norm of each head and the rotary positions in one pass: each row of x [T, H, D] BF16 (strided in tokens and heads,
    e.g. the q or the k heads of a fused projection) over its root mean square (eps under the root) times weight_offset +
    weight [D] (None: ones), rotated by positions [T] int32 (rotation and positions None: the norm alone).  Returns out
    [T, H, D] (contiguous unless given; x itself works in place).  Where x or weight requires a gradient, autograd calls
    norm_rope_backward (out cannot be given then; a backward pass is captured into a graph, as torch wants it, while no eager
    graph of the same leaves lives); the rotation has to be open still when it does.  There is no second gradient and no
    forward-mode one: both are refused."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)):
        if out is not None:
            raise ValueError("out: no gradient can pass through a tensor that is given; call under torch.no_grad() or let norm_rope make it")
        if stream is None:
            done = pd.quick().norm_rope_grad(pd._handle(rotation) or 0, 0 if rotation is None else rotation.head_dim, rotation, x, weight,
                                             positions, eps, weight_offset)
            if done is not NotImplemented:
                return done
        _no_tangent("norm_rope", x, weight)
        return _NormRotation.apply(x, weight, rotation, positions, eps, weight_offset, stream)
    if stream is None:
        done = pd.quick().norm_rope(pd._handle(rotation) or 0, 0 if rotation is None else rotation.head_dim, x, weight, positions, out, eps,
                                    weight_offset)
        if done is not NotImplemented:
            return done
    _no_tangent("norm_rope", x, weight)
    dev = pd.current_device()
    _check_norm(rotation, x, weight, positions, dev)
    if out is not None:
        _rows("out", out, *x.shape, dev, False)
    else:
        out = _fresh(x.shape, _BF16, x.device, stream)
    pd.pd_norm_rope_apply(rotation, x, weight, positions, out, eps, weight_offset, stream)
    return out


def norm_rope_backward(rotation, x, weight, positions, grad, eps: float = 1e-6, weight_offset: float = 0.0, weight_grad: bool = True,
                       stream=None):
    """The gradients of norm_rope from the gradient of its out [T, H, D]: (grad_x [T, H, D], grad_weight [D]), the second None
    where it is not wanted or there is no weight.  No gradient passes through it."""
    dev = pd.current_device()
    _check_norm(rotation, x, weight, positions, dev)
    _rows("grad", grad, *x.shape, dev, False)
    grad_x = _fresh(x.shape, _BF16, x.device, stream)
    grad_weight = ws = None
    if weight_grad and weight is not None:
        grad_weight = _fresh(weight.shape, _BF16, x.device, stream)
        ws = _fresh(pd.pd_norm_rope_workspace_bytes(x.shape[2]), _U8, x.device, stream)
    pd.pd_norm_rope_backward(rotation, x, weight, positions, grad, grad_x, grad_weight, ws, eps, weight_offset, stream)
    return grad_x, grad_weight


def append_kv_normed(rotation, q, k, v, q_weight, k_weight, k_cache, v_cache, block_table, context_lens, token_starts=None, q_out=None,
                     eps: float = 1e-6, weight_offset: float = 0.0, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """append_kv with the RMS norm of each head of q and k, as norm_rope's, before the rotation: q_weight and k_weight [D] BF16
    (None: ones).  Everything else, the rows that get nothing among it, is append_kv's."""
    if stream is None and q is not None:
        done = pd.quick().append_kv_normed(pd._handle(rotation) or 0, 0 if rotation is None else rotation.head_dim, q, k, v, q_weight,
                                           k_weight, k_cache, v_cache, block_table, context_lens, token_starts, q_out, eps, weight_offset,
                                           k_scale, v_scale)
        if done is not NotImplemented:
            return done
    dev = pd.current_device()
    _check_append(q, k, v, k_cache, v_cache, block_table, context_lens, token_starts, q_out, dev)
    _weight("q_weight", q_weight, k.shape[2], dev)
    _weight("k_weight", k_weight, k.shape[2], dev)
    if q is not None and q_out is None:
        q_out = _fresh(q.shape, _BF16, q.device, stream)
    if k_cache.dtype is _U8:
        pd.pd_append_kv_normed_fp8(rotation, q, k, v, q_weight, k_weight, q_out, k_cache, v_cache, k_scale, v_scale, block_table,
                                   context_lens, token_starts, eps, weight_offset, stream)
    else:
        pd.pd_append_kv_normed(rotation, q, k, v, q_weight, k_weight, q_out, k_cache, v_cache, block_table, context_lens, token_starts, eps,
                               weight_offset, stream)
    return q_out


def prefix_workspace(num_seqs: int, num_groups: int, num_q_heads: int, num_kv_heads: int, head_dim: int, num_splits: int,
                     device, stream=None) -> torch.Tensor:
    """The workspace of a decode_attn_prefix; stream: of a call on another stream than the current one."""
    n = pd.pd_prefix_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, num_splits)
    return _fresh(n, _U8, device, stream)


def _check_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table, context_lens, out, ws, dev: int) -> None:
    if q.dim() != 3 or not q.is_contiguous():
        _refuse("q", q, "contiguous BF16", (None, None, None), dev)
    S, Hq, D = q.shape
    _rows("q", q, S, Hq, D, dev, True)
    _caches(k_cache, v_cache, k_cache.shape[2] if k_cache.dim() == 4 else 0, D, dev)
    _indices("prefix_lens", prefix_lens, (None,), dev)
    G = prefix_lens.shape[0]
    _indices("prefix_table", prefix_table, (G, None), dev)
    if group_starts is not None:
        _indices("group_starts", group_starts, (G + 1,), dev)
    _indices("context_lens", context_lens, (S,), dev)
    _indices("block_table", block_table, (S, None), dev)
    if out is not None:
        _rows("out", out, S, Hq, D, dev, True)
        if not out.is_contiguous():
            raise ValueError("out has to be contiguous")
    if ws is not None and not (ws.is_contiguous() and ws.get_device() == dev):
        _refuse("ws", ws, "a contiguous buffer", (None,), dev)


def decode_attn_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table, context_lens,
                       inv_sqrt_d: float, num_splits: int, out=None, ws=None, stream=None, k_scale: float = 1.0,
                       v_scale: float = 1.0):
    """Decode attention behind shared prefixes: sequences group_starts[g] to group_starts[g + 1] - 1 (None: the whole
    batch, one group) attend to the prefix_lens[g] tokens prefix_table[g] names, then to their own context_lens
    tokens; a prefix is read once for its group.  Returns out [S, Hq, D] BF16.  uint8 caches are FP8 E4M3 codes
    with per-tensor scales.  A serving call: no gradient passes through it."""
    if stream is None:
        done = pd.quick().decode_attn_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table,
                                             context_lens, inv_sqrt_d, num_splits, out, ws, k_scale, v_scale)
        if done is not NotImplemented:
            return done
    _check_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table, context_lens, out, ws,
                  pd.current_device())
    S, Hq, D = q.shape
    if out is None:
        out = _fresh(q.shape, _BF16, q.device, stream)
    if ws is None:
        ws = prefix_workspace(S, prefix_lens.shape[0], Hq, max(1, k_cache.shape[2]), D, num_splits, q.device, stream)
    if k_cache.dtype is _U8:
        pd.pd_decode_attn_prefix_fp8(q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_lens, group_starts,
                                     block_table, context_lens, out, inv_sqrt_d, num_splits, ws, stream)
    else:
        pd.pd_decode_attn_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table, context_lens,
                                 out, inv_sqrt_d, num_splits, ws, stream)
    return out


def chunk_workspace(num_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int, device, stream=None) -> torch.Tensor:
    """The workspace of a chunk_attn; stream: of a call on another stream than the current one."""
    return _fresh(pd.pd_chunk_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, head_dim), _U8, device, stream)


def _check_chunk(q, k_cache, v_cache, block_table, context_lens, token_starts, out, lse, ws, dev: int) -> None:
    _rows("q", q, None, None, q.shape[-1] if q.dim() == 3 else None, dev, True)
    T, Hq, D = q.shape
    _caches(k_cache, v_cache, k_cache.shape[2] if k_cache.dim() == 4 else 0, D, dev)
    _indices("context_lens", context_lens, (None,), dev)
    S = context_lens.shape[0]
    _indices("block_table", block_table, (S, None), dev)
    if token_starts is not None:
        _indices("token_starts", token_starts, (S + 1,), dev)
    if out is not None:
        _rows("out", out, T, Hq, D, dev, True)
        if not out.is_contiguous():
            raise ValueError("out has to be contiguous")
    if lse is not None and not (lse.dtype is torch.float32 and lse.shape == (T, Hq) and lse.is_contiguous() and lse.get_device() == dev):
        _refuse("lse", lse, "contiguous FP32", (T, Hq), dev)
    if ws is not None and not (ws.is_contiguous() and ws.get_device() == dev):
        _refuse("ws", ws, "a contiguous buffer", (None,), dev)


def chunk_attn(q, k_cache, v_cache, block_table, context_lens, inv_sqrt_d: float, token_starts=None, window: int = 0, out=None,
               lse=None, return_lse: bool = False, ws=None, stream=None, k_scale: float = 1.0, v_scale: float = 1.0):
    """Attention of new tokens over the paged cache that holds them already: rows token_starts[s] to token_starts[s + 1] - 1
    of q [T, Hq, D] (None: one each) are the last tokens of sequence s, whose context_lens [S] count them, and each sees the
    keys up to its own, the last `window` of them (0: all).  Returns out [T, Hq, D] BF16, and with return_lse (or an lse
    that is given) also lse [T, Hq], the logarithm of each row's sum.  Rows of no sequence get nothing: an out or lse made
    here holds anything there.  uint8 caches are FP8 E4M3 codes with per-tensor scales.  Keys and values that a token of the
    call sees are finite; weights are rounded to BF16 (over FP8 to f16) before they meet V, but for single tokens alone that go
    to the decode's kernels, which keep 16 bits.  A serving call: no gradient passes through it."""
    if lse is None and return_lse and q.dim() == 3:
        lse = _fresh(q.shape[:2], torch.float32, q.device, stream)
    if stream is None:
        done = pd.quick().chunk_attn(q, k_cache, v_cache, block_table, context_lens, token_starts, inv_sqrt_d, window, out, lse, ws,
                                     k_scale, v_scale)
        if done is not NotImplemented:
            return done if lse is None else (done, lse)
    _check_chunk(q, k_cache, v_cache, block_table, context_lens, token_starts, out, lse, ws, pd.current_device())
    T, Hq, D = q.shape
    if out is None:
        out = _fresh(q.shape, _BF16, q.device, stream)
    if ws is None:
        ws = chunk_workspace(T, Hq, max(1, k_cache.shape[2]), D, q.device, stream)
    if k_cache.dtype is _U8:
        pd.pd_chunk_attn_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, token_starts, out, lse, inv_sqrt_d, window,
                             ws, stream)
    else:
        pd.pd_chunk_attn(q, k_cache, v_cache, block_table, context_lens, token_starts, out, lse, inv_sqrt_d, window, ws, stream)
    return out if lse is None else (out, lse)


class TiledInputs:
    """Device copies of a workloads.TiledWorkload."""

    def __init__(self, tw, device="cuda"):
        self.w = tw
        self.device = torch.device(device)
        self.q = bf16_tensor(tw.q, self.device)
        self.pool = bf16_tensor(tw.pool, self.device)
        if tw.layout == "scratch":
            flat = self.pool.view(-1)
            stripe = tw.num_kv_heads * tw.block_size * tw.head_dim
            self.k_pool = flat
            self.v_pool = flat[stripe:]
        else:
            self.k_pool = self.pool
            self.v_pool = bf16_tensor(tw.v_pool, self.device)
        self.tile_blocks = [i32_tensor(tw.tile_blocks[c], self.device) for c in range(tw.num_calls)]
        self.tile_counts = [i32_tensor(tw.tile_block_counts[c], self.device) for c in range(tw.num_calls)]


def run_tiled(inp: TiledInputs, tiled: pd.Tiled | None = None, out=None, stream=None):
    """begin_step, one step_tile per call, finalize; returns out [S, Hq, D] BF16."""
    tw = inp.w
    own = tiled is None
    if own:
        tiled = pd.Tiled(tw.num_seqs, tw.num_q_heads, tw.num_kv_heads, tw.head_dim, tw.block_size,
                         tw.tile_capacity)
    try:
        strides = tiled.scratch_pool_strides() if tw.layout == "scratch" else tiled.paged_strides()
        if out is None:
            out = _fresh((tw.num_seqs, tw.num_q_heads, tw.head_dim), torch.bfloat16, inp.device, stream)
        tiled.begin(tw.num_seqs, stream)
        for c in range(tw.num_calls):
            tiled.step(inp.q, inp.k_pool, inp.v_pool, inp.tile_blocks[c], inp.tile_counts[c],
                       tw.num_seqs, strides, int(tw.last_block_valid_slots[c]), stream)
        tiled.finalize(out, tw.num_seqs, stream)
    finally:
        if own:
            torch.cuda.current_stream().synchronize()
            tiled.close()
    return out


class MixedTiledInputs:
    """Device copies of a workloads.MixedTiledWorkload."""

    def __init__(self, mw, device="cuda"):
        self.w = mw
        self.device = torch.device(device)
        self.q = bf16_tensor(mw.q, self.device)
        self.paged_k = bf16_tensor(mw.paged_k, self.device)
        self.paged_v = bf16_tensor(mw.paged_v, self.device)
        self.scratch = bf16_tensor(mw.scratch, self.device)
        flat = self.scratch.view(-1)
        stripe = mw.num_kv_heads * mw.block_size * mw.head_dim
        self.scratch_k = flat
        self.scratch_v = flat[stripe:]
        self.tile_blocks = [i32_tensor(c[1], self.device) for c in mw.calls]
        self.tile_counts = [i32_tensor(c[2], self.device) for c in mw.calls]

    def sources(self, tiled: pd.Tiled):
        out = []
        for i, (kind, _, _, lbvs) in enumerate(self.w.calls):
            if kind == "paged":
                k, v, st = self.paged_k, self.paged_v, tiled.paged_strides()
            else:
                k, v, st = self.scratch_k, self.scratch_v, tiled.scratch_pool_strides()
            out.append((k, v, self.tile_blocks[i], self.tile_counts[i], st, int(lbvs)))
        return out


def run_tiled_mixed(inp: MixedTiledInputs, tiled: pd.Tiled | None = None, out=None, stream=None):
    """One pd_tiled_run: begin, one step per source (paged, then scratch pool), finalize."""
    mw = inp.w
    own = tiled is None
    if own:
        tiled = pd.Tiled(mw.num_seqs, mw.num_q_heads, mw.num_kv_heads, mw.head_dim, mw.block_size,
                         mw.tile_capacity)
    try:
        if out is None:
            out = _fresh((mw.num_seqs, mw.num_q_heads, mw.head_dim), torch.bfloat16, inp.device, stream)
        tiled.run(inp.q, inp.sources(tiled), out, mw.num_seqs, stream)
    finally:
        if own:
            torch.cuda.current_stream().synchronize()
            tiled.close()
    return out
