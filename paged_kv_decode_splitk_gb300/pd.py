"""ctypes binding of libpd (include/pd.h), argument marshalling only.

Every function keeps the C name.  Tensors are torch tensors on the device;
their data pointers, sizes and the current CUDA stream go to the library
unchanged.  Every step of the computation runs in libpd's kernels: there is
no Python or CPU fallback, and a missing library raises `PdLibraryError`.

Negative return codes raise `PdError` (with pd_last_error()'s message);
PD_NOT_APPLICABLE is returned as the value 1 so that the caller can take
another path, like the C convention.
"""

from __future__ import annotations

import ctypes
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libpd.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "pd.h")

PD_OK = 0
PD_NOT_APPLICABLE = 1
PD_ERR_INVALID = -1
PD_ERR_CAPACITY = -2
PD_ERR_WORKSPACE = -3
PD_ERR_CUDA = -4
PD_ERR_ALLOC = -5
PD_ERR_UNSUPPORTED = -6

PD_GQA_PACK_OFF = 0
PD_GQA_PACK_ON = 1
PD_GQA_PACK_SPLITK = 2

PD_POLICY_LEGACY = 0
PD_POLICY_AUTO = 1
PD_POLICY_PINNED = 2

PD_DEV_BAD_BLOCK_ID = 1
PD_DEV_BAD_CONTEXT_LEN = 2
PD_DEV_BAD_TILE_COUNT = 4
PD_DEV_WAIT_TIMEOUT = 8
PD_DEV_BAD_GROUPS = 16

PD_ROPE_HALF = 0
PD_ROPE_INTERLEAVED = 1
PD_ROPE_NONE = 0
PD_ROPE_LINEAR = 1
PD_ROPE_NTK = 2
PD_ROPE_BANDED = 3
PD_ROPE_YARN = 4
PD_ROPE_TABLE = 5

ROPE_LAYOUTS = {"half": PD_ROPE_HALF, "interleaved": PD_ROPE_INTERLEAVED}
ROPE_SCALINGS = {"none": PD_ROPE_NONE, "linear": PD_ROPE_LINEAR, "ntk": PD_ROPE_NTK, "banded": PD_ROPE_BANDED,
                 "yarn": PD_ROPE_YARN, "table": PD_ROPE_TABLE}
POLICY_NAMES = {"legacy": PD_POLICY_LEGACY, "auto": PD_POLICY_AUTO, "pinned": PD_POLICY_PINNED}


class PdLibraryError(RuntimeError):
    """libpd.so is missing or unloadable."""


class PdError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"libpd error {code}: {message}")
        self.code = code


class pd_tiled_dims(ctypes.Structure):
    _fields_ = [("max_seqs", ctypes.c_int), ("num_q_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("block_size", ctypes.c_int), ("tile_capacity", ctypes.c_int)]


class pd_tiled_source(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("tile_blocks", ctypes.c_void_p), ("tile_block_counts", ctypes.c_void_p),
                ("blk_stride", ctypes.c_int64), ("tok_stride", ctypes.c_int64),
                ("kvh_stride", ctypes.c_int64), ("last_block_valid_slots", ctypes.c_int)]


class pd_rope_desc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("scaling", ctypes.c_int), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_context", ctypes.c_double), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double), ("attention_factor", ctypes.c_double),
                ("frequencies", ctypes.POINTER(ctypes.c_double))]


_lock = threading.Lock()
_lib = None

_VP = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_SIGS = {
    "pd_last_error": (ctypes.c_char_p, []),
    "pd_build_info": (_I, [_VP, _VP, _VP, _VP]),
    "pd_parse_policy": (_I, [ctypes.c_char_p, _VP, _VP]),
    "pd_parse_gqa_pack": (_I, [ctypes.c_char_p, _VP]),
    "pd_resolve_policy": (_I, [ctypes.c_char_p, ctypes.c_char_p, _VP, _VP]),
    "pd_policy_from_env": (_I, [ctypes.c_char_p, _VP, _VP]),
    "pd_gqa_pack_enabled": (_I, []),
    "pd_split_ref_seqs": (_I, [_I, _I]),
    "pd_legacy_splits": (_I, [_I, _I, _I]),
    "pd_auto_splits": (_I, [_I, _I]),
    "pd_num_splits": (_I, [_I, _I, _I, _I, _I, _I]),
    "pd_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "pd_gqa_pack_shape_ok": (_I, [_I, _I, _I]),
    "pd_gqa_pack_ctas": (_I, [_I, _I]),
    "pd_split_chunk_tokens": (_I, [_I, _I, _I]),
    "pd_decode_attn": (_I, [_VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I,
                            ctypes.c_float, _I, _VP, _SZ, _I, _VP]),
    "pd_decode_attn_fp8": (_I, [_VP, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP, _I, _VP, _VP, _I, _I,
                                _I, _I, _I, _I, ctypes.c_float, _I, _VP, _SZ, _I, _VP]),
    "pd_decode_attn_noalloc": (_I, [_VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                    ctypes.c_float, _I, _I, _VP]),
    "pd_prefix_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "pd_decode_attn_prefix": (_I, [_VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                   ctypes.c_float, _I, _VP, _SZ, _VP]),
    "pd_decode_attn_prefix_fp8": (_I, [_VP, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP, _I, _VP, _VP, _I, _VP, _I, _VP,
                                       _VP, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _VP, _SZ, _VP]),
    "pd_debug_prefix_walk": (_I, [_I, _I, _VP, _VP, _I, _I, _I, _I, ctypes.c_float, _I, _VP, _I, _VP, _VP, _VP]),
    "pd_chunk_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "pd_chunk_attn": (_I, [_VP, _I64, _VP, _VP, _VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _I,
                           _VP, _SZ, _VP]),
    "pd_chunk_attn_fp8": (_I, [_VP, _I64, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I,
                               _I, _I, _I, ctypes.c_float, _I, _VP, _SZ, _VP]),
    "pd_debug_chunk_walk": (_I, [_I, _VP, _VP, _I, _I, _I, _I, _I, _VP, _I, _VP, _VP]),
    "pd_rope_frequencies": (_I, [_VP, _VP, _VP]),
    "pd_rope_create": (_I, [_VP, _VP]),
    "pd_rope_destroy": (None, [_VP]),
    "pd_rope_apply": (_I, [_VP, _VP, _I64, _I64, _VP, _VP, _I64, _I64, _I, _I, _I, _VP]),
    "pd_norm_rope_apply": (_I, [_VP, _VP, _I64, _I64, _VP, ctypes.c_float, ctypes.c_float, _VP, _VP, _I64, _I64, _I, _I, _I, _VP]),
    "pd_norm_rope_workspace_bytes": (_SZ, [_I]),
    "pd_norm_rope_backward": (_I, [_VP, _VP, _I64, _I64, _VP, ctypes.c_float, ctypes.c_float, _VP, _VP, _I64, _I64, _VP, _I64, _I64, _VP,
                                   _I, _I, _I, _VP, _SZ, _VP]),
    "pd_append_kv_normed": (_I, [_VP, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP, _VP, _VP, _VP, _I,
                                 _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP]),
    "pd_append_kv_normed_fp8": (_I, [_VP, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP, _VP, _VP,
                                     ctypes.c_float, ctypes.c_float, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP]),
    "pd_append_kv": (_I, [_VP, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I,
                          _I, _I, _I, _VP]),
    "pd_append_kv_fp8": (_I, [_VP, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _VP, ctypes.c_float, ctypes.c_float,
                              _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP]),
    "pd_tiled_validate": (_I, [_VP]),
    "pd_tiled_state_bytes": (_I, [_VP, _VP, _VP, _VP, _VP]),
    "pd_tiled_create": (_I, [_VP, _VP]),
    "pd_tiled_destroy": (None, [_VP]),
    "pd_tiled_get_dims": (_I, [_VP, _VP]),
    "pd_tiled_state": (_I, [_VP, _VP, _VP, _VP]),
    "pd_tiled_paged_strides": (None, [_VP, _VP]),
    "pd_tiled_scratch_pool_strides": (None, [_VP, _VP]),
    "pd_tiled_begin": (_I, [_VP, _I, _VP]),
    "pd_tiled_step": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I64, _I64, _I64, _I, _VP]),
    "pd_tiled_finalize": (_I, [_VP, _VP, _I, _VP]),
    "pd_tiled_run": (_I, [_VP, _VP, _VP, _I, _VP, _I, _VP]),
    "pd_device_status": (_I, [_VP]),
    "pd_debug_fail_next_allocs": (None, [_I]),
    "pd_debug_set_tuning": (None, [_I, _I, _I]),
}


def lib():
    """Load libpd.so (built by `__graft_entry__.build()` / `build.py`)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise PdLibraryError(f"{LIB_PATH} is missing: build it with "
                                     "`python -m paged_kv_decode_splitk_gb300.build`")
            try:
                L = ctypes.CDLL(LIB_PATH)
            except OSError as e:
                raise PdLibraryError(f"cannot load {LIB_PATH}: {e}") from e
            for name, (res, args) in _SIGS.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


_quick = None


class _Declined:
    """In the module's place where it cannot be used: declines every call."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


def quick():
    """The CPython module over the library (csrc/pd_binding.cpp), built beside it: api.py's first try at a call.  Where it
    is missing or was built for another torch, every call takes the ctypes binding to the same library, with a warning."""
    global _quick
    if _quick is None:
        import importlib.machinery
        import importlib.util
        import warnings

        import torch  # (its libraries, which the module is linked to)

        lib()
        path = os.path.join(PKG, "_build", "pd_binding.so")
        why = "is missing"
        if os.path.exists(path):
            try:
                loader = importlib.machinery.ExtensionFileLoader("pd_binding", path)
                module = importlib.util.module_from_spec(importlib.util.spec_from_loader("pd_binding", loader))
                loader.exec_module(module)
                if module.built_for == torch.__version__:
                    _quick = module
                why = f"was built for torch {module.built_for}"
            except ImportError as e:
                why = f"does not load ({e})"
        if _quick is None:
            warnings.warn(f"{path} {why}: calls take some 10 us more; build it with `python -m paged_kv_decode_splitk_gb300.build`",
                          RuntimeWarning, stacklevel=3)
            _quick = _Declined()
    return _quick


def header_symbols() -> list[str]:
    """Function names include/pd.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pd_[a-z0-9_]+)\s*\(", text)))


def last_error() -> str:
    return lib().pd_last_error().decode(errors="replace")


def _check(rc: int) -> int:
    if rc < 0:
        raise PdError(rc, last_error())
    return rc


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _wrote(rc: int, *tensors) -> int:
    """_check, and torch learns of the caller's tensors that the library has written, as of its own writes: a gradient that
    has saved one refuses it.  (Tensors of the inference mode have no version.)"""
    if _check(rc) == PD_OK:
        from torch.autograd.graph import increment_version
        for t in tensors:
            if t is not None and not t.is_inference():
                increment_version(t)
    return rc


_torch_device = None  # () -> the current device's number
_torch_stream = None  # (device) -> its current stream's address


def _bind_torch():
    """The two lookups every call makes, by the cheapest way torch has (0.1 us where the public ones, which build
    objects, cost 0.2 and 3)."""
    global _torch_device, _torch_stream
    import torch
    device = getattr(torch._C, "_cuda_getDevice", None) if torch.cuda.is_available() else lambda: 0
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if torch.cuda.is_available():
        torch.cuda.current_device()  # (initialises CUDA, once)
    _torch_device = device or torch.cuda.current_device
    _torch_stream = stream or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def current_device() -> int:
    """Number of the current CUDA device (0 where there is none)."""
    if _torch_device is None:
        _bind_torch()
    return _torch_device()


def _stream(stream) -> int | None:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _torch_stream(current_device()) if _torch_stream is not None else _torch_stream_first()


def _torch_stream_first() -> int:
    _bind_torch()
    return _torch_stream(_torch_device())


# ---- policy -----------------------------------------------------------------

def pd_build_info() -> dict:
    v = [ctypes.c_int() for _ in range(4)]
    _check(lib().pd_build_info(*[ctypes.byref(x) for x in v]))
    return {"max_splits": v[0].value, "pack_width": v[1].value, "pack_head_dim": v[2].value,
            "min_kv_per_split": v[3].value}


def pd_parse_policy(text: str) -> tuple[int, int]:
    pol, pin = ctypes.c_int(), ctypes.c_int()
    _check(lib().pd_parse_policy(text.encode(), ctypes.byref(pol), ctypes.byref(pin)))
    return pol.value, pin.value


def pd_parse_gqa_pack(text: str) -> bool:
    e = ctypes.c_int()
    _check(lib().pd_parse_gqa_pack(text.encode(), ctypes.byref(e)))
    return bool(e.value)


def pd_resolve_policy(declared: str | None, override: str | None) -> tuple[int, int]:
    pol, pin = ctypes.c_int(), ctypes.c_int()
    _check(lib().pd_resolve_policy(None if declared is None else declared.encode(),
                                   None if override is None else override.encode(),
                                   ctypes.byref(pol), ctypes.byref(pin)))
    return pol.value, pin.value


def pd_policy_from_env(declared: str | None) -> tuple[int, int]:
    pol, pin = ctypes.c_int(), ctypes.c_int()
    _check(lib().pd_policy_from_env(None if declared is None else declared.encode(),
                                    ctypes.byref(pol), ctypes.byref(pin)))
    return pol.value, pin.value


def pd_gqa_pack_enabled() -> bool:
    return bool(lib().pd_gqa_pack_enabled())


def pd_split_ref_seqs(num_seqs: int, max_decode_seqs: int) -> int:
    return lib().pd_split_ref_seqs(num_seqs, max_decode_seqs)


def pd_legacy_splits(sm_count: int, num_q_heads: int, ref_seqs: int) -> int:
    return _check(lib().pd_legacy_splits(sm_count, num_q_heads, ref_seqs))


def pd_auto_splits(sm_count: int, num_q_heads: int) -> int:
    return _check(lib().pd_auto_splits(sm_count, num_q_heads))


def pd_num_splits(policy, pin: int, sm_count: int, num_q_heads: int, num_seqs: int,
                  max_decode_seqs: int) -> int:
    if isinstance(policy, str):
        policy = POLICY_NAMES[policy]
    return _check(lib().pd_num_splits(policy, pin, sm_count, num_q_heads, num_seqs, max_decode_seqs))


def pd_workspace_bytes(rows: int, num_q_heads: int, head_dim: int, num_splits: int) -> int:
    return lib().pd_workspace_bytes(rows, num_q_heads, head_dim, num_splits)


def pd_gqa_pack_shape_ok(num_q_heads: int, num_kv_heads: int, head_dim: int) -> bool:
    return bool(lib().pd_gqa_pack_shape_ok(num_q_heads, num_kv_heads, head_dim))


def pd_gqa_pack_ctas(num_kv_heads: int, num_seqs: int) -> int:
    return lib().pd_gqa_pack_ctas(num_kv_heads, num_seqs)


def pd_split_chunk_tokens(context_len: int, num_splits: int, block_size: int) -> int:
    return _check(lib().pd_split_chunk_tokens(context_len, num_splits, block_size))


# ---- paged decode -----------------------------------------------------------------

def pd_decode_attn(q, k_cache, v_cache, block_table, context_lens, out, inv_sqrt_d: float,
                   num_splits: int, workspace=None, gqa_pack: int = 0, stream=None,
                   num_blocks: int | None = None) -> int:
    """out[S, Hq, D] <- paged-decode attention (see pd.h).  Shapes come from the tensors:
    q [S, Hq, D]; k_cache / v_cache [num_blocks, block_size, Hkv, D] BF16; block_table
    [S, max_blocks] int32; context_lens [S] int32; workspace a byte/float tensor or None."""
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_cache.shape
    assert D2 == D, "head_dim mismatch"
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().pd_decode_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                              int(block_table.shape[1]), _ptr(context_lens), _ptr(out), S, Hq, Hkv,
                              D, bs, nb if num_blocks is None else num_blocks, float(inv_sqrt_d),
                              int(num_splits), _ptr(workspace), ws_bytes, int(gqa_pack),
                              _stream(stream))
    return _wrote(rc, out, workspace)


def pd_decode_attn_fp8(q, k_cache, v_cache, k_scale: float, v_scale: float, block_table, context_lens,
                       out, inv_sqrt_d: float, num_splits: int, workspace=None, gqa_pack: int = 0,
                       stream=None, num_blocks: int | None = None) -> int:
    """pd_decode_attn over an FP8 E4M3 cache: k_cache / v_cache uint8 tensors
    [num_blocks, block_size, Hkv, D] of E4M3 codes, K = value * k_scale, V = value * v_scale."""
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_cache.shape
    assert D2 == D, "head_dim mismatch"
    assert k_cache.element_size() == 1 and v_cache.element_size() == 1, "FP8 caches are 1-byte codes"
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().pd_decode_attn_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale),
                                  _ptr(block_table), int(block_table.shape[1]), _ptr(context_lens), _ptr(out),
                                  S, Hq, Hkv, D, bs, nb if num_blocks is None else num_blocks,
                                  float(inv_sqrt_d), int(num_splits), _ptr(workspace), ws_bytes,
                                  int(gqa_pack), _stream(stream))
    return _wrote(rc, out, workspace)


def pd_decode_attn_noalloc(q, k_cache, v_cache, block_table, context_lens, out, inv_sqrt_d: float,
                           num_splits: int, gqa_pack: int = 0, stream=None,
                           num_blocks: int | None = None) -> int:
    """pd_decode_attn with the split-K workspace held by the library (see pd.h): for
    callers that cannot allocate device memory.  Same tensors, shapes and gqa_pack
    modes (0 off, 1 packed non-split, 2 packed with splits), no workspace."""
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_cache.shape
    assert D2 == D, "head_dim mismatch"
    rc = lib().pd_decode_attn_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                      int(block_table.shape[1]), _ptr(context_lens), _ptr(out), S, Hq,
                                      Hkv, D, bs, nb if num_blocks is None else num_blocks,
                                      float(inv_sqrt_d), int(num_splits), int(gqa_pack),
                                      _stream(stream))
    return _wrote(rc, out)


# ---- decode behind shared prefixes ----------------------------------------------------

def pd_prefix_workspace_bytes(num_seqs: int, num_groups: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                              num_splits: int) -> int:
    return lib().pd_prefix_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, num_splits)


def pd_decode_attn_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table, context_lens, out,
                          inv_sqrt_d: float, num_splits: int, workspace, stream=None, num_blocks: int | None = None) -> int:
    """out[S, Hq, D] <- decode attention behind shared prefixes (see pd.h): prefix_table [G, max_prefix_blocks],
    prefix_lens [G], group_starts [G + 1] or None (one group), the rest as for pd_decode_attn."""
    S, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    G, mpb = prefix_table.shape
    return _wrote(lib().pd_decode_attn_prefix(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), prefix_table.data_ptr(), mpb, prefix_lens.data_ptr(),
        _ptr(group_starts), G, block_table.data_ptr(), block_table.shape[1], context_lens.data_ptr(), out.data_ptr(), S, Hq,
        Hkv, D, bs, nb if num_blocks is None else num_blocks, inv_sqrt_d, num_splits, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)), out, workspace)


def pd_decode_attn_prefix_fp8(q, k_cache, v_cache, k_scale: float, v_scale: float, prefix_table, prefix_lens, group_starts,
                              block_table, context_lens, out, inv_sqrt_d: float, num_splits: int, workspace, stream=None,
                              num_blocks: int | None = None) -> int:
    """pd_decode_attn_prefix over an FP8 cache (uint8 E4M3 codes, K = value * k_scale, V = value * v_scale)."""
    S, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    G, mpb = prefix_table.shape
    return _wrote(lib().pd_decode_attn_prefix_fp8(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, prefix_table.data_ptr(), mpb,
        prefix_lens.data_ptr(), _ptr(group_starts), G, block_table.data_ptr(), block_table.shape[1], context_lens.data_ptr(),
        out.data_ptr(), S, Hq, Hkv, D, bs, nb if num_blocks is None else num_blocks, inv_sqrt_d, num_splits, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)), out, workspace)


def pd_debug_prefix_walk(group_starts, prefix_lens, num_q_heads: int, num_kv_heads: int, head_dim: int, fp8: bool = False,
                         own_us: float = 0.0, max_teams: int = 76):
    """The division of a shared-prefix call's work (see pd.h): (segments, parts, totals), lists of tuples and a tuple."""
    G, group = len(prefix_lens), num_q_heads // num_kv_heads
    rows = [(b - a) * group for a, b in zip(group_starts, group_starts[1:])]
    starts, lens = (ctypes.c_int32 * (G + 1))(*group_starts), (ctypes.c_int32 * G)(*prefix_lens)
    most = 4 * max_teams + 2 * sum(num_kv_heads * (r // 128 + 1) for r in rows)  # (a team's run ends an item, or ends itself)
    segments, n = (ctypes.c_int32 * (10 * most))(), ctypes.c_int()
    parts, totals = (ctypes.c_int64 * (3 * num_kv_heads * max(1, sum(rows))))(), (ctypes.c_int32 * 4)()
    _check(lib().pd_debug_prefix_walk(group_starts[-1], G, starts, lens, num_q_heads, num_kv_heads, head_dim, int(fp8), own_us, max_teams,
                                      segments, most, ctypes.byref(n), parts, totals))
    return ([tuple(segments[10 * i:10 * i + 10]) for i in range(n.value)],
            [tuple(parts[3 * i:3 * i + 3]) for i in range(num_kv_heads * sum(rows))], tuple(totals))


# ---- attention of new tokens over the paged cache ---------------------------------------

def pd_chunk_workspace_bytes(num_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return lib().pd_chunk_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, head_dim)


def _window(window: int) -> int:
    """A window as the library takes it: one above 31 bits is more than any table holds."""
    return max(-1, min(window, 2**31 - 1))


def pd_chunk_attn(q, k_cache, v_cache, block_table, context_lens, token_starts, out, lse, inv_sqrt_d: float, window: int, workspace,
                  stream=None, num_blocks: int | None = None) -> int:
    """out[T, Hq, D] (and lse[T, Hq], or None) <- attention of new tokens over a BF16 cache (see pd.h): q [T, Hq, D]
    strided in tokens, token_starts [S + 1] or None (one each), the rest as for pd_decode_attn."""
    T, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    S, mb = block_table.shape
    return _wrote(lib().pd_chunk_attn(
        q.data_ptr(), _token_stride(q), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), mb, context_lens.data_ptr(),
        _ptr(token_starts), out.data_ptr(), _ptr(lse), T, S, Hq, Hkv, D, bs, nb if num_blocks is None else num_blocks, inv_sqrt_d,
        _window(window), _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)),
        out, lse, workspace)


def pd_chunk_attn_fp8(q, k_cache, v_cache, k_scale: float, v_scale: float, block_table, context_lens, token_starts, out, lse,
                      inv_sqrt_d: float, window: int, workspace, stream=None, num_blocks: int | None = None) -> int:
    """pd_chunk_attn over an FP8 cache (uint8 E4M3 codes, K = value * k_scale, V = value * v_scale)."""
    T, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    S, mb = block_table.shape
    return _wrote(lib().pd_chunk_attn_fp8(
        q.data_ptr(), _token_stride(q), k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, block_table.data_ptr(), mb,
        context_lens.data_ptr(), _ptr(token_starts), out.data_ptr(), _ptr(lse), T, S, Hq, Hkv, D, bs,
        nb if num_blocks is None else num_blocks, inv_sqrt_d, _window(window), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)), out, lse, workspace)


def pd_debug_chunk_walk(token_starts, context_lens, num_q_heads: int, num_kv_heads: int, head_dim: int, window: int = 0,
                        max_ctas: int = 152):
    """The division of a chunk attention's work (see pd.h): (segments, totals), a list of tuples and a tuple."""
    S = len(context_lens)
    starts = None if token_starts is None else (ctypes.c_int32 * (S + 1))(*token_starts)
    new = S if token_starts is None else sum(b - a for a, b in zip(token_starts, token_starts[1:]))
    most = max_ctas + num_q_heads * (S + new)  # (an item a query head, block and sequence, and a border's cut)
    segments, n, totals = (ctypes.c_int32 * (11 * most))(), ctypes.c_int(), (ctypes.c_int64 * 6)()
    _check(lib().pd_debug_chunk_walk(S, starts, (ctypes.c_int32 * max(1, S))(*context_lens), num_q_heads, num_kv_heads, head_dim, window,
                                     max_ctas, segments, most, ctypes.byref(n), totals))
    return [tuple(segments[11 * i:11 * i + 11]) for i in range(n.value)], tuple(totals)


# ---- rotary positions and the append to the paged cache ------------------------------

def rope_desc(head_dim: int, rot_dim: int | None = None, *, layout="half", base: float = 10000.0, scaling="none",
              factor: float = 1.0, original_context: float = 0.0, low_turns: float = 0.0, high_turns: float = 0.0,
              attention_factor: float = 0.0, frequencies=None) -> pd_rope_desc:
    """A pd_rope_desc (see pd.h).  layout and scaling by name or value; frequencies (a sequence of
    rot_dim/2 floats) choose the table rule."""
    rot = head_dim if rot_dim is None else rot_dim
    if frequencies is not None:
        scaling = PD_ROPE_TABLE
        freq = [float(f) for f in frequencies]
        if len(freq) != rot // 2:
            raise ValueError(f"rope: {len(freq)} frequencies for rot_dim {rot}: rot_dim/2 are wanted")
        table = (ctypes.c_double * max(1, len(freq)))(*freq)
    else:
        table = None
    for name, value, names in (("layout", layout, ROPE_LAYOUTS), ("scaling", scaling, ROPE_SCALINGS)):
        if isinstance(value, str) and value not in names:
            raise ValueError(f"rope: unknown {name} {value!r}: one of {', '.join(names)}")
    return pd_rope_desc(head_dim, rot, ROPE_LAYOUTS.get(layout, layout), ROPE_SCALINGS.get(scaling, scaling), base, factor,
                        original_context, low_turns, high_turns, attention_factor,
                        ctypes.cast(table, ctypes.POINTER(ctypes.c_double)) if table is not None else None)


def pd_rope_frequencies(desc: pd_rope_desc) -> tuple[list[float], float]:
    """The angles per position (rot_dim/2) and the factor on cosine and sine of a description."""
    f = (ctypes.c_double * max(1, desc.rot_dim // 2))()
    c = ctypes.c_double()
    _check(lib().pd_rope_frequencies(ctypes.byref(desc), f, ctypes.byref(c)))
    return list(f)[: desc.rot_dim // 2], c.value


def pd_rope_create(desc: pd_rope_desc) -> int:
    h = ctypes.c_void_p()
    _check(lib().pd_rope_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def pd_rope_destroy(handle: int) -> None:
    lib().pd_rope_destroy(handle)


class Rope:
    """Owner of a pd_rope handle: one model's rotary positions on the current device."""

    def __init__(self, head_dim, rot_dim=None, **options):
        self.handle = None
        self.desc = rope_desc(head_dim, rot_dim, **options)
        self.head_dim, self.rot_dim = self.desc.head_dim, self.desc.rot_dim
        self.handle = pd_rope_create(self.desc)

    def frequencies(self):
        return pd_rope_frequencies(self.desc)

    def close(self):
        handle, self.handle = self.handle, None  # (from here on nobody is given it)
        if handle:
            pd_rope_destroy(handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _handle(rope):
    if rope is None:
        return None
    h = rope.handle if isinstance(rope, Rope) else rope
    if not h:
        raise ValueError("the rotation's handle is closed")
    return h


def _token_stride(t) -> int:
    """Elements from one token's rows to the next of [T, H, D] (any value serves a single token)."""
    n, h, d = t.shape
    return t.stride(0) if n > 1 else h * d


def pd_rope_apply(rope, x, positions, out, inverse: bool = False, stream=None) -> int:
    """out [T, H, D] <- x [T, H, D] rotated by positions [T] (see pd.h); strided in tokens and heads."""
    T, H, D = x.shape
    return _wrote(lib().pd_rope_apply(_handle(rope), x.data_ptr(), _token_stride(x), x.stride(1) if H > 1 else D,
                                      positions.data_ptr(), out.data_ptr(), _token_stride(out),
                                      out.stride(1) if H > 1 else D, T, H, inverse, _stream(stream)), out)


def pd_append_kv(rope, q, k, v, q_out, k_cache, v_cache, block_table, context_lens, token_starts=None, stream=None,
                 num_blocks: int | None = None) -> int:
    """New tokens' keys (rotated) and values into a BF16 cache, q rotated into q_out (see pd.h).  q, k, v
    [T, H, D] strided in tokens; rope a Rope or None; q and q_out None for keys and values alone."""
    T, Hkv, D = k.shape
    nb, bs = k_cache.shape[:2]
    S, mb = block_table.shape
    return _wrote(lib().pd_append_kv(
        _handle(rope), _ptr(q), 0 if q is None else _token_stride(q), k.data_ptr(), _token_stride(k), v.data_ptr(),
        _token_stride(v), _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), mb,
        context_lens.data_ptr(), _ptr(token_starts), T, S, 0 if q is None else q.shape[1], Hkv, D, bs,
        nb if num_blocks is None else num_blocks, _stream(stream)), q_out, k_cache, v_cache)


def pd_append_kv_fp8(rope, q, k, v, q_out, k_cache, v_cache, k_scale: float, v_scale: float, block_table, context_lens,
                     token_starts=None, stream=None, num_blocks: int | None = None) -> int:
    """pd_append_kv into an FP8 cache (uint8 E4M3 codes of x * (1 / k_scale) and x * (1 / v_scale))."""
    T, Hkv, D = k.shape
    nb, bs = k_cache.shape[:2]
    S, mb = block_table.shape
    return _wrote(lib().pd_append_kv_fp8(
        _handle(rope), _ptr(q), 0 if q is None else _token_stride(q), k.data_ptr(), _token_stride(k), v.data_ptr(),
        _token_stride(v), _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, block_table.data_ptr(),
        mb, context_lens.data_ptr(), _ptr(token_starts), T, S, 0 if q is None else q.shape[1], Hkv, D, bs,
        nb if num_blocks is None else num_blocks, _stream(stream)), q_out, k_cache, v_cache)


def _head_stride(t) -> int:
    """Elements from one head's row to the next of [T, H, D] (any value serves a single head)."""
    return t.stride(1) if t.shape[1] > 1 else t.shape[2]


def pd_norm_rope_apply(rope, x, weight, positions, out, eps: float = 1e-6, weight_offset: float = 0.0, stream=None) -> int:
    """out [T, H, D] <- x [T, H, D], each row's RMS norm times (weight_offset + weight [D]) rotated by positions [T] (see
    pd.h); strided in tokens and heads; rope and positions None for the norm alone, weight None for ones."""
    T, H, D = x.shape
    return _wrote(lib().pd_norm_rope_apply(_handle(rope), x.data_ptr(), _token_stride(x), _head_stride(x), _ptr(weight), eps, weight_offset,
                                           _ptr(positions), out.data_ptr(), _token_stride(out), _head_stride(out), T, H, D,
                                           _stream(stream)), out)


def pd_norm_rope_workspace_bytes(head_dim: int) -> int:
    return lib().pd_norm_rope_workspace_bytes(head_dim)


def pd_norm_rope_backward(rope, x, weight, positions, grad, grad_x, grad_weight, workspace, eps: float = 1e-6, weight_offset: float = 0.0,
                          stream=None) -> int:
    """grad_x [T, H, D] and grad_weight [D] (or None) <- the gradients of pd_norm_rope_apply from the gradient of its out."""
    T, H, D = x.shape
    return _wrote(lib().pd_norm_rope_backward(
        _handle(rope), x.data_ptr(), _token_stride(x), _head_stride(x), _ptr(weight), eps, weight_offset, _ptr(positions), grad.data_ptr(),
        _token_stride(grad), _head_stride(grad), grad_x.data_ptr(), _token_stride(grad_x), _head_stride(grad_x), _ptr(grad_weight), T, H, D,
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)),
        grad_x, grad_weight, workspace)


def pd_append_kv_normed(rope, q, k, v, q_weight, k_weight, q_out, k_cache, v_cache, block_table, context_lens, token_starts=None,
                        eps: float = 1e-6, weight_offset: float = 0.0, stream=None, num_blocks: int | None = None) -> int:
    """pd_append_kv with the RMS norm of each head of q and k before the rotation (weights [D] BF16, or None for ones)."""
    T, Hkv, D = k.shape
    nb, bs = k_cache.shape[:2]
    S, mb = block_table.shape
    return _wrote(lib().pd_append_kv_normed(
        _handle(rope), _ptr(q), 0 if q is None else _token_stride(q), k.data_ptr(), _token_stride(k), v.data_ptr(), _token_stride(v),
        _ptr(q_weight), _ptr(k_weight), eps, weight_offset, _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), mb,
        context_lens.data_ptr(), _ptr(token_starts), T, S, 0 if q is None else q.shape[1], Hkv, D, bs,
        nb if num_blocks is None else num_blocks, _stream(stream)), q_out, k_cache, v_cache)


def pd_append_kv_normed_fp8(rope, q, k, v, q_weight, k_weight, q_out, k_cache, v_cache, k_scale: float, v_scale: float, block_table,
                            context_lens, token_starts=None, eps: float = 1e-6, weight_offset: float = 0.0, stream=None,
                            num_blocks: int | None = None) -> int:
    """pd_append_kv_normed into an FP8 cache (uint8 E4M3 codes of x * (1 / k_scale) and x * (1 / v_scale))."""
    T, Hkv, D = k.shape
    nb, bs = k_cache.shape[:2]
    S, mb = block_table.shape
    return _wrote(lib().pd_append_kv_normed_fp8(
        _handle(rope), _ptr(q), 0 if q is None else _token_stride(q), k.data_ptr(), _token_stride(k), v.data_ptr(), _token_stride(v),
        _ptr(q_weight), _ptr(k_weight), eps, weight_offset, _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale,
        block_table.data_ptr(), mb, context_lens.data_ptr(), _ptr(token_starts), T, S, 0 if q is None else q.shape[1], Hkv, D, bs,
        nb if num_blocks is None else num_blocks, _stream(stream)), q_out, k_cache, v_cache)


# ---- tiled ---------------------------------------------------------------------------

def pd_tiled_validate(dims: pd_tiled_dims) -> None:
    _check(lib().pd_tiled_validate(ctypes.byref(dims)))


def pd_tiled_state_bytes(dims: pd_tiled_dims) -> dict:
    v = [ctypes.c_size_t() for _ in range(4)]
    _check(lib().pd_tiled_state_bytes(ctypes.byref(dims), *[ctypes.byref(x) for x in v]))
    return {"m": v[0].value, "l": v[1].value, "o": v[2].value, "output": v[3].value}


class Tiled:
    """Owner of a pd_tiled handle (TiledAttention): create / begin / step / finalize."""

    def __init__(self, max_seqs, num_q_heads, num_kv_heads, head_dim, block_size, tile_capacity):
        self.dims = pd_tiled_dims(max_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                  tile_capacity)
        self.handle = pd_tiled_create(self.dims)

    def close(self):
        if self.handle:
            pd_tiled_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def paged_strides(self):
        return pd_tiled_paged_strides(self.handle)

    def scratch_pool_strides(self):
        return pd_tiled_scratch_pool_strides(self.handle)

    def begin(self, num_seqs, stream=None):
        return pd_tiled_begin(self.handle, num_seqs, stream)

    def step(self, q, k_pool, v_pool, tile_blocks, tile_block_counts, num_seqs, strides,
             last_block_valid_slots, stream=None):
        return pd_tiled_step(self.handle, q, k_pool, v_pool, tile_blocks, tile_block_counts,
                             num_seqs, strides, last_block_valid_slots, stream)

    def finalize(self, out, num_seqs, stream=None):
        return pd_tiled_finalize(self.handle, out, num_seqs, stream)

    def run(self, q, sources, out, num_seqs, stream=None):
        return pd_tiled_run(self.handle, q, sources, out, num_seqs, stream)

    def state(self):
        return pd_tiled_state(self.handle)


def pd_tiled_create(dims: pd_tiled_dims) -> int:
    h = ctypes.c_void_p()
    _check(lib().pd_tiled_create(ctypes.byref(dims), ctypes.byref(h)))
    return h.value


def pd_tiled_destroy(handle: int) -> None:
    lib().pd_tiled_destroy(handle)


def pd_tiled_get_dims(handle: int) -> pd_tiled_dims:
    d = pd_tiled_dims()
    _check(lib().pd_tiled_get_dims(handle, ctypes.byref(d)))
    return d


def pd_tiled_state(handle: int) -> tuple[int, int, int]:
    m, l_, o = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().pd_tiled_state(handle, ctypes.byref(m), ctypes.byref(l_), ctypes.byref(o)))
    return m.value, l_.value, o.value


def pd_tiled_paged_strides(handle: int) -> tuple[int, int, int]:
    s = (ctypes.c_int64 * 3)()
    lib().pd_tiled_paged_strides(handle, s)
    return tuple(s)


def pd_tiled_scratch_pool_strides(handle: int) -> tuple[int, int, int]:
    s = (ctypes.c_int64 * 3)()
    lib().pd_tiled_scratch_pool_strides(handle, s)
    return tuple(s)


def pd_tiled_begin(handle: int, num_seqs: int, stream=None) -> int:
    return _check(lib().pd_tiled_begin(handle, num_seqs, _stream(stream)))


def pd_tiled_step(handle: int, q, k_pool, v_pool, tile_blocks, tile_block_counts, num_seqs: int,
                  strides, last_block_valid_slots: int, stream=None) -> int:
    blk, tok, kvh = (int(x) for x in strides)
    return _check(lib().pd_tiled_step(handle, _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(tile_blocks),
                                      _ptr(tile_block_counts), num_seqs, blk, tok, kvh,
                                      int(last_block_valid_slots), _stream(stream)))


def pd_tiled_run(handle: int, q, sources, out, num_seqs: int, stream=None) -> int:
    """begin, one step per source, finalize.  sources: sequence of
    (k_pool, v_pool, tile_blocks, tile_block_counts, strides, last_block_valid_slots)."""
    arr = (pd_tiled_source * max(1, len(sources)))()
    for i, (k, v, tb, tc, strides, lbvs) in enumerate(sources):
        blk, tok, kvh = (int(x) for x in strides)
        arr[i] = pd_tiled_source(_ptr(k), _ptr(v), _ptr(tb), _ptr(tc), blk, tok, kvh, int(lbvs))
    return _wrote(lib().pd_tiled_run(handle, _ptr(q), ctypes.cast(arr, _VP) if sources else None,
                                     len(sources), _ptr(out), num_seqs, _stream(stream)), out)


def pd_tiled_finalize(handle: int, out, num_seqs: int, stream=None) -> int:
    return _wrote(lib().pd_tiled_finalize(handle, _ptr(out), num_seqs, _stream(stream)), out)


# ---- diagnostics -------------------------------------------------------------------

def pd_device_status() -> int:
    f = ctypes.c_int()
    _check(lib().pd_device_status(ctypes.byref(f)))
    return f.value


def pd_debug_fail_next_allocs(count: int) -> None:
    lib().pd_debug_fail_next_allocs(count)


def pd_debug_set_tuning(stages_per_warp: int = 0, cluster: int = 0, longest_first: int = -1) -> None:
    lib().pd_debug_set_tuning(stages_per_warp, cluster, longest_first)
