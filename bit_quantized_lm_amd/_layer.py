"""ctypes binding of the draft layer's attention (include/draftlayer.h), same names as the C ABI.

As in `_binding`: argument marshalling only, torch for device memory and
streams, outputs allocated where the caller passes none, errors as ValueError
(an argument) or DraftHeadError (the runtime).  Shapes, types and devices of the
tensors are checked here, since the library sees only pointers.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

import numpy as np

from . import _binding as B

_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "draftlayer.h")
PAGES = (32, 64, 128, 256)     # tokens a page may hold
HEAD_DIMS = (64, 128, 256)
WORKSPACE_ZERO_BYTES = 6144    # DL_WORKSPACE_ZERO_BYTES

_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = B.load_library()
        P, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                     ctypes.c_size_t)
        for name, types in (
                ("draft_layer_rope_table", [i32, i32, f64, f64, i32, f64, f64, f64, P]),
                ("draft_layer_append", [P, i64, P, i64, P, i64, P, i32, i32, i32, P, P, P, P, i32, i32, P, P, P, i32, i32,
                                        i32, i32, i32, i32, P, P]),
                ("draft_layer_read", [P, P, P, P, i32, i32, P, P, P, i32, i32, i32, i32, i32, P, P, P]),
                ("draft_layer_workspace_bytes", [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]),
                ("draft_layer_attend", [P, i64, P, P, P, P, i32, i32, P, P, P, i32, i32, i32, i32, i32, i32, f32, i32, i32, P,
                                        P, P, sz, P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = i32, types
        _lib = lib
    return _lib


torch = None     # set by the first device call
_U8 = _F32 = _I32 = _BF16 = None


def _device_lib():
    """The library, with torch at hand (host functions need none)."""
    global torch, _U8, _F32, _I32, _BF16
    if torch is None:
        import torch as t
        torch, _U8, _F32, _I32, _BF16 = t, t.uint8, t.float32, t.int32, t.bfloat16
    return _load()


def layer_header_functions() -> list[str]:
    """Names of the functions include/draftlayer.h declares."""
    with open(_HEADER) as f:
        return re.findall(r"^int (draft_layer_\w+)\s*\(", f.read(), flags=re.M)


# ------------------------------------------------------------------ host side
def draft_layer_rope_table(positions: int, rot: int, base: float = 10000.0, factor: float = 1.0, original: int = 0,
                           beta_fast: float = 32.0, beta_slow: float = 1.0, mscale: float | None = None) -> np.ndarray:
    """(cos, sin) of the rotary angles, fp32 [positions][rot/2][2].

    factor > 1 stretches them for contexts longer than the trained one: all
    alike (original = 0), or by YaRN's ramp for a model trained on `original`
    positions.  mscale: the factor on both (None: 1, and YaRN's
    0.1 ln(factor) + 1 where its ramp is used)."""
    lib = _load()
    if mscale is None:
        mscale = 0.1 * math.log(factor) + 1.0 if original > 0 and factor > 1.0 else 1.0
    out = np.empty((max(positions, 0), max(rot // 2, 0), 2), dtype=np.float32)
    B._check(lib.draft_layer_rope_table(positions, rot, base, factor, original, beta_fast, beta_slow, mscale, B._ptr(out)))
    return out


# ------------------------------------------------------------------ device side
# The checks run before every launch: each is one expression of the cheapest
# calls, and says what is wrong only once something is.
def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _wrong(name, t, dtype, shape, dev):
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {dev}, "
                     f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _is(t, dtype, shape, dev):
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape


def _rows3(name, t, dev, heads, d):
    """Row stride of a bf16 [T][heads][D] tensor whose rows may have gaps (heads None: any number)."""
    shape = t.shape
    if t.dtype is not _BF16 or len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads) or t.get_device() != dev:
        _wrong(name, t, _BF16, ("T", "heads" if heads is None else heads, d), dev)
    if shape[0] == 0:
        return shape[1] * d
    row, head, one = t.stride()
    if one != 1 or (head != d and shape[1] != 1):
        raise ValueError(f"{name}'s heads must be contiguous in a row")
    return row if shape[0] > 1 else shape[1] * d


def _cache(k_codes, v_codes, k_scale, v_scale):
    """Checks a cache's four tensors; (GPU index, pages, kv heads, page, D)."""
    shape = k_codes.shape
    if len(shape) != 4:
        raise ValueError("k_codes must be [pages][heads][page][D]")
    dev = k_codes.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"the cache must be on the current GPU, not on {k_codes.device}")
    pages, heads, page, d = shape
    flat = (pages, heads)
    if (k_codes.dtype is _U8 and v_codes.dtype is _U8 and k_scale.dtype is _F32 and v_scale.dtype is _F32
            and v_codes.get_device() == dev and k_scale.get_device() == dev and v_scale.get_device() == dev
            and k_codes.is_contiguous() and v_codes.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()
            and v_codes.shape == shape and k_scale.shape == flat and v_scale.shape == flat):
        return dev, pages, heads, page, d
    for name, t, dtype, want in (("k_codes", k_codes, _U8, shape), ("v_codes", v_codes, _U8, shape),
                                 ("k_scale", k_scale, _F32, flat), ("v_scale", v_scale, _F32, flat)):
        if not _is(t, dtype, want, dev):
            _wrong(name, t, dtype, want, dev)


def _batch(q_start, kv_len, table, dev):
    """Checks a batch's tensors; (sequences, pages a sequence)."""
    shape = table.shape
    if len(shape) != 2:
        raise ValueError("table must be [sequences][pages]")
    n = shape[0]
    if (q_start.dtype is _I32 and kv_len.dtype is _I32 and table.dtype is _I32
            and q_start.get_device() == dev and kv_len.get_device() == dev and table.get_device() == dev
            and q_start.is_contiguous() and kv_len.is_contiguous() and table.is_contiguous()
            and q_start.shape == (n + 1,) and kv_len.shape == (n,)):
        return shape
    for name, t, want in (("q_start", q_start, (n + 1,)), ("kv_len", kv_len, (n,)), ("table", table, shape)):
        if not _is(t, _I32, want, dev):
            _wrong(name, t, _I32, want, dev)


def _raw_stream(stream, dev):
    """The hipStream_t of `stream` (None: the current one, without building torch's object for it)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else B._stream(stream)


def _out(given, name, like, shape, dtype, dev, stream):
    """The caller's tensor, checked, or a new one (kept for `stream`, if that is not the current one)."""
    if given is not None:
        if not _is(given, dtype, shape, dev):
            _wrong(name, given, dtype, shape, dev)
        return given
    t = like.new_empty(shape) if like.dtype is dtype else like.new_empty(shape, dtype=dtype)
    if stream is not None:
        B._keep_for((t,), stream)
    return t


def draft_layer_append(q, k, v, rope, k_codes, v_codes, k_scale, v_scale, q_start, kv_len, table, interleaved: bool = False,
                       q_out=None, stream=None):
    """Rotate q and k by their positions and write k and v to the cache in 8 bits.

    q: CUDA bf16 [T][hq][D] (or None: keys and values only), k, v: bf16
    [T][hkv][D], rows with gaps allowed (slices of one projection); rope: fp32
    [positions][rot/2][2] (None: no rotation); the cache and the batch as
    include/draftlayer.h has them.  Returns the rotated q, bf16 [T][hq][D]
    (q_out may be q itself where q has no gaps)."""
    lib = _device_lib()
    dev, n_pages, hkv, page, d = _cache(k_codes, v_codes, k_scale, v_scale)
    n_seq, max_pages = _batch(q_start, kv_len, table, dev)
    ldk, ldv = _rows3("k", k, dev, hkv, d), _rows3("v", v, dev, hkv, d)
    rows = k.shape[0]
    _need(v.shape[0] == rows, "k and v must have as many rows")
    hq, ldq = hkv, 0
    if q is None:
        _need(q_out is None, "q_out needs q")
    else:
        ldq, hq = _rows3("q", q, dev, None, d), q.shape[1]
        _need(q.shape[0] == rows, "q and k must have as many rows")
        q_out = _out(q_out, "q_out", q, (rows, hq, d), _BF16, dev, stream)
    positions = rot = 0
    if rope is not None:
        if rope.dim() != 3 or rope.shape[2] != 2 or not _is(rope, _F32, rope.shape, dev):
            _wrong("rope", rope, _F32, ("positions", "rot/2", 2), dev)
        positions, rot = rope.shape[0], rope.shape[1] * 2
    B._check(lib.draft_layer_append(
        None if q is None else q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, None if rope is None else rope.data_ptr(),
        positions, rot, 1 if interleaved else 0, k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        n_pages, page, q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), n_seq, max_pages, rows, hq, hkv, d,
        None if q is None else q_out.data_ptr(), _raw_stream(stream, dev)))
    return q_out


def draft_layer_read(k_codes, v_codes, k_scale, v_scale, q_start, kv_len, table, rows: int, k_out=None, v_out=None, stream=None):
    """The last tokens of each sequence out of the cache: sequence s's
    q_start[s+1] - q_start[s] last ones, `rows` in all.  Returns (k, v), bf16
    [rows][hkv][D]; rows from q_start[-1] on are not written."""
    lib = _device_lib()
    dev, n_pages, hkv, page, d = _cache(k_codes, v_codes, k_scale, v_scale)
    n_seq, max_pages = _batch(q_start, kv_len, table, dev)
    shape = (max(rows, 0), hkv, d)
    k_out = _out(k_out, "k_out", k_codes, shape, _BF16, dev, stream)
    v_out = _out(v_out, "v_out", k_codes, shape, _BF16, dev, stream)
    B._check(lib.draft_layer_read(
        k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n_pages, page, q_start.data_ptr(),
        kv_len.data_ptr(), table.data_ptr(), n_seq, max_pages, rows, hkv, d, k_out.data_ptr(), v_out.data_ptr(),
        _raw_stream(stream, dev)))
    return k_out, v_out


def draft_layer_workspace_bytes(rows: int, n_seq: int, hq: int, hkv: int, d: int) -> int:
    """Device workspace bytes draft_layer_attend needs at most for calls of up to
    `rows` rows of up to n_seq sequences."""
    lib = _load()
    out = ctypes.c_size_t()
    B._check(lib.draft_layer_workspace_bytes(rows, n_seq, hq, hkv, d, ctypes.byref(out)))
    return out.value


def draft_layer_workspace(rows: int, n_seq: int, hq: int, hkv: int, d: int, device):
    """A device workspace for draft_layer_attend's calls of up to `rows` rows of up
    to n_seq sequences (the part that must start at zero is cleared here; the
    library keeps it at zero)."""
    import torch
    size = draft_layer_workspace_bytes(rows, n_seq, hq, hkv, d)
    if size <= 16 << 20:
        # few rows (8.5 MB): clearing all hides behind the host's call, 17.3 us, which a view of the counters makes 18.6
        return torch.zeros(size, dtype=torch.uint8, device=device)
    t = torch.empty(size, dtype=torch.uint8, device=device)
    t.narrow(0, 0, WORKSPACE_ZERO_BYTES).zero_()
    return t


def draft_layer_attend(q, k_codes, v_codes, k_scale, v_scale, q_start, kv_len, table, scale: float | None = None, window: int = 0,
                       sinks: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of the rows over the cache.

    q: CUDA bf16 [T][hq][D], rows with gaps allowed; scale: None for
    1/sqrt(D); window > 0: a row sees the last `window` tokens up to its own and
    the first `sinks`; workspace: from draft_layer_workspace (allocated when
    None).  Returns (out bf16 [T][hq][D], lse fp32 [T][hq]); rows from
    q_start[-1] on are not written."""
    lib = _device_lib()
    dev, n_pages, hkv, page, d = _cache(k_codes, v_codes, k_scale, v_scale)
    n_seq, max_pages = _batch(q_start, kv_len, table, dev)
    ldq = _rows3("q", q, dev, None, d)
    rows, hq = q.shape[0], q.shape[1]
    out = _out(out, "out", q, (rows, hq, d), _BF16, dev, stream)
    lse = _out(lse, "lse", k_scale, (rows, hq), _F32, dev, stream)
    if workspace is None:
        workspace = draft_layer_workspace(rows, n_seq, hq, hkv, d, dev)
        if stream is not None:
            B._keep_for((workspace,), stream)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on GPU {dev}")
    B._check(lib.draft_layer_attend(
        q.data_ptr(), ldq, k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n_pages, page,
        q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), n_seq, max_pages, rows, hq, hkv, d,
        1.0 / math.sqrt(d) if scale is None else scale, window, sinks, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)))
    return out, lse


class DraftCache:
    """A paged cache in 8 bits: codes and scales of `n_pages` pages of `page`
    tokens for one layer.  Which page belongs to which sequence is the caller's
    to say, in each call's table."""

    def __init__(self, n_pages: int, hkv: int, d: int, page: int = 64, device="cuda"):
        import torch
        _need(page in PAGES, f"page must be one of {PAGES}")
        _need(d in HEAD_DIMS, f"d must be one of {HEAD_DIMS}")
        _need(n_pages > 0 and hkv > 0, "n_pages and hkv must be positive")
        self.n_pages, self.hkv, self.d, self.page = n_pages, hkv, d, page
        self.k_codes, self.v_codes = (torch.full((n_pages, hkv, page, d), 128, dtype=torch.uint8, device=device) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones((n_pages, hkv), dtype=torch.float32, device=device) for _ in range(2))

    @property
    def tensors(self):
        return self.k_codes, self.v_codes, self.k_scale, self.v_scale

    def append(self, q, k, v, rope, q_start, kv_len, table, interleaved=False, q_out=None, stream=None):
        return draft_layer_append(q, k, v, rope, *self.tensors, q_start, kv_len, table, interleaved=interleaved, q_out=q_out,
                                  stream=stream)

    def read(self, q_start, kv_len, table, rows, stream=None):
        return draft_layer_read(*self.tensors, q_start, kv_len, table, rows, stream=stream)

    def attend(self, q, q_start, kv_len, table, scale=None, window=0, sinks=0, out=None, lse=None, workspace=None, stream=None):
        return draft_layer_attend(q, *self.tensors, q_start, kv_len, table, scale=scale, window=window, sinks=sinks, out=out,
                                  lse=lse, workspace=workspace, stream=stream)

    def attend_branches(self, q, q_start, kv_len, table, group_start, prefix_len, scale=None, window=0, sinks=0, out=None, lse=None,
                        workspace=None, stream=None):
        from ._branch import draft_branch_attend
        return draft_branch_attend(q, *self.tensors, q_start, kv_len, table, group_start, prefix_len, scale=scale, window=window,
                                   sinks=sinks, out=out, lse=lse, workspace=workspace, stream=stream)

    def fork(self, uses, table, kv_len, parents, need, uses_out=None, table_out=None, status=None, workspace=None, stream=None):
        from ._branch import draft_branch_fork
        return draft_branch_fork(*self.tensors, uses, table, kv_len, parents, need, uses_out=uses_out, table_out=table_out,
                                 status=status, workspace=workspace, stream=stream)

    def compact(self, uses, table, uses_out=None, table_out=None, status=None, workspace=None, stream=None):
        from ._branch import draft_branch_compact
        return draft_branch_compact(*self.tensors, uses, table, uses_out=uses_out, table_out=table_out, status=status,
                                    workspace=workspace, stream=stream)
