"""ctypes binding of the operators on several branches of one context
(include/draftbranch.h), same names as the C ABI.

As in `_layer`: argument marshalling only, shapes, types and devices checked
here, outputs and workspaces allocated where the caller passes none, errors as
ValueError (an argument) or DraftHeadError (the runtime).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re

from . import _binding as B
from . import _layer as L

_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "draftbranch.h")
DB_BF16, DB_FP32 = 0, 1
MAX_TOP = 64          # DB_MAX_TOP

_lib = None
torch = None          # set by the first device call


def _load():
    global _lib
    if _lib is None:
        lib = B.load_library()
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        for name, types in (
                ("draft_branch_pages_workspace_bytes", [i32, i32, ctypes.POINTER(sz)]),
                ("draft_branch_fork", [P, P, P, P, i32, i32, i32, i32, P, P, P, i32, P, P, i32, i32, P, P, P, P, sz, P]),
                ("draft_branch_compact", [P, P, P, P, i32, i32, i32, i32, P, P, i32, i32, P, P, P, P, sz, P]),
                ("draft_branch_attend_workspace_bytes", [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]),
                ("draft_branch_attend", [P, i64, P, P, P, P, i32, i32, P, P, P, i32, i32, P, P, i32, i32, i32, i32, i32, f32, i32, i32, P,
                                         P, P, sz, P]),
                ("draft_branch_logprobs_workspace_bytes", [i32, i32, i32, ctypes.POINTER(sz)]),
                ("draft_branch_logprobs", [P, i32, i64, i32, i32, f32, P, P, i32, i32, P, P, P, P, P, P, sz, P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = i32, types
        _lib = lib
    return _lib


def _device_lib():
    """The library, with torch at hand (the sizes of workspaces need none)."""
    global torch
    if torch is None:
        L._device_lib()
        torch = L.torch
    return _load()


def branch_header_functions() -> list[str]:
    """Names of the functions include/draftbranch.h declares."""
    with open(_HEADER) as f:
        return re.findall(r"^int (draft_branch_\w+)\s*\(", f.read(), flags=re.M)


@functools.lru_cache(maxsize=256, typed=True)
def _size(name, *args) -> int:
    out = ctypes.c_size_t()
    B._check(getattr(_load(), name)(*args, ctypes.byref(out)))
    return out.value


def _workspace(given, size, dev, stream):
    """(address, bytes) of the caller's workspace, checked, or of a new one of size() bytes; the tensor itself."""
    if given is None:
        given = torch.empty(size(), dtype=torch.uint8, device=f"cuda:{dev}")
        if stream is not None:
            B._keep_for((given,), stream)
    elif given.get_device() != dev or not given.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on GPU {dev}")
    return given.data_ptr(), given.numel() * given.element_size(), given


def _ints(name, t, shape, dev):
    if not L._is(t, L._I32, shape, dev):
        L._wrong(name, t, L._I32, shape, dev)


# --------------------------------------------------------------------- pages
def draft_branch_pages_workspace_bytes(n_pages: int, n_new: int) -> int:
    """Device workspace bytes of draft_branch_fork (to at most n_new rows) and
    draft_branch_compact over a pool of n_pages."""
    return _size("draft_branch_pages_workspace_bytes", n_pages, n_new)


def draft_branch_pages_workspace(n_pages: int, n_new: int, device):
    """A device workspace for them; it may hold anything."""
    import torch
    return torch.empty(draft_branch_pages_workspace_bytes(n_pages, n_new), dtype=torch.uint8, device=device)


def _pages(k_codes, v_codes, k_scale, v_scale, uses, table, made, uses_out, table_out, status, stream):
    """Checks what fork and compact have in common; makes the outputs that are not given."""
    dev, n_pages, hkv, page, d = L._cache(k_codes, v_codes, k_scale, v_scale)
    if len(table.shape) != 2:
        raise ValueError("table must be [sequences][pages]")
    _ints("table", table, table.shape, dev)
    _ints("uses", uses, (n_pages,), dev)
    wide = table.shape[1]
    if uses_out is None and table_out is None and status is None:      # one allocation, 1.4 us of the host's time each
        uses_out, table_out, status = L._out(None, "", uses, (n_pages + made * wide + 2,), L._I32, dev, stream).split_with_sizes(
            (n_pages, made * wide, 2))
        table_out = table_out.view(made, wide)
    else:
        uses_out = L._out(uses_out, "uses_out", uses, (n_pages,), L._I32, dev, stream)
        table_out = L._out(table_out, "table_out", table, (made, wide), L._I32, dev, stream)
        status = L._out(status, "status", uses, (2,), L._I32, dev, stream)
    return dev, (k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n_pages, page, hkv, d), uses_out, table_out, status


def draft_branch_fork(k_codes, v_codes, k_scale, v_scale, uses, table, kv_len, parents, need, uses_out=None, table_out=None,
                      status=None, workspace=None, stream=None):
    """The next batch's page table from the present one.

    uses: CUDA int32 [pages], table entries that name each page; table, kv_len:
    the present batch's; parents: int32 [rows], the present sequence that each new
    row goes on from (another number: none, the row starts empty); need: int32
    [rows], positions that it has to have pages for.  Returns (table_out int32
    [rows][max_pages], uses_out, status int32 [2]: free pages after the call,
    pages that were lacking, with nothing done where that is not 0)."""
    lib = _device_lib()
    L._need(len(parents.shape) == 1, "parents must be [rows]")
    made = parents.shape[0]
    dev, pool, uses_out, table_out, status = _pages(k_codes, v_codes, k_scale, v_scale, uses, table, made, uses_out, table_out, status, stream)
    n_seq, wide = table.shape
    _ints("kv_len", kv_len, (n_seq,), dev)
    _ints("parents", parents, (made,), dev)
    _ints("need", need, (made,), dev)
    at, size, _held = _workspace(workspace, lambda: draft_branch_pages_workspace_bytes(pool[4], made), dev, stream)
    B._check(lib.draft_branch_fork(
        *pool, uses.data_ptr(), table.data_ptr(), kv_len.data_ptr(), n_seq, parents.data_ptr(), need.data_ptr(), made, wide,
        uses_out.data_ptr(), table_out.data_ptr(), status.data_ptr(), at, size, L._raw_stream(stream, dev)))
    return table_out, uses_out, status


def draft_branch_compact(k_codes, v_codes, k_scale, v_scale, uses, table, uses_out=None, table_out=None, status=None, workspace=None,
                         stream=None):
    """Moves the pages in use to the pool's front.  table: CUDA int32
    [rows][max_pages], every row that names a page of the pool.  Returns
    (table_out, uses_out, status int32 [2]: pages in use, pages moved)."""
    lib = _device_lib()
    dev, pool, uses_out, table_out, status = _pages(k_codes, v_codes, k_scale, v_scale, uses, table, table.shape[0], uses_out, table_out,
                                                    status, stream)
    at, size, _held = _workspace(workspace, lambda: draft_branch_pages_workspace_bytes(pool[4], 1), dev, stream)
    B._check(lib.draft_branch_compact(
        *pool, uses.data_ptr(), table.data_ptr(), table.shape[0], table.shape[1], uses_out.data_ptr(), table_out.data_ptr(),
        status.data_ptr(), at, size, L._raw_stream(stream, dev)))
    return table_out, uses_out, status


# ----------------------------------------------------------------- attention
def draft_branch_attend_workspace_bytes(rows: int, n_seq: int, hq: int, hkv: int, d: int) -> int:
    """Device workspace bytes of draft_branch_attend's calls of up to `rows` rows
    of up to n_seq sequences."""
    return _size("draft_branch_attend_workspace_bytes", rows, n_seq, hq, hkv, d)


def draft_branch_attend_workspace(rows: int, n_seq: int, hq: int, hkv: int, d: int, device):
    """A device workspace for them; it may hold anything."""
    import torch
    return torch.empty(draft_branch_attend_workspace_bytes(rows, n_seq, hq, hkv, d), dtype=torch.uint8, device=device)


def draft_branch_attend(q, k_codes, v_codes, k_scale, v_scale, q_start, kv_len, table, group_start, prefix_len, scale: float | None = None,
                        window: int = 0, sinks: int = 0, out=None, lse=None, workspace=None, stream=None):
    """draft_layer_attend for sequences that share prefixes, each read once but
    for short contexts and groups of long members (include/draftbranch.h).

    group_start: CUDA int32 [groups + 1]: sequences group_start[g] ..
    group_start[g+1] - 1 share the tokens of the positions below prefix_len[g]
    (int32 [groups]), which are read from the pages of the first one's table row.
    The rest as draft_layer_attend.  Returns (out bf16 [T][hq][D], lse fp32
    [T][hq]); rows from q_start[-1] on are not written."""
    lib = _device_lib()
    dev, n_pages, hkv, page, d = L._cache(k_codes, v_codes, k_scale, v_scale)
    n_seq, max_pages = L._batch(q_start, kv_len, table, dev)
    n_groups = prefix_len.shape[0] if len(prefix_len.shape) == 1 else 0
    if not (L._is(group_start, L._I32, (n_groups + 1,), dev) and L._is(prefix_len, L._I32, (n_groups,), dev)):
        _ints("prefix_len", prefix_len, (n_groups,), dev)
        _ints("group_start", group_start, (n_groups + 1,), dev)
    ldq = L._rows3("q", q, dev, None, d)
    rows, hq = q.shape[0], q.shape[1]
    out = L._out(out, "out", q, (rows, hq, d), L._BF16, dev, stream)
    lse = L._out(lse, "lse", k_scale, (rows, hq), L._F32, dev, stream)
    at, size, _held = _workspace(workspace, lambda: draft_branch_attend_workspace_bytes(rows, n_seq, hq, hkv, d), dev, stream)
    B._check(lib.draft_branch_attend(
        q.data_ptr(), ldq, k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n_pages, page,
        q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), n_seq, max_pages, group_start.data_ptr(), prefix_len.data_ptr(), n_groups,
        rows, hq, hkv, d, 1.0 / math.sqrt(d) if scale is None else scale, window, sinks, out.data_ptr(), lse.data_ptr(), at, size,
        L._raw_stream(stream, dev)))
    return out, lse


# ---------------------------------------------------------- log probabilities
def draft_branch_logprobs_workspace_bytes(rows: int, vocab: int, top: int = 0) -> int:
    """Device workspace bytes of draft_branch_logprobs' calls of up to `rows`
    rows of up to `vocab` logits with up to `top` alternatives."""
    return _size("draft_branch_logprobs_workspace_bytes", rows, vocab, top)


def draft_branch_logprobs_workspace(rows: int, vocab: int, top: int, device):
    """A device workspace for them; it may hold anything."""
    import torch
    return torch.empty(draft_branch_logprobs_workspace_bytes(rows, vocab, top), dtype=torch.uint8, device=device)


def draft_branch_logprobs(logits, tokens=None, top: int = 0, scale: float = 1.0, scales=None, logprob=None, top_id=None,
                          top_logprob=None, lse=None, entropy=None, workspace=None, stream=None):
    """Log probabilities under the softmax of scale * (scales[m]) * logits.

    logits: CUDA bf16, int16 (bf16 bits, as the head's row has them) or fp32
    [M][N], rows with gaps allowed; tokens: int32 [M][any] (None: none asked
    for); top: how many best alternatives; scales: fp32 [M], a factor a row.
    Returns (logprob fp32 [M][any], top_id int32 [M][top], top_logprob fp32
    [M][top], lse fp32 [M], entropy fp32 [M])."""
    lib = _device_lib()
    shape, dtype = logits.shape, logits.dtype
    dev = logits.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"logits must be on the current GPU, not on {logits.device}")
    kind = DB_FP32 if dtype is L._F32 else DB_BF16
    if len(shape) != 2 or (dtype is not L._BF16 and dtype is not torch.int16 and dtype is not L._F32) or (
            shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be bf16, int16 (bf16 bits) or fp32 rows [M][N] without gaps in a row, not {dtype} {tuple(shape)}")
    rows, n = shape
    ld = logits.stride(0) if rows > 1 else n
    if scales is not None and not L._is(scales, L._F32, (rows,), dev):
        L._wrong("scales", scales, L._F32, (rows,), dev)
    n_tok = 0
    if tokens is not None:
        if len(tokens.shape) != 2:
            raise ValueError("tokens must be [M][any]")
        n_tok = tokens.shape[1]
        _ints("tokens", tokens, (rows, n_tok), dev)
    L._need(top >= 0, "top must be >= 0")
    like = logits
    if logprob is None and top_logprob is None and lse is None and entropy is None:      # one allocation, 1.4 us of the host's time each
        logprob, top_logprob, lse, entropy = L._out(None, "", like, (rows * (n_tok + top + 2),), L._F32, dev, stream).split_with_sizes(
            (rows * n_tok, rows * top, rows, rows))
        logprob, top_logprob = logprob.view(rows, n_tok), top_logprob.view(rows, top)
    else:
        logprob = L._out(logprob, "logprob", like, (rows, n_tok), L._F32, dev, stream)
        top_logprob = L._out(top_logprob, "top_logprob", like, (rows, top), L._F32, dev, stream)
        lse = L._out(lse, "lse", like, (rows,), L._F32, dev, stream)
        entropy = L._out(entropy, "entropy", like, (rows,), L._F32, dev, stream)
    top_id = L._out(top_id, "top_id", like, (rows, top), L._I32, dev, stream)
    at, size, _held = _workspace(workspace, lambda: draft_branch_logprobs_workspace_bytes(rows, n, top), dev, stream)
    B._check(lib.draft_branch_logprobs(
        logits.data_ptr(), kind, ld, rows, n, scale, None if scales is None else scales.data_ptr(), None if tokens is None else tokens.data_ptr(),
        n_tok, top, logprob.data_ptr(), lse.data_ptr(), entropy.data_ptr(), top_id.data_ptr(), top_logprob.data_ptr(), at, size,
        L._raw_stream(stream, dev)))
    return logprob, top_id, top_logprob, lse, entropy
