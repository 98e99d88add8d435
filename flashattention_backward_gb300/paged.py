"""Paged key-value cache: the attention of one new token, and its pages.

Argument marshalling for the ``fa_decode``, ``fa_cache_*`` and ``fa_pages_*``
entry points of ``include/fa.h``, whose kernels do all the work.

A cache is two pools ``k_pages`` and ``v_pages`` of shape
``[pages, kv_heads, page_rows, d]`` (bf16 or fp32; ``[pages, page_rows,
kv_heads, d]`` storage works through ``.permute(0, 2, 1, 3)`` views), and three
int32 tensors: ``page_table [sequences, columns]``, ``lengths [sequences]``
and, for the page calls, ``refs [pages]``.  Row ``j`` of a sequence is row
``j % page_rows`` of page ``page_table[s, j // page_rows]``.  An empty cache is
a table of -1, lengths of 0 and refs of 0::

    start = fa.pages_extend(table, lengths, refs, n_new, page_rows)
    fa.cache_append(k_new, v_new, k_pages, v_pages, table, start, n_new)
    o, L = fa.attention_decode(q, k_pages, v_pages, table, lengths)

Nothing here waits for the GPU or reads back from it, so a whole step can be
captured into a graph.  What is wrong on the device (a page or index out of
range, too few free pages) is never followed; it is recorded in the device
status word, which :func:`get_device_status` reads and ``check_status=True``
raises as :class:`FaError`.

No call here has a gradient.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

import flashattention_backward_gb300 as _pkg

_BF16, _FP32 = 0, 1
_i32, _i64, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class FaCache(ctypes.Structure):
    _fields_ = [
        ("num_pages", _i32),
        ("page_rows", _i32),
        ("H_kv", _i32),
        ("d", _i32),
        ("dtype", _i32),
        ("S", _i32),
        ("max_pages", _i32),
        ("reserved", _i32),
        ("stride_page", _i64),
        ("stride_h", _i64),
        ("stride_n", _i64),
        ("table_stride", _i64),
    ]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the paged-cache entry points."""
    P = ctypes.POINTER(FaCache)
    lib.fa_decode_workspace_bytes.argtypes = [P, _i32]
    lib.fa_decode_workspace_bytes.restype = _sz
    lib.fa_decode.argtypes = [P, _i32, ctypes.c_float, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                              _sz, _vp]
    lib.fa_cache_append.argtypes = [P, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.fa_cache_copy_pages.argtypes = [P, _i32, _vp, _vp, _vp, _vp, _vp]
    lib.fa_pages_extend.argtypes = [P] + [_vp] * 6
    lib.fa_pages_fork.argtypes = [P, _i32] + [_vp] * 7
    lib.fa_pages_free.argtypes = [P, _i32] + [_vp] * 5
    lib.fa_pages_compact.argtypes = [P] + [_vp] * 8
    for name in ("decode", "cache_append", "cache_copy_pages", "pages_extend", "pages_fork", "pages_free",
                 "pages_compact"):
        getattr(lib, "fa_" + name).restype = ctypes.c_int


def _done(code: int, what: str, stream, check_status: bool) -> None:
    if code != 0:
        raise _pkg.FaError(code, what)
    if check_status:
        _pkg._raise_on_device_error(stream, what + " (device)")


def _raw_stream(device: torch.device, stream) -> int:
    """The stream as a number, after checking that `device` is the current one."""
    index = torch.cuda.current_device()
    if device.index != index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{index}")
    if stream is None:
        # the number alone: torch.cuda.current_stream() takes 3 us to wrap it
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _lend(stream, *tensors) -> None:
    """Tensors of this call and a stream given by the caller: their memory may
    not be handed out again before that stream is done with it."""
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        for t in tensors:
            t.record_stream(stream)


def _row_strides(t: torch.Tensor):
    """The first three strides of a 4-D tensor with contiguous rows; the stride
    of a dimension of one element, which torch leaves open, is set to a
    packed one."""
    s0, s1, s2, s3 = t.stride()
    n0, n1, n2, d = t.shape
    if s3 != 1:
        raise ValueError("the last dimension must be contiguous")
    if n2 == 1:
        s2 = d
    if n1 == 1:
        s1 = n2 * s2 if s2 >= d else d
    if n0 == 1:
        s0 = max(n1 * s1, n2 * s2, d)
    return s0, s1, s2


def _ints(what: str, t: torch.Tensor, shape, device) -> int:
    """Address of a dense int32 tensor of that shape on that device."""
    if t.dtype != torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _table(page_table: torch.Tensor, device):
    """Sequences, columns, row stride and address of a page table."""
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.device != device:
        raise ValueError(f"page_table must be a 2-D int32 tensor on {device}")
    S, columns = page_table.shape
    row, column = page_table.stride()
    if column != 1 and columns > 1:
        raise ValueError("the rows of page_table must be contiguous")
    return S, columns, row if S > 1 else columns, page_table.data_ptr()


_DTYPES = {torch.bfloat16: _BF16, torch.float32: _FP32}


def _cache(k_pages, v_pages, page_table):
    """Descriptor, device and address of the page table (which may be None)."""
    shape, strides, dtype, device = k_pages.shape, k_pages.stride(), k_pages.dtype, k_pages.device
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [pages, kv_heads, page_rows, d] tensors of one shape")
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    if v_pages.dtype != dtype:
        raise ValueError("k_pages and v_pages must share the dtype")
    if device.type != "cuda" or v_pages.device != device:
        raise ValueError("the pools must be on one CUDA device")
    same = v_pages.stride() == strides
    strides = _row_strides(k_pages)
    if not same and _row_strides(v_pages) != strides:
        raise ValueError("k_pages and v_pages must share their strides")
    S, columns, row, table = (1, 1, 1, 0) if page_table is None else _table(page_table, device)
    pages, heads, rows, d = shape
    return FaCache(pages, rows, heads, d, code, S, columns, 0, *strides, row), device, table


def cache_for(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: Optional[torch.Tensor] = None) -> FaCache:
    """Descriptor of two pools and, if given, the page table over them."""
    return _cache(k_pages, v_pages, page_table)[0]


def _library():
    return _pkg._LIB or _pkg.load_library()


def fa_decode_workspace_bytes(c: FaCache, heads: int) -> int:
    return int(_library().fa_decode_workspace_bytes(ctypes.byref(c), int(heads)))


def attention_decode(q, k_pages, v_pages, page_table, lengths, scale: Optional[float] = None, workspace=None, out=None,
                     stream=None, check_status: bool = False):
    """O, L of one new token a sequence: ``q`` is [S, H, 1, d], with H a
    multiple of the cache's heads (query head h reads key-value head
    h // (H // kv_heads)), and attends to all ``lengths[s]`` rows of sequence
    s, the new token's own among them once it is appended.  An empty sequence
    gives O = 0, L = +inf.  ``scale`` defaults to 1/sqrt(d).

    ``out`` may pass (o, L) to write to; ``workspace`` a uint8 tensor of
    :func:`fa_decode_workspace_bytes`, otherwise one is allocated for the
    call.  Calls that may run at the same time, replays of captured graphs
    among them, need a workspace each."""
    c, device, table = _cache(k_pages, v_pages, page_table)
    shape = q.shape
    S, d = c.S, c.d
    if len(shape) != 4 or shape[0] != S or shape[2] != 1 or shape[3] != d:
        raise ValueError(f"q must be a [{S}, heads, 1, {d}] tensor")
    if q.dtype != k_pages.dtype or q.device != device:
        raise ValueError("q must have the dtype and device of the pools")
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("attention_decode has no gradient: call it under torch.no_grad()")
    heads = shape[1]
    raw = _raw_stream(device, stream)
    lens = _ints("lengths", lengths, (S,), device)
    qs, qh, _ = _row_strides(q)
    lib = _library()
    ref = ctypes.byref(c)
    need = lib.fa_decode_workspace_bytes(ref, heads)
    if out is not None:
        o, L = out
        if o.shape != shape or o.dtype != q.dtype or o.device != device:
            raise ValueError("out[0] must have the shape, dtype and device of q")
        if L.shape != shape[:3] or L.dtype != torch.float32 or L.device != device or not L.is_contiguous():
            raise ValueError(f"out[1] must be a contiguous float32 tensor of shape {tuple(shape[:3])}")
        os, oh, _ = _row_strides(o)
    else:
        o = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=q.dtype, device=device)
        L = torch.empty(shape[:3], dtype=torch.float32, device=device)
        os, oh = heads * d, d
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        ws, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        ws = workspace.data_ptr()
    else:
        ws = 0
    if stream is not None:
        _lend(stream, *(t for t in (o, L, workspace) if t is not None))
    code = lib.fa_decode(ref, heads, d ** -0.5 if scale is None else scale, q.data_ptr(), qs, qh, k_pages.data_ptr(),
                         v_pages.data_ptr(), table, lens, o.data_ptr(), os, oh, L.data_ptr(), ws, need, raw)
    if code or check_status:
        _done(code, "fa_decode", stream, check_status)
    return o, L


def cache_append(k, v, k_pages, v_pages, page_table, start, counts=None, stream=None,
                 check_status: bool = False) -> None:
    """Rows of new tokens into their pages: ``k[s, :, i]`` and ``v[s, :, i]``
    ([S, kv_heads, rows, d]) become row ``start[s] + i`` of sequence s, for
    i < ``counts[s]`` (all rows without counts).  The pages must be there
    (:func:`pages_extend`, which also gives ``start``); a sequence with a
    negative start is left alone."""
    c, device, table = _cache(k_pages, v_pages, page_table)
    if k.dim() != 4 or k.shape[0] != c.S or k.shape[1] != c.H_kv or k.shape[3] != c.d or v.shape != k.shape:
        raise ValueError(f"k and v must be [{c.S}, {c.H_kv}, rows, {c.d}] tensors")
    if k.dtype != k_pages.dtype or v.dtype != k.dtype or k.device != device or v.device != device:
        raise ValueError("k and v must have the dtype and device of the pools")
    rows = k.shape[2]
    if rows == 0:
        return
    strides = _row_strides(k)
    if v.stride() != k.stride() and _row_strides(v) != strides:
        raise ValueError("k and v must share their strides")
    raw = _raw_stream(device, stream)
    at = _ints("start", start, (c.S,), device)
    n = 0 if counts is None else _ints("counts", counts, (c.S,), device)
    code = _library().fa_cache_append(ctypes.byref(c), rows, k.data_ptr(), v.data_ptr(), *strides, k_pages.data_ptr(),
                                      v_pages.data_ptr(), table, at, n, raw)
    if code or check_status:
        _done(code, "fa_cache_append", stream, check_status)


def cache_copy_pages(k_pages, v_pages, moves, count=None, stream=None, check_status: bool = False) -> None:
    """Copies rows between pages of both pools: ``moves`` is int32 [n, 3] of
    (src, dst, rows), with src -1 skipped, as :func:`pages_fork` and
    :func:`pages_compact` return it; ``count`` (int32 [1]) says how many of
    them count.  No dst may be the dst or src of another move."""
    c, device, _ = _cache(k_pages, v_pages, None)
    if moves.dim() != 2:
        raise ValueError("moves must be an [n, 3] tensor")
    raw = _raw_stream(device, stream)
    m = _ints("moves", moves, (moves.shape[0], 3), device)
    n = 0 if count is None else _ints("count", count, (1,), device)
    code = _library().fa_cache_copy_pages(ctypes.byref(c), moves.shape[0], m, n, k_pages.data_ptr(),
                                          v_pages.data_ptr(), raw)
    if code or check_status:
        _done(code, "fa_cache_copy_pages", stream, check_status)


def _pages(page_table, lengths, refs, page_rows: int, stream):
    """Descriptor, device, stream and addresses for the page calls."""
    if refs.dim() != 1 or not refs.is_cuda:
        raise ValueError("refs must be a 1-D CUDA tensor")
    device = refs.device
    pages = refs.shape[0]
    S, columns, row, table = _table(page_table, device)
    c = FaCache(pages, int(page_rows), 1, 0, 0, S, columns, 0, 0, 0, 0, row)
    raw = _raw_stream(device, stream)
    return c, device, raw, table, _ints("lengths", lengths, (S,), device), _ints("refs", refs, (pages,), device)


def pages_extend(page_table, lengths, refs, n_new, page_rows: int, stream=None, check_status: bool = False):
    """Makes room for ``n_new[s]`` (int32 [S]) more rows of every sequence:
    updates the table, ``lengths`` and ``refs`` and returns ``start``, the
    lengths before.  If there are too few free pages, or a sequence would pass
    the table, nothing changes and every start is -1."""
    c, device, raw, table, lens, r = _pages(page_table, lengths, refs, page_rows, stream)
    n = _ints("n_new", n_new, (c.S,), device)
    start = torch.empty_like(lengths)
    if stream is not None:
        _lend(stream, start)
    code = _library().fa_pages_extend(ctypes.byref(c), table, lens, r, n, start.data_ptr(), raw)
    if code or check_status:
        _done(code, "fa_pages_extend", stream, check_status)
    return start


def pages_fork(page_table, lengths, refs, src, dst, page_rows: int, stream=None, check_status: bool = False):
    """Makes each empty sequence ``dst[i]`` a copy of ``src[i]`` (int32 [n]):
    full pages are shared, a partly filled last page is replaced by a free
    one.  Returns the moves ([n, 3]) that :func:`cache_copy_pages` has to make
    in every pool of the cache.  If anything is wrong with the pairs, or there
    are too few free pages, nothing changes and all moves are -1."""
    c, device, raw, table, lens, r = _pages(page_table, lengths, refs, page_rows, stream)
    if src.dim() != 1:
        raise ValueError("src must be a 1-D tensor")
    n = src.shape[0]
    a, b = _ints("src", src, (n,), device), _ints("dst", dst, (n,), device)
    if n == 0:
        return torch.empty((0, 3), dtype=torch.int32, device=device)
    moves = torch.empty((n, 3), dtype=torch.int32, device=device)
    if stream is not None:
        _lend(stream, moves)
    code = _library().fa_pages_fork(ctypes.byref(c), n, a, b, table, lens, r, moves.data_ptr(), raw)
    if code or check_status:
        _done(code, "fa_pages_fork", stream, check_status)
    return moves


def pages_free(page_table, lengths, refs, sequences, page_rows: int, stream=None, check_status: bool = False) -> None:
    """Empties the listed sequences (int32 [n]; -1 is skipped): their pages
    lose a reference, their table entries become -1, their lengths 0."""
    c, device, raw, table, lens, r = _pages(page_table, lengths, refs, page_rows, stream)
    if sequences.dim() != 1:
        raise ValueError("sequences must be a 1-D tensor")
    n = sequences.shape[0]
    code = _library().fa_pages_free(ctypes.byref(c), n, _ints("sequences", sequences, (n,), device), table, lens, r,
                                    raw)
    if code or check_status:
        _done(code, "fa_pages_free", stream, check_status)


def pages_compact(page_table, lengths, refs, page_rows: int, out=None, stream=None, check_status: bool = False):
    """Moves the pages in use to the front of the pool.  Returns the moves
    ([pages // 2, 3], the rest -1) and their number (int32 [1]) for
    :func:`cache_copy_pages`.  The table and refs are updated in place, or
    written to ``out`` = (table, refs) of the same shapes and strides, so that
    work in flight can go on with the old ones."""
    c, device, raw, table, lens, r = _pages(page_table, lengths, refs, page_rows, stream)
    table_out, refs_out = table, r
    if out is not None:
        if out[0].shape != page_table.shape or out[0].stride() != page_table.stride() or \
                out[0].dtype != torch.int32 or out[0].device != device:
            raise ValueError("out[0] must have the shape, strides, dtype and device of page_table")
        table_out, refs_out = out[0].data_ptr(), _ints("out[1]", out[1], (c.num_pages,), device)
    moves = torch.empty((c.num_pages // 2, 3), dtype=torch.int32, device=device)
    count = torch.empty(1, dtype=torch.int32, device=device)
    if stream is not None:
        _lend(stream, moves, count)
    code = _library().fa_pages_compact(ctypes.byref(c), table, lens, r, table_out, refs_out, moves.data_ptr(),
                                       count.data_ptr(), raw)
    if code or check_status:
        _done(code, "fa_pages_compact", stream, check_status)
    return moves, count
