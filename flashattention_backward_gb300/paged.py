"""Paged key-value cache: the attention of one new token, and its pages.

The ``fa_decode``, ``fa_cache_*`` and ``fa_pages_*`` entry points of
``include/fa.h``, whose kernels do all the work.  Arguments are checked and
marshalled by a small compiled binding (``csrc/fa_torch.cpp``): these calls
are short enough for that to count.

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

A call runs on the current stream, or on ``stream``, whose work is in order
with the call's; what it allocates is memory of that stream.  Its results may
be used on the current stream too, once that has waited for the other.

No call here has a gradient; one whose tensors need one is refused unless
gradients are switched off (``torch.no_grad()``).
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

import torch

import flashattention_backward_gb300 as _pkg

from . import _build

# the library's entry points, in the order in which the binding takes them
_ENTRIES = ("decode_workspace_bytes", "decode", "cache_append", "cache_copy_pages", "pages_extend", "pages_fork",
            "pages_free", "pages_compact")
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


_EXT = None


def _binding():
    """The compiled binding (csrc/fa_torch.cpp), with the library's entry points handed over."""
    global _EXT
    if _EXT is None:
        lib = _pkg.load_library()
        path = _build.torch_binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"the PyTorch binding was not found at {path}: run __graft_entry__.build(), which says why "
                               "where it cannot be compiled")
        spec = importlib.util.spec_from_file_location("_fa_torch", path)
        ext = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(ext)
        ext.bind(_pkg.FaError, *(ctypes.cast(getattr(lib, "fa_" + name), _vp).value for name in _ENTRIES))
        _EXT = ext
    return _EXT


def _raw(stream):
    """The caller's stream as a number; None is the current one."""
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _status(what: str, stream) -> None:
    _pkg._raise_on_device_error(stream, what + " (device)")


def cache_for(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: Optional[torch.Tensor] = None) -> FaCache:
    """Descriptor of two pools and, if given, the page table over them."""
    return FaCache(*_binding().describe(k_pages, v_pages, page_table))


def fa_decode_workspace_bytes(c: FaCache, heads: int) -> int:
    return int(_pkg.load_library().fa_decode_workspace_bytes(ctypes.byref(c), int(heads)))


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
    among them, need a workspace each.

    The same call gives the same bits.  The order of its sums goes by the
    lengths, the heads, the dtype and the shapes of pools and table, so a table
    with more columns may give other last bits."""
    got = (_EXT or _binding()).decode(q, k_pages, v_pages, page_table, lengths, scale, workspace,
                                      None if out is None else tuple(out), _raw(stream))
    if check_status:
        _status("fa_decode", stream)
    return got


def cache_append(k, v, k_pages, v_pages, page_table, start, counts=None, stream=None,
                 check_status: bool = False) -> None:
    """Rows of new tokens into their pages: ``k[s, :, i]`` and ``v[s, :, i]``
    ([S, kv_heads, rows, d]) become row ``start[s] + i`` of sequence s, for
    i < ``counts[s]`` (all rows without counts).  The pages must be there
    (:func:`pages_extend`, which also gives ``start``); a sequence with a
    negative start is left alone."""
    (_EXT or _binding()).append(k, v, k_pages, v_pages, page_table, start, counts, _raw(stream))
    if check_status:
        _status("fa_cache_append", stream)


def cache_copy_pages(k_pages, v_pages, moves, count=None, stream=None, check_status: bool = False) -> None:
    """Copies rows between pages of both pools: ``moves`` is int32 [n, 3] of
    (src, dst, rows), with src -1 skipped, as :func:`pages_fork` and
    :func:`pages_compact` return it; ``count`` (int32 [1]) says how many of
    them count.  No dst may be the dst or src of another move."""
    (_EXT or _binding()).copy(k_pages, v_pages, moves, count, _raw(stream))
    if check_status:
        _status("fa_cache_copy_pages", stream)


def pages_extend(page_table, lengths, refs, n_new, page_rows: int, stream=None, check_status: bool = False):
    """Makes room for ``n_new[s]`` (int32 [S]) more rows of every sequence:
    updates the table, ``lengths`` and ``refs`` and returns ``start``, the
    lengths before.  If there are too few free pages, or a sequence would pass
    the table, nothing changes and every start is -1."""
    start = (_EXT or _binding()).extend(page_table, lengths, refs, n_new, page_rows, _raw(stream))
    if check_status:
        _status("fa_pages_extend", stream)
    return start


def pages_fork(page_table, lengths, refs, src, dst, page_rows: int, stream=None, check_status: bool = False):
    """Makes each empty sequence ``dst[i]`` a copy of ``src[i]`` (int32 [n]):
    full pages are shared, a partly filled last page is replaced by a free
    one.  Returns the moves ([n, 3]) that :func:`cache_copy_pages` has to make
    in every pool of the cache.  If anything is wrong with the pairs, or there
    are too few free pages, nothing changes and all moves are -1."""
    moves = (_EXT or _binding()).fork(page_table, lengths, refs, src, dst, page_rows, _raw(stream))
    if check_status:
        _status("fa_pages_fork", stream)
    return moves


def pages_free(page_table, lengths, refs, sequences, page_rows: int, stream=None, check_status: bool = False) -> None:
    """Empties the listed sequences (int32 [n]; -1 is skipped): their pages
    lose a reference, their table entries become -1, their lengths 0."""
    (_EXT or _binding()).free(page_table, lengths, refs, sequences, page_rows, _raw(stream))
    if check_status:
        _status("fa_pages_free", stream)


def pages_compact(page_table, lengths, refs, page_rows: int, out=None, stream=None, check_status: bool = False):
    """Moves the pages in use to the front of the pool.  Returns the moves
    ([pages // 2, 3], the rest -1) and their number (int32 [1]) for
    :func:`cache_copy_pages`.  The table and refs are updated in place, or
    written to ``out`` = (table, refs) of the same shapes and strides, so that
    work in flight can go on with the old ones."""
    got = (_EXT or _binding()).compact(page_table, lengths, refs, page_rows, None if out is None else tuple(out),
                                       _raw(stream))
    if check_status:
        _status("fa_pages_compact", stream)
    return got
