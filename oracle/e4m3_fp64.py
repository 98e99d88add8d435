"""A paged key-value cache in 8 bits, restated plainly for the tests: e4m3
numbers and their scales in float64, appends as loops over sequences, heads and
blocks.  Shares no code with the CUDA path."""

from __future__ import annotations

import numpy as np

__all__ = ["TOP", "nearest", "scale_for", "append", "values"]

TOP = 448.0


def nearest(x):
    """float64 numbers, |x| <= 448, to the nearest e4m3 number, ties to even; what is not finite becomes NaN."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.where(np.isfinite(x), x, 0.0)
    _, e = np.frexp(finite)  # |x| = m 2^e, 1/2 <= m < 1: four significant bits are steps of 2^(e - 4), 2^-9 at least
    step = np.ldexp(1.0, np.maximum(np.where(finite == 0, -100, e) - 4, -9))
    return np.where(np.isfinite(x), np.rint(finite / step) * step, np.nan)


def scale_for(x):
    """The smallest power of two s >= 2^-126 with max |x| <= 448 s, over the finite x."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    top = np.where(np.isfinite(x), x, 0.0).max(initial=0.0)
    s = 2.0 ** -126
    while TOP * s < top:
        s *= 2
    return s


def append(x, pages, scales, table, start, counts, block):
    """Rows x [S, H, rows, d] into pages [pages, H, page_rows, d] (stored values) and scales [pages, H, blocks], in place.

    Rows that are dropped: a negative start, a page that does not exist, a place behind the table."""
    S, H, rows, _ = x.shape
    page_rows, columns = pages.shape[2], table.shape[1]
    for s in range(S):
        n = rows if counts is None else min(max(int(counts[s]), 0), rows)
        if start[s] < 0:
            continue
        at, end = int(start[s]), int(start[s]) + n
        while at < end:
            lo = at // block * block
            to = min(end, lo + block)
            column = lo // page_rows
            p = int(table[s, column]) if column < columns else -1
            if 0 <= p < pages.shape[0]:
                r, b = lo % page_rows, lo % page_rows // block
                for h in range(H):
                    new = x[s, h, at - start[s]:to - start[s]]
                    scale = scale_for(new)
                    if at > lo:
                        old = scales[p, h, b]
                        scale = max(scale, old)
                        pages[p, h, r:r + at - lo] = nearest(pages[p, h, r:r + at - lo] * (old / scale))
                    pages[p, h, r + at - lo:r + to - lo] = nearest(new / scale)
                    scales[p, h, b] = scale
            at = to


def values(pages, scales):
    """What the stored values stand for."""
    return pages * np.repeat(scales, pages.shape[2] // scales.shape[2], 2)[..., None]
