"""The paged cache without a GPU: what the C entry points refuse before they
touch CUDA, what the binding refuses, the arithmetic that the kernels find a
row with, and the model that the GPU tests hold the page calls to."""

import ctypes
import random

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from flashattention_backward_gb300 import _build, paged
from oracle.paged_fp64 import PageModel, decode

BAD = 0x1000  # a 16-byte aligned dummy address; validation fails before any use
INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def _cache(**kw):
    base = dict(num_pages=100, page_rows=16, H_kv=2, d=64, dtype=fa.FA_BF16, S=3, max_pages=20, reserved=0,
                stride_page=2 * 16 * 64, stride_h=16 * 64, stride_n=64, table_stride=20)
    base.update(kw)
    return fa.FaCache(**base)


def _calls(lib, c):
    """Every entry point that takes the pools, then those that take the table alone."""
    ref = ctypes.byref(c) if c is not None else None
    yield lib.fa_decode(ref, 4, 0.125, BAD, 256, 64, BAD, BAD, BAD, BAD, 2 * BAD, 256, 64, BAD, BAD, 1 << 40, None)
    yield lib.fa_cache_append(ref, 1, BAD, BAD, 128, 64, 64, BAD, BAD, BAD, BAD, BAD, None)
    yield lib.fa_cache_copy_pages(ref, 1, BAD, BAD, BAD, BAD, None)


def _page_calls(lib, c):
    ref = ctypes.byref(c) if c is not None else None
    yield lib.fa_pages_extend(ref, BAD, BAD, BAD, BAD, BAD, None)
    yield lib.fa_pages_fork(ref, 1, BAD, BAD, BAD, BAD, BAD, BAD, None)
    yield lib.fa_pages_free(ref, 1, BAD, BAD, BAD, BAD, None)
    yield lib.fa_pages_compact(ref, BAD, BAD, BAD, BAD, BAD, BAD, BAD, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_pages=0), INVALID), (dict(page_rows=0), INVALID), (dict(S=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(H_kv=0), INVALID), (dict(reserved=1), INVALID), (dict(table_stride=19), INVALID),
    (dict(num_pages=(1 << 30) + 1), UNSUPPORTED),
    (dict(page_rows=1 << 20, max_pages=1 << 11, table_stride=1 << 11), UNSUPPORTED),
    (dict(S=1 << 24), UNSUPPORTED),
])
def test_geometry_is_checked_by_every_call(lib, kw, code):
    c = _cache(**kw)
    for r in list(_calls(lib, c)) + list(_page_calls(lib, c)):
        assert r == code
    assert fa.fa_decode_workspace_bytes(c, 4) == 0
    assert all(r == INVALID for r in list(_calls(lib, None)) + list(_page_calls(lib, None)))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=16), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
    (dict(stride_n=60), INVALID), (dict(stride_n=68), INVALID), (dict(stride_h=0), INVALID),
    (dict(stride_page=0), INVALID), (dict(stride_page=-64), INVALID), (dict(stride_h=16 * 64 + 4), INVALID),
])
def test_pools_are_checked(lib, kw, code):
    for r in _calls(lib, _cache(**kw)):
        assert r == code


def test_pointers_and_sizes_are_checked(lib):
    c = ctypes.byref(_cache())
    ok = [c, 4, 0.125, BAD, 256, 64, BAD, BAD, BAD, BAD, 2 * BAD, 256, 64, BAD, BAD, 1 << 40, None]
    for i, x in [(1, 0), (1, 3), (1, -2), (2, 0.0), (2, float("nan")), (2, float("inf")), (2, 3e38), (2, -1.0), (3, 0), (3, BAD + 8),
                 (4, 4), (5, -64), (6, BAD + 2), (7, 0), (8, 0), (8, BAD + 2), (9, 0), (10, BAD + 4), (10, BAD), (11, 60), (12, 0),
                 (13, 0)]:
        args = list(ok)
        args[i] = x
        assert lib.fa_decode(*args) == INVALID, i
    ok = [c, 1, BAD, BAD, 128, 64, 64, BAD, BAD, BAD, BAD, BAD, None]
    for i, x in [(1, 0), (2, 0), (3, BAD + 4), (4, 4), (5, 4), (6, -64), (7, 0), (8, BAD + 8), (9, 0), (10, 0),
                 (11, BAD + 1)]:
        args = list(ok)
        args[i] = x
        assert lib.fa_cache_append(*args) == INVALID, i
    ok[1] = 1 << 30
    assert lib.fa_cache_append(*ok) == UNSUPPORTED
    for args in ([c, -1, BAD, BAD, BAD, BAD, None], [c, 1, 0, BAD, BAD, BAD, None], [c, 1, BAD, BAD + 2, BAD, BAD, None],
                 [c, 1, BAD, BAD, 0, BAD, None], [c, 1, BAD, BAD, BAD, BAD + 8, None]):
        assert lib.fa_cache_copy_pages(*args) == INVALID
    for f, n in ((lib.fa_pages_extend, 5), (lib.fa_pages_compact, 7)):
        for i in range(n):
            assert f(c, *[BAD if j != i else 0 for j in range(n)], None) == INVALID
    for i in range(6):
        assert lib.fa_pages_fork(c, 1, *[BAD if j != i else BAD + 2 for j in range(6)], None) == INVALID
    assert lib.fa_pages_fork(c, 0, *[BAD] * 6, None) == INVALID
    assert lib.fa_pages_fork(c, 4, *[BAD] * 6, None) == INVALID  # more pairs than sequences
    many = ctypes.byref(_cache(S=65537, H_kv=1))
    assert lib.fa_pages_fork(many, 1, *[BAD] * 6, None) == UNSUPPORTED
    assert lib.fa_pages_free(c, -1, *[BAD] * 4, None) == INVALID
    for i in range(4):
        assert lib.fa_pages_free(c, 1, *[BAD if j != i else 0 for j in range(4)], None) == INVALID


def test_size_of_the_workspace(lib):
    assert fa.fa_decode_workspace_bytes(_cache(), 3) == 0  # not a multiple of the cache's heads
    # what passes through it is bounded by the GPU, not by the lengths
    big = _cache(S=1000, max_pages=1 << 20, table_stride=1 << 20)
    assert fa.fa_decode_workspace_bytes(big, 64) < 256 << 20
    assert fa.fa_decode_workspace_bytes(_cache(max_pages=1, table_stride=1), 4) == 0  # 16 rows: nothing to join
    assert fa.status_string(fa.FA_ERR_PAGES).startswith("page")


def test_division_by_multiplication():
    """FastDiv's formula, over its whole range of divisors and the numerators where it could go wrong."""
    rng = random.Random(1)
    divisors = [1, 2, 3, 5, 7, 12, 13, 16, 24, 100, 255, 256, 257, 641, 1000, 65535, 65537, (1 << 30) - 1, 1 << 30]
    for d in divisors + [rng.randrange(1, 1 << rng.randrange(1, 31)) for _ in range(500)]:
        s = 0
        while (1 << s) < d:
            s += 1
        m = ((((1 << s) - d) << 32) // d + 1) & 0xFFFFFFFF
        assert m == (((1 << s) - d) << 32) // d + 1
        top = (1 << 31) - 1
        for n in [0, 1, d - 1, d, d + 1, 2 * d - 1, top, top - 1, top // d * d, max(0, top // d * d - 1)] + \
                 [rng.randrange(1 << 31) for _ in range(50)]:
            if n <= top:
                t = (n * m >> 32) + n
                assert t < 1 << 32 and t >> s == n // d


def test_binding_refuses(lib):
    pools = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):  # CPU tensors: no CPU path exists
        fa.cache_for(pools, pools)
    for bad in ((pools.half(), pools.half()), (pools, None), ("pools", pools)):
        with pytest.raises(TypeError):
            fa.cache_for(*bad)
    for bad in ((pools, pools.float()), (pools, pools[:3]), (pools[0], pools[0])):
        with pytest.raises(ValueError):
            fa.cache_for(*bad)
    table = torch.zeros(3, 5, dtype=torch.int32)
    refs = torch.zeros(9, dtype=torch.int32)
    for call in (lambda: fa.attention_decode(torch.zeros(3, 2, 1, 64), pools, pools, table, table[:, 0]),
                 lambda: fa.cache_append(pools, pools, pools, pools, table, refs),
                 lambda: fa.cache_copy_pages(pools, pools, table[:, :3]),
                 lambda: fa.pages_extend(table, table[:, 0], refs, table[:, 0], 16),
                 lambda: fa.pages_fork(table, table[:, 0], refs, refs, refs, 16),
                 lambda: fa.pages_free(table, table[:, 0], refs, refs, 16),
                 lambda: fa.pages_compact(table, table[:, 0], refs, 16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fa.pages_extend(table, table[:, 0], None, table[:, 0], 16)


def test_missing_binding_fails_loudly(lib, monkeypatch):
    monkeypatch.setattr(paged, "_EXT", None)
    monkeypatch.setattr(_build, "torch_binding_path", lambda: "/nonexistent/_fa_torch.so")
    with pytest.raises(RuntimeError, match="build"):
        fa.pages_free(*[torch.zeros(1, dtype=torch.int32)] * 4, 16)


def test_oracle_is_a_softmax():
    """Against torch in float64 on a dense copy, an empty sequence and one with a missing page among them."""
    gen = torch.Generator().manual_seed(0)
    S, H, hk, d, rows = 3, 4, 2, 16, 5
    kp, vp = (torch.randn(9, hk, rows, d, generator=gen, dtype=torch.float64) for _ in range(2))
    q = torch.randn(S, H, d, generator=gen, dtype=torch.float64)
    table = torch.tensor([[3, 1, 8], [0, -1, 7], [-1, -1, -1]])
    o, L, A, V = decode(q.numpy(), kp.numpy(), vp.numpy(), table.numpy(), [13, 15, 0], 0.25)
    for s, (ids, n) in enumerate((([3, 1, 8], 13), ([0, 7], 10))):
        for h in range(H):
            k, v = (t[ids, h // 2].reshape(-1, d)[:n] for t in (kp, vp))
            x = 0.25 * k @ q[s, h]
            assert np.allclose(o[s, h], torch.softmax(x, 0) @ v, atol=1e-14)
            assert np.isclose(L[s, h], torch.logsumexp(x, 0))
    assert (o[2] == 0).all() and np.isposinf(L[2]).all()


def test_page_model_keeps_its_books():
    """Whatever is called in whatever order: every reference is counted, no free page is named."""
    rng = random.Random(7)
    for _ in range(60):
        rows, S = rng.choice([1, 3, 8]), rng.randint(1, 9)
        m = PageModel(rng.randint(1, 40), rows, S, 6)
        for _ in range(30):
            what = rng.randrange(4)
            if what == 0:
                m.extend([rng.choice([0, 0, 1, rng.randint(0, 3 * rows)]) for _ in range(S)])
            elif what == 1:
                m.fork([rng.randrange(S)], [rng.randrange(S)])
            elif what == 2:
                m.free([rng.randrange(S)])
            else:
                m.compact()
                used = sum(r > 0 for r in m.refs)
                assert all(r > 0 for r in m.refs[:used]) and not any(m.refs[used:])
            named = [p for row in m.table for p in row if p >= 0]
            assert all(m.refs[p] == named.count(p) for p in range(len(m.refs)))
            assert all(sum(p >= 0 for p in row) == m.held(n) for row, n in zip(m.table, m.lengths))
