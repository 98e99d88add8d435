"""The paged cache in 8 bits without a GPU: what the C entry points and the
binding refuse before they touch CUDA, and the restatement that the GPU tests
hold the kernels to."""

import ctypes
import math

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from flashattention_backward_gb300 import _build
from oracle.e4m3_fp64 import append, nearest, scale_for, values

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


def _args(c, block=8):
    """Each entry point's arguments, all good."""
    c = ctypes.byref(c) if c is not None else None
    k, v, ks, vs, x, y = BAD, 2 * BAD, 3 * BAD, 4 * BAD, 5 * BAD, 6 * BAD
    return dict(
        fa_decode_e4m3=[c, block, 4, 0.125, x, 256, 64, k, v, ks, vs, BAD, BAD, y, 256, 64, BAD, BAD, 1 << 40, None],
        fa_cache_append_e4m3=[c, block, 1, x, y, 128, 64, 64, k, v, ks, vs, BAD, BAD, BAD, None],
        fa_cache_read_e4m3=[c, block, 1, k, v, ks, vs, BAD, BAD, BAD, x, y, 128, 64, 64, None],
        fa_cache_copy_pages_e4m3=[c, block, 1, BAD, BAD, k, v, ks, vs, None])


@pytest.mark.parametrize("kw,code", [
    (dict(num_pages=0), INVALID), (dict(page_rows=0), INVALID), (dict(S=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(H_kv=0), INVALID), (dict(reserved=1), INVALID), (dict(table_stride=19), INVALID),
    (dict(num_pages=(1 << 30) + 1), UNSUPPORTED),
    (dict(page_rows=1 << 20, max_pages=1 << 11, table_stride=1 << 11), UNSUPPORTED), (dict(S=1 << 24), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=16), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
    (dict(stride_n=60), INVALID), (dict(stride_n=72), INVALID), (dict(stride_h=0), INVALID),
    (dict(stride_page=0), INVALID), (dict(stride_page=-64), INVALID), (dict(stride_h=16 * 64 + 8), INVALID),
])
def test_the_cache_is_checked_by_every_call(lib, kw, code):
    c = _cache(**kw)
    for name, args in _args(c).items():
        assert getattr(lib, name)(*args) == code, name
    assert fa.fa_decode_e4m3_workspace_bytes(c, 4) == 0
    for name, args in _args(None).items():
        assert getattr(lib, name)(*args) == INVALID, name


@pytest.mark.parametrize("block", [0, -1, 3, 5, 32, 1 << 20])
def test_blocks_divide_a_page(lib, block):
    for name, args in _args(_cache(), block).items():
        assert getattr(lib, name)(*args) == INVALID, name


def test_a_page_has_fewer_scales_than_32_bits_count(lib):
    big = dict(H_kv=4, page_rows=1 << 29, max_pages=1, stride_n=64, stride_h=64 << 29, stride_page=64 << 31)
    for name, args in _args(_cache(**big), 1).items():
        assert getattr(lib, name)(*args) == UNSUPPORTED, name


def test_pointers_and_sizes_are_checked(lib):
    wrong = dict(
        fa_decode_e4m3=[(2, 0), (2, 3), (2, -2), (3, 0.0), (3, math.nan), (3, math.inf), (3, 3e38), (3, -1.0), (4, 0),
                        (4, BAD + 8), (5, 4), (6, -64), (7, BAD + 2), (8, 0), (9, 0), (9, BAD + 2), (10, 0), (10, BAD + 1),
                        (11, 0), (12, BAD + 2), (13, BAD + 4), (13, 5 * BAD), (14, 60), (15, 0), (16, 0)],
        fa_cache_append_e4m3=[(2, 0), (3, 0), (4, BAD + 4), (5, 4), (6, 4), (7, -64), (8, 0), (8, 2 * BAD), (9, BAD + 8),
                              (10, 0), (10, 4 * BAD), (11, BAD + 2), (12, 0), (13, 0), (14, BAD + 1)],
        fa_cache_read_e4m3=[(2, 0), (3, BAD + 8), (4, 0), (5, BAD + 2), (6, 0), (7, 0), (8, BAD + 2), (9, BAD + 2), (10, 0),
                            (10, 6 * BAD), (11, BAD + 8), (12, 60), (13, 0), (14, -64)],
        fa_cache_copy_pages_e4m3=[(2, -1), (3, 0), (4, BAD + 2), (5, 0), (5, 2 * BAD), (6, BAD + 8), (7, 0), (7, 4 * BAD),
                                  (8, BAD + 1)])
    for name, args in _args(_cache()).items():
        for i, x in wrong[name]:
            bad = list(args)
            bad[i] = x
            assert getattr(lib, name)(*bad) == INVALID, (name, i, x)
    for name in ("fa_cache_append_e4m3", "fa_cache_read_e4m3"):
        args = _args(_cache())[name]
        args[2] = 1 << 30
        assert getattr(lib, name)(*args) == UNSUPPORTED
    many = _args(_cache(H_kv=1, stride_page=16 * 64))["fa_decode_e4m3"]
    many[2] = 513
    assert lib.fa_decode_e4m3(*many) == UNSUPPORTED


def test_nothing_to_copy_is_no_error(lib):
    args = _args(_cache())["fa_cache_copy_pages_e4m3"]
    args[2:5] = 0, 0, 0
    assert lib.fa_cache_copy_pages_e4m3(*args) == fa.FA_OK


def test_size_of_the_workspace(lib):
    assert fa.fa_decode_e4m3_workspace_bytes(_cache(), 3) == 0  # not a multiple of the cache's heads
    big = _cache(S=1000, max_pages=1 << 20, table_stride=1 << 20)  # bounded by the GPU, not by the lengths
    assert fa.fa_decode_e4m3_workspace_bytes(big, 64) < 256 << 20
    assert fa.fa_decode_e4m3_workspace_bytes(_cache(max_pages=1, table_stride=1), 4) == 0  # 16 rows: nothing to join


def _tensors(dev="cpu"):
    pools = [torch.zeros(4, 2, 16, 64, device=dev).to(torch.float8_e4m3fn) for _ in range(2)]
    return pools + [torch.ones(4, 2, 2, device=dev) for _ in range(2)]


def test_binding_refuses(lib):
    kp, vp, ks, vs = _tensors()
    table, q = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, 2, 1, 64)
    n = table[:, 0].contiguous()
    calls = (lambda *c: fa.attention_decode_e4m3(q, *c, table, n), lambda *c: fa.cache_append_e4m3(q, q, *c, table, n),
             lambda *c: fa.cache_read_e4m3(*c, table, 3), lambda *c: fa.cache_copy_pages_e4m3(*c, table[:, :3].contiguous()),
             lambda *c: fa.cache_for_e4m3(*c))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):  # CPU tensors: no CPU path exists
            call(kp, vp, ks, vs)
        for bad in ((None, vp, ks, vs), (kp, "v", ks, vs), (kp, vp, None, vs), (kp, vp, ks, 1.0)):
            with pytest.raises(TypeError):
                call(*bad)
        for bad in ((kp, vp[:3], ks, vs), (kp[0], vp[0], ks, vs)):
            with pytest.raises(ValueError):
                call(*bad)
    for dtype in (torch.float16, torch.float8_e4m3fn, torch.int32):
        with pytest.raises(TypeError, match="dtype"):
            fa.cache_read_e4m3(kp, vp, ks, vs, table, 3, dtype=dtype)
        with pytest.raises(TypeError, match="dtype"):
            fa.attention_decode_e4m3(q.to(dtype), kp, vp, ks, vs, table, n)
    with pytest.raises(TypeError):
        fa.cache_read_e4m3(kp, vp, ks, vs, table, 3, dtype="bf16")
    # pools in 8 bits do not go to the calls that know nothing of scales
    for call in (lambda: fa.attention_decode(q, kp, vp, table, n), lambda: fa.cache_append(q, q, kp, vp, table, n),
                 lambda: fa.cache_copy_pages(kp, vp, table[:, :3]), lambda: fa.cache_for(kp, vp)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("name", ["q", "k", "v", "k_scales", "v_scales"])
def test_a_tensor_that_needs_a_gradient_is_refused(lib, name):
    kp, vp, ks, vs = _tensors()
    table = torch.zeros(3, 5, dtype=torch.int32)
    n = table[:, 0].contiguous()
    x = torch.zeros(3, 2, 1, 64)
    scales = dict(k_scales=ks, v_scales=vs)
    calls = [(lambda q, k_scales, v_scales: fa.attention_decode_e4m3(q, kp, vp, k_scales, v_scales, table, n), dict(q=x)),
             (lambda k, v, k_scales, v_scales: fa.cache_append_e4m3(k, v, kp, vp, k_scales, v_scales, table, n),
              dict(k=x, v=x)),
             (lambda k_scales, v_scales: fa.cache_read_e4m3(kp, vp, k_scales, v_scales, table, 3), {}),
             (lambda k_scales, v_scales: fa.cache_copy_pages_e4m3(kp, vp, k_scales, v_scales, table[:, :3]), {})]
    for call, args in calls:
        args = {**args, **scales}
        if name in args:
            args[name] = args[name].clone().requires_grad_()
            with pytest.raises(ValueError, match="no gradient"):
                call(**args)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(**args)


# ------------------------------------------------------------ the restatement
def test_nearest_is_the_cast():
    """Against PyTorch's own cast: every e4m3 number, the middles between neighbours, and beside those."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    grid = np.unique(codes[codes.isfinite()].numpy())
    assert len(grid) == 253 and grid[-1] == 448  # 256 codes, two of them NaN and two of them 0
    middles = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, middles, middles * (1 + 2.0 ** -20), middles * (1 - 2.0 ** -20),
                        np.random.default_rng(0).uniform(-448, 448, 5000), np.random.default_rng(1).normal(size=5000) / 50])
    x = x.astype(np.float32).astype(np.float64)
    assert np.array_equal(nearest(x), torch.tensor(x).float().to(torch.float8_e4m3fn).double().numpy())
    assert np.isnan(nearest([math.nan, math.inf, -math.inf])).all()


def test_scale_is_the_smallest():
    rng = np.random.default_rng(2)
    for top in np.concatenate([2.0 ** rng.uniform(-130, 127.9, 300), [448.0, 448.0000001, 449, 896, 3.3895e38, 1e-45]]):
        s = scale_for([top, -top / 3, math.inf, math.nan])
        assert top <= 448 * s and math.frexp(s)[0] == 0.5
        assert s == 2.0 ** -126 or 448 * s / 2 < top
    assert scale_for([0.0, math.nan]) == 2.0 ** -126 == scale_for([])


def test_growing_scale_moves_rows():
    pages, scales = np.zeros((2, 1, 4, 2)), np.full((2, 1, 2), 7.0)
    table = np.array([[1]])
    x = np.array([[[[1.0, -3.0], [100.0, 0.001], [900.0, 2.0]]]])
    append(x[:, :, :1], pages, scales, table, [0], None, 2)
    assert scales[1, 0, 0] == 2.0 ** -7 and np.array_equal(pages[1, 0, 0], [128, -384])  # 3 * 128 <= 448
    append(x[:, :, 1:], pages, scales, table, [1], None, 2)
    assert scales[1, 0].tolist() == [0.25, 4.0]  # 448 / 4 >= 100, 448 * 4 >= 900
    assert np.array_equal(pages[1, 0], [[4, -12], [400 - 16, 0.00390625], [224, 0.5], [0, 0]])
    assert np.array_equal(values(pages, scales)[1, 0, 2], [896, 2])
    assert (pages[0] == 0).all() and (scales[0] == 7).all()
