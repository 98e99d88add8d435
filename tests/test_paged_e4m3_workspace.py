"""The paged cache in 8 bits at the largest pages, on the host: the size of fa_decode_e4m3's workspace where some numbers
of scales alone are allowed, and blocks that fa_cache_append_e4m3 could not count its way through."""

import ctypes

import pytest

import flashattention_backward_gb300 as fa
from flashattention_backward_gb300 import _build

BAD = 0x1000  # a 16-byte aligned dummy address; validation fails before any use


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


@pytest.mark.parametrize("H_kv,log_rows", [(4, 29), (2, 30), (64, 25)])
def test_the_workspace_does_not_go_by_the_scales(lib, H_kv, log_rows):
    """H_kv * page_rows = 2^31: too many scales with one a row, but half of that, and one a page, are allowed."""
    page_rows = 1 << log_rows
    c = fa.FaCache(num_pages=2, page_rows=page_rows, H_kv=H_kv, d=64, dtype=fa.FA_BF16, S=1, max_pages=1, reserved=0,
                   stride_page=H_kv * page_rows * 64, stride_h=page_rows * 64, stride_n=64, table_stride=1)
    need = fa.fa_decode_e4m3_workspace_bytes(c, 2 * H_kv)
    assert need == 2 * 1280 * 8 * (8 + 4 * 64)  # as many parts as there may be

    def call(block, have):
        return lib.fa_decode_e4m3(ctypes.byref(c), block, 2 * H_kv, 0.125, 5 * BAD, 64, 64, BAD, 2 * BAD, 3 * BAD, 4 * BAD, BAD, BAD,
                                  6 * BAD, 64, 64, BAD, BAD, have, None)

    assert call(1, need) == fa.FA_ERR_UNSUPPORTED
    for block in (2, page_rows):  # what is asked for is what the query says
        assert call(block, need - 1) == fa.FA_ERR_INVALID_ARG


def test_a_cache_or_heads_that_are_refused_have_none(lib):
    good = dict(num_pages=2, page_rows=16, H_kv=2, d=64, dtype=fa.FA_BF16, S=1, max_pages=1 << 20, reserved=0,
                stride_page=2 * 16 * 64, stride_h=16 * 64, stride_n=64, table_stride=1 << 20)
    assert fa.fa_decode_e4m3_workspace_bytes(fa.FaCache(**good), 4) > 0
    for bad in (dict(S=0), dict(d=48), dict(stride_n=72), dict(reserved=1), dict(page_rows=1 << 20)):
        assert fa.fa_decode_e4m3_workspace_bytes(fa.FaCache(**{**good, **bad}), 4) == 0
    for heads in (0, 3, -2, 2 * 513):
        assert fa.fa_decode_e4m3_workspace_bytes(fa.FaCache(**good), heads) == 0


@pytest.mark.parametrize("d,dtype", [(16, fa.FA_FP32), (32, fa.FA_BF16), (64, fa.FA_FP32), (96, fa.FA_BF16), (128, fa.FA_BF16),
                                     (256, fa.FA_FP32), (256, fa.FA_BF16)])
def test_an_append_into_too_large_a_block_is_refused(lib, d, dtype):
    """With 2^31 units of 16 numbers or more in a block their count, or its way round 32 bits, would not end. Rows outside
    may have a stride of 0, so that little memory is needed to ask for it."""
    for log_rows in (26, 27, 28, 29, 30):
        rows = 1 << log_rows
        c = fa.FaCache(num_pages=1, page_rows=rows, H_kv=1, d=d, dtype=dtype, S=1, max_pages=1, reserved=0,
                       stride_page=rows * d, stride_h=rows * d, stride_n=d, table_stride=1)
        for block in (rows, rows // 2, rows // 4):
            # no place for the new rows: what fits is refused for that, before it reaches a device
            args = [ctypes.byref(c), block, 1, 0, 0, 0, 0, 0, BAD, 2 * BAD, 3 * BAD, 4 * BAD, BAD, BAD, BAD, None]
            assert lib.fa_cache_append_e4m3(*args) == fa.FA_ERR_INVALID_ARG
            if block * d >= 1 << 35:
                args[3:5] = 5 * BAD, 6 * BAD
                assert lib.fa_cache_append_e4m3(*args) == fa.FA_ERR_UNSUPPORTED
