"""fa_pages_extend: results that may not stand where its inputs do, and what a
refused call leaves as it was."""

import ctypes

import pytest
import torch

import flashattention_backward_gb300 as fa
from flashattention_backward_gb300 import _build

A, B, C, D, E = (0x1000 * k for k in range(1, 6))  # aligned dummy addresses; refused before any use


def test_start_may_not_be_an_input():
    _build.build()
    lib = fa.load_library()
    c = ctypes.byref(fa.FaCache(num_pages=100, page_rows=16, H_kv=2, d=64, dtype=fa.FA_BF16, S=3, max_pages=20,
                                stride_page=2048, stride_h=1024, stride_n=64, table_stride=20))
    assert lib.fa_pages_extend(c, A, B, C, D, B, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_pages_extend(c, A, B, C, D, D, None) == fa.FA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("S", [3, 1500])
def test_too_few_pages(S):
    """Also with entries behind the sequences' pages that are not -1, and counts below 0: whatever a sequence holds, and
    every page's being used or free, is as it was."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
    table = torch.full((S, 6), 7, dtype=torch.int32, device="cuda:0")
    lengths, n_new = ints([0] * S), ints([0] * S)
    table[0, :2], table[S - 1, 0] = ints([4, 1]), 2
    lengths[0], lengths[S - 1] = 7, 4
    refs = ints([0, 1, 1, -2, 1, 0, 0, 0])
    n_new[1], n_new[S - 1] = 12, 11  # 3 + 3 pages of the 5 that are free
    held = table.clone(), lengths.clone(), refs.clone()
    start = fa.pages_extend(table, lengths, refs, n_new, 4)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert (start == -1).all() and torch.equal(lengths, held[1])
    assert table[0, :2].tolist() == [4, 1] and table[S - 1, 0].item() == 2
    assert torch.equal(refs.clamp(min=0), held[2].clamp(min=0))
    n_new[S - 1] = 0  # three pages: as many as there are before page 6, lowest first
    start = fa.pages_extend(table, lengths, refs, n_new, 4)
    assert fa.get_device_status() == 0
    assert start.tolist() == held[1].tolist() and table[1, :3].tolist() == [0, 3, 5]
    assert refs.tolist() == [1, 1, 1, 1, 1, 1, 0, 0] and lengths[1].item() == 12
