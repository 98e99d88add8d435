"""When two calls of fa_decode give the same bits: the same lengths in the same
geometry, whatever else is in the pools and wherever the pages lie.  Another
width of the table may sum in another order."""

import pytest
import torch

import flashattention_backward_gb300 as fa
from test_gpu_decode import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths", [[2000], [1900, 0, 3, 777, 64]])
def test_bits_go_by_the_geometry(dtype, lengths):
    q, kp, vp, table, n = make(len(lengths), 8, 1, 128, 16, lengths, dtype, seed=6, junk=False)
    wider = [torch.nn.functional.pad(table, (0, w - table.shape[1]), value=-1) for w in (128, 129, 4000)]
    sizes = [fa.fa_decode_workspace_bytes(fa.cache_for(kp, vp, t), 8) for t in wider]
    if len(lengths) == 1 and dtype == torch.bfloat16:  # 128 columns: a cluster of blocks; one more: runs and a join
        assert sizes[0] == 0 < sizes[1]
    order = torch.randperm(kp.shape[0], device=kp.device)
    back = torch.argsort(order).int()
    for t in wider:
        want = fa.attention_decode(q, kp, vp, t, n)
        check(want, q, kp, vp, t, n, 128 ** -0.5)
        moved = torch.where(t >= 0, back[t.clamp(min=0).long()], t)
        for args in ((q, kp, vp, t, n), (q, kp[order], vp[order], moved, n)):
            got = fa.attention_decode(*args)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.get_device_status() == 0
