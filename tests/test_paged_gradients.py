"""The paged cache's calls have no gradient: tensors that need one are refused,
wherever they stand, unless gradients are switched off."""

import pytest
import torch

import flashattention_backward_gb300 as fa
from flashattention_backward_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def calls(dev):
    """Every call on pools, its floating-point tensors by name."""
    kp, vp = (torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    q = torch.zeros(3, 4, 1, 64, dtype=torch.bfloat16, device=dev)
    k, v = (torch.zeros(3, 2, 5, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    table = torch.arange(3, dtype=torch.int32, device=dev)[:, None]
    lengths = torch.ones(3, dtype=torch.int32, device=dev)
    moves = torch.full((2, 3), -1, dtype=torch.int32, device=dev)
    o, L = torch.zeros_like(q), torch.zeros(3, 4, 1, device=dev)
    yield (lambda q, k_pages, v_pages, o, L: fa.attention_decode(q, k_pages, v_pages, table, lengths, out=(o, L)),
           dict(q=q, k_pages=kp, v_pages=vp, o=o, L=L))
    yield (lambda k, v, k_pages, v_pages: fa.cache_append(k, v, k_pages, v_pages, table, lengths),
           dict(k=k, v=v, k_pages=kp, v_pages=vp))
    yield (lambda k_pages, v_pages: fa.cache_copy_pages(k_pages, v_pages, moves), dict(k_pages=kp, v_pages=vp))


@pytest.mark.parametrize("name", ["q", "k", "v", "k_pages", "v_pages"])
def test_a_tensor_that_needs_a_gradient_is_refused(name):
    """The refusal comes first, so it needs no GPU."""
    for call, args in calls("cpu"):
        if name in args:
            for t in (args[name].clone().requires_grad_(), args[name].clone().requires_grad_() * 1):
                with pytest.raises(ValueError, match="no gradient"):
                    call(**{**args, name: t})
                with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                    call(**{**args, name: t})


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["q", "k", "v", "k_pages", "v_pages", "o", "L"])
def test_on_a_gpu(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    for call, args in calls("cuda:0"):
        call(**args)
        if name in args:
            t = args[name].clone().requires_grad_()
            with pytest.raises(ValueError, match="no gradient"):
                call(**{**args, name: t})
            with torch.no_grad():
                call(**{**args, name: t})
    assert fa.get_device_status() == 0


@pytest.mark.gpu
def test_a_descriptor_needs_no_gradient():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kp = torch.zeros(4, 2, 16, 64, device="cuda:0", requires_grad=True)
    assert fa.cache_for(kp, kp).num_pages == 4
