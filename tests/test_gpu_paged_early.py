"""Calls of the paged cache that directly follow the call whose results they
read, behind slow work, in a captured graph and outside of one: their blocks
are on the GPU before that work has ended, and must not use what they read
before it is there."""

import pytest
import torch

import flashattention_backward_gb300 as fa
from test_gpu_cache_pages import Cache, ints, pools
from test_gpu_decode import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def captured(step):
    """step() once outside a graph, then as a graph on a stream of its own: (replay, results)."""
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
    torch.cuda.synchronize()
    return graph.replay, got


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("graph", [False, True])
def test_extend_then_decode(dtype, wide, graph):
    """The lengths and table that a decode reads come from the kernel in front of it, which waits for slow work itself."""
    S, H, Hk, d, page = 5, 8, 2, 64, 16
    c = Cache(96, page, S, 12 + wide)
    kp, vp = pools(96, Hk, page, d, dtype)
    q = torch.randn(S, H, 1, d, device=DEV).to(dtype)
    plan, n_new = ints([0] * S), ints([0] * S)
    big = torch.zeros(1 << 24, device=DEV)

    def step():
        big.add_(1)
        n_new.copy_(plan)
        fa.pages_extend(*c.args(), n_new, page)
        return fa.attention_decode(q, kp, vp, c.table, c.lengths)

    replay, got = captured(step) if graph else (None, None)
    for more in ([30, 1, 0, 64, 16], [0, 0, 0, 0, 0], [1, 1, 3, 1, 1], [33, 15, 0, 80, 2]):
        q.normal_()
        plan.copy_(ints(more))
        torch.cuda.synchronize()
        if graph:
            replay()
        else:
            got = step()
        torch.cuda.synchronize()
        assert fa.get_device_status() == 0
        assert c.m.extend(more) is not None
        c.same()
        check(got, q, kp, vp, c.table, c.lengths, d ** -0.5)


@pytest.mark.parametrize("graph", [False, True])
def test_fork_copy_extend_append_free_compact_copy(graph):
    """Every call reads what the one in front of it wrote: moves, start, table, lengths, counts."""
    S, Hk, d, page = 6, 2, 64, 8
    c = Cache(64, page, S, 9)
    kp, vp = pools(64, Hk, page, d, torch.bfloat16)
    k, v = (torch.randn(S, Hk, 3, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    src, dst, gone = ints([0, 1, 1]), ints([2, 3, 4]), ints([0, 1])
    n_new = ints([0, 0, 3, 1, 0, 0])
    big = torch.zeros(1 << 24, device=DEV)
    kept = [t.clone() for t in (kp, vp)]
    c.extend([13, 20, 0, 0, 0, 0])
    before = [t.clone() for t in c.args()]

    def back():
        for t, x in zip((kp, vp, *c.args()), (*kept, *before)):
            t.copy_(x)

    def step():
        back()
        big.add_(1)
        fa.cache_copy_pages(kp, vp, fa.pages_fork(*c.args(), src, dst, page))
        fa.cache_append(k, v, kp, vp, c.table, fa.pages_extend(*c.args(), n_new, page), n_new)
        fa.pages_free(*c.args(), gone, page)
        moves, count = fa.pages_compact(*c.args(), page)
        fa.cache_copy_pages(kp, vp, moves, count)
        return moves, count

    m = c.m
    dense = [[[t[m.table[a][j // page], :, j % page] for j in range(m.lengths[a])] for t in kept] for a in (0, 1, 1)]
    for i, n in ((0, 3), (1, 1)):
        for t, x in zip(dense[i], (k, v)):
            t.extend(x[2 + i, :, j] for j in range(n))
    m.fork([0, 1, 1], [2, 3, 4])
    m.extend([0, 0, 3, 1, 0, 0])
    m.free([0, 1])
    want = m.compact()
    replay, got = captured(step) if graph else (None, None)
    for _ in range(5):
        if graph:
            replay()
        else:
            got = step()
        torch.cuda.synchronize()
        assert fa.get_device_status() == 0
        c.same()
        assert got[1].item() == len(want) > 0 and got[0][:len(want)].tolist() == [list(x) for x in want]
        for i in range(3):
            for t, rows in zip((kp, vp), dense[i]):
                for j, x in enumerate(rows):
                    assert torch.equal(t[m.table[2 + i][j // page], :, j % page], x)
