"""Memory of the paged cache's calls on a stream given by the caller, while the
current stream is another and busy: what was freed there with work still to
come must not be written to, and neither what that stream still reads."""

import pytest
import torch

import flashattention_backward_gb300 as fa
from test_gpu_cache_pages import Cache, ints
from test_gpu_decode import make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def busy():
    """Some milliseconds of work on the current stream."""
    big = torch.zeros(1 << 27, device=DEV)
    for _ in range(20):
        big.add_(1)


def sizes(args):
    """Bytes of o, L and the workspace of a decode."""
    q, kp, vp, table, _ = args
    ws = fa.fa_decode_workspace_bytes(fa.cache_for(kp, vp, table), q.shape[1])
    return [q.numel() * q.element_size(), 4 * q.shape[0] * q.shape[1], ws]


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_memory_freed_on_the_current_stream(wide, dtype):
    """Temporaries of the sizes that a decode allocates, read by work that is still to come when they are freed."""
    args = make(4, 8, 2, 128, 16, [4000, 100, 1700, 64], dtype, seed=1, wide=wide)
    want = fa.attention_decode(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(10):
        held = [torch.full((n,), i + 1, dtype=torch.uint8, device=DEV) for n in sizes(args) if n > 0 for _ in range(3)]
        torch.cuda.synchronize()
        busy()
        read = [t + 1 for t in held]
        freed = [t.data_ptr() for t in held]
        del held
        got = fa.attention_decode(*args, stream=side)
        assert not {t.data_ptr() for t in got} & set(freed)
        torch.cuda.synchronize()
        assert all((t == i + 2).all() for t in read)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_call_with_and_one_without_a_stream(wide, dtype):
    """At the same time, each with a workspace that the call allocates."""
    args = [make(4, 8, 2, 128, 16, [4000, 100, 1700, 64], dtype, seed=20 + i, wide=wide) for i in range(2)]
    want = [fa.attention_decode(*a) for a in args]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(40):
        got.append((fa.attention_decode(*args[0]), fa.attention_decode(*args[1], stream=side)))
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
def test_results_read_on_the_current_stream(wide):
    """Results of a call on another stream, let go while the current stream has still to read them."""
    args = [make(4, 8, 2, 128, 16, [4000, 100, 1700, 64], seed=30 + i, wide=wide) for i in range(2)]
    want = [fa.attention_decode(*a) for a in args]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        o, L = fa.attention_decode(*args[0], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        busy()
        read = o.clone(), L.clone()
        del o, L
        for _ in range(3):
            again = fa.attention_decode(*args[1], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(read[0], want[0][0]) and torch.equal(read[1], want[0][1])
        assert torch.equal(again[0], want[1][0]) and torch.equal(again[1], want[1][1])


def test_page_calls_on_a_stream_of_their_own():
    """start, moves and count beside memory of their sizes that the current stream has still to read."""
    side = torch.cuda.Stream()
    src, dst, n, one = ints([0, 1]), ints([2, 3]), ints([9, 3, 0, 0]), ints([0, 0, 1, 1])
    for i in range(10):
        c = Cache(40, 4, 4, 6)
        held = [torch.full((b,), i + 1, dtype=torch.uint8, device=DEV) for b in (4, 16, 24, 240, 512) for _ in range(4)]
        torch.cuda.synchronize()
        busy()
        read = [t + 1 for t in held]
        del held
        start = [fa.pages_extend(*c.args(), n, 4, stream=side)]
        moves = fa.pages_fork(*c.args(), src, dst, 4, stream=side)
        start.append(fa.pages_extend(*c.args(), one, 4, stream=side))
        fa.pages_free(*c.args(), src, 4, stream=side)
        again, count = fa.pages_compact(*c.args(), 4, stream=side)
        torch.cuda.synchronize()
        assert all((t == i + 2).all() for t in read)
        want = [c.m.extend([9, 3, 0, 0]), c.m.fork([0, 1], [2, 3]), c.m.extend([0, 0, 1, 1])]
        c.m.free([0, 1])
        left = c.m.compact()
        c.same()
        assert [start[0].tolist(), [tuple(x) for x in moves.tolist()], start[1].tolist()] == want
        assert again[:len(left)].tolist() == [list(x) for x in left] and count.item() == len(left)
    assert fa.get_device_status(side) == 0


@pytest.mark.parametrize("wide", [0, 3000])
def test_a_stream_given_as_a_number(wide):
    """Also the default stream's number, 0, while another one is current."""
    args = make(3, 8, 2, 64, 16, [900, 0, 65], seed=40, wide=wide)
    want = fa.attention_decode(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side.cuda_stream, side, 0):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = fa.attention_decode(*args, stream=given)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("wide", [0, 3000])
def test_a_graph_of_another_stream(wide):
    """Captured on the stream that is given, which is not the current one inside of the capture."""
    args = make(3, 8, 2, 64, 16, [900, 0, 65], seed=41, wide=wide)
    want = fa.attention_decode(*args)
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        got = fa.attention_decode(*args, stream=side)
        main.wait_stream(side)
        out = got[0] + 0
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(out, want[0])
