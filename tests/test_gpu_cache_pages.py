"""Rows and pages of the paged cache on the GPU: appends and copies bit by bit
against plain indexing, the page calls against a model of Python lists, and a
run of them together."""

import random

import pytest
import torch

import flashattention_backward_gb300 as fa
from oracle.paged_fp64 import PageModel
from test_gpu_decode import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pools(pages, heads, rows, d, dtype, rows_first=False):
    shape = (pages, rows, heads, d) if rows_first else (pages, heads, rows, d)
    out = [torch.randn(shape, device=DEV).to(dtype) for _ in range(2)]
    return [t.permute(0, 2, 1, 3) if rows_first else t for t in out]


class Cache:
    """Device tensors beside the model, compared after every call."""

    def __init__(self, pages, rows, sequences, columns, pad=0):
        self.m = PageModel(pages, rows, sequences, columns)
        self.full = torch.full((sequences, columns + pad), -1, dtype=torch.int32, device=DEV)
        self.table = self.full[:, :columns]
        self.lengths, self.refs = ints([0] * sequences), ints([0] * pages)
        self.rows = rows

    def args(self):
        return self.table, self.lengths, self.refs

    def same(self):
        assert self.table.tolist() == self.m.table
        assert self.lengths.tolist() == self.m.lengths
        assert self.refs.tolist() == self.m.refs
        assert (self.full[:, self.m.columns:] == -1).all()

    def refused(self, want):
        code = fa.get_device_status()
        assert code == (fa.FA_ERR_PAGES if want is None else 0)

    def extend(self, n_new):
        want = self.m.extend(n_new)
        start = fa.pages_extend(*self.args(), ints(n_new), self.rows)
        assert start.tolist() == (want if want is not None else [-1] * len(n_new))
        self.refused(want)
        self.same()
        return start

    def fork(self, src, dst):
        want = self.m.fork(src, dst)
        moves = fa.pages_fork(*self.args(), ints(src), ints(dst), self.rows)
        assert moves.tolist() == [list(x) for x in (want if want is not None else [(-1, -1, -1)] * len(src))]
        self.refused(want)
        self.same()
        return moves

    def free(self, sequences):
        self.m.free(dict.fromkeys(sequences))
        fa.pages_free(*self.args(), ints(sequences), self.rows)
        assert fa.get_device_status() == 0
        self.same()

    def compact(self):
        want = self.m.compact()
        moves, count = fa.pages_compact(*self.args(), self.rows)
        assert fa.get_device_status() == 0
        assert count.item() == len(want)
        assert moves[:len(want)].tolist() == [list(x) for x in want] and (moves[len(want):] == -1).all()
        self.same()
        return moves, count


@pytest.mark.parametrize("rows", [1, 3, 16, 64])
@pytest.mark.parametrize("pages,sequences", [(40, 12), (5000, 40), (9001, 1100)])
def test_page_calls_follow_the_model(rows, pages, sequences):
    rng = random.Random(rows * 100003 + pages)
    c = Cache(pages, rows, sequences, 23, pad=3)
    for step in range(25):
        live = [s for s in range(sequences) if c.m.lengths[s]]
        empty = [s for s in range(sequences) if not c.m.lengths[s]]
        what = rng.choice(["extend", "extend", "fork", "free", "compact"])
        if what == "extend":
            c.extend([rng.choice([0, 0, 1, rng.randint(0, 9 * rows)]) if c.m.lengths[s] < 12 * rows else 0
                      for s in range(sequences)])
        elif what == "fork" and live and empty:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            c.fork([rng.choice(live) for _ in dst], dst)
        elif what == "free" and live:
            c.free(rng.sample(live, rng.randint(1, len(live))) + [-1])
        elif what == "compact":
            c.compact()


def test_refused_calls_change_nothing():
    c = Cache(10, 4, 6, 5)
    c.extend([9, 4, 0, 0, 0, 0])   # 3 + 1 pages
    c.extend([0, 0, 21, 0, 0, 0])  # behind the table
    c.extend([0, 0, -1, 0, 0, 0])
    c.extend([0, 0, 20, 8, 0, 0])  # 7 pages of the 6 left
    c.fork([0], [6])
    c.fork([-1], [2])
    c.fork([0, 1], [2, 2])         # the same destination twice
    c.fork([0, 2], [2, 3])         # a destination that is a source
    c.fork([0], [1])               # a destination in use
    c.fork([1], [0])
    c.extend([0, 0, 20, 0, 0, 0])  # one page left
    c.fork([0, 0], [3, 4])         # wants two
    c.fork([0], [3])
    c.free([3, 3, 0, 3, -1])       # listed more than once: emptied once
    table = c.table.clone()
    fa.pages_free(*c.args(), ints([6, -2, 100]), 4)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    c.same()
    assert torch.equal(table, c.table)


def test_damaged_tables_are_not_followed():
    c = Cache(10, 4, 3, 5)
    c.extend([9, 4, 0])
    c.table[0, 1] = 77
    before = [t.clone() for t in c.args()]
    moves = fa.pages_fork(*c.args(), ints([0]), ints([2]), 4)
    assert fa.get_device_status() == fa.FA_ERR_PAGES and (moves == -1).all()
    assert all(torch.equal(a, b) for a, b in zip(before, c.args()))
    out = (torch.empty_like(c.table), torch.empty_like(c.refs))
    fa.pages_compact(*c.args(), 4, out=out)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert out[0].tolist() == [[0, -1, 2, -1, -1], [3, -1, -1, -1, -1], [-1] * 5]
    fa.pages_free(*c.args(), ints([0]), 4)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert c.refs.tolist() == [0, 1, 0, 1, 0, 0, 0, 0, 0, 0] and c.lengths.tolist() == [0, 4, 0]
    fa.pages_free(*c.args(), ints([0, 0]), 4)  # empty by now
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_drops_entries_of_free_pages(in_place):
    """A damaged entry that names a free page, which the compaction gives to
    another sequence: it becomes -1, it does not come to share that page."""
    c = Cache(10, 4, 3, 5)
    c.extend([9, 4, 8])   # pages 0 1 2, 3 and 4 5
    c.free([1])           # page 3 is free: page 5 will go there
    c.table[0, 1] = 3
    out = (c.table, c.refs) if in_place else (torch.empty_like(c.full)[:, :5], torch.empty_like(c.refs))
    moves, count = fa.pages_compact(*c.args(), 4, out=out)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert count.item() == 1 and moves[0].tolist() == [5, 3, 4]
    assert out[0].tolist() == [[0, -1, 2, -1, -1], [-1] * 5, [4, 3, -1, -1, -1]]


def test_compact_into_copies_leaves_the_old_ones():
    c = Cache(50, 4, 6, 7)
    c.extend([20, 3, 9, 28, 0, 1])
    c.free([0, 2])
    before = [t.clone() for t in c.args()]
    out = (torch.empty_like(c.table), torch.empty_like(c.refs))
    moves, count = fa.pages_compact(*c.args(), 4, out=out)
    assert all(torch.equal(a, b) for a, b in zip(before, c.args()))
    want = c.m.compact()
    assert count.item() == len(want) > 0 and out[0].tolist() == c.m.table and out[1].tolist() == c.m.refs


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 32), (torch.bfloat16, 96), (torch.bfloat16, 256),
                                     (torch.float32, 16), (torch.float32, 128), (torch.float32, 256)])
@pytest.mark.parametrize("rows_first", [False, True])
@pytest.mark.parametrize("page", [1, 13, 16])
def test_append_writes_its_rows_alone(dtype, d, rows_first, page):
    S, H, n = 5, 3, 37
    start, counts = [0, 5, 12, -1, 30], [37, 0, 20, 7, 1]
    columns = -(-70 // page)
    kp, vp = pools(S * columns + 1, H, page, d, dtype, rows_first)
    table = torch.randperm(S * columns + 1, device=DEV)[: S * columns].int().reshape(S, columns)
    k = torch.randn(S, n, H, 2 * d, device=DEV).to(dtype).permute(0, 2, 1, 3)[..., :d]  # padded rows
    v = torch.randn(S, n, H, 2 * d, device=DEV).to(dtype).permute(0, 2, 1, 3)[..., :d]
    want = [kp.clone(), vp.clone()]
    for s in range(S):
        for i in range(counts[s] if start[s] >= 0 else 0):
            j = start[s] + i
            p = table[s, j // page].long()
            want[0][p, :, j % page], want[1][p, :, j % page] = k[s, :, i], v[s, :, i]
    fa.cache_append(k, v, kp, vp, table, ints(start), ints(counts))
    assert fa.get_device_status() == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_without_counts_and_single_rows():
    kp, vp = pools(9, 2, 16, 64, torch.bfloat16)
    table = ints([[3, 1], [0, 8]])
    k, v = (torch.randn(2, 2, 1, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    want = [kp.clone(), vp.clone()]
    for s, (p, r) in enumerate(((1, 0), (0, 15))):
        want[0][p, :, r], want[1][p, :, r] = k[s, :, 0], v[s, :, 0]
    fa.cache_append(k, v, kp, vp, table, ints([16, 15]))
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_drops_rows_without_a_page():
    kp, vp = pools(4, 2, 8, 64, torch.bfloat16)
    k, v = (torch.randn(3, 2, 12, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    want = [kp.clone(), vp.clone()]
    table = ints([[0, 99], [-1, 1], [2, 3]])
    for s, i, p, r in ([(0, i, 0, i) for i in range(8)] + [(1, 8 + i, 1, i) for i in range(4)] +
                       [(2, i, 3, 6 + i) for i in range(2)]):
        want[0][p, :, r], want[1][p, :, r] = k[s, :, i], v[s, :, i]
    fa.cache_append(k, v, kp, vp, table, ints([0, 0, 14]), ints([12, 12, 50]))  # 50: cut to the 12 rows there are
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    fa.cache_append(k, v, kp, vp, table, ints([2 ** 31 - 1, 2 ** 31 - 5, 16]))
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("dtype,H,d,page,rows_first", [(torch.bfloat16, 3, 96, 13, False),
                                                       (torch.bfloat16, 8, 128, 64, True),
                                                       (torch.float32, 1, 16, 1, False),
                                                       (torch.float32, 5, 256, 16, True)])
def test_copy_moves_its_rows_alone(dtype, H, d, page, rows_first):
    kp, vp = pools(30, H, page, d, dtype, rows_first)
    moves = [(0, 10, page), (0, 11, 1), (5, 12, 0), (-1, -1, -1), (29, 2, max(1, page // 2)), (3, 28, page)]
    want = [kp.clone(), vp.clone()]
    for a, b, n in moves:
        for t in want:
            if a >= 0:
                t[b, :, :n] = t[a, :, :n]
    left = [kp.clone(), vp.clone()]
    fa.cache_copy_pages(kp, vp, ints(moves))
    assert fa.get_device_status() == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    kp, vp = left[0].clone(), left[1].clone()
    fa.cache_copy_pages(kp, vp, ints(moves), ints([1]))
    left[0][10], left[1][10] = left[0][0], left[1][0]
    assert torch.equal(kp, left[0]) and torch.equal(vp, left[1])
    fa.cache_copy_pages(kp, vp, ints(moves), ints([0]))
    assert fa.get_device_status() == 0
    bad = ints([(30, 1, 1), (1, 30, 1), (1, 2, page + 1), (1, 2, -1), (-2, 4, 1), (1, -1, 1)])
    fa.cache_copy_pages(kp, vp, bad)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    fa.cache_copy_pages(kp, vp, ints(moves), ints([7]))  # more than there are: all of them
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_large_copies():
    kp, vp = pools(600, 8, 16, 128, torch.bfloat16)
    order = torch.randperm(600, device=DEV)
    src, dst = order[:300], order[300:]
    want = [t.clone() for t in (kp, vp)]
    for t in want:
        t[dst] = t[src]
    fa.cache_copy_pages(kp, vp, torch.stack([src, dst, torch.full_like(src, 16)], 1).int())
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("captured", [False, True])
def test_a_generation_together(captured):
    """Prompts, single tokens, forks, sequences dropped and the pool compacted, with the attention of each step checked
    against dense copies kept on the side; the step of one token also captured and replayed."""
    S, H, Hk, d, page, pages, columns = 6, 8, 2, 64, 5, 60, 12
    rng = random.Random(4)
    gen = torch.Generator().manual_seed(4)
    c = Cache(pages, page, S, columns)
    kp, vp = (torch.full((pages, Hk, page, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dense = [[torch.zeros(Hk, 0, d, dtype=torch.bfloat16) for _ in range(2)] for _ in range(S)]

    def rand(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16)

    def grow(n_new):
        rows = max(n_new)
        k, v = rand(S, Hk, rows, d), rand(S, Hk, rows, d)
        start = c.extend(n_new)
        fa.cache_append(k.to(DEV), v.to(DEV), kp, vp, c.table, start, ints(n_new))
        for s in range(S):
            for i, t in enumerate((k, v)):
                dense[s][i] = torch.cat([dense[s][i], t[s, :, :n_new[s]]], 1)

    def look(q, got):
        n = max(1, max(x[0].shape[1] for x in dense))
        kd, vd = torch.zeros(S, Hk, n, d).bfloat16(), torch.zeros(S, Hk, n, d).bfloat16()
        for s in range(S):
            kd[s, :, :dense[s][0].shape[1]], vd[s, :, :dense[s][1].shape[1]] = dense[s]
        check(got, q, kd, vd, torch.arange(S, dtype=torch.int32)[:, None],
              torch.tensor([x[0].shape[1] for x in dense], dtype=torch.int32), d ** -0.5)

    def attend():
        q = rand(S, H, 1, d).to(DEV)
        got = fa.attention_decode(q, kp, vp, c.table, c.lengths)
        assert fa.get_device_status() == 0
        look(q, got)

    grow([11, 5, 0, 1, 0, 0])
    attend()
    one, q1 = ints([0] * S), torch.zeros(S, H, 1, d, dtype=torch.bfloat16, device=DEV)
    k1, v1 = (torch.zeros(S, Hk, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        start = fa.pages_extend(*c.args(), one, page)
        fa.cache_append(k1, v1, kp, vp, c.table, start, one)
        return fa.attention_decode(q1, kp, vp, c.table, c.lengths)

    if captured:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            step()  # no new rows: changes nothing
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                held = step()
        torch.cuda.synchronize()

    def token(live):
        n_new = [1 if s in live else 0 for s in range(S)]
        k, v, q = rand(S, Hk, 1, d), rand(S, Hk, 1, d), rand(S, H, 1, d)
        for t, x in ((k1, k), (v1, v), (q1, q), (one, torch.tensor(n_new, dtype=torch.int32))):
            t.copy_(x)
        torch.cuda.synchronize()
        if captured:
            graph.replay()
            got = held
        else:
            got = step()
        assert fa.get_device_status() == 0
        assert c.m.extend(n_new) is not None
        c.same()
        for s in live:
            dense[s] = [torch.cat([dense[s][i], t[s]], 1) for i, t in enumerate((k, v))]
        look(q1, got)

    for _ in range(7):
        token([0, 1, 3])
    fa.cache_copy_pages(kp, vp, c.fork([0, 0, 1], [2, 4, 5]))
    for a, b in ((0, 2), (0, 4), (1, 5)):
        dense[b] = list(dense[a])
    attend()
    for _ in range(6):
        token(list(range(S)))
    gone = rng.sample(range(S), 3)
    c.free(gone)
    for s in gone:
        dense[s] = [torch.zeros(Hk, 0, d, dtype=torch.bfloat16) for _ in range(2)]
    fa.cache_copy_pages(kp, vp, *c.compact())
    attend()
    grow([0 if s not in gone else 13 for s in range(S)])
    for _ in range(4):
        token(list(range(S)))


def test_refusals():
    kp, vp = pools(9, 2, 16, 64, torch.bfloat16)
    table, start = ints([[3, 1], [0, 8]]), ints([0, 0])
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device=DEV)
    before = kp.clone()
    for args in ((k[:1], k[:1], kp, vp, table, start), (k, k[:, :, :2], kp, vp, table, start),
                 (k.float(), k.float(), kp, vp, table, start), (k, k.transpose(1, 2).contiguous().transpose(1, 2), kp, vp, table, start),
                 (k[..., :32], k[..., :32], kp, vp, table, start), (k, k, kp, vp, table, start.long()),
                 (k, k, kp, vp, table, start[:1]), (k, k, kp, vp, table[0], start), (k, k, kp, vp, table, start, start[:1]),
                 (k.cpu(), k.cpu(), kp, vp, table, start)):
        with pytest.raises(ValueError):
            fa.cache_append(*args)
    fa.cache_append(k[:, :, :0], k[:, :, :0], kp, vp, table, start)  # no rows: nothing to do
    for moves in (ints([0, 1, 2]), ints([[0, 1]]), ints([[0, 1, 2]]).long(), ints([[0, 1, 2]]).cpu()):
        with pytest.raises(ValueError):
            fa.cache_copy_pages(kp, vp, moves)
    with pytest.raises(ValueError):
        fa.cache_copy_pages(kp, vp, ints([[0, 1, 2]]), ints([1, 2]))
    fa.cache_copy_pages(kp, vp, torch.empty(0, 3, dtype=torch.int32, device=DEV))
    assert torch.equal(kp, before)
    c = Cache(9, 4, 3, 5)
    one = ints([1, 0, 0])
    for call in (lambda: fa.pages_extend(c.table, c.lengths, c.refs, one[:2], 4),
                 lambda: fa.pages_extend(c.table, c.lengths.long(), c.refs, one, 4),
                 lambda: fa.pages_extend(c.table.long(), c.lengths, c.refs, one, 4),
                 lambda: fa.pages_extend(c.table, c.lengths, c.refs.cpu(), one, 4),
                 lambda: fa.pages_fork(c.table, c.lengths, c.refs, one, one[:2], 4),
                 lambda: fa.pages_fork(c.table, c.lengths, c.refs, one.long(), one, 4),
                 lambda: fa.pages_free(c.table, c.lengths, c.refs, one[None], 4),
                 lambda: fa.pages_compact(c.table, c.lengths, c.refs, 4, out=(c.table[:2], c.refs)),
                 lambda: fa.pages_compact(c.table, c.lengths, c.refs, 4, out=(c.table, c.refs[:2]))):
        with pytest.raises(ValueError):
            call()
    for rows in (0, -1):
        with pytest.raises(fa.FaError):
            fa.pages_extend(c.table, c.lengths, c.refs, one, rows)
    with pytest.raises(fa.FaError):
        fa.pages_extend(c.table, c.lengths, c.refs, ints([99, 0, 0]), 4, check_status=True)
    assert fa.pages_fork(c.table, c.lengths, c.refs, one[:0], one[:0], 4).shape == (0, 3)
    fa.pages_free(c.table, c.lengths, c.refs, one[:0], 4)
    c.same()
    assert fa.get_device_status() == 0


def test_calls_on_another_stream():
    """A stream given by the caller, while the current one is another."""
    stream = torch.cuda.Stream()
    c = Cache(40, 4, 4, 6)
    kp, vp = pools(40, 2, 4, 64, torch.bfloat16)
    k = torch.randn(4, 2, 9, 64, device=DEV).to(torch.bfloat16)
    n = ints([9, 3, 0, 0])
    src, dst = ints([0, 1]), ints([2, 3])
    torch.cuda.synchronize()
    start = fa.pages_extend(*c.args(), n, 4, stream=stream)
    fa.cache_append(k, k, kp, vp, c.table, start, n, stream=stream)
    moves = fa.pages_fork(*c.args(), src, dst, 4, stream=stream)
    fa.cache_copy_pages(kp, vp, moves, stream=stream)
    fa.pages_free(*c.args(), src, 4, stream=stream)
    again, count = fa.pages_compact(*c.args(), 4, stream=stream)
    fa.cache_copy_pages(kp, vp, again, count, stream=stream.cuda_stream)
    stream.synchronize()
    assert fa.get_device_status(stream) == 0
    c.m.extend([9, 3, 0, 0])
    c.m.fork([0, 1], [2, 3])
    c.m.free([0, 1])
    c.m.compact()
    c.same()
    for s, n in ((2, 9), (3, 3)):
        for j in range(n):
            assert torch.equal(kp[c.m.table[s][j // 4], :, j % 4], k[s - 2, :, j])


def test_a_step_captured_between_other_work():
    """Copies, kernels of PyTorch's own and another stream's work in front of, between and behind the calls of a captured
    step: the calls' blocks may line up early, but must not look at anything before it is there."""
    S, H, Hk, d, page = 4, 8, 2, 64, 16
    c = Cache(64, page, S, 12)
    kp, vp = pools(64, Hk, page, d, torch.bfloat16)
    src = [torch.randn(S, n, 1, d, device=DEV).to(torch.bfloat16) for n in (Hk, Hk, H)]
    k, v, q = (torch.zeros_like(t) for t in src)
    plan, one = ints([1, 1, 0, 1]), ints([0] * S)
    big = torch.zeros(1 << 24, device=DEV)
    host = torch.zeros(S, dtype=torch.int32).pin_memory()
    c.extend([30, 15, 0, 1])
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def step():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big.add_(1)                # something slow, and then what the step reads
            one.copy_(plan)
            k.copy_(src[0])
            v.copy_(src[1])
        torch.cuda.current_stream().wait_stream(side)
        q.copy_(src[2])
        start = fa.pages_extend(*c.args(), one, page)
        big.mul_(2)
        fa.cache_append(k, v, kp, vp, c.table, start, one)
        got = fa.attention_decode(q, kp, vp, c.table, c.lengths)
        out = got[0] * 2
        host.copy_(start, non_blocking=True)
        return got[0], got[1], out

    with torch.cuda.stream(main):
        step()
        torch.cuda.synchronize()
        c.m.extend([1, 1, 0, 1])
        with torch.cuda.graph(graph, stream=main):
            got = step()
    torch.cuda.synchronize()
    for i in range(20):
        for t in src:
            t.normal_()
        plan.copy_(ints([1, i % 2, i // 3 % 2, 1]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert fa.get_device_status() == 0
        want = c.m.extend([1, i % 2, i // 3 % 2, 1])
        c.same()
        assert host.tolist() == want
        check(got[:2], src[2], kp, vp, c.table, c.lengths, d ** -0.5)
        assert torch.equal(got[2], got[0] * 2)
        for s in range(S):
            n = c.m.lengths[s] - 1
            if want[s] == n:
                assert torch.equal(kp[c.m.table[s][n // page], :, n % page], src[0][s, :, 0])
