"""Rows of the paged cache in 8 bits on the GPU: appends, reads and copies bit
by bit against the restatement, damaged tables, other streams, graphs, and a run of all calls
together."""

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from oracle import e4m3_fp64 as oracle
from test_gpu_cache_pages import Cache, ints

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def f64(t):
    return t.detach().cpu().float().double().numpy()


def pool(gen, pages, heads, rows, d, block, rows_first=False):
    """A pool full of values, and scales: [values, scales]."""
    shape = (pages, rows, heads, d) if rows_first else (pages, heads, rows, d)
    x = (torch.randn(shape, generator=gen) * 112).clamp(-448, 448).to(F8).to(DEV)
    e = torch.randint(-9, -5, (pages, heads, rows // block), generator=gen)
    return [x.permute(0, 2, 1, 3) if rows_first else x, torch.exp2(e.float()).to(DEV)]


class Quantised:
    """Pools and scales of K and V, beside the restatement's."""

    def __init__(self, pages, heads, rows, d, block, seed=0, rows_first=False):
        gen = torch.Generator().manual_seed(seed)
        (self.kp, self.ks), (self.vp, self.vs) = (pool(gen, pages, heads, rows, d, block, rows_first) for _ in range(2))
        self.block = block
        self.want = [[f64(self.kp), f64(self.ks)], [f64(self.vp), f64(self.vs)]]

    def args(self):
        return self.kp, self.vp, self.ks, self.vs

    def append(self, k, v, table, start, counts=None, status=0, **kw):
        fa.cache_append_e4m3(k, v, *self.args(), table, start, counts, **kw)
        torch.cuda.synchronize()
        assert fa.get_device_status() == status
        for x, (p, s) in zip((k, v), self.want):
            oracle.append(f64(x), p, s, table.cpu().numpy(), start.tolist(), None if counts is None else counts.tolist(),
                          self.block)

    def same(self):
        for got, want in zip((self.kp, self.ks, self.vp, self.vs), (w for pair in self.want for w in pair)):
            assert np.array_equal(f64(got), want, equal_nan=True)


def table_of(gen, held, columns, pages):
    order = torch.randperm(pages, generator=gen)
    table = torch.full((len(held), columns), -1, dtype=torch.int32)
    k = 0
    for s, n in enumerate(held):
        table[s, :n] = order[k:k + n].int()
        k += n
    return table.to(DEV)


def rows_like(gen, shape, dtype, layout="bhnd"):
    S, H, n, d = shape
    x = torch.randn((S, n, H, d) if layout == "bnhd" else shape, generator=gen)
    x *= torch.exp2(torch.randint(-3, 4, x.shape[:-1] + (1,), generator=gen).float())  # rows of different size
    x = x.to(dtype).to(DEV)
    return x.permute(0, 2, 1, 3) if layout == "bnhd" else x


@pytest.mark.parametrize("page,block", [(1, 1), (8, 2), (13, 1), (13, 13), (16, 16), (48, 24), (64, 8), (100, 100), (256, 256)])
@pytest.mark.parametrize("d,dtype", [(32, torch.bfloat16), (64, torch.float32), (96, torch.bfloat16), (128, torch.bfloat16),
                                     (256, torch.bfloat16), (16, torch.float32), (256, torch.float32)])
def test_append(page, block, d, dtype):
    """From the front, from the middle of a block and behind its end; counts from nothing to all; then one row more."""
    gen = torch.Generator().manual_seed(page * 1000 + d)
    start, counts, n = [0, 5, page - 1, page, 3 * page + block // 2], [37, 0, 1, 36, 20], 37
    held = [-(-(a + c + 1) // page) for a, c in zip(start, counts)]
    c = Quantised(sum(held) + 2, 3, page, d, block, seed=d, rows_first=d == 64)
    table = table_of(gen, held, max(held) + 1, sum(held) + 2)
    k, v = (rows_like(gen, (5, 3, n, d), dtype, "bnhd" if d == 128 else "bhnd") for _ in range(2))
    c.append(k, v, table, ints(start), ints(counts))
    c.same()
    k, v = (rows_like(gen, (5, 3, 1, d), dtype) for _ in range(2))
    c.append(k, v, table, ints([a + m for a, m in zip(start, counts)]))
    c.same()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_row_by_row(dtype):
    """A block whose scale grows again and again, and one whose scale does not."""
    gen = torch.Generator().manual_seed(1)
    c = Quantised(4, 2, 32, 64, 16, seed=1)
    table = ints([[2, 0], [3, 1]])
    for i in range(40):
        k, v = (torch.randn(2, 2, 1, 64, generator=gen) for _ in range(2))
        k *= 2.0 ** (i % 16 - 8)
        v *= 2.0 ** -(i % 16)
        c.append(k.to(dtype).to(DEV), v.to(dtype).to(DEV), table, ints([i, i]))
        c.same()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_extremes(dtype):
    """The type's lowest and smallest values, rows of zeros, infinities and NaN, values at the border of a scale."""
    low = torch.finfo(dtype).min
    step = torch.finfo(dtype).eps
    kinds = [[low, 1.0], [0.0, -0.0], [2.0 ** -126, -2.0 ** -133], [float("inf"), 3.0], [float("nan"), -3.0],
             [float("-inf"), float("nan")], [448.0, -0.001], [448 * (1 + 2 * step), 17.0], [1.75 * 2.0 ** -100, 2.0 ** -109],
             [float("-inf"), low]]
    x = torch.zeros(len(kinds), 1, 4, 32)
    for i, (a, b) in enumerate(kinds):
        x[i, 0, 1, 3], x[i, 0, 2, 30] = a, b
        x[i, 0, 3] = b / 3
    x = x.to(dtype).to(DEV)
    c = Quantised(len(kinds), 1, 8, 32, 4)
    table = ints([[i] for i in range(len(kinds))])
    c.append(x, -x, table, ints([0] * len(kinds)))
    c.same()
    c.append(x, x.flip(2), table, ints([2] * len(kinds)))  # into a block that holds rows, and the next one
    c.same()


def test_append_leaves_the_rest_alone():
    """Rows before and behind, heads and pages beside, blocks that get no rows, sequences with a negative start or none."""
    gen = torch.Generator().manual_seed(3)
    c = Quantised(9, 2, 16, 64, 4, seed=3)
    before = [t.clone() for t in c.args()]
    table = ints([[0, 1], [2, 3], [4, 5]])
    k, v = (rows_like(gen, (3, 2, 5, 64), torch.bfloat16) for _ in range(2))
    c.append(k, v, table, ints([14, -1, 0]), ints([5, 5, 0]))
    c.same()
    for t, old in zip(c.args(), before):
        assert torch.equal(t.view(torch.uint8)[2:], old.view(torch.uint8)[2:])


def test_append_strides():
    """Keys and values of one projection, a pool that is part of a larger one."""
    gen = torch.Generator().manual_seed(4)
    S, H, n, d = 3, 2, 7, 64
    fused = torch.randn(S, n, 3, H, d, generator=gen).to(torch.bfloat16).to(DEV)
    k, v = fused[:, :, 1].permute(0, 2, 1, 3), fused[:, :, 2].permute(0, 2, 1, 3)
    c = Quantised(6, H, 8, d, 8, seed=4)
    big = torch.zeros(6, H + 1, 8, 2 * d, device=DEV).to(F8)
    kp, vp = big[:, :H, :, :d], big[:, :H, :, d:]
    kp.copy_(c.kp), vp.copy_(c.vp)
    c.kp, c.vp = kp, vp
    c.append(k, v, ints([[0, 1], [2, 3], [4, 5]]), ints([0, 3, 9]))
    c.same()
    assert (big[:, H].float() == 0).all()


def test_bad_pages_starts_and_counts():
    gen = torch.Generator().manual_seed(5)
    c = Quantised(6, 2, 8, 64, 4, seed=5)
    table = ints([[0, 1 << 20, 2], [-7, 3, 4], [5, -1, -1]])
    k, v = (rows_like(gen, (3, 2, 20, 64), torch.bfloat16) for _ in range(2))
    c.append(k, v, table, ints([2, 5, 0]), ints([20, 19, 8]), status=fa.FA_ERR_PAGES)
    c.same()
    c.append(k, v, table, ints([0, 0, 2]), ints([-3, 0, 30]), status=fa.FA_ERR_PAGES)  # counts are cut
    c.same()
    for start in (20, 24, 1 << 30, (1 << 31) - 1):  # at and behind the table's end
        c.append(k, v, table, ints([start, 24, 24]), ints([20, 1, 0]), status=fa.FA_ERR_PAGES)
        c.same()
    x = [torch.full((3, 2, 20, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for start, counts in (([2, 0, 0], [20, 20, 8]), ([-1, 8, 3], [5, 30, -2]), ([(1 << 31) - 1, 23, 24], [20, 2, 1])):
        fa.cache_read_e4m3(*c.args(), table, 20, ints(start), ints(counts), out=tuple(x))
        assert fa.get_device_status() == fa.FA_ERR_PAGES
        for got, (p, s) in zip(x, c.want):
            assert np.array_equal(f64(got), dense(p, s, table.tolist(), start, counts, 20))
    with pytest.raises(fa.FaError) as err:
        fa.cache_read_e4m3(*c.args(), table, 20, ints([-1, 0, 0]), ints([1, 0, 0]), check_status=True)
    assert err.value.code == fa.FA_ERR_PAGES and fa.get_device_status() == 0


def dense(pages, scales, table, start, counts, rows):
    """What is read: zeros behind the counts and where there is no page."""
    x = oracle.values(pages, scales)
    P, H, R, d = x.shape
    out = np.zeros((len(table), H, rows, d))
    for s, ids in enumerate(table):
        a = 0 if start is None else start[s]
        for i in range(rows if counts is None else min(max(counts[s], 0), rows)):
            column = (a + i) // R
            if a >= 0 and column < len(ids) and 0 <= ids[column] < P:
                out[s, :, i] = x[ids[column], :, (a + i) % R]
    return out


@pytest.mark.parametrize("page,block", [(1, 1), (13, 13), (16, 4), (64, 64), (256, 32)])
@pytest.mark.parametrize("d,dtype", [(32, torch.bfloat16), (128, torch.bfloat16), (96, torch.bfloat16), (16, torch.float32),
                                     (256, torch.float32)])
def test_read(page, block, d, dtype):
    """Every stored value times its scale is exact in both types."""
    gen = torch.Generator().manual_seed(page + d)
    c = Quantised(40, 3, page, d, block, seed=d, rows_first=page == 16)
    columns = 9
    table = torch.randint(0, 40, (4, columns), generator=gen).int().to(DEV)
    n = page * columns
    for rows, start, counts in ((min(n, 300), None, None), (min(n, 300), [0, 1, n // 2, n], [min(n, 300), 0, n // 3, 0]),
                                (1, [n - 1, 0, 3 % n, 0], None)):
        if counts is not None:
            counts = [min(x, rows) for x in counts]
        got = fa.cache_read_e4m3(*c.args(), table, rows, None if start is None else ints(start),
                                 None if counts is None else ints(counts), dtype=dtype)
        assert fa.get_device_status() == 0
        for x, (p, s) in zip(got, c.want):
            assert x.shape == (4, 3, rows, d) and x.dtype == dtype
            assert np.array_equal(f64(x), dense(p, s, table.tolist(), start, counts, rows))


def test_read_into_given_rows():
    c = Quantised(8, 2, 16, 64, 16, seed=6)
    table = ints([[0, 3], [5, 1]])
    big = torch.full((2, 30, 3, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    other = torch.full_like(big, 7.0)
    out = tuple(t[:, :25, :2].permute(0, 2, 1, 3) for t in (big, other))
    got = fa.cache_read_e4m3(*c.args(), table, 25, counts=ints([25, 4]), out=out)
    assert got[0].data_ptr() == big.data_ptr()
    for t, (p, s) in zip((big, other), c.want):
        assert np.array_equal(f64(t[:, :25, :2].permute(0, 2, 1, 3)), dense(p, s, table.tolist(), None, [25, 4], 25))
        assert (t[:, 25:] == 7).all() and (t[:, :, 2] == 7).all()
    assert fa.get_device_status() == 0
    assert fa.cache_read_e4m3(*c.args(), table, 0)[0].shape == (2, 2, 0, 64)


def test_nan_is_read_back():
    """Both codes of NaN, whatever their scale; zeros where nothing is asked for."""
    c = Quantised(2, 1, 4, 32, 4, seed=7)
    c.kp.view(torch.uint8)[0, 0, 1, 3], c.kp.view(torch.uint8)[0, 0, 2, 4] = 0x7f, 0xff
    k, _ = fa.cache_read_e4m3(*c.args(), ints([[0]]), 4, counts=ints([2]))
    want = torch.zeros(4, 32, dtype=torch.bool, device=DEV)
    want[1, 3] = True
    assert torch.equal(k[0, 0].isnan(), want) and (k[0, 0, 2:] == 0).all()


def move_rows(c, moves):
    for p, s in c.want:
        for src, dst, rows in moves:
            if src >= 0:
                p[dst, :, :rows] = p[src, :, :rows]
                held = -(-rows // c.block)
                s[dst, :, :held] = s[src, :, :held]


@pytest.mark.parametrize("page,block,d,heads", [(1, 1, 16, 1), (13, 1, 96, 3), (16, 4, 64, 2), (100, 50, 256, 5), (256, 1, 128, 32)])
def test_copy(page, block, d, heads):
    c = Quantised(30, heads, page, d, block, seed=page, rows_first=page == 16)
    order = np.random.default_rng(page).permutation(30)
    moves = [(int(a), int(b), r) for a, b, r in zip(order[:10], order[10:20], [page, 1, 0, page // 2, page] * 2)]
    moves[4] = (-1, -1, -1)
    fa.cache_copy_pages_e4m3(*c.args(), ints(moves))
    move_rows(c, moves)
    assert fa.get_device_status() == 0
    c.same()
    rest = [(int(order[20 + i]), int(order[i]), page) for i in range(5)]
    fa.cache_copy_pages_e4m3(*c.args(), ints(rest), ints([3]))
    move_rows(c, rest[:3])
    c.same()


def test_bad_moves_are_skipped():
    c = Quantised(6, 2, 8, 64, 4, seed=8)
    moves = [(0, 6, 8), (-2, 1, 8), (0, 2, 9), (1, 3, -1), (0, 4, 5)]
    fa.cache_copy_pages_e4m3(*c.args(), ints(moves))
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    move_rows(c, moves[4:])
    c.same()
    fa.cache_copy_pages_e4m3(*c.args(), ints([(1, 5, 8)]), ints([2]))
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    move_rows(c, [(1, 5, 8)])
    c.same()


def test_offsets_beyond_32_bits():
    """Pages further than 2^32 bytes into the pools, scales further than 2^31 floats' bytes."""
    pages, page, d = 140000, 256, 128  # 4.6e9 bytes a pool
    kp, vp = (torch.empty(pages, 1, page, d, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    ks, vs = (torch.empty(pages, 1, page, device=DEV) for _ in range(2))
    ids = [139999, 3, 135000, 139990]
    gen = torch.Generator().manual_seed(9)
    k, v = (rows_like(gen, (1, 1, 1000, d), torch.bfloat16) for _ in range(2))
    fa.cache_append_e4m3(k, v, kp, vp, ks, vs, ints([ids]), ints([0]))
    fa.cache_copy_pages_e4m3(kp, vp, ks, vs, ints([[139999, 139998, 256]]))
    ids[0] = 139998
    got = fa.cache_read_e4m3(kp, vp, ks, vs, ints([ids]), 1000)
    assert fa.get_device_status() == 0
    small = Quantised(4, 1, page, d, 1)
    for x, y, (p, s) in zip((k, v), got, small.want):
        oracle.append(f64(x), p, s, np.array([[0, 1, 2, 3]]), [0], None, 1)
        assert np.array_equal(f64(y), dense(p, s, [[0, 1, 2, 3]], None, None, 1000))


def test_more_blocks_than_32_bits_count_threads():
    """One row over and over, each a block of its own."""
    n, page = (1 << 27) + 50, 1 << 20
    pages = n // page + 1
    kp, vp = (torch.zeros(pages, 1, page, 16, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    ks, vs = (torch.zeros(pages, 1, page, device=DEV) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    x = torch.arange(1.0, 17.0, device=DEV)
    fa.cache_append_e4m3(x.expand(1, 1, n, 16), (-x).expand(1, 1, n, 16), kp, vp, ks, vs, table, ints([0]))
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    # 16 is below 448 * 2^-4 = 28 and above 14; all of 1 ... 16 have four significant bits
    for scales in (ks, vs):
        assert (scales.view(-1)[:n] == 2.0 ** -4).all() and (scales.view(-1)[n:] == 0).all()
    for pool, sign in ((kp, 1), (vp, -1)):
        rows = pool.view(torch.uint8).view(-1, 16)
        for part in (rows[:50], rows[n - 100:n]):
            assert torch.equal(part.view(F8).float(), (sign * 16 * x).expand(len(part), 16))
        assert (rows[n:] == 0).all()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("block", [1, 4, 8])
def test_a_run_of_all_calls(graph, block):
    """Prompts, forks, further tokens, compaction and reading, behind slow work and in a captured graph: every call reads
    what the one in front of it wrote."""
    S, Hk, d, page = 6, 2, 64, 8
    gen = torch.Generator().manual_seed(10 + block)
    c = Cache(64, page, S, 9)
    x = Quantised(64, Hk, page, d, block, seed=10)
    prompts = [rows_like(gen, (S, Hk, 20, d), torch.bfloat16) for _ in range(2)]
    k, v = (rows_like(gen, (S, Hk, 3, d), torch.bfloat16) for _ in range(2))
    q = torch.randn(S, 4, 1, d, generator=gen).to(torch.bfloat16).to(DEV)
    lens, n_new = ints([13, 20, 0, 0, 0, 0]), ints([0, 0, 3, 1, 0, 0])
    src, dst, gone = ints([0, 1, 1]), ints([2, 3, 4]), ints([0, 1])
    big = torch.zeros(1 << 24, device=DEV)
    kept = [t.clone() for t in (*x.args(), *c.args())]

    def step():
        for t, old in zip((*x.args(), *c.args()), kept):
            t.view(torch.uint8).copy_(old.view(torch.uint8)) if t.dtype == F8 else t.copy_(old)
        big.add_(1)
        start = fa.pages_extend(*c.args(), lens, page)
        fa.cache_append_e4m3(*prompts, *x.args(), c.table, start, lens)
        fa.cache_copy_pages_e4m3(*x.args(), fa.pages_fork(*c.args(), src, dst, page))
        start = fa.pages_extend(*c.args(), n_new, page)
        fa.cache_append_e4m3(k, v, *x.args(), c.table, start, n_new)
        fa.pages_free(*c.args(), gone, page)
        moves, count = fa.pages_compact(*c.args(), page)
        fa.cache_copy_pages_e4m3(*x.args(), moves, count)
        o, L = fa.attention_decode_e4m3(q, *x.args(), c.table, c.lengths)
        return o, L, fa.cache_read_e4m3(*x.args(), c.table, 24, counts=c.lengths)

    m = c.m
    want = x.want

    def append(rows, start, counts):
        for r, (p, s) in zip(rows, want):
            oracle.append(f64(r), p, s, np.array(m.table), start, counts, block)

    append(prompts, m.extend(lens.tolist()), lens.tolist())
    move_rows(x, m.fork([0, 1, 1], [2, 3, 4]))
    append((k, v), m.extend(n_new.tolist()), n_new.tolist())
    m.free([0, 1])
    move_rows(x, m.compact())
    stream = torch.cuda.Stream()
    if graph:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            step()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=stream):
                got = step()
        torch.cuda.synchronize()
    for _ in range(4):
        if graph:
            g.replay()
        else:
            got = step()
        torch.cuda.synchronize()
        assert fa.get_device_status() == 0
        c.same()
        o, L, read = got
        for y, (p, s) in zip(read, want):
            assert np.array_equal(f64(y), dense(p, s, m.table, None, m.lengths, 24))
        # the attention of the rows read back, which bf16 holds exactly, is that of the rows in the cache
        keys, values = (y.double() for y in read)
        seen = torch.arange(24, device=DEV)[None, :] < c.lengths[:, None]
        w = (q.double().view(S, Hk, 2, d) @ keys.transpose(2, 3) * d ** -0.5).masked_fill(~seen[:, None, None], -np.inf)
        ref = (torch.nan_to_num(torch.softmax(w, 3)) @ values).view(S, 4, 1, d)
        assert (o.double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 1e-4 * values.abs().max()
        assert torch.equal(L.isinf(), (c.lengths == 0)[:, None, None].expand_as(L))


def test_prompts_go_on_from_the_cache():
    """The forward over rows read back, queries of the last tokens against all of them, as the next part of a prompt."""
    gen = torch.Generator().manual_seed(12)
    S, H, d, n, page = 2, 3, 128, 200, 16
    c = Quantised(40, H, page, d, page, seed=12)
    table = table_of(gen, [13, 13], 13, 40)
    k, v = (rows_like(gen, (S, H, n, d), torch.bfloat16, "bnhd") for _ in range(2))
    c.append(k, v, table, ints([0, 0]))
    c.same()
    keys, values = fa.cache_read_e4m3(*c.args(), table, n)
    q = torch.randn(S, H, 1, d, generator=gen).to(torch.bfloat16).to(DEV)
    o, L = fa.attention_forward(q, keys, values, d ** -0.5, causal=True)
    o2, L2 = fa.attention_decode_e4m3(q, *c.args(), table, ints([n, n]))
    # the forward rounds its weights to bf16 (2^-8 of each, at most 2^-8 of max |v| in the sum) and its output
    assert (o.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * values.float().abs().max()
    assert (L.reshape(S, H) - L2.reshape(S, H)).abs().max() <= 1e-3


def test_calls_on_another_stream():
    """Memory that a call allocates is that of the stream it is given, while the current one is busy."""
    gen = torch.Generator().manual_seed(13)
    side = torch.cuda.Stream()
    c = Quantised(8, 2, 16, 64, 16, seed=13)
    table = ints([[0, 3], [5, 1]])
    k, v = (rows_like(gen, (2, 2, 20, 64), torch.bfloat16) for _ in range(2))
    big = torch.zeros(1 << 27, device=DEV)
    for i in range(5):
        held = [torch.full((2 * 2 * 20 * 64 * 2,), i + 1, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        for _ in range(10):
            big.add_(1)
        read = [t + 1 for t in held]
        freed = {t.data_ptr() for t in held}
        del held
        fa.cache_append_e4m3(k, v, *c.args(), table, ints([3, 0]) if i == 0 else start, stream=side)
        start = ints([3, 0])
        got = fa.cache_read_e4m3(*c.args(), table, 20, start, stream=side)
        assert not {t.data_ptr() for t in got} & freed
        torch.cuda.synchronize()
        assert all((t == i + 2).all() for t in read)
        if i == 0:
            for x, (p, s) in zip((k, v), c.want):
                oracle.append(f64(x), p, s, table.cpu().numpy(), [3, 0], None, 16)
        c.same()
        for x, (p, s) in zip(got, c.want):
            assert np.array_equal(f64(x), dense(p, s, table.tolist(), [3, 0], None, 20))
    assert fa.get_device_status(side) == 0


def test_refusals():
    c = Quantised(8, 2, 16, 64, 4, seed=14)
    kp, vp, ks, vs = c.args()
    table, start = ints([[0, 3], [5, 1]]), ints([0, 0])
    k, v = (torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    o = [torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    cache = dict(k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs)
    calls = [(fa.cache_append_e4m3, dict(cache, k=k, v=v, page_table=table, start=start)),
             (fa.cache_read_e4m3, dict(cache, page_table=table, rows=3, start=start, out=tuple(o))),
             (fa.cache_copy_pages_e4m3, dict(cache, moves=ints([[0, 1, 16]]))),
             (fa.attention_decode_e4m3, dict(cache, q=k[:, :, :1], page_table=table, lengths=start))]
    bad = [dict(v_pages=vp[:-1]), dict(v_pages=vp.transpose(1, 2).contiguous().transpose(1, 2)), dict(k_pages=kp.cpu()),
           dict(k_scales=ks[:-1]), dict(v_scales=vs[:, :1]), dict(k_scales=ks[..., :3]), dict(v_scales=vs[..., :2]),
           dict(k_scales=ks.double()), dict(v_scales=vs.cpu()), dict(k_scales=ks.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(k_scales=torch.zeros(8, 2, 0, device=DEV)), dict(k_scales=torch.ones(8, 2, 32, device=DEV)),
           dict(page_table=table.long()), dict(page_table=table.cpu()), dict(page_table=table.t()), dict(start=start.long()),
           dict(start=start[:1]), dict(counts=ints([1])), dict(counts=start.cpu()), dict(k=k[:, :1]), dict(v=v[:1]),
           dict(v=v.float()), dict(k=k[..., :32]), dict(v=v.transpose(1, 2).contiguous().transpose(1, 2)), dict(rows=-1),
           dict(out=(o[0], o[1].float())), dict(out=(o[0][:, :, :2], o[1])), dict(q=k), dict(q=k[:1, :, :1]),
           dict(moves=ints([[0, 1]])), dict(moves=ints([[0, 1, 2]]).long()), dict(moves=ints([0, 1, 2])), dict(count=ints([1, 1]))]
    for call, good in calls:
        call(**good)
        names = set(good) | ({"counts"} if "start" in good else set()) | ({"count"} if "moves" in good else set())
        for x in bad:
            if set(x) <= names:
                with pytest.raises(ValueError):
                    call(**{**good, **x})
        for x in (dict(k_pages=kp.float(), v_pages=vp.float()), dict(k_pages=kp.view(torch.uint8)), dict(v_scales=None)):
            with pytest.raises(TypeError):
                call(**{**good, **x})
    for call, good, x in ((*calls[0], dict(v_pages=kp)), (*calls[0], dict(v_scales=ks)), (*calls[2], dict(v_pages=kp)),
                          (*calls[2], dict(k_scales=vs)), (*calls[1], dict(out=(o[0], o[0])))):
        with pytest.raises(fa.FaError) as err:
            call(**{**good, **x})
        assert err.value.code == fa.FA_ERR_INVALID_ARG
    for n in ((1 << 31) // 4, (1 << 31) - 1):
        with pytest.raises(fa.FaError) as err:
            fa.cache_read_e4m3(*c.args(), table, n)
        assert err.value.code == fa.FA_ERR_UNSUPPORTED
    fa.cache_append_e4m3(k[:, :, :0], v[:, :, :0], *c.args(), table, start)
    d, block = fa.cache_for_e4m3(*c.args(), table, torch.float32)
    assert (block, d.dtype, d.S, d.max_pages, d.page_rows, d.stride_n) == (4, fa.FA_FP32, 2, 2, 16, 64)
    assert fa.get_device_status() == 0
