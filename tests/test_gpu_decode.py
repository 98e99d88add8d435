"""fa_decode against the float64 restatement: head layouts, head dims, page
sizes, lengths from nothing to tens of thousands, splits and joins, strides,
streams and graphs.

Tolerances are bounds, not fits.  With u = 2^-24, a score is a sum of d
products whose absolute sum is at most A (as the oracle returns it), summed in
fp32 with at most 2u of the sum an addition, so it is off by
e_s <= 2 d u A + 4 u |s|, |s| <= A.  A weight exp(s - m) is then off by e_s plus the
rounding of its exponent's product (4 u |s|), 2^-21 of the hardware exponential and,
in bf16, 2^-16 (it is multiplied as the sum of two bf16 numbers, each rounded to
2^-8 of its value).  Both the weighted sum and the sum of weights carry that
error and at most 2 u n of their additions, so
  |O - ref| <= half a step of the output type * |ref| + 2 V (e_w + 2 (n + 64) u)
  |L - ref| <= e_s + e_w + 2 (n + 64) u + 8 u |L|
with V the largest |v|, n the number of rows and 64 for the joining of parts."""

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from oracle.paged_fp64 import decode

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def make(S, H, Hk, d, page, lengths, dtype=torch.bfloat16, seed=0, rows_first=False, spare=2, junk=True, q_std=1.0, wide=0):
    """A cache with pages in random order; what no row reads is NaN.  wide: more columns of the table.  How the work is
    shared out goes by the rows that the table could hold: an item of a narrow one is read by a cluster of blocks, those
    of a wide one by equal runs of all of them and a second kernel."""
    gen = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lengths]
    pages, columns = sum(held) + spare, max(held + [1]) + 1 + wide
    order = torch.randperm(pages, generator=gen)
    table = torch.full((S, columns), -1, dtype=torch.int32)
    shape = (pages, page, Hk, d) if rows_first else (pages, Hk, page, d)
    pools = []
    for _ in range(2):
        t = torch.randn(shape, generator=gen).to(dtype)
        pools.append(t.permute(0, 2, 1, 3) if rows_first else t)
    live = torch.zeros(pages, page, dtype=torch.bool)
    k = 0
    for s, n in enumerate(lengths):
        ids = order[k:k + held[s]]
        k += held[s]
        table[s, :held[s]] = ids.int()
        for c in range(held[s]):
            live[ids[c], :max(0, min(page, n - c * page))] = True
    if junk:
        for t in pools:
            t[~live[:, None, :].expand(-1, Hk, -1)] = float("nan")
    q = (torch.randn(S, H, 1, d, generator=gen) * q_std).to(dtype)
    lens = torch.tensor(lengths, dtype=torch.int32)
    return [t.to(DEV) for t in (q, *pools, table, lens)]


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, q, kp, vp, table, lengths, scale):
    o, L = got
    d = q.shape[3]
    ref, Lr, A, V = decode(f64(q)[:, :, 0], np.nan_to_num(f64(kp)), np.nan_to_num(f64(vp)), table.cpu().numpy(),
                           lengths.cpu().numpy(), float(np.float32(scale)))
    n = lengths.cpu().clamp(min=0).numpy()[:, None]
    e_s = 2 * d * U * A + 4 * U * A
    e_w = e_s + 4 * U * A + 2.0 ** -21 + (2.0 ** -16 if q.dtype == torch.bfloat16 else 0)
    tol_o = HALF_STEP[q.dtype] * np.abs(ref) + (2 * V * (e_w + 2 * (n + 64) * U))[:, :, None]
    x, y = f64(o)[:, :, 0], f64(L)[:, :, 0]
    assert np.isfinite(x).all()
    assert (np.abs(x - ref) <= tol_o).all(), float((np.abs(x - ref) - tol_o).max())
    empty = np.isinf(Lr)
    assert (x[empty] == 0).all() and np.array_equal(np.isposinf(y), empty)
    tol_l = e_s + e_w + 2 * (n + 64) * U + 8 * U * np.abs(np.where(empty, 0, Lr))
    assert (np.abs(y[~empty] - Lr[~empty]) <= tol_l[~empty]).all(), float(np.abs(y[~empty] - Lr[~empty]).max())


def run_and_check(args, scale=None, **kw):
    q, kp, vp, table, lengths = args
    scale = q.shape[3] ** -0.5 if scale is None else scale
    got = fa.attention_decode(q, kp, vp, table, lengths, scale, **kw)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    check(got, q, kp, vp, table, lengths, scale)
    return got


BF16_DIMS, FP32_DIMS = (32, 64, 96, 128, 256), (16, 32, 64, 96, 128, 256)


@pytest.mark.parametrize("d", BF16_DIMS)
@pytest.mark.parametrize("H,Hk", [(4, 4), (6, 2), (16, 2), (12, 1), (16, 1), (40, 2)])
@pytest.mark.parametrize("wide", [0, 3000])
def test_head_layouts_bf16(d, H, Hk, wide):
    lengths = [0, 1, 15, 16, 17, 63, 64, 65, 300]
    run_and_check(make(len(lengths), H, Hk, d, 16, lengths, seed=d + H, wide=wide))


@pytest.mark.parametrize("d", FP32_DIMS)
@pytest.mark.parametrize("H,Hk", [(3, 3), (6, 2), (9, 1), (16, 2)])
@pytest.mark.parametrize("wide", [0, 3000])
def test_head_layouts_fp32(d, H, Hk, wide):
    lengths = [0, 1, 15, 16, 17, 63, 64, 65, 300]
    run_and_check(make(len(lengths), H, Hk, d, 16, lengths, torch.float32, seed=d + H, wide=wide))


@pytest.mark.parametrize("page", [1, 2, 3, 7, 13, 16, 48, 64, 100, 256, 1000])
@pytest.mark.parametrize("rows_first", [False, True])
def test_page_sizes(page, rows_first):
    lengths = [page - 1, page, page + 1, 2 * page, 259, 1]
    for dtype in (torch.bfloat16, torch.float32):
        run_and_check(make(6, 4, 2, 64, page, lengths, dtype, seed=page, rows_first=rows_first))


@pytest.mark.parametrize("n", [1, 64, 65, 2048, 4000, 32768])
@pytest.mark.parametrize("H,Hk,d,dtype", [(8, 1, 128, torch.bfloat16), (2, 2, 64, torch.bfloat16),
                                          (2, 1, 256, torch.bfloat16), (2, 1, 96, torch.float32)])
@pytest.mark.parametrize("wide", [0, 600])
def test_one_sequence_over_the_whole_gpu(n, H, Hk, d, dtype, wide):
    run_and_check(make(1, H, Hk, d, 64, [n], dtype, seed=n, wide=wide))


def test_many_short_and_one_long():
    lengths = [4000] + [i % 5 for i in range(300)] + [1999]
    run_and_check(make(len(lengths), 4, 2, 64, 16, lengths, seed=3))


@pytest.mark.parametrize("d,dtype,H,Hk", [(32, torch.bfloat16, 2, 2), (64, torch.bfloat16, 32, 2), (128, torch.float32, 8, 2)])
def test_more_items_than_runs(d, dtype, H, Hk):
    """The join goes by runs then, and takes several heads a block."""
    lengths = [700 if i % 97 == 0 else (i * 37) % 130 for i in range(700)]
    run_and_check(make(len(lengths), H, Hk, d, 16, lengths, dtype, seed=4))


@pytest.mark.parametrize("d,dtype,Hk,S,n", [(128, torch.bfloat16, 1, 9, 150000), (256, torch.bfloat16, 2, 40, 12000),
                                            (32, torch.float32, 2, 40, 30000)])
def test_enough_rows_for_small_runs(d, dtype, Hk, S, n):
    """Past 64 tiles for each resident block the work ends in small runs.  All sequences read the same pages, each a
    different number of them; two of the sequences are compared."""
    q, kp, vp, table, _ = make(1, 4, Hk, d, 64, [n], dtype, seed=21)
    q = torch.randn(S, 4, 1, d, generator=torch.Generator().manual_seed(22)).to(dtype).to(DEV)
    lengths = torch.tensor([n - 77 * s for s in range(S)], dtype=torch.int32, device=DEV)
    blocks = torch.cuda.get_device_properties(0).multi_processor_count * (1 if d == 256 else 2 if d == 128 else 3)
    assert S * Hk * (n - 77 * S) / 64 > 64 * blocks
    o, L = fa.attention_decode(q, kp, vp, table.expand(S, -1).contiguous(), lengths)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    for s in (0, S - 1):
        one = slice(s, s + 1)
        check((o[one], L[one]), q[one], kp, vp, table, lengths[one], d ** -0.5)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_all_empty(wide, dtype):
    run_and_check(make(3, 4, 2, 64, 16, [0, 0, 0], dtype, wide=wide))


@pytest.mark.parametrize("S,n", [(1, 1900), (7, 1000), (18, 500), (36, 250), (74, 180), (148, 100), (300, 60), (700, 60)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_clusters_of_every_size(S, n, dtype):
    """As many blocks an item as the GPU holds at a time: 16, 8, 4, 2, 1, or more
    items than that, with full and partly empty shares."""
    lengths = [max(0, n - 7 * (i % 50)) for i in range(S)]
    run_and_check(make(S, 4, 1, 128, 64, lengths, dtype, seed=S))


def test_peaked_scores():
    """Scores with a deviation of 4: the running maximum moves, most weights vanish."""
    for dtype in (torch.bfloat16, torch.float32):
        run_and_check(make(4, 8, 2, 128, 16, [3, 500, 2000, 77], dtype, seed=5, q_std=4.0))


def test_rising_scores():
    """Each key scores above the one before, so that every row raises the maximum."""
    q, kp, vp, table, lengths = make(1, 4, 1, 64, 16, [700], seed=6, junk=False)
    q.fill_(1.0)
    for j in range(700):
        kp[table[0, j // 16].item(), :, j % 16] = j / 64
    run_and_check((q, kp, vp, table, lengths))


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_reaches_its_heads_alone(wide, dtype):
    """A NaN in a query makes every score of its head NaN, one in a key a score of
    each head that reads it, however the rows are shared out; the other heads
    and an empty sequence with a NaN query know nothing of it."""
    args = make(3, 4, 2, 64, 16, [200, 0, 130], dtype, seed=31, wide=wide)
    clean = fa.attention_decode(*args)
    q, kp, vp, table, lengths = args
    q[0, 1, 0, 5] = float("nan")
    q[1, 2, 0, 0] = float("nan")
    kp[table[2, 100 // 16].item(), 1, 100 % 16, 63] = float("nan")  # key head 1: query heads 2, 3
    o, L = fa.attention_decode(*args)
    assert fa.get_device_status() == 0
    hit = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    hit[0, 1] = hit[2, 2] = hit[2, 3] = True
    assert o[hit].isnan().all() and L[hit].isnan().all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(L[~hit], clean[1][~hit])


@pytest.mark.parametrize("scale", [1e-3, 1.0])
def test_scale(scale):
    run_and_check(make(3, 4, 2, 64, 16, [100, 7, 64], seed=8), scale)


def test_strided_queries_and_given_outputs():
    q, kp, vp, table, lengths = make(5, 8, 2, 64, 16, [100, 0, 7, 64, 1000], seed=9, wide=3000)
    fused = torch.randn(5, 12, 64, device=DEV).to(torch.bfloat16)  # queries, keys and values of one projection
    view = fused[:, 2:10, None, :]
    o_all = torch.full((5, 10, 1, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    out = (o_all[:, 1:9], torch.empty(5, 8, 1, device=DEV))
    ws = torch.empty(fa.fa_decode_workspace_bytes(fa.cache_for(kp, vp, table), 8), dtype=torch.uint8, device=DEV)
    got = run_and_check((view, kp, vp, table, lengths), out=out, workspace=ws)
    assert got[0].data_ptr() == out[0].data_ptr()
    assert (o_all[:, 0] == 7).all() and (o_all[:, 9] == 7).all()


def test_shared_pages():
    """Sequences that name the same pages, as forks do."""
    q, kp, vp, table, lengths = make(4, 8, 2, 128, 16, [320, 320, 320, 320], seed=10)
    table[1:, :10] = table[0, :10]
    run_and_check((q, kp, vp, table, lengths))


def test_offsets_beyond_32_bits():
    """Pages further than 2^31 elements (and 2^32 bytes) into the pools."""
    pages, page, d = 70000, 256, 128  # 2.29e9 elements a pool
    kp, vp = (torch.empty(pages, 1, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ids = [69999, 3, 65600, 69990]
    gen = torch.Generator().manual_seed(11)
    small = [torch.randn(4, 1, page, d, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    for i, p in enumerate(ids):
        kp[p], vp[p] = small[0][i], small[1][i]
    q = torch.randn(1, 4, 1, d, generator=gen).to(torch.bfloat16).to(DEV)
    lengths = torch.tensor([1000], dtype=torch.int32, device=DEV)
    got = fa.attention_decode(q, kp, vp, torch.tensor([ids], dtype=torch.int32, device=DEV), lengths)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    check(got, q, *small, torch.tensor([[0, 1, 2, 3]], dtype=torch.int32), lengths, d ** -0.5)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_pages_and_lengths_are_not_followed(dtype, wide):
    q, kp, vp, table, lengths = make(4, 4, 2, 64, 16, [100, 50, 300, 20], dtype, seed=12, wide=wide)
    table[0, 2], table[2, 5] = 1 << 20, -7
    got = fa.attention_decode(q, kp, vp, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    check(got, q, kp, vp, table, lengths, 64 ** -0.5)
    lengths = torch.tensor([-5, 50, 1 << 30, 20], dtype=torch.int32, device=DEV)
    got = fa.attention_decode(q, kp, vp, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    check((got[0][[0, 1, 3]], got[1][[0, 1, 3]]), q[[0, 1, 3]], kp, vp, table[[0, 1, 3]], lengths[[0, 1, 3]], 64 ** -0.5)
    with pytest.raises(fa.FaError) as err:
        fa.attention_decode(q, kp, vp, table, lengths, check_status=True)
    assert err.value.code == fa.FA_ERR_PAGES
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
def test_same_call_same_bits(wide):
    args = make(7, 8, 2, 128, 16, [4000, 1, 900, 0, 77, 3333, 512], seed=13, wide=wide)
    a = fa.attention_decode(*args)
    for _ in range(5):
        b = fa.attention_decode(*args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("wide", [0, 3000])
def test_two_streams_at_once(wide):
    args = [make(4, 8, 2, 128, 16, [4000, 100, 1700, 64], seed=20 + i, wide=wide) for i in range(2)]
    want = [fa.attention_decode(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for a, st in zip(args, streams):
            got.append(fa.attention_decode(*a, stream=st))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
def test_graph_follows_lengths_that_change(wide):
    """A captured call reads lengths and table at each replay; two graphs replayed at once have workspaces of their own."""
    q, kp, vp, table, lengths = make(3, 8, 2, 64, 16, [2000, 900, 50], seed=30, junk=False, wide=wide)
    pairs = []
    torch.cuda.synchronize()
    for _ in range(2):
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            fa.attention_decode(q, kp, vp, table, lengths)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                got = fa.attention_decode(q, kp, vp, table, lengths)
        pairs.append((stream, graph, got))
    for new in ([2000, 900, 50], [1, 0, 16], [700, 777, 50]):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        for stream, graph, _ in pairs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, got in pairs:
            check(got, q, kp, vp, table, lengths, 64 ** -0.5)
    assert fa.get_device_status() == 0


def test_agrees_with_the_forward_over_the_same_rows():
    """fa_fwd of one query row (causal, aligned bottom-right: it sees all keys) over a dense copy of the cache."""
    S, H, d, n = 2, 4, 128, 1000
    q, kp, vp, table, lengths = make(S, H, H, d, 8, [n] * S, seed=31)
    at = table[:, : n // 8].long()
    k, v = (t[at].permute(0, 2, 1, 3, 4).reshape(S, H, n, d).contiguous() for t in (kp, vp))
    o, L = fa.attention_forward(q, k, v, d ** -0.5, causal=True)
    o2, L2 = run_and_check((q, kp, vp, table, lengths))
    # the forward rounds its weights to bf16 (2^-8 of each, at most 2^-8 of max |v| in the sum) and its output
    assert (o.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * v.float().abs().max()
    assert (L.reshape(S, H) - L2.reshape(S, H)).abs().max() <= 1e-3


def test_refusals():
    q, kp, vp, table, lengths = make(3, 8, 2, 64, 16, [100, 7, 64], seed=40, wide=3000)
    good = dict(q=q, k_pages=kp, v_pages=vp, page_table=table, lengths=lengths)
    fa.attention_decode(**good)
    o, L = torch.empty_like(q), torch.empty(3, 8, 1, device=DEV)
    for bad in (dict(q=q[:2]), dict(q=q[:, :, 0]), dict(q=q.expand(-1, -1, 2, -1)), dict(q=q[..., :32]), dict(q=q.float()),
                dict(q=q.cpu()), dict(q=q.detach().requires_grad_()), dict(v_pages=vp.float()), dict(v_pages=vp[:-1]),
                dict(v_pages=vp.transpose(1, 2).contiguous().transpose(1, 2)), dict(k_pages=kp.cpu()),
                dict(page_table=table.long()), dict(page_table=table.t()), dict(page_table=table.cpu()),
                dict(lengths=lengths.long()), dict(lengths=lengths[:2]), dict(lengths=lengths.cpu()),
                dict(out=(o.float(), L)), dict(out=(o, L[:, :, 0])), dict(out=(o, L.half())),
                dict(workspace=torch.empty(1 << 20, 2, device=DEV)[:, 0])):
        with pytest.raises(ValueError):
            fa.attention_decode(**{**good, **bad})
    small = torch.empty(fa.fa_decode_workspace_bytes(fa.cache_for(kp, vp, table), 8) - 1, dtype=torch.uint8, device=DEV)
    for bad in (dict(q=q[:, :7]), dict(scale=0.0), dict(scale=float("nan")), dict(workspace=small), dict(out=(q, L))):
        with pytest.raises(fa.FaError) as err:
            fa.attention_decode(**{**good, **bad})
        assert err.value.code == fa.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FaError) as err:  # more than 512 query heads a key-value head
        fa.attention_decode(torch.empty(3, 1026, 1, 64, dtype=torch.bfloat16, device=DEV), kp, vp, table, lengths)
    assert err.value.code == fa.FA_ERR_UNSUPPORTED
    with torch.no_grad():
        fa.attention_decode(**{**good, "q": q.detach().requires_grad_()})
    assert fa.get_device_status() == 0


def test_largest_group_of_heads():
    """512 query heads on one key-value head, in pieces of 16 (8 in fp32)."""
    for dtype in (torch.bfloat16, torch.float32):
        for wide in (0, 3000):
            run_and_check(make(2, 512, 1, 32, 16, [300, 65], dtype, seed=41, wide=wide))


def test_strides_of_dimensions_of_one():
    """PyTorch leaves the stride of a dimension of one element open; the descriptor holds a packed one."""
    def strides(shape, st, table=None):
        t = torch.zeros(1 << 16, dtype=torch.bfloat16, device=DEV).as_strided(shape, st)
        c = fa.cache_for(t, t, table)
        return c.stride_page, c.stride_h, c.stride_n, c.table_stride

    assert strides((1, 1, 1, 64), (3, 5, 7, 1))[:3] == (64, 64, 64)
    assert strides((2, 1, 16, 64), (1024, 1, 64, 1))[:3] == (1024, 1024, 64)
    assert strides((5, 3, 16, 64), (16 * 3 * 64, 64, 3 * 64, 1))[:3] == (16 * 3 * 64, 64, 3 * 64)
    table = torch.zeros(3, 5, dtype=torch.int32, device=DEV)
    c = fa.cache_for(*[torch.zeros(2, 1, 16, 64, device=DEV)] * 2, table[:, :4])
    assert (c.S, c.max_pages, c.table_stride, c.dtype) == (3, 4, 5, fa.FA_FP32)
    c = fa.cache_for(*[torch.zeros(2, 1, 16, 64, device=DEV)] * 2, table[:1, :4])
    assert (c.S, c.max_pages, c.table_stride) == (1, 4, 4)
    with pytest.raises(ValueError):
        strides((2, 2, 4, 64), (1024, 512, 128, 2))


def test_grouped_single_page_strides():
    """Single sequences, heads, pages and rows, in storages that leave their strides open."""
    for shape in ((1, 1, 1), (1, 4, 1), (1, 4, 4), (3, 4, 1)):
        S, H, Hk = shape
        for page, n in ((1, 1), (16, 16), (64, 5)):
            run_and_check(make(S, H, Hk, 64, page, [n] * S, seed=50, spare=0, rows_first=True))
