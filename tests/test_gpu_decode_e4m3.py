"""fa_decode_e4m3 against the float64 restatement over the values that the
stored numbers stand for: head layouts, head dims, page and block sizes,
lengths from nothing to tens of thousands, scales far apart, strides, streams
and graphs.

Tolerances are bounds, not fits.  With u = 2^-24, a score is a sum of d
products whose absolute sum is at most A (as the oracle returns it), summed in
fp32 with at most 2u of the sum an addition.  Queries are multiplied in units of a
common power of two of their head: bf16 ones (8 bits) as an fp16 number, or three e4m3 numbers
on the tensor-memory path, exactly where they are within 2^-19 of the largest; fp32 ones as the sum
of two fp16 numbers, off by at most 2^-23.  Adding the two up and three products
follow, which leaves four of the eight below, one for the other half of 2^-23.  So
  e_s <= (2 d + 8) u A + e_q A,  e_q = 2^-24 in fp32, 0 in bf16.
A weight is off by e_s plus the rounding of its exponent's product (4 u A), 2^-21 of
the hardware exponential and what it loses as it is multiplied, for which 2^-11 +
2^-12 are allowed in bf16 and 3u in fp32 here.  The kernels are off by less: 2^-15 with four e5m2
numbers (tensor memory), 2^-23 with two fp16 numbers (the others), or a share of the
largest weight; test_gpu_decode_e4m3_weights.py holds them to that.  Both the weighted sum and the sum of weights carry
that error and at most 2 u n of their additions, so
  |O - ref| <= half a step of the output type * |ref| + 2 V (e_w + 2 (n + 64) u)
  |L - ref| <= e_s + e_l + 2 (n + 64) u + 8 u |L|,  e_l as e_w without the multiplied weights' loss
with V the largest |v|, n the number of rows and 64 for the joining of parts."""

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from oracle.e4m3_fp64 import values
from oracle.paged_fp64 import decode

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def make(S, H, Hk, d, page, lengths, dtype=torch.bfloat16, seed=0, block=None, rows_first=False, spare=2, junk=True, q_std=1.0,
         wide=0, exponents=(-9, -5)):
    """A cache with pages in random order; what no row reads is NaN, and so are the scales of blocks that hold no row.
    wide: more columns of the table.  How the work is shared out goes by the rows that the table could hold: an item of a
    narrow one is read by a cluster of blocks, those of a wide one by equal runs of all of them and a second kernel."""
    gen = torch.Generator().manual_seed(seed)
    block = page if block is None else block
    held = [-(-n // page) for n in lengths]
    pages, columns = sum(held) + spare, max(held + [1]) + 1 + wide
    order = torch.randperm(pages, generator=gen)
    table = torch.full((S, columns), -1, dtype=torch.int32)
    live = torch.zeros(pages, page, dtype=torch.bool)
    k = 0
    for s, n in enumerate(lengths):
        ids = order[k:k + held[s]]
        k += held[s]
        table[s, :held[s]] = ids.int()
        for c in range(held[s]):
            live[ids[c], :max(0, min(page, n - c * page))] = True
    pools = []
    for _ in range(2):
        t = (torch.randn(pages, Hk, page, d, generator=gen) * 112).clamp(-448, 448)
        s = torch.exp2(torch.randint(*exponents, (pages, Hk, page // block), generator=gen).float())
        if junk:
            t[~live[:, None, :].expand(-1, Hk, -1)] = float("nan")
            s[~live.view(pages, 1, -1, block).any(3).expand(-1, Hk, -1)] = float("nan")
        t = t.to(F8)
        if rows_first:
            t = t.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(F8)
        pools.append((t, s))
    q = (torch.rand(S, H, 1, d, generator=gen) * 1.75 + 0.25) * (torch.randint(0, 2, (S, H, 1, d), generator=gen) * 2 - 1)
    (kp, ks), (vp, vs) = pools
    lens = torch.tensor(lengths, dtype=torch.int32)
    # a clone keeps the strides of a tensor that is dense in memory
    return [t.to(DEV) for t in ((q * q_std).to(dtype), kp, vp, ks, vs, table, lens)]


def f64(t):
    return t.detach().cpu().float().double().numpy()


def check(got, q, kp, vp, ks, vs, table, lengths, scale):
    o, L = got
    d = q.shape[3]
    k, v = (np.nan_to_num(values(f64(p), f64(s))) for p, s in ((kp, ks), (vp, vs)))
    ref, Lr, A, V = decode(f64(q)[:, :, 0], k, v, table.cpu().numpy(), lengths.cpu().numpy(), float(np.float32(scale)))
    n = lengths.cpu().clamp(min=0).numpy()[:, None]
    e_s = (2 * d + 8) * U * A + (U * A if q.dtype == torch.float32 else 0)
    e_l = e_s + 4 * U * A + 2.0 ** -21
    e_w = e_l + (2 * U + U if q.dtype == torch.float32 else 2.0 ** -11 + 2.0 ** -12)
    tol_o = HALF_STEP[q.dtype] * np.abs(ref) + (2 * V * (e_w + 2 * (n + 64) * U))[:, :, None]
    x, y = f64(o)[:, :, 0], f64(L)[:, :, 0]
    assert np.isfinite(x).all()
    assert (np.abs(x - ref) <= tol_o).all(), float((np.abs(x - ref) - tol_o).max())
    empty = np.isinf(Lr)
    assert (x[empty] == 0).all() and np.array_equal(np.isposinf(y), empty)
    tol_l = e_s + e_l + 2 * (n + 64) * U + 8 * U * np.abs(np.where(empty, 0, Lr))
    assert (np.abs(y[~empty] - Lr[~empty]) <= tol_l[~empty]).all(), float(np.abs(y[~empty] - Lr[~empty]).max())


def run_and_check(args, scale=None, **kw):
    scale = args[0].shape[3] ** -0.5 if scale is None else scale
    got = fa.attention_decode_e4m3(*args, scale, **kw)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    check(got, *args, scale)
    return got


BF16_DIMS, FP32_DIMS = (32, 64, 96, 128, 256), (16, 32, 64, 96, 128, 256)
BOTH = [torch.bfloat16, torch.float32]


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


@pytest.mark.parametrize("page,block", [(1, 1), (2, 1), (3, 3), (7, 1), (13, 13), (16, 2), (48, 16), (64, 64), (100, 5),
                                        (256, 128), (1000, 8)])
@pytest.mark.parametrize("rows_first", [False, True])
def test_page_and_block_sizes(page, block, rows_first):
    lengths = [page - 1, page, page + 1, 2 * page, 259, 1]
    for dtype in BOTH:
        run_and_check(make(6, 4, 2, 64, page, lengths, dtype, seed=page, block=block, rows_first=rows_first))


@pytest.mark.parametrize("n", [1, 64, 65, 2048, 4000, 32768])
@pytest.mark.parametrize("H,Hk,d,dtype", [(8, 1, 128, torch.bfloat16), (2, 2, 64, torch.bfloat16),
                                          (2, 1, 256, torch.bfloat16), (2, 1, 96, torch.float32)])
@pytest.mark.parametrize("wide", [0, 600])
def test_one_sequence_over_the_whole_gpu(n, H, Hk, d, dtype, wide):
    run_and_check(make(1, H, Hk, d, 64, [n], dtype, seed=n, block=16, wide=wide))


def test_many_short_and_one_long():
    lengths = [4000] + [i % 5 for i in range(300)] + [1999]
    run_and_check(make(len(lengths), 4, 2, 64, 16, lengths, seed=3))


@pytest.mark.parametrize("d,dtype,H,Hk", [(32, torch.bfloat16, 2, 2), (64, torch.bfloat16, 32, 2), (128, torch.float32, 8, 2)])
def test_more_items_than_runs(d, dtype, H, Hk):
    """The join goes by runs then, and takes several heads a block."""
    lengths = [700 if i % 97 == 0 else (i * 37) % 130 for i in range(700)]
    run_and_check(make(len(lengths), H, Hk, d, 16, lengths, dtype, seed=4))


@pytest.mark.parametrize("d,dtype,Hk,S,n", [(128, torch.bfloat16, 1, 9, 150000), (256, torch.bfloat16, 2, 40, 16000),
                                            (32, torch.float32, 2, 40, 60000)])
def test_enough_rows_for_small_runs(d, dtype, Hk, S, n):
    """A problem of many tiles for each resident block ends in small runs.  All sequences read the same pages, each a
    different number of them; two of the sequences are compared."""
    q, *pools, table, _ = make(1, 4, Hk, d, 64, [n], dtype, seed=21)
    q = (torch.randn(S, 4, 1, d, generator=torch.Generator().manual_seed(22)).clamp(-2, 2) + 3).to(dtype).to(DEV)
    lengths = torch.tensor([n - 77 * s for s in range(S)], dtype=torch.int32, device=DEV)
    o, L = fa.attention_decode_e4m3(q, *pools, table.expand(S, -1).contiguous(), lengths)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    for s in (0, S - 1):
        one = slice(s, s + 1)
        check((o[one], L[one]), q[one], *pools, table, lengths[one], d ** -0.5)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", BOTH)
def test_all_empty(wide, dtype):
    run_and_check(make(3, 4, 2, 64, 16, [0, 0, 0], dtype, wide=wide))


@pytest.mark.parametrize("S,n", [(1, 1900), (7, 1000), (18, 500), (36, 250), (74, 180), (148, 100), (300, 60), (700, 60)])
@pytest.mark.parametrize("dtype", BOTH)
def test_clusters_of_every_size(S, n, dtype):
    """As many blocks an item as the GPU holds at a time, with full and partly empty shares."""
    lengths = [max(0, n - 7 * (i % 50)) for i in range(S)]
    run_and_check(make(S, 4, 1, 128, 64, lengths, dtype, seed=S, block=32))


@pytest.mark.parametrize("S,n", [(30, 2900), (100, 1400), (200, 760), (400, 740)])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (128, torch.float32)])
def test_clusters_of_several_tiles_a_block(S, n, d, dtype):
    """8, 4 and 2 blocks an item and one alone, as many tiles a block as there may be and one more, and none."""
    lengths = [max(0, n - 31 * (i % 100)) for i in range(S)]
    run_and_check(make(S, 2, 1, d, 64, lengths, dtype, seed=S, block=32))


@pytest.mark.parametrize("dtype", BOTH)
def test_peaked_scores(dtype):
    """Scores with a deviation of 4: the running maximum moves, most weights vanish."""
    run_and_check(make(4, 8, 2, 128, 16, [3, 500, 2000, 77], dtype, seed=5, q_std=4.0))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("wide", [0, 3000])
def test_rising_and_falling_scores(dtype, wide):
    """Each key scores above the one before, so that every row raises the maximum; or below."""
    q, kp, vp, ks, vs, table, lengths = make(1, 4, 1, 64, 16, [700], dtype, seed=6, block=1, junk=False, wide=wide)
    q.fill_(1.0)
    kp.view(torch.uint8).fill_(0x38)  # 1.0: the scales alone tell the keys apart
    for sign in (1, -1):
        for j in range(700):
            ks[table[0, j // 16].item(), :, j % 16] = (j if sign > 0 else 700 - j) / 64
        run_and_check((q, kp, vp, ks, vs, table, lengths))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("block", [1, 16])
def test_scales_far_apart(dtype, block):
    """Blocks of V whose scales differ by up to 2^80 and whose weights do not go by that."""
    q, kp, vp, ks, vs, table, lengths = make(2, 4, 2, 64, 16, [900, 130], dtype, seed=7, block=block, junk=False)
    gen = torch.Generator().manual_seed(7)
    vs.copy_(torch.exp2(torch.randint(-40, 41, vs.shape, generator=gen).float()))
    run_and_check((q, kp, vp, ks, vs, table, lengths))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("wide", [0, 3000])
def test_a_large_value_that_no_weight_reaches(dtype, wide):
    """A page of V of 2^100 times the others' size, whose keys score so low that its weights are 0: the others' sum is
    held as if it were not there, wherever it stands.  And one of 2^-100 of their size that has all the weight."""
    d = 64
    for where in (0, 30, 62):
        args = make(1, 4, 1, d, 16, [1000], dtype, seed=8, junk=False, wide=wide)
        q, kp, vp, ks, vs, table, lengths = args
        q.fill_(1.0)
        page = table[0, where].item()
        kp[page] = torch.full((1, 16, d), -448.0).to(F8)
        ks[page], vs[page] = 1.0, 2.0 ** 93
        got = fa.attention_decode_e4m3(*args)
        assert fa.get_device_status() == 0
        without = table.clone()
        without[0, where] = -1
        check(got, q, kp, vp, ks, vs, without, lengths, d ** -0.5)
        kp[page] = torch.full((1, 16, d), 448.0).to(F8)
        vs[page] = 2.0 ** -107
        o, _ = fa.attention_decode_e4m3(*args)
        assert fa.get_device_status() == 0
        # 448 a column against keys of about 1: the other rows' weights are exp(-3500), the page's all the same
        rows = min(16, 1000 - 16 * where)
        want = torch.tensor(values(f64(vp), f64(vs))[page, :, :rows].mean(1))[:, None].expand(1, 4, 1, d)
        assert (o.cpu().double() - want).abs().max() <= (HALF_STEP[dtype] + 2.0 ** -19) * 2.0 ** -107 * 448


@pytest.mark.parametrize("dtype", BOTH)
def test_values_of_nothing(dtype):
    """Rows of zeros, whose scale is the smallest there is, with all the weight and with some."""
    q, kp, vp, ks, vs, table, lengths = make(2, 4, 2, 64, 16, [40, 16], dtype, seed=9, junk=False)
    first = table[:, 0].long()
    vp.view(torch.uint8)[first] = 0
    vs[first] = 2.0 ** -126
    o, _ = run_and_check((q, kp, vp, ks, vs, table, lengths))
    assert (o[1] == 0).all()
    kp.view(torch.uint8).fill_(0)
    ks.fill_(2.0 ** -126)
    run_and_check((q, kp, vp, ks, vs, table, lengths))


@pytest.mark.parametrize("dtype", BOTH)
def test_queries_of_every_size(dtype):
    """Heads whose queries differ by many powers of two; columns that do within a head, where only the small ones meet keys."""
    args = make(3, 8, 2, 64, 16, [100, 7, 300], dtype, seed=10, junk=False)
    q, kp, ks = args[0], args[1], args[3]
    base = q.clone()
    q.mul_(torch.exp2(torch.arange(-60, 60, 15, device=DEV).float())[None, :, None, None].to(dtype))
    ks.mul_(2.0 ** -4)
    run_and_check(args, 1e-16)
    q.copy_(base)
    q[..., ::2] *= 2.0 ** -12
    kp.view(torch.uint8)[..., 1::2] = 0
    run_and_check(args, 100.0)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", BOTH)
def test_nan_reaches_its_heads_alone(wide, dtype):
    """A NaN in a query makes every score of its head NaN, one in a key a score of each head that reads it, one in a value
    its column, however the rows are shared out; the other heads and an empty sequence know nothing of it."""
    args = make(3, 4, 2, 64, 16, [200, 0, 130], dtype, seed=31, wide=wide)
    clean = fa.attention_decode_e4m3(*args)
    q, kp, vp, ks, vs, table, lengths = args
    q[0, 1, 0, 5] = float("nan")
    q[1, 2, 0, 0] = float("nan")
    kp.view(torch.uint8)[table[2, 100 // 16].item(), 1, 100 % 16, 63] = 0x7f  # key head 1: query heads 2, 3
    vp.view(torch.uint8)[table[2, 0].item(), 0, 3, 17] = 0xff                 # key head 0: query heads 0, 1
    o, L = fa.attention_decode_e4m3(*args)
    assert fa.get_device_status() == 0
    hit = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    hit[0, 1] = hit[2, 2] = hit[2, 3] = True
    column = torch.zeros(3, 4, 1, 64, dtype=torch.bool, device=DEV)
    column[hit] = True
    column[2, :2, :, 17] = True
    assert o[column].isnan().all() and L[hit].isnan().all()
    assert torch.equal(o[~column], clean[0][~column]) and torch.equal(L[~hit], clean[1][~hit])


@pytest.mark.parametrize("scale", [1e-3, 1.0])
def test_scale(scale):
    run_and_check(make(3, 4, 2, 64, 16, [100, 7, 64], seed=8), scale)


def test_scales_that_are_no_powers_of_two():
    """As another program may have quantised: any positive scale counts as it is."""
    for dtype in BOTH:
        args = make(3, 4, 2, 64, 16, [100, 7, 300], dtype, seed=11, block=4, junk=False)
        gen = torch.Generator().manual_seed(11)
        for t in args[3:5]:
            t.copy_(torch.rand(t.shape, generator=gen) / 100 + 1e-4)
        run_and_check(args)


def test_strided_queries_and_given_outputs():
    q, *cache, table, lengths = make(5, 8, 2, 64, 16, [100, 0, 7, 64, 1000], seed=9, wide=3000)
    fused = torch.rand(5, 12, 64, device=DEV).add_(0.25).to(torch.bfloat16)  # queries, keys and values of one projection
    view = fused[:, 2:10, None, :]
    o_all = torch.full((5, 10, 1, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    out = (o_all[:, 1:9], torch.empty(5, 8, 1, device=DEV))
    c, _ = fa.cache_for_e4m3(*cache, table)
    ws = torch.empty(fa.fa_decode_e4m3_workspace_bytes(c, 8), dtype=torch.uint8, device=DEV)
    got = run_and_check((view, *cache, table, lengths), out=out, workspace=ws)
    assert got[0].data_ptr() == out[0].data_ptr()
    assert (o_all[:, 0] == 7).all() and (o_all[:, 9] == 7).all()


def test_shared_pages():
    """Sequences that name the same pages, as forks do."""
    args = make(4, 8, 2, 128, 16, [320, 320, 320, 320], seed=10)
    args[5][1:, :10] = args[5][0, :10]
    run_and_check(args)


@pytest.mark.parametrize("wide", [0, 3000])
def test_offsets_beyond_32_bits(wide):
    """Pages further than 2^32 bytes into the pools, scales further than 2^31 bytes into theirs."""
    pages, page, d = 140000, 256, 128  # 4.6e9 bytes a pool
    ids = [139999, 3, 135000, 139990]
    q, *small, table, lengths = make(1, 4, 1, d, page, [1000], seed=11, block=1, spare=0, junk=False)
    large = [torch.empty(pages, 1, page, d, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    large += [torch.empty(pages, 1, page, device=DEV) for _ in range(2)]
    for t, x in zip(large, small):
        for i, p in enumerate(ids):
            t[p] = x[table[0, i].item()]
    big = torch.full((1, 4 + wide), -1, dtype=torch.int32, device=DEV)
    big[0, :4] = torch.tensor(ids)
    got = fa.attention_decode_e4m3(q, *large, big, lengths)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    check(got, q, *small, table, lengths, d ** -0.5)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", BOTH)
def test_bad_pages_and_lengths_are_not_followed(dtype, wide):
    q, *cache, table, lengths = make(4, 4, 2, 64, 16, [100, 50, 300, 20], dtype, seed=12, block=4, wide=wide)
    table[0, 2], table[2, 5] = 1 << 20, -7
    got = fa.attention_decode_e4m3(q, *cache, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    check(got, q, *cache, table, lengths, 64 ** -0.5)
    lengths = torch.tensor([-5, 50, 1 << 30, 20], dtype=torch.int32, device=DEV)
    got = fa.attention_decode_e4m3(q, *cache, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    some = [0, 1, 3]
    check((got[0][some], got[1][some]), q[some], *cache, table[some], lengths[some], 64 ** -0.5)
    with pytest.raises(fa.FaError) as err:
        fa.attention_decode_e4m3(q, *cache, table, lengths, check_status=True)
    assert err.value.code == fa.FA_ERR_PAGES
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", BOTH)
def test_same_call_same_bits(wide, dtype):
    args = make(7, 8, 2, 128, 16, [4000, 1, 900, 0, 77, 3333, 512], dtype, seed=13, wide=wide)
    a = fa.attention_decode_e4m3(*args)
    for _ in range(5):
        b = fa.attention_decode_e4m3(*args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("wide", [0, 3000])
def test_two_streams_at_once(wide):
    args = [make(4, 8, 2, 128, 16, [4000, 100, 1700, 64], seed=20 + i, wide=wide) for i in range(2)]
    want = [fa.attention_decode_e4m3(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for a, st in zip(args, streams):
            got.append(fa.attention_decode_e4m3(*a, stream=st))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", BOTH)
def test_memory_freed_on_the_current_stream(wide, dtype):
    """Temporaries of the sizes that a decode allocates, read by work that is still to come when they are freed."""
    args = make(4, 8, 2, 128, 16, [4000, 100, 1700, 64], dtype, seed=1, wide=wide)
    want = fa.attention_decode_e4m3(*args)
    c, _ = fa.cache_for_e4m3(*args[1:6], dtype)
    sizes = [args[0].numel() * args[0].element_size(), 4 * 4 * 8, fa.fa_decode_e4m3_workspace_bytes(c, 8)]
    side, big = torch.cuda.Stream(), torch.zeros(1 << 27, device=DEV)
    for i in range(6):
        held = [torch.full((n,), i + 1, dtype=torch.uint8, device=DEV) for n in sizes if n > 0 for _ in range(3)]
        torch.cuda.synchronize()
        for _ in range(20):
            big.add_(1)
        read = [t + 1 for t in held]
        freed = {t.data_ptr() for t in held}
        del held
        got = fa.attention_decode_e4m3(*args, stream=side)
        assert not {t.data_ptr() for t in got} & freed
        torch.cuda.synchronize()
        assert all((t == i + 2).all() for t in read)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("wide", [0, 3000])
def test_graph_follows_lengths_that_change(wide):
    """A captured call reads lengths, scales and table at each replay; two graphs replayed at once have workspaces of their own."""
    q, *cache, table, lengths = make(3, 8, 2, 64, 16, [2000, 900, 50], seed=30, junk=False, wide=wide)
    pairs = []
    torch.cuda.synchronize()
    for _ in range(2):
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            fa.attention_decode_e4m3(q, *cache, table, lengths)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                got = fa.attention_decode_e4m3(q, *cache, table, lengths)
        pairs.append((stream, graph, got))
    for new in ([2000, 900, 50], [1, 0, 16], [700, 777, 50]):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        cache[2].mul_(2), cache[3].mul_(0.5)
        torch.cuda.synchronize()
        for stream, graph, _ in pairs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, got in pairs:
            check(got, q, *cache, table, lengths, 64 ** -0.5)
    assert fa.get_device_status() == 0


def test_agrees_with_the_decode_of_the_same_values():
    """fa_decode over a cache that holds the values themselves, which fp32 does exactly."""
    for d, H, Hk in ((64, 4, 4), (128, 12, 2)):
        q, kp, vp, ks, vs, table, lengths = make(4, H, Hk, d, 16, [700, 0, 33, 16], torch.float32, seed=32, block=8, junk=False)
        plain = [p.float() * s.repeat_interleave(8, 2)[..., None] for p, s in ((kp, ks), (vp, vs))]
        want = fa.attention_decode(q, *plain, table, lengths)
        got = fa.attention_decode_e4m3(q, kp, vp, ks, vs, table, lengths)
        assert (got[0] - want[0]).abs().max() <= 2e-5 * plain[1].abs().max()
        seen = (lengths > 0)[:, None, None].expand_as(got[1])
        assert (got[1][seen] - want[1][seen]).abs().max() <= 2e-5 * want[1][seen].abs().max()


def test_refusals():
    q, *cache, table, lengths = make(3, 8, 2, 64, 16, [100, 7, 64], seed=40, wide=3000)
    names = dict(zip(("k_pages", "v_pages", "k_scales", "v_scales"), cache))
    good = dict(names, q=q, page_table=table, lengths=lengths)
    fa.attention_decode_e4m3(**good)
    o, L = torch.empty_like(q), torch.empty(3, 8, 1, device=DEV)
    for bad in (dict(q=q[:2]), dict(q=q[:, :, 0]), dict(q=q.expand(-1, -1, 2, -1)), dict(q=q[..., :32]), dict(q=q.cpu()),
                dict(q=q.detach().requires_grad_()), dict(lengths=lengths.long()), dict(lengths=lengths[:2]),
                dict(lengths=lengths.cpu()), dict(out=(o.float(), L)), dict(out=(o, L[:, :, 0])), dict(out=(o, L.half())),
                dict(k_scales=cache[2].requires_grad_(False).clone().requires_grad_()),
                dict(workspace=torch.empty(1 << 20, 2, device=DEV)[:, 0])):
        with pytest.raises(ValueError):
            fa.attention_decode_e4m3(**{**good, **bad})
    c, _ = fa.cache_for_e4m3(*cache, table)
    small = torch.empty(fa.fa_decode_e4m3_workspace_bytes(c, 8) - 1, dtype=torch.uint8, device=DEV)
    for bad in (dict(q=q[:, :7]), dict(scale=0.0), dict(scale=float("nan")), dict(workspace=small), dict(out=(q, L))):
        with pytest.raises(fa.FaError) as err:
            fa.attention_decode_e4m3(**{**good, **bad})
        assert err.value.code == fa.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FaError) as err:  # more than 512 query heads a key-value head
        fa.attention_decode_e4m3(**{**good, "q": torch.empty(3, 1026, 1, 64, dtype=torch.bfloat16, device=DEV)})
    assert err.value.code == fa.FA_ERR_UNSUPPORTED
    assert fa.get_device_status() == 0


def test_largest_group_of_heads():
    """512 query heads on one key-value head, in pieces."""
    for dtype in BOTH:
        for wide in (0, 3000):
            run_and_check(make(2, 512, 1, 32, 16, [300, 65], dtype, seed=41, wide=wide))


def test_grouped_single_page_strides():
    """Single sequences, heads, pages and rows, in storages that leave their strides open."""
    for S, H, Hk in ((1, 1, 1), (1, 4, 1), (1, 4, 4), (3, 4, 1)):
        for page, n in ((1, 1), (16, 16), (64, 5)):
            run_and_check(make(S, H, Hk, 64, page, [n] * S, seed=50, spare=0, rows_first=True))
