"""fa_decode_e4m3 where the table has room for so many rows that the tensor-memory
kernels take the problem (bf16, d 128 or 256, up to four query heads a key head):
what test_gpu_decode_e4m3.py asks of the others."""

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from test_gpu_decode_e4m3 import DEV, F8, HALF_STEP, check, make, run_and_check, values, f64

pytestmark = pytest.mark.gpu
SM = 152  # of a GB300


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def is_large(args):
    """By the workspace: 1 or 4 heads a part, 8 at least elsewhere."""
    q, *cache, table, _ = args
    c, _ = fa.cache_for_e4m3(*cache, table)
    n = fa.fa_decode_e4m3_workspace_bytes(c, q.shape[1])
    part = 8 + 4 * q.shape[3]
    return n == 2 * 1280 * part * (1 if q.shape[1] == c.H_kv else 4)


def large(S, H, Hk, d, page, lengths, **kw):
    """More columns than the rows need."""
    rows = SM * (2 * 56 if d == 128 else 40) * 128 // (S * Hk) + 128
    args = make(S, H, Hk, d, page, lengths, wide=rows // page + 1, **kw)
    assert is_large(args)
    return args


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("H,Hk", [(4, 4), (3, 3), (4, 2), (6, 2), (8, 2), (1, 1), (4, 1)])
def test_head_layouts(d, H, Hk):
    lengths = [0, 1, 15, 16, 17, 127, 128, 129, 300, 511]
    run_and_check(large(len(lengths), H, Hk, d, 16, lengths, seed=d + H))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page,block", [(1, 1), (3, 3), (13, 13), (16, 2), (48, 16), (64, 64), (100, 5), (256, 128), (1000, 8)])
@pytest.mark.parametrize("rows_first", [False, True])
def test_page_and_block_sizes(d, page, block, rows_first):
    lengths = [page - 1, page, page + 1, 2 * page, 259, 1]
    run_and_check(large(6, 4, 2, d, page, lengths, seed=page, block=block, rows_first=rows_first))


@pytest.mark.parametrize("n", [1, 128, 129, 2048, 32768])
@pytest.mark.parametrize("H,Hk,d", [(4, 1, 128), (2, 2, 256), (1, 1, 128), (2, 1, 256)])
def test_one_sequence_over_the_whole_gpu(n, H, Hk, d):
    run_and_check(large(1, H, Hk, d, 64, [n], seed=n, block=16))


def test_many_short_and_one_long():
    lengths = [4000] + [i % 5 for i in range(300)] + [1999]
    run_and_check(large(len(lengths), 4, 2, 128, 16, lengths, seed=3))


@pytest.mark.parametrize("d,H,Hk,S", [(128, 2, 2, 700), (256, 8, 2, 700), (128, 8, 4, 1300)])
def test_more_items_than_runs(d, H, Hk, S):
    """More sequences than a block has threads, too; the join goes by runs then."""
    lengths = [700 if i % 97 == 0 else (i * 37) % 130 for i in range(S)]
    run_and_check(large(S, H, Hk, d, 16, lengths, seed=4))


@pytest.mark.parametrize("d,H,S,n", [(128, 4, 40, 60000), (256, 1, 40, 40000)])
def test_enough_rows_for_small_runs(d, H, S, n):
    """A problem of many tiles for each group ends in small runs.  All sequences read the same pages, each a different
    number of them; two of the sequences are compared."""
    q, *pools, table, _ = make(1, H, 1, d, 64, [n], seed=21)
    q = (torch.randn(S, H, 1, d, generator=torch.Generator().manual_seed(22)).clamp(-2, 2) + 3).to(torch.bfloat16).to(DEV)
    lengths = torch.tensor([n - 77 * s for s in range(S)], dtype=torch.int32, device=DEV)
    args = (q, *pools, table.expand(S, -1).contiguous(), lengths)
    assert is_large(args)
    o, L = fa.attention_decode_e4m3(*args)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    for s in (0, S - 1):
        one = slice(s, s + 1)
        check((o[one], L[one]), q[one], *pools, table, lengths[one], d ** -0.5)


def test_all_empty():
    run_and_check(large(3, 4, 2, 128, 16, [0, 0, 0]))


@pytest.mark.parametrize("d", [128, 256])
def test_peaked_scores(d):
    run_and_check(large(4, 8, 2, d, 16, [3, 500, 2000, 77], seed=5, q_std=4.0))


@pytest.mark.parametrize("H", [1, 4])
@pytest.mark.parametrize("d", [128, 256])
def test_rising_and_falling_scores(d, H):
    """Each key scores above the one before, so that the maximum moves in every tile; or below."""
    q, kp, vp, ks, vs, table, lengths = large(1, H, 1, d, 16, [700], seed=6, block=1, junk=False)
    q.fill_(1.0)
    kp.view(torch.uint8).fill_(0x38)  # 1.0: the scales alone tell the keys apart
    for sign in (1, -1):
        for j in range(700):
            ks[table[0, j // 16].item(), :, j % 16] = (j if sign > 0 else 700 - j) / 64
        run_and_check((q, kp, vp, ks, vs, table, lengths))


@pytest.mark.parametrize("d,block", [(128, 1), (128, 16), (256, 16)])
def test_scales_far_apart(d, block):
    q, kp, vp, ks, vs, table, lengths = large(2, 4, 2, d, 16, [900, 130], seed=7, block=block, junk=False)
    gen = torch.Generator().manual_seed(7)
    vs.copy_(torch.exp2(torch.randint(-40, 41, vs.shape, generator=gen).float()))
    run_and_check((q, kp, vp, ks, vs, table, lengths))


@pytest.mark.parametrize("d,H", [(128, 4), (128, 1), (256, 4)])
def test_a_large_value_that_no_weight_reaches(d, H):
    """A page of V of 2^100 times the others' size, whose keys score so low that its weights are 0: the others' sum is
    held as if it were not there, wherever it stands.  And one of 2^-100 of their size that has all the weight."""
    dtype = torch.bfloat16
    for where in (0, 30, 62):
        args = large(1, H, 1, d, 16, [1000], seed=8, junk=False)
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
        rows = min(16, 1000 - 16 * where)
        want = torch.tensor(values(f64(vp), f64(vs))[page, :, :rows].mean(1))[:, None].expand(1, H, 1, d)
        # weights of 2^-4 are held exactly
        assert (o.cpu().double() - want).abs().max() <= (HALF_STEP[dtype] + 2.0 ** -19) * 2.0 ** -107 * 448


def test_values_of_nothing():
    q, kp, vp, ks, vs, table, lengths = large(2, 4, 2, 128, 16, [40, 16], seed=9, junk=False)
    first = table[:, 0].long()
    vp.view(torch.uint8)[first] = 0
    vs[first] = 2.0 ** -126
    o, _ = run_and_check((q, kp, vp, ks, vs, table, lengths))
    assert (o[1] == 0).all()
    kp.view(torch.uint8).fill_(0)
    ks.fill_(2.0 ** -126)
    run_and_check((q, kp, vp, ks, vs, table, lengths))


def test_queries_of_every_size():
    args = large(3, 8, 2, 128, 16, [100, 7, 300], seed=10, junk=False)
    q, kp, ks = args[0], args[1], args[3]
    base = q.clone()
    q.mul_(torch.exp2(torch.arange(-60, 60, 15, device=DEV).float())[None, :, None, None].to(q.dtype))
    ks.mul_(2.0 ** -4)
    run_and_check(args, 1e-16)
    q.copy_(base)
    q[..., ::2] *= 2.0 ** -12
    kp.view(torch.uint8)[..., 1::2] = 0
    run_and_check(args, 100.0)


@pytest.mark.parametrize("d,H,Hk", [(128, 4, 2), (128, 2, 2), (256, 6, 2)])
def test_nan_reaches_its_heads_alone(d, H, Hk):
    args = large(3, H, Hk, d, 16, [200, 0, 130], seed=31)
    clean = fa.attention_decode_e4m3(*args)
    q, kp, vp, ks, vs, table, lengths = args
    group = H // Hk
    q[0, 1, 0, 5] = float("nan")
    q[1, 0, 0, 0] = float("inf")
    kp.view(torch.uint8)[table[2, 100 // 16].item(), 1, 100 % 16, 63] = 0x7f
    vp.view(torch.uint8)[table[2, 0].item(), 0, 3, 17] = 0xff
    o, L = fa.attention_decode_e4m3(*args)
    assert fa.get_device_status() == 0
    hit = torch.zeros(3, H, dtype=torch.bool, device=DEV)
    hit[0, 1] = True
    hit[2, group:] = True
    column = torch.zeros(3, H, 1, d, dtype=torch.bool, device=DEV)
    column[hit] = True
    column[2, :group, :, 17] = True
    assert o[column].isnan().all() and L[hit].isnan().all()
    assert torch.equal(o[~column], clean[0][~column]) and torch.equal(L[~hit], clean[1][~hit])


def test_shared_pages():
    args = large(4, 8, 2, 128, 16, [320, 320, 320, 320], seed=10)
    args[5][1:, :10] = args[5][0, :10]
    run_and_check(args)


def test_offsets_beyond_32_bits():
    """Pages further than 2^32 bytes into the pools, scales further than 2^31 bytes into theirs."""
    pages, page, d = 140000, 256, 128  # 4.6e9 bytes a pool
    ids = [139999, 3, 135000, 139990]
    q, *small, table, lengths = make(1, 4, 1, d, page, [1000], seed=11, block=1, spare=0, junk=False)
    far = [torch.empty(pages, 1, page, d, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    far += [torch.empty(pages, 1, page, device=DEV) for _ in range(2)]
    for t, x in zip(far, small):
        for i, p in enumerate(ids):
            t[p] = x[table[0, i].item()]
    wide = torch.full((1, SM * 2 * 56 * 128 // page + 1), -1, dtype=torch.int32, device=DEV)
    wide[0, :4] = torch.tensor(ids)
    assert is_large((q, *far, wide, lengths))
    got = fa.attention_decode_e4m3(q, *far, wide, lengths)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    check(got, q, *small, table, lengths, d ** -0.5)


def test_strided_queries_and_given_outputs():
    q, *cache, table, lengths = large(5, 8, 2, 128, 16, [100, 0, 7, 64, 1000], seed=9)
    fused = torch.rand(5, 12, 128, device=DEV).add_(0.25).to(torch.bfloat16)  # queries, keys and values of one projection
    view = fused[:, 2:10, None, :]
    o_all = torch.full((5, 10, 1, 128), 7.0, device=DEV, dtype=torch.bfloat16)
    out = (o_all[:, 1:9], torch.empty(5, 8, 1, device=DEV))
    c, _ = fa.cache_for_e4m3(*cache, table)
    ws = torch.full((fa.fa_decode_e4m3_workspace_bytes(c, 8),), 255, dtype=torch.uint8, device=DEV)
    run_and_check((view, *cache, table, lengths), out=out, workspace=ws)
    assert (o_all[:, 0] == 7).all() and (o_all[:, 9] == 7).all()


def test_bad_pages_and_lengths_are_not_followed():
    q, *cache, table, lengths = large(4, 4, 2, 128, 16, [100, 50, 300, 20], seed=12, block=4)
    table[0, 2], table[2, 5] = 1 << 20, -7
    got = fa.attention_decode_e4m3(q, *cache, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    check(got, q, *cache, table, lengths, 128 ** -0.5)
    lengths = torch.tensor([-5, 50, 1 << 30, 20], dtype=torch.int32, device=DEV)
    got = fa.attention_decode_e4m3(q, *cache, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    some = [0, 1, 3]
    check((got[0][some], got[1][some]), q[some], *cache, table[some], lengths[some], 128 ** -0.5)
    table.fill_(-1)
    lengths = torch.tensor([500, 50, 0, 20], dtype=torch.int32, device=DEV)
    o, L = fa.attention_decode_e4m3(q, *cache, table, lengths)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert (o == 0).all() and torch.isposinf(L).all()


@pytest.mark.parametrize("d", [128, 256])
def test_same_call_same_bits_on_any_stream(d):
    args = large(7, 8, 2, d, 16, [4000, 1, 900, 0, 77, 3333, 512], seed=13)
    want = fa.attention_decode_e4m3(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [fa.attention_decode_e4m3(*args, stream=st) for _ in range(10) for st in streams]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    assert fa.get_device_status() == 0


def test_beside_the_forward_on_another_stream():
    """Both hold tensor memory; each waits for the other's blocks to give theirs back."""
    args = large(7, 8, 2, 128, 16, [4000, 1, 900, 0, 77, 3333, 512], seed=14)
    want = fa.attention_decode_e4m3(*args)
    x = torch.randn(2, 8, 2048, 128, device=DEV).to(torch.bfloat16)
    forward = fa.attention_forward(x, x, x, 0.1, causal=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        got.append((fa.attention_decode_e4m3(*args, stream=streams[0]), fa.attention_forward(x, x, x, 0.1, causal=True, stream=streams[1])))
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    for a, b in got:
        assert torch.equal(a[0], want[0]) and torch.equal(b[0], forward[0])


def test_graph_follows_lengths_that_change():
    q, *cache, table, lengths = large(3, 8, 2, 128, 16, [2000, 900, 50], seed=30, junk=False)
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
            check(got, q, *cache, table, lengths, 128 ** -0.5)
    assert fa.get_device_status() == 0


def test_agrees_with_the_small_kernels():
    """The same cache with a table that is no wider than it has to be."""
    q, kp, vp, ks, vs, table, lengths = large(3, 8, 2, 128, 16, [300, 65, 1], seed=33)
    narrow = table[:, :20].contiguous()
    assert not is_large((q, kp, vp, ks, vs, narrow, lengths))
    a = fa.attention_decode_e4m3(q, kp, vp, ks, vs, table, lengths)
    b = fa.attention_decode_e4m3(q, kp, vp, ks, vs, narrow, lengths)
    assert (a[0].float() - b[0].float()).abs().max() <= 2.0 ** -7 * b[0].abs().max()
    assert (a[1] - b[1]).abs().max() <= 2.0 ** -18 * b[1].abs().max()


@pytest.mark.parametrize("d,H,Hk", [(128, 8, 2), (128, 2, 2), (256, 8, 2), (256, 2, 2)])
def test_again_and_again(d, H, Hk):
    """Items of one tile to some, in runs that begin and end inside of them, the same bits each time."""
    lengths = [700 if i % 97 == 0 else (i * 37) % 130 for i in range(700)]
    args = large(700, H, Hk, d, 16, lengths, seed=4)
    want = run_and_check(args)
    for _ in range(30):
        o, L = fa.attention_decode_e4m3(*args)
        assert torch.equal(o, want[0]) and torch.equal(L, want[1])
    assert fa.get_device_status() == 0
