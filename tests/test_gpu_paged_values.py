"""fa_decode where the cache holds infinities and NaN in rows that are read.

Tolerances are those of test_gpu_decode.py."""

import pytest
import torch

import flashattention_backward_gb300 as fa
from test_gpu_decode import check, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def put(pool, table, s, j, head, col, x, page=16):
    pool[table[s, j // page].item(), head, j % page, col] = x


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype,H,d", [(torch.bfloat16, 4, 32), (torch.bfloat16, 4, 64), (torch.bfloat16, 32, 96),
                                       (torch.bfloat16, 40, 128), (torch.bfloat16, 4, 256), (torch.bfloat16, 32, 256),
                                       (torch.float32, 4, 64), (torch.float32, 16, 128)])
def test_infinite_values(dtype, H, d, wide):
    """An infinity in a row of V comes out in its column, for each query head that reads it; infinities of both signs in
    a column, or a NaN, come out as NaN.  Other columns, heads and sequences know nothing of them."""
    n = [300, 0, 130, 5, 2000]
    q, kp, vp, table, lengths = make(5, H, 2, d, 16, n, dtype, seed=d + H, wide=wide)
    g = H // 2
    clean = vp.clone()
    want = {}  # (sequence, key head, column): value
    for s, head, col, rows, x in ((0, 0, 3, [0], INF), (0, 1, d - 1, [299], -INF), (2, 1, 0, [63, 64, 129], INF),
                                  (3, 0, 17, [4], -INF), (4, 0, 9, [700], INF), (4, 0, 10, [1999], INF),
                                  (4, 1, 31, [0, 1024], -INF)):
        want[s, head, col] = x
        for j in rows:
            put(vp, table, s, j, head, col, x)
    for s, head, col, rows in ((0, 0, 8, [5, 290]), (2, 1, 7, [1, 2])):
        want[s, head, col] = NAN
        put(vp, table, s, rows[0], head, col, INF)
        put(vp, table, s, rows[1], head, col, -INF)
    want[4, 1, 2] = NAN
    put(vp, table, 4, 1500, 1, 2, NAN)
    o, L = fa.attention_decode(q, kp, vp, table, lengths)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    ref = fa.attention_decode(q, kp, clean, table, lengths)
    for (s, head, col), x in want.items():
        at = (s, slice(head * g, (head + 1) * g), 0, col)
        got = o[at].float()
        assert got.isnan().all() if x != x else (got == x).all(), (s, head, col, x, got)
        o[at] = ref[0][at]
    check((o, L), q, kp, clean, table, lengths, d ** -0.5)
    assert torch.equal(o, ref[0]) and torch.equal(L, ref[1])


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_value_infinite(dtype, wide):
    args = make(3, 8, 2, 64, 16, [1000, 0, 17], dtype, seed=3, wide=wide, junk=False)
    args[2].fill_(INF)
    o, L = fa.attention_decode(*args)
    assert fa.get_device_status() == 0
    assert (o[[0, 2]] == INF).all() and (o[1] == 0).all()
    assert L[[0, 2]].isfinite().all() and (L[1] == INF).all()


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_up_to_the_limit(wide, dtype):
    """Sums are taken before they are divided by the sum of the weights, which is at most the number of rows (the largest
    weight is 1): with n rows, values up to the largest float32 / (2 n) cannot overflow them, and none is taken for an
    infinity."""
    q, kp, vp, table, lengths = make(3, 8, 2, 64, 16, [300, 1, 17], dtype, seed=4, wide=wide, junk=False)
    x = 2.0 ** 127 / 512
    vp.fill_(x)
    o, L = fa.attention_decode(q, kp, vp, table, lengths)
    assert fa.get_device_status() == 0
    # the sum of weights and the weighted sum carry at most 2^-16 + 2^-21 each and 300 additions; x itself is exact
    assert ((o.double() - x).abs() <= x * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -14)).all()


@pytest.mark.parametrize("wide", [0, 3000])
def test_infinite_values_in_runs_that_go_on(wide):
    """Many sequences a block, some of them with an infinity: nothing but its own column changes."""
    n = [(i * 37) % 300 for i in range(400)]
    q, kp, vp, table, lengths = make(400, 4, 2, 64, 16, n, seed=5, wide=wide)
    ref = fa.attention_decode(q, kp, vp, table, lengths)
    hit = [s for s in range(400) if n[s] > 10 and s % 7 == 0]
    for s in hit:
        put(vp, table, s, n[s] // 2, s % 2, 5, INF)
    o, L = fa.attention_decode(q, kp, vp, table, lengths)
    assert fa.get_device_status() == 0
    assert torch.equal(L, ref[1])
    for s in hit:
        own = slice(2 * (s % 2), 2 * (s % 2) + 2)
        assert (o[s, own, 0, 5] == INF).all()
        o[s, own, 0, 5] = ref[0][s, own, 0, 5]
    assert torch.equal(o, ref[0])
