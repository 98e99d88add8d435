"""fa_decode_e4m3 at the ends of its range, on every path: blocks of V with the smallest scales that there are and with
the largest.

Bounds as in test_gpu_decode_e4m3.py, with what weights are held in as in test_gpu_decode_e4m3_weights.py.  At a scale b
below 2^-115 the largest weight is 2^126 b (2^123 b on tensor memory) when a unit is set, not 2^10 (2^7) or more, so that
weights are off by up to 2^-25 / 2^126 = 2^-151 (2^-29 / 2^123), and their products with b, below 2^-126, by 2^-150: together
less than 2^-149 / b of the largest.
The weighted sums of a warp or a part, below 2^-126 too, are rounded to 2^-149."""

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa
from oracle.e4m3_fp64 import values
from oracle.paged_fp64 import decode
from test_gpu_decode_e4m3 import F8, HALF_STEP, U, f64, make

pytestmark = pytest.mark.gpu
# d, heads a key head, type, columns of the table more than the rows need: none for clusters
PATHS = [(64, 2, torch.bfloat16, 0), (64, 2, torch.bfloat16, 3000), (128, 16, torch.bfloat16, 3000), (96, 3, torch.float32, 0),
         (64, 8, torch.float32, 3000), (128, 4, torch.bfloat16, 80000), (128, 1, torch.bfloat16, 80000), (256, 4, torch.bfloat16, 80000)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


def cache(path, lengths, **kw):
    d, group, dtype, wide = path
    return make(len(lengths), 2 * group, 2, d, 16, lengths, dtype, wide=wide, junk=False, **kw)


def check(args, b):
    q, kp, vp, ks, vs, table, lengths = args
    scale = np.float64(np.float32(q.shape[3] ** -0.5))
    o, L = fa.attention_decode_e4m3(*args)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    k, v = values(f64(kp), f64(ks)), values(f64(vp), f64(vs))
    ref, Lr, A, V = decode(f64(q)[:, :, 0], k, v, table.cpu().numpy(), lengths.cpu().numpy(), scale)
    d, n = q.shape[3], lengths.cpu().numpy()[:, None]
    e_s = (2 * d + 9) * U * A
    e_w = e_s + 4 * U * A + 2.0 ** -21 + 2.0 ** -15 + max(2.0 ** -35, 2.0 ** -149 / b)
    tol = HALF_STEP[q.dtype] * np.abs(ref) + (2 * V * (e_w + 2 * (n + 64) * U))[:, :, None] + 2.0 ** -140
    if q.dtype == torch.float32:
        tol -= (2 * V * 2.0 ** -15 * (1 - 2.0 ** -7))[:, :, None]  # weights of 22 bits
    off = np.abs(f64(o)[:, :, 0] - ref)
    assert (off <= tol).all(), (float((off / tol).max()), float((off / V.clip(1e-300)[:, :, None]).max()))
    seen = np.isfinite(Lr)
    tol = 2 * e_s + 4 * U * A + 2.0 ** -20 + 2 * (n + 64) * U
    assert (np.abs(f64(L)[:, :, 0][seen] - Lr[seen]) <= tol[seen] + 8 * U * np.abs(Lr[seen])).all()


@pytest.mark.parametrize("e", [-126, -125, -122, -120, -118, -117, -115, -114, -101, -99])
@pytest.mark.parametrize("path", PATHS)
def test_smallest_scales_of_values(path, e):
    args = cache(path, [300, 0, 17, 1], seed=1)
    args[4].fill_(2.0 ** e)
    check(args, 2.0 ** e)


@pytest.mark.parametrize("e", [110, 118, 119, 126, 127])
@pytest.mark.parametrize("path", PATHS)
def test_largest_scales_of_values(path, e):
    """With stored values that are small enough for sums of as many rows."""
    args = cache(path, [300, 0, 17, 1], seed=2)
    gen = torch.Generator().manual_seed(3)
    args[2].copy_((torch.randint(-4, 5, args[2].shape, generator=gen) * 2.0 ** -9).to(F8))  # the smallest there are
    args[4].fill_(2.0 ** e)
    check(args, 2.0 ** e)


@pytest.mark.parametrize("path", PATHS)
def test_smallest_scales_beside_large_ones(path):
    """Rows with all the weight on the smallest scales, after rows on the largest that score far below."""
    args = cache(path, [200, 40], seed=4)
    q, kp, vp, ks, vs, table, lengths = args
    q.fill_(1.0)
    kp.view(torch.uint8).fill_(0xb8)  # -1
    ks.fill_(2.0 ** 6)
    vs.fill_(2.0 ** 100)
    last = [table[0, 12].item(), table[1, 2].item()]  # rows 192 ... and 32 ...
    kp.view(torch.uint8)[last] = 0x38  # 1
    vs[last] = 2.0 ** -126
    o, _ = fa.attention_decode_e4m3(*args)
    assert fa.get_device_status() == 0
    d = q.shape[3]
    for s in range(2):
        want = values(f64(vp), f64(vs))[last[s], :, :8].mean(1)  # the others' weights are exp(-128 sqrt(d))
        got = f64(o)[s, :, 0].reshape(2, -1, d)
        assert np.abs(got - want[:, None]).max() <= (HALF_STEP[q.dtype] + 2.0 ** -14) * 448 * 2.0 ** -126


@pytest.mark.parametrize("key", [1.0, -1.0, None])
@pytest.mark.parametrize("path", PATHS)
def test_an_infinite_query_makes_nan_of_its_head(path, key):
    """Of any sign, whatever the keys' signs are (None: as they come) and however few there are; all scores may be
    -inf by it. The other heads, and a sequence without rows, know nothing of it."""
    args = cache(path, [300, 0, 17, 1, 1], seed=5)
    if key:
        args[1].view(torch.uint8).fill_(0x38 if key > 0 else 0xb8)
    clean = fa.attention_decode_e4m3(*args)
    q = args[0]
    inf, d = float("inf"), q.shape[3]
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=q.device)
    for s, h, c, x in ((0, 0, 0, inf), (0, -1, d - 1, -inf), (1, 0, 1, -inf), (2, 1, 17, -inf), (2, 0, 5, inf), (3, 0, 8, inf),
                       (3, 1, 15, -inf), (4, 1, 3, inf), (4, 0, d // 2, -inf)):
        q[s, h, 0, c] = x
        hit[s, h] = s != 1
    o, L = fa.attention_decode_e4m3(*args)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    assert o[hit].isnan().all() and L[hit].isnan().all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(L[~hit], clean[1][~hit])


@pytest.mark.parametrize("e", [126, 118, -118, -126])
@pytest.mark.parametrize("path", PATHS)
def test_queries_and_keys_at_opposite_ends(path, e):
    """Queries of up to 2^e and keys with scales that take the scores back to some units."""
    args = cache(path, [300, 0, 17, 1], seed=6)
    q, ks = args[0], args[3]
    q.mul_(2.0 ** (e - 1))
    ks.mul_(2.0 ** (1 - e if e > 0 else -e - 8))
    check(args, 2.0 ** -9)
