"""fa_decode_e4m3: what its weights are held in.  Data on which lost bits of the
weights show: many small weights that matter together behind one that is large,
and sums in which the weights' errors do not cancel but the values do.

Bounds.  A key's weight is p b, p = exp(score - the largest score), b its block's
scale of V.  As a factor of the product with V it is held with a relative error of
at most r, or, if that is more, with an absolute one of at most a of the run's
largest weight; the sum l that O is divided by has p in fp32.  So
  |O - ref| <= half a step of O + (r + e) sum_j p_j |v_j| / l + a n max_j(p_j b_j) max |q| / l
with q the stored values and e what every path has: 2^-22 of the hardware exponential, rounding errors of
the scores (4 of 2^-24 of the largest score, in the exponent), in the weighted sum and in l, and the additions.  These are
made tile by tile: at most 4 of a product's partial sums a tile of 64 rows or more, and 64 for the
joining, each off by at most 2^-23 of the sum of absolute values.
  tensor-memory path, bf16:  r = 2^-15, a = 2^-36 (four terms of e5m2, the largest weight at 2^7 or more of 2^-29)
  the other path:            r = 2^-22, a = 2^-35 (two fp16 numbers, the largest weight at 2^10 or more of 2^-25)"""

import numpy as np
import pytest
import torch

import flashattention_backward_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
HK = 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


# S sequences read the same pages, so many that a run holds most of an item; the last number says which path
PATHS = {
    "sm103 128, 4 heads": (128, 4, torch.bfloat16, 304, True),
    "sm103 128, 1 head": (128, 1, torch.bfloat16, 304, True),
    "sm103 256, 3 heads": (256, 3, torch.bfloat16, 152, True),
    "sm103 256, 1 head": (256, 1, torch.bfloat16, 152, True),
    "mma 128, 5 heads": (128, 5, torch.bfloat16, 304, False),
    "mma 64, 1 head": (64, 1, torch.bfloat16, 400, False),
    "mma 64, 16 heads": (64, 16, torch.bfloat16, 400, False),
    "mma 256, 9 heads": (256, 9, torch.bfloat16, 152, False),
    "mma 32, 2 heads": (32, 2, torch.bfloat16, 400, False),
    "fp32 128, 4 heads": (128, 4, torch.float32, 304, False),
    "fp32 64, 8 heads": (64, 8, torch.float32, 400, False),
}


def cache(path, n, gaps, v, v_scales, top=30, columns=0, page=64, heads=None):
    """One sequence's rows with scores `gaps` (in bits) below `top` bits, a scale a row: q = 1, keys 1 times their scales.
    heads: factors of the scores, for each query head of a key head."""
    d, group, dtype, S, _ = PATHS[path]
    pages = -(-n // page)
    kp = torch.full((pages, HK, page, d), 0x38, dtype=torch.uint8)  # 1.0
    vp = torch.zeros(pages, HK, page, d)
    ks, vs = torch.ones(pages, HK, page), torch.ones(pages, HK, page)
    scale = d ** -0.5
    bits = top - np.asarray(gaps, dtype=np.float64)
    at = torch.tensor(bits * np.log(2) / (d * np.float64(np.float32(scale)))).float()
    for t, x in ((ks, at), (vs, v_scales)):
        flat = torch.ones(pages * page)
        flat[:n] = torch.as_tensor(x, dtype=torch.float32)
        t.copy_(flat.view(pages, 1, page).expand(-1, HK, -1))
    flat = torch.zeros(pages * page, d)
    flat[:n] = torch.as_tensor(v, dtype=torch.float32)
    vp.copy_(flat.view(pages, 1, page, d).expand(-1, HK, -1, -1))
    q = torch.ones(S, HK * group, 1, d, dtype=dtype)
    if heads is not None:
        q *= torch.tensor(heads, dtype=dtype).repeat(HK)[:, None, None]
    table = torch.full((S, max(pages, columns)), -1, dtype=torch.int32)
    table[:, :pages] = torch.arange(pages)
    lengths = torch.full((S,), n, dtype=torch.int32)
    return [t.to(DEV) for t in (q, kp.view(F8), vp.to(F8), ks, vs, table, lengths)]


def check(path, args, n):
    d, group, dtype, S, sm103 = PATHS[path]
    q, kp, vp, ks, vs, table, lengths = args
    c, _ = fa.cache_for_e4m3(*args[1:6], dtype)
    takes = fa.fa_decode_e4m3_workspace_bytes(c, HK * group) == 2 * 1280 * (8 + 4 * d) * (1 if group == 1 else 4)
    assert takes == sm103
    o, L = fa.attention_decode_e4m3(*args)
    torch.cuda.synchronize()
    assert fa.get_device_status() == 0
    rows = lambda t: t[:, 0].reshape(-1, *t.shape[3:])[:n].cpu().float().double().numpy()
    k, v, b = rows(ks), rows(vp), rows(vs)
    r, a = (2.0 ** -15, 2.0 ** -36) if sm103 else (2.0 ** -22, 2.0 ** -35)
    for h in range(group):
        score = k * (d * np.float64(np.float32(d ** -0.5)) * q[0, h, 0, 0].item())
        p = np.exp(score - score.max())
        w, l = p * b, p.sum()
        ref, total = (w @ v) / l, (w @ np.abs(v)) / l
        e = 2 * (2.0 ** -22 + np.abs(score).max() * 4 * 2.0 ** -24) + 2 * (4 * n / 64 + 64) * 2.0 ** -23
        tol = HALF_STEP[dtype] * np.abs(ref) + (r + e) * total + a * n * w.max() * np.abs(v).max() / l
        off = np.abs(o[:, h::group].cpu().double().numpy() - ref)
        assert (off <= tol).all(), (h, float((off / tol).max()), float((off.max((0, 1, 2)) / np.abs(ref).clip(1e-300)).max()))
        want = score.max() + np.log(l)
        off = np.abs(L[:, h::group].cpu().double().numpy() - want)
        assert (off <= np.abs(score).max() * 8 * 2.0 ** -24 + e + 2.0 ** -22 * abs(want)).all()


def some_values(n, d, seed, mean):
    return (torch.randn(n, d, generator=torch.Generator().manual_seed(seed)) + mean).clamp(-448, 448).to(F8).float()


@pytest.mark.parametrize("gap", [10, 17, 19, 20.5, 22])
@pytest.mark.parametrize("by", ["score", "scale"])
@pytest.mark.parametrize("path", list(PATHS))
def test_many_small_weights_behind_a_large_one(path, by, gap):
    """The first row's weight is 2^gap times that of each other, by its score or by its scale, and its value is 0: O is the
    others'.  In half of the columns their mean is as large as their deviation, in the others it is 0."""
    n, d = 12000, PATHS[path][0]
    v = some_values(n, d, 1, torch.arange(d) % 2)
    v[0] = 0
    gaps, scales = np.zeros(n), np.ones(n)
    if by == "score":
        gaps[1:] = gap
    else:
        scales[0] = 2.0 ** gap
    check(path, cache(path, n, gaps, v, scales), n)


@pytest.mark.parametrize("gap", [26.5, 28.5])
@pytest.mark.parametrize("path", list(PATHS))
def test_weights_at_the_end_of_their_range(path, gap):
    """As above, with weights that are a few steps of what they are held in, the value 1 for all, and large ones for each
    warp, which has a unit of its own, of the first tile."""
    n, d = 12000, PATHS[path][0]
    v = torch.ones(n, d)
    v[:128:16] = 0
    gaps = np.full(n, gap)
    gaps[:128:16] = 0
    check(path, cache(path, n, gaps, v, np.ones(n), top=32), n)


@pytest.mark.parametrize("path", list(PATHS))
def test_scores_as_they_come_behind_a_large_weight(path):
    """A first row with nearly all of the weight and a value of 0, the others' scores with a deviation of 1."""
    n, d = 12000, PATHS[path][0]
    v = some_values(n, d, 2, 0)
    v[0] = 0
    gaps = np.zeros(n)
    gaps[1:] = 20 - np.random.default_rng(2).normal(size=n - 1).clip(-3, 3) / np.log(2)
    check(path, cache(path, n, gaps, v, np.ones(n)), n)


@pytest.mark.parametrize("path", list(PATHS))
def test_values_that_cancel(path):
    """Two kinds of rows, one with half the weight and twice the value of the other and the opposite sign: but for 0.9 of
    half a step of 11 bits, which is what O is."""
    n, d = 128, PATHS[path][0]
    gaps = np.where(np.arange(n) % 2, -np.log2((1 + 0.9 * 2.0 ** -11) / 2), 0.0)
    v = torch.where(torch.arange(n) % 2 > 0, 1.0, -0.5)[:, None].expand(-1, d)
    check(path, cache(path, n, gaps, v, np.ones(n), top=2, columns=3800 // 64 if PATHS[path][4] else 0), n)


@pytest.mark.parametrize("path", [p for p in PATHS if PATHS[p][1] > 1])
def test_a_large_scale_that_is_left_behind(path):
    """The first row's scale is 2^80 times the others' and its value 0.  The scores rise from tile to tile: by 8 bits and more in
    one head, so that the maxima of all move, and by 0.9 in the others, whose first row has as much weight as any at last."""
    n, (d, group) = 12000, PATHS[path][:2]
    v = some_values(n, d, 3, torch.arange(d) % 2)
    v[0] = 0
    scales = np.ones(n)
    scales[0] = 2.0 ** 80
    top = 0.9 * (n // 128)
    check(path, cache(path, n, top - 0.9 * (np.arange(n) // 128), v, scales, top=top, heads=[9.5] + [1] * (group - 1)), n)
