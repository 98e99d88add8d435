"""Measured cases of a paged key-value cache held in 8 bits: rows quantised as
they are written, the attention of one new token over them, rows read back, and
pages copied.

The pools ``k_pages`` and ``v_pages`` are float8_e4m3fn [pages, kv_heads,
page_rows, d].  ``k_scales`` and ``v_scales`` (float32 [pages, kv_heads,
blocks]) hold a power of two for every block of page_rows / blocks rows of a
page and head: a stored value times its block's scale is the value it stands
for.  ``page_table`` (int32 [sequences, columns]) says which page holds which
rows of a sequence; entries behind its pages are -1.

``run`` computes every operator in its plain form (elementary torch operations
in 32 bits, rounded once) or, with ``own``, through this repository's calls.
"""

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
_F8 = torch.float8_e4m3fn
_TOP = 448.0  # the largest value of the type
_DEV = "cuda"


def listed():
    return [
        # One answer's first tokens: almost nothing to read, the call's own latency counts.
        dict(name="decode_first_tokens", op="decode", batch=1, heads=32, kv_heads=32, dim=64, longest=48,
             spread="equal", page=16, block=16, dtype="bf16", mix=1),
        # A batch of short dialogues, a key-value head for each query head, lengths from nothing to 2048.
        dict(name="decode_dialogues", op="decode", batch=32, heads=32, kv_heads=32, dim=64, longest=2048,
             spread="ragged", page=16, block=16, dtype="bf16", mix=2),
        # A full serving batch, four query heads to a key-value head, a scale for each page: the largest cache.
        dict(name="decode_serving_batch", op="decode", batch=64, heads=32, kv_heads=8, dim=128, longest=8192,
             spread="ragged", page=64, block=64, dtype="bf16", mix=3),
        # One long document: a single sequence has to fill the whole GPU.
        dict(name="decode_long_document", op="decode", batch=1, heads=8, kv_heads=8, dim=128, longest=32768,
             spread="equal", page=256, block=32, dtype="bf16", mix=4),
        # All sixteen query heads on one key-value head, pages of an odd number of rows, a scale for each token.
        dict(name="decode_one_kv_head", op="decode", batch=4, heads=16, kv_heads=1, dim=128, longest=4000,
             spread="ragged", page=13, block=1, dtype="bf16", mix=5),
        # Queries and outputs in full precision, as for telling what the 8 bits of the cache cost.
        dict(name="decode_fp32", op="decode", batch=8, heads=8, kv_heads=2, dim=96, longest=4000,
             spread="ragged", page=16, block=8, dtype="fp32", mix=6),
        # The step of a serving batch: one new row a sequence, in the middle of a block.
        dict(name="append_step", op="append", batch=64, kv_heads=8, dim=128, rows=1, held=4000, spread="equal",
             page=64, block=64, layout="bhnd", dtype="bf16", mix=7),
        # Prompts that have just been computed go into their pages.
        dict(name="append_prompts", op="append", batch=4, kv_heads=16, dim=128, rows=4000, held=0, spread="ragged",
             page=16, block=16, layout="bnhd", dtype="bf16", mix=8),
        # A short answer is read back, to look at it.
        dict(name="read_answer", op="read", batch=1, kv_heads=32, dim=64, rows=48, skip=5, spread="equal", page=16,
             block=16, dtype="fp32", mix=9),
        # Cached prompts come back for the attention of the prompts' next parts.
        dict(name="read_prompts", op="read", batch=4, kv_heads=16, dim=128, rows=4000, skip=0, spread="ragged",
             page=64, block=32, dtype="bf16", mix=10),
        # Four samples from one prompt: each gets its own last page.
        dict(name="copy_tails", op="copy", moves=4, pages=64, partly=True, kv_heads=32, dim=64, page=16, block=16, mix=11),
        # A pool is compacted: what lives behind moves to free pages in front.
        dict(name="copy_compacted", op="copy", moves=2048, pages=8192, partly=False, kv_heads=8, dim=128, page=16,
             block=8, mix=12),
    ]


def _between(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choices(["decode", "append", "read", "copy"], [10, 5, 3, 2])[0]
    dtype = rng.choices(["bf16", "fp32"], [3, 1])[0]
    dim = rng.choice([32, 64, 96, 128, 256] if dtype == "bf16" else [16, 32, 64, 96, 128, 256])
    page = rng.choice([1, 8, 13, 16, 16, 32, 48, 64, 100, 128, 256])
    block = rng.choice([b for b in range(1, page + 1) if page % b == 0])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    mix = rng.randrange(1 << 30)
    row = kv_heads * dim  # bytes of a row of one pool, all its heads
    if op == "decode":
        group = rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16, 20, 32])
        longest = _between(rng, 1, 32768)
        most = max(1, (1 << 29) // (2 * row * longest))
        return dict(op=op, batch=_between(rng, 1, min(64, most)), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    longest=longest, spread=rng.choice(["equal", "ragged", "ragged"]), page=page, block=block, dtype=dtype,
                    mix=mix)
    if op in ("append", "read"):
        rows = rng.choice([1, 1, _between(rng, 1, 4000)]) if op == "append" else _between(rng, 1, 4000)
        most = max(1, (1 << 25) // (row * rows))
        case = dict(op=op, batch=_between(rng, 1, min(64, most)), kv_heads=kv_heads, dim=dim, rows=rows)
        case["held" if op == "append" else "skip"] = _between(rng, 1, 2000) - 1
        if op == "append":
            case["layout"] = rng.choice(["bhnd", "bnhd"])
        return dict(case, spread=rng.choice(["equal", "ragged"]), page=page, block=block, dtype=dtype, mix=mix)
    moves = _between(rng, 1, max(1, min(2048, (1 << 25) // (row * page))))
    return dict(op=op, moves=moves, pages=2 * moves + rng.randrange(1, 64), partly=rng.random() < 0.5, kv_heads=kv_heads,
                dim=dim, page=page, block=block, mix=mix)


def _amounts(mix, count, longest, spread):
    """Rows of each sequence.  Ragged: the first has them all, every eighth is an empty slot, the others lie between."""
    if spread == "equal":
        return [longest] * count
    rng = random.Random(mix)
    return [longest if i == 0 else 0 if i % 8 == 7 else rng.randint(1, longest) for i in range(count)]


def _new_rows(case):
    return [max(1, n) for n in _amounts(case["mix"], case["batch"], case["rows"], case["spread"])]


def _moved(case):
    """Rows of each page that is copied."""
    rng = random.Random(case["mix"])
    return [rng.randint(1, case["page"]) if case["partly"] else case["page"] for _ in range(case["moves"])]


def work(case):
    page, block, hk = case["page"], case["block"], case["kv_heads"]
    row = hk * case["dim"]  # a row of one pool, all its heads
    if case["op"] == "copy":
        rows = _moved(case)
        return {"bytes": 4 * row * sum(rows) + 16 * hk * sum(-(-n // block) for n in rows) + 12 * len(rows), "flops": 0}
    es = _BYTES[case["dtype"]]
    if case["op"] == "decode":
        lens = _amounts(case["mix"], case["batch"], case["longest"], case["spread"])
        vec = case["batch"] * case["heads"] * case["dim"]
        small = 4 * case["batch"] * (case["heads"] + 1) + 4 * sum(-(-n // page) for n in lens)
        return {"bytes": 2 * row * sum(lens) + 8 * hk * sum(-(-n // block) for n in lens) + 2 * vec * es + small,
                "flops": 4 * case["heads"] * case["dim"] * sum(lens)}
    b = case["batch"]
    if case["op"] == "append":
        rows = _new_rows(case)
        blocks = sum((case["held"] + n - 1) // block - case["held"] // block + 1 for n in rows)
        return {"bytes": 2 * row * (es + 1) * sum(rows) + 8 * hk * blocks + 8 * b + 4 * (sum(rows) // page + b), "flops": 0}
    rows = _amounts(case["mix"], b, case["rows"], case["spread"])
    blocks = sum(-(-n // block) for n in rows)
    return {"bytes": 2 * row * (sum(rows) + es * b * case["rows"]) + 8 * hk * blocks + 8 * b + 4 * (sum(rows) // page + b),
            "flops": 0}


def _rand(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=_DEV, dtype=_TYPES[dtype])


def _pool(gen, case, pages):
    """Values as a quantised row has them, up to the type's largest, and scales that make them about 1 in size."""
    hk, page, d = case["kv_heads"], case["page"], case["dim"]
    values = torch.randn((pages, hk, page, d), generator=gen, device=_DEV).mul_(112.0).clamp_(-_TOP, _TOP).to(_F8)
    exponents = torch.randint(-9, -5, (pages, hk, page // case["block"]), generator=gen, device=_DEV)
    return values, torch.exp2(exponents.float())


def _table(gen, lens, columns, page, pages):
    """A table of `columns` columns whose sequences hold pages in no order."""
    held = torch.tensor([-(-n // page) for n in lens], device=_DEV)
    mine = torch.arange(columns, device=_DEV)[None, :] < held[:, None]
    table = torch.full((len(lens), columns), -1, dtype=torch.int32, device=_DEV)
    table[mine] = torch.randperm(pages, generator=gen, device=_DEV)[: int(mine.sum())].int()
    return table


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(int(seed) * 1000003 + case["mix"] % 1000003)
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    ints = dict(dtype=torch.int32, device=_DEV)
    st = {"case": case, "scale": d ** -0.5}
    if case["op"] == "decode":
        lens = _amounts(case["mix"], case["batch"], case["longest"], case["spread"])
        held = sum(-(-n // page) for n in lens)
        pages = held + held // 8 + 1
        st["table"] = _table(gen, lens, -(-case["longest"] // page), page, pages)
        st["lengths"] = torch.tensor(lens, **ints)
        st["q"] = _rand(gen, (case["batch"], case["heads"], 1, d), case["dtype"])
    elif case["op"] in ("append", "read"):
        writes = case["op"] == "append"
        held = case["held" if writes else "skip"]
        rows = _new_rows(case) if writes else _amounts(case["mix"], case["batch"], case["rows"], case["spread"])
        full = [held + n for n in rows]
        pages = sum(-(-n // page) for n in full) + 1
        st["table"] = _table(gen, full, max(1, -(-max(full) // page)), page, pages)
        st["start"] = torch.full((case["batch"],), held, **ints)
        st["counts"] = torch.tensor(rows, **ints)
        b, n = case["batch"], case["rows"]
        if writes:
            shape = (b, hk, n, d) if case["layout"] == "bhnd" else (b, n, hk, d)
            st["k"], st["v"] = (_rand(gen, shape, case["dtype"]) for _ in range(2))
            st["k"] *= torch.where(torch.arange(d, device=_DEV) % 32 == 5, 6.0, 1.0).to(st["k"].dtype)  # keys have large columns
            if case["layout"] == "bnhd":
                st["k"], st["v"] = st["k"].permute(0, 2, 1, 3), st["v"].permute(0, 2, 1, 3)
    else:
        pages, moves = case["pages"], case["moves"]
        order = torch.randperm(pages, generator=gen, device=_DEV)
        st["moves"] = torch.stack([order[:moves], order[moves: 2 * moves], torch.tensor(_moved(case), device=_DEV)], 1).int()
    st["k_pages"], st["k_scales"] = _pool(gen, case, pages)
    st["v_pages"], st["v_scales"] = _pool(gen, case, pages)
    return st


def _rows(pages, scales, table, block):
    """The values of all rows that the table names, [sequences, kv_heads, rows, d] in 32 bits."""
    at = table.clamp(min=0).long()
    x = pages.view(torch.uint8)[at].view(_F8).float() * scales[at].repeat_interleave(block, 3)[..., None]
    s, columns, hk, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, hk, columns * page, d)


def _decode(st):
    q, block = st["q"], st["case"]["block"]
    b, heads, _, d = q.shape
    k = _rows(st["k_pages"], st["k_scales"], st["table"], block)
    hk, n = k.shape[1:3]
    seen = (torch.arange(n, device=q.device)[None, :] < st["lengths"][:, None])[:, None, None, :]
    s = torch.where(seen, q.float().view(b, hk, heads // hk, d) @ k.transpose(2, 3) * st["scale"], -math.inf)
    del k
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    z = p.sum(3, keepdim=True)
    v = torch.where(seen.transpose(2, 3), _rows(st["v_pages"], st["v_scales"], st["table"], block), 0.0)
    o = torch.where(z > 0, p @ v / z, 0.0)
    lse = torch.where(z > 0, m + torch.log(z), math.inf)
    return o.reshape(b, heads, 1, d).to(q.dtype), lse.reshape(b, heads, 1)


def _scale_for(top):
    """The smallest power of two that takes values up to `top` to at most 448 (2^-126 at least)."""
    mantissa, exponent = torch.frexp(top)  # top = mantissa 2^exponent, 1/2 <= mantissa < 1, and 448 = 7/8 2^9
    exponent = (exponent - 9 + (mantissa > 0.875).int()).clamp(-126, 120)
    return ((exponent + 127) << 23).int().view(torch.float32)


def _to_e4m3(x):
    """In 32 bits, |x| <= 448: rounded to the nearest, ties to even; what is not finite becomes NaN."""
    return torch.where(torch.isfinite(x), x, math.nan).to(_F8)


def _append_to(x, pages, scales, st):
    """New rows into one pool.  What lies behind a sequence's rows is its last row once more: the same values to the same place."""
    block, page = st["case"]["block"], st["case"]["page"]
    start, end = st["start"].long(), (st["start"] + st["counts"]).long()
    first, last = start // block, (end - 1) // block
    many = (x.shape[2] + block - 2) // block + 1
    at = torch.minimum(first[:, None] + torch.arange(many, device=x.device), last[:, None])  # blocks [sequences, many]
    pos = torch.minimum(at[:, :, None] * block + torch.arange(block, device=x.device), end[:, None, None] - 1)
    new = (pos >= start[:, None, None])[:, :, None, :, None]
    seq = torch.arange(x.shape[0], device=x.device)[:, None, None]
    rows = x.permute(0, 2, 1, 3)[seq, (pos - start[:, None, None]).clamp(min=0)].float().permute(0, 1, 3, 2, 4)
    on = st["table"].gather(1, (pos // page).flatten(1)).view(pos.shape).long()  # pages [sequences, many, block]
    held = pages.view(torch.uint8)[on, :, pos % page].view(_F8).float().permute(0, 1, 3, 2, 4)
    top = torch.where(new & torch.isfinite(rows), rows.abs(), 0.0).amax((3, 4))  # [sequences, many, kv_heads]
    in_page = (pos[:, :, 0] % page) // block
    old = torch.where((at * block < start[:, None])[:, :, None], scales[on[:, :, 0], :, in_page], 0.0)
    scale = torch.maximum(_scale_for(top), old)
    values = torch.where(new, rows * (1 / scale)[..., None, None], held * (old / scale)[..., None, None])
    values = _to_e4m3(values).view(torch.uint8).permute(0, 1, 3, 2, 4)
    pages.view(torch.uint8)[on, :, pos % page] = values
    scales[on[:, :, 0], :, in_page] = scale


def _read(pages, scales, st):
    """Rows behind a sequence's count are zeros."""
    case = st["case"]
    i = torch.arange(case["rows"], device=pages.device)[None, :]
    there = i < st["counts"][:, None]
    pos = torch.where(there, st["start"][:, None] + i, 0).long()
    on = st["table"].gather(1, pos // case["page"]).clamp(min=0).long()
    x = pages.view(torch.uint8)[on, :, pos % case["page"]].view(_F8).float()
    x = x * scales[on, :, pos % case["page"] // case["block"]][..., None]
    return torch.where(there[:, :, None, None], x, 0.0).permute(0, 2, 1, 3).to(_TYPES[case["dtype"]])


def _copy(pages, scales, st):
    src, dst, rows = st["moves"].long().unbind(1)
    block = st["case"]["block"]
    values, row = pages.view(torch.uint8), torch.arange(st["case"]["page"], device=pages.device)
    keep = (row[None, :] >= rows[:, None])[:, None, :, None]
    values[dst] = torch.where(keep, values[dst], values[src])
    keep = (row[None, ::block] >= rows[:, None])[:, None, :]
    scales[dst] = torch.where(keep, scales[dst], scales[src])


def run(state):
    op, st = state["case"]["op"], state
    cache = st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"]
    if own:
        import flashattention_backward_gb300 as fa

        if op == "decode":
            return fa.attention_decode_e4m3(st["q"], *cache, st["table"], st["lengths"], st["scale"])
        if op == "read":
            return fa.cache_read_e4m3(*cache, st["table"], st["case"]["rows"], st["start"], st["counts"],
                                      dtype=_TYPES[st["case"]["dtype"]])
        if op == "append":
            fa.cache_append_e4m3(st["k"], st["v"], *cache, st["table"], st["start"], st["counts"])
        else:
            fa.cache_copy_pages_e4m3(*cache, st["moves"])
    else:
        if op == "decode":
            return _decode(st)
        if op == "read":
            return _read(st["k_pages"], st["k_scales"], st), _read(st["v_pages"], st["v_scales"], st)
        if op == "append":
            _append_to(st["k"], st["k_pages"], st["k_scales"], st)
            _append_to(st["v"], st["v_pages"], st["v_scales"], st)
        else:
            _copy(st["k_pages"], st["k_scales"], st)
            _copy(st["v_pages"], st["v_scales"], st)
    return cache


def _sequence(st, which, s, n):
    """Rows 0 ... n - 1 of a sequence in 64 bits, [kv_heads, n, d]."""
    case = st["case"]
    ids = st["table"][s, : -(-n // case["page"])].long()
    x = st[which + "_pages"].view(torch.uint8)[ids].view(_F8).double()
    pages, hk, page, d = x.shape
    by_block = x.view(pages, hk, page // case["block"], case["block"], d) * st[which + "_scales"][ids].double()[..., None, None]
    return by_block.view(pages, hk, page, d).transpose(0, 1).reshape(hk, pages * page, d)[:, :n]


def _nearest(x):
    """64-bit numbers to the nearest of 4 significant bits and exponents from -6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(st, which):
    """The pool's stored values and scales after the rows are in it, block by block of each sequence's table row."""
    case = st["case"]
    page, block, hk, d = case["page"], case["block"], case["kv_heads"], case["dim"]
    values, scales = st[which + "_pages"].float().double(), st[which + "_scales"].double()
    for s, (start, count) in enumerate(zip(st["start"].tolist(), st["counts"].tolist())):
        b0, b1 = start // block, -(-(start + count) // block)
        blocks = torch.arange(b0, b1, device=_DEV)
        ids, rest = st["table"][s].long()[blocks * block // page], blocks % (page // block)
        by_block = values.view(-1, hk, page // block, block, d)
        held, old = by_block[ids, :, rest], scales[ids, :, rest]  # [blocks, kv_heads, block, d], [blocks, kv_heads]
        rows = torch.zeros((b1 - b0) * block, hk, d, dtype=torch.float64, device=_DEV)
        rows[start - b0 * block: start - b0 * block + count] = st[which][s, :, :count].double().transpose(0, 1)
        rows = rows.view(b1 - b0, block, hk, d).transpose(1, 2)
        at = (blocks[:, None] * block + torch.arange(block, device=_DEV))[:, None, :, None]
        # a logarithm of a power of two may be off by its last bit, and no other value of 32 bits is as near to one as 1e-9
        need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((2, 3)) / _TOP) - 1e-9).clamp(min=-126))
        scale = torch.where((blocks * block < start)[:, None], torch.maximum(old, need), need)
        by = scale[..., None, None]
        stored = torch.where(at < start, _nearest(held * old[..., None, None] / by), _nearest(rows / by))
        by_block[ids, :, rest] = torch.where(at < start + count, stored, held)
        scales[ids, :, rest] = scale
    return values, scales


def exact(case, seed):
    """The operators sequence by sequence in 64 bits.  Copied pages are moved, not computed."""
    if case["op"] == "copy":
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        (kv, ks), (vv, vs) = _exact_append(st, "k"), _exact_append(st, "v")
        return kv, vv, ks, vs
    if case["op"] == "read":
        got = []
        for which in "kv":
            x = torch.zeros(case["batch"], case["kv_heads"], case["rows"], case["dim"], dtype=torch.float64, device=_DEV)
            for s, n in enumerate(st["counts"].tolist()):
                x[s, :, :n] = _sequence(st, which, s, case["skip"] + n)[:, case["skip"]:]
            got.append(x)
        return tuple(got)
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(case["batch"], case["heads"], 1, case["dim"], dtype=torch.float64, device=_DEV)
    lse = torch.full((case["batch"], case["heads"], 1), math.inf, dtype=torch.float64, device=_DEV)
    for b, n in enumerate(st["lengths"].tolist()):
        if n == 0:
            continue
        keys, values = _sequence(st, "k", b, n), _sequence(st, "v", b, n)
        q = st["q"][b, :, 0].double().view(case["kv_heads"], group, case["dim"])
        scores = torch.einsum("ghd,gnd->ghn", q, keys) * st["scale"]
        top = torch.logsumexp(scores, 2)
        out[b, :, 0] = torch.einsum("ghn,gnd->ghd", torch.exp(scores - top[..., None]), values).reshape(-1, case["dim"])
        lse[b, :, 0] = top.reshape(-1)
    return out, lse
