"""Measured cases of the paged key-value cache: the attention of one new token
over it, the rows written into it, and the pages that are forked, freed and
compacted.

A cache is two pools, ``k_pages`` and ``v_pages`` of shape
[pages, kv_heads, page_rows, d].  ``page_table`` (int32 [sequences, columns])
says which page holds rows c * page_rows ... of a sequence, ``lengths`` (int32)
how many rows it has, and ``refs`` (int32 [pages]) how many table entries name
a page.  Entries behind a sequence's pages are -1.

``run`` computes every operator in its plain form (elementary torch operations
in 32 bits, rounded once) or, with ``own``, through this repository's calls.
"""

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
_DEV = "cuda"


def listed():
    return [
        # One answer's first tokens: almost nothing to read, the call's own latency counts.
        dict(name="decode_first_tokens", op="decode", batch=1, heads=32, kv_heads=32, dim=64, longest=48,
             spread="equal", page=16, dtype="bf16", mix=1),
        # A batch of short dialogues, a key-value head for each query head, lengths from nothing to 2048.
        dict(name="decode_dialogues", op="decode", batch=32, heads=32, kv_heads=32, dim=64, longest=2048,
             spread="ragged", page=16, dtype="bf16", mix=2),
        # A full serving batch, four query heads to a key-value head: the largest cache.
        dict(name="decode_serving_batch", op="decode", batch=64, heads=32, kv_heads=8, dim=128, longest=8192,
             spread="ragged", page=64, dtype="bf16", mix=3),
        # One long document: a single sequence has to fill the whole GPU.
        dict(name="decode_long_document", op="decode", batch=1, heads=8, kv_heads=8, dim=128, longest=32768,
             spread="equal", page=256, dtype="bf16", mix=4),
        # All sixteen query heads on one key-value head, and pages of an odd number of rows.
        dict(name="decode_one_kv_head", op="decode", batch=4, heads=16, kv_heads=1, dim=128, longest=4000,
             spread="ragged", page=13, dtype="bf16", mix=5),
        # The widest head dim.
        dict(name="decode_wide_heads", op="decode", batch=4, heads=16, kv_heads=16, dim=256, longest=8192,
             spread="equal", page=32, dtype="bf16", mix=6),
        # A cache in full precision, as for checking a model's answers.
        dict(name="decode_fp32", op="decode", batch=8, heads=8, kv_heads=2, dim=96, longest=4000,
             spread="ragged", page=16, dtype="fp32", mix=7),
        # The step of a serving batch: one new row a sequence.
        dict(name="append_step", op="append", batch=64, kv_heads=8, dim=128, rows=1, held=4000, spread="equal",
             page=16, layout="bhnd", dtype="bf16", mix=8),
        # Prompts that have just been computed go into their pages.
        dict(name="append_prompts", op="append", batch=4, kv_heads=16, dim=128, rows=4000, held=0, spread="ragged",
             page=16, layout="bnhd", dtype="bf16", mix=9),
        # Four samples from one prompt: each takes its pages, gets its own last page, one row, and is dropped.
        dict(name="fork_samples", op="fork", live=1, forks=4, kv_heads=32, dim=64, longest=300, page=16,
             dtype="bf16", mix=10),
        # A search that branches every sequence of a batch seven times.
        dict(name="fork_search", op="fork", live=32, forks=224, kv_heads=8, dim=128, longest=4000, page=64,
             dtype="bf16", mix=11),
        # Half of a pool is free, in scattered places: what lives moves to the front.
        dict(name="compact_pool", op="compact", pages=8192, sequences=64, columns=64, kv_heads=8, dim=128, page=16,
             dtype="bf16", mix=12),
    ]


def _between(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choices(["decode", "append", "fork", "compact"], [12, 3, 3, 2])[0]
    dtype = rng.choices(["bf16", "fp32"], [4, 1])[0]
    dim = rng.choice([32, 64, 96, 128, 256] if dtype == "bf16" else [16, 32, 64, 96, 128, 256])
    page = rng.choice([1, 8, 13, 16, 16, 32, 48, 64, 100, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    mix = rng.randrange(1 << 30)
    row = kv_heads * dim * _BYTES[dtype]
    if op == "decode":
        group = rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16, 20, 32])
        longest = _between(rng, 1, 32768)
        most = max(1, (1 << 30) // (2 * row * longest))
        return dict(op=op, batch=_between(rng, 1, min(64, most)), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    longest=longest, spread=rng.choice(["equal", "ragged", "ragged"]), page=page, dtype=dtype, mix=mix)
    if op == "append":
        rows = rng.choice([1, 1, _between(rng, 1, 4000)])
        most = max(1, (1 << 27) // (2 * row * rows))
        return dict(op=op, batch=_between(rng, 1, min(64, most)), kv_heads=kv_heads, dim=dim, rows=rows,
                    held=_between(rng, 1, 2000) - 1, spread=rng.choice(["equal", "ragged"]), page=page,
                    layout=rng.choice(["bhnd", "bnhd"]), dtype=dtype, mix=mix)
    if op == "fork":
        live = _between(rng, 1, 32)
        longest = _between(rng, 1, max(1, min(4000, (1 << 28) // (row * live))))
        most = max(1, (1 << 27) // (row * page))
        return dict(op=op, live=live, forks=_between(rng, 1, min(224, most)), kv_heads=kv_heads, dim=dim,
                    longest=longest, page=page, dtype=dtype, mix=mix)
    most = max(16, min(8192, (1 << 28) // (row * page)))
    pages = _between(rng, 16, most)
    sequences = _between(rng, 1, min(64, pages // 2))
    columns = max(1, int(pages * rng.uniform(0.2, 0.9)) // sequences)
    return dict(op=op, pages=pages, sequences=sequences, columns=columns, kv_heads=kv_heads, dim=dim, page=page,
                dtype=dtype, mix=mix)


def _amounts(mix, count, longest, spread):
    """Rows of each sequence.  Ragged: the first has them all, every eighth is an empty slot, the others lie between."""
    if spread == "equal":
        return [longest] * count
    rng = random.Random(mix)
    return [longest if i == 0 else 0 if i % 8 == 7 else rng.randint(1, longest) for i in range(count)]


def _tails(case):
    return _amounts(case["mix"], case["live"], case["longest"], "ragged")


def work(case):
    es = _BYTES[case["dtype"]]
    row = case["kv_heads"] * case["dim"] * es  # a row of one pool, all its heads
    page = case["page"]
    if case["op"] == "decode":
        lens = _amounts(case["mix"], case["batch"], case["longest"], case["spread"])
        vec = case["batch"] * case["heads"] * case["dim"]
        table = sum(-(-n // page) for n in lens)
        return {"bytes": 2 * row * sum(lens) + 2 * vec * es + 4 * case["batch"] * (case["heads"] + 1) + 4 * table,
                "flops": 4 * case["heads"] * case["dim"] * sum(lens)}
    if case["op"] == "append":
        rows = sum(max(1, n) for n in _amounts(case["mix"], case["batch"], case["rows"], case["spread"]))
        return {"bytes": 4 * row * rows + 8 * case["batch"] + 4 * (rows // page + case["batch"]), "flops": 0}
    if case["op"] == "fork":
        lens = _tails(case)
        of = [lens[i % case["live"]] for i in range(case["forks"])]
        # the rows of the last pages, the new rows, and the entries of the tables and of refs
        moved = sum(n % page for n in of) + case["forks"]
        return {"bytes": 4 * row * moved + 4 * 6 * sum(-(-n // page) for n in of) + 4 * 8 * case["forks"], "flops": 0}
    live = case["sequences"] * case["columns"]
    moved = live * (case["pages"] - live) / case["pages"]
    return {"bytes": 4 * row * page * moved + 4 * (2 * case["pages"] + 2 * live) + 12 * moved, "flops": 0}


def _rand(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=_DEV, dtype=_TYPES[dtype])


def _table(gen, lens, columns, page, pages):
    """A table of `columns` columns whose sequences hold pages in no order, and how often each page is named."""
    held = torch.tensor([-(-n // page) for n in lens], device=_DEV)
    mine = torch.arange(columns, device=_DEV)[None, :] < held[:, None]
    order = torch.randperm(pages, generator=gen, device=_DEV)[: int(mine.sum())].int()
    table = torch.full((len(lens), columns), -1, dtype=torch.int32, device=_DEV)
    table[mine] = order
    refs = torch.zeros(pages, dtype=torch.int32, device=_DEV)
    refs[order.long()] = 1
    return table, refs


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(int(seed) * 1000003 + case["mix"] % 1000003)
    page, hk, d, dt = case["page"], case["kv_heads"], case["dim"], case["dtype"]
    ints = dict(dtype=torch.int32, device=_DEV)
    st = {"case": case, "page": page, "scale": d ** -0.5}
    if case["op"] == "decode":
        lens = _amounts(case["mix"], case["batch"], case["longest"], case["spread"])
        held = sum(-(-n // page) for n in lens)
        pages = held + held // 8 + 1
        st["table"], st["refs"] = _table(gen, lens, -(-case["longest"] // page), page, pages)
        st["lengths"] = torch.tensor(lens, **ints)
        st["q"] = _rand(gen, (case["batch"], case["heads"], 1, d), dt)
    elif case["op"] == "append":
        held = case["held"]
        rows = [max(1, n) for n in _amounts(case["mix"], case["batch"], case["rows"], case["spread"])]
        full = [held + n for n in rows]
        pages = sum(-(-n // page) for n in full) + 1
        st["table"], st["refs"] = _table(gen, full, -(-max(full) // page), page, pages)
        st["start"] = torch.full((case["batch"],), held, **ints)
        st["counts"] = torch.tensor(rows, **ints)
        b, n = case["batch"], case["rows"]
        if case["layout"] == "bhnd":
            st["k"], st["v"] = (_rand(gen, (b, hk, n, d), dt) for _ in range(2))
        else:
            st["k"], st["v"] = (_rand(gen, (b, n, hk, d), dt).permute(0, 2, 1, 3) for _ in range(2))
    elif case["op"] == "fork":
        live, forks = case["live"], case["forks"]
        lens = _tails(case) + [0] * forks
        pages = sum(-(-n // page) for n in lens) + 2 * forks
        st["table"], st["refs"] = _table(gen, lens, -(-(case["longest"] + 1) // page), page, pages)
        st["lengths"] = torch.tensor(lens, **ints)
        st["src"] = torch.arange(forks, **ints) % live
        st["dst"] = torch.arange(forks, **ints) + live
        st["new"] = torch.tensor([0] * live + [1] * forks, **ints)
        st["k"], st["v"] = (_rand(gen, (live + forks, hk, 1, d), dt) for _ in range(2))
    else:
        pages, s, columns = case["pages"], case["sequences"], case["columns"]
        lens = [columns * page] * s
        st["table"], st["refs"] = _table(gen, lens, columns, page, pages)
        st["lengths"] = torch.tensor(lens, **ints)
        st["table_out"], st["refs_out"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
    st["k_pages"], st["v_pages"] = (_rand(gen, (pages, hk, page, d), dt) for _ in range(2))
    return st


def _decode(q, k_pages, v_pages, table, lengths, scale):
    b, heads, _, d = q.shape
    hk, page = k_pages.shape[1:3]
    n = table.shape[1] * page
    at = table.clamp(min=0).long()
    seen = (torch.arange(n, device=q.device)[None, :] < lengths[:, None])[:, None, None, :]
    k = k_pages[at].permute(0, 2, 1, 3, 4).reshape(b, hk, n, d).float()
    s = torch.where(seen, q.float().view(b, hk, heads // hk, d) @ k.transpose(2, 3) * scale, -math.inf)
    del k
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    z = p.sum(3, keepdim=True)
    v = v_pages[at].permute(0, 2, 1, 3, 4).reshape(b, hk, n, d).float()
    v = torch.where(seen.transpose(2, 3), v, 0.0)
    o = torch.where(z > 0, p @ v / z, 0.0)
    lse = torch.where(z > 0, m + torch.log(z), math.inf)
    return o.reshape(b, heads, 1, d).to(q.dtype), lse.reshape(b, heads, 1)


def _append(k, v, k_pages, v_pages, table, start, counts, page):
    # rows behind a sequence's count are written as its last row once more: the same values to the same place
    i = torch.minimum(torch.arange(k.shape[2], device=k.device)[None, :], counts[:, None].long() - 1)
    at = start[:, None].long() + i
    pages = table.gather(1, at // page).long()
    pick = i[:, :, None, None].expand(-1, -1, k.shape[1], k.shape[3])
    k_pages[pages, :, at % page] = k.permute(0, 2, 1, 3).gather(1, pick)
    v_pages[pages, :, at % page] = v.permute(0, 2, 1, 3).gather(1, pick)


def _copy(k_pages, v_pages, moves):
    src, dst, rows = moves[moves[:, 0] >= 0].long().unbind(1)
    keep = (torch.arange(k_pages.shape[2], device=src.device)[None, :] >= rows[:, None])[:, None, :, None]
    k_pages[dst] = torch.where(keep, k_pages[dst], k_pages[src])
    v_pages[dst] = torch.where(keep, v_pages[dst], v_pages[src])


def _lowest_free(refs):
    return torch.argsort((refs > 0).int(), stable=True)


def _mine(lengths, table, page):
    held = (lengths.long() + page - 1) // page
    return torch.arange(table.shape[1], device=table.device)[None, :] < held[:, None]


def _fork(table, lengths, refs, src, dst, page):
    src, dst = src.long(), dst.long()
    n = lengths[src]
    tail = (n % page) > 0
    new = _lowest_free(refs)[torch.cumsum(tail, 0) - tail.long()]
    mine = _mine(n, table, page)
    last = (n.long() // page).clamp(max=table.shape[1] - 1)
    old = table[src].gather(1, last[:, None])[:, 0]
    moves = torch.where(tail[:, None], torch.stack([old.long(), new, (n % page).long()], 1), -1).int()
    rows = torch.where(mine, table[src], -1)
    is_tail = tail[:, None] & (torch.arange(table.shape[1], device=table.device)[None, :] == last[:, None])
    rows = torch.where(is_tail, new[:, None].int(), rows)
    refs.index_add_(0, rows.clamp(min=0).long().flatten(), mine.int().flatten())
    table[dst] = rows
    lengths[dst] = n
    return moves


def _extend_by_one(table, lengths, refs, new, page):
    """At most one row a sequence, so at most one page."""
    start = lengths.clone()
    takes = ((start + new + page - 1) // page) > ((start + page - 1) // page)
    got = _lowest_free(refs)[torch.cumsum(takes, 0) - takes.long()]
    column = (start.long() // page).clamp(max=table.shape[1] - 1)[:, None]
    table.scatter_(1, column, torch.where(takes[:, None], got[:, None].int(), table.gather(1, column)))
    refs.index_add_(0, got, takes.int())
    lengths += new
    return start


def _free(table, lengths, refs, gone, page):
    gone = gone.long()
    mine = _mine(lengths[gone], table, page)
    refs.index_add_(0, table[gone].clamp(min=0).long().flatten(), -mine.int().flatten())
    table[gone] = -1
    lengths[gone] = 0


def _compact(table, lengths, refs, table_out, refs_out, page):
    pages = refs.shape[0]
    ids = torch.arange(pages, device=refs.device)
    live = refs > 0
    n_live = live.sum()
    mover, hole = live & (ids >= n_live), ~live & (ids < n_live)
    count = mover.sum()
    movers = torch.argsort((~mover).int(), stable=True)
    holes = torch.argsort((~hole).int(), stable=True)
    goes = ids < count
    to = ids.scatter(0, movers, torch.where(goes, holes, movers))
    moves = torch.stack([movers, holes, torch.full_like(ids, page)], 1)
    moves = torch.where(goes[:, None], moves, -1)[: pages // 2].int()
    table_out.copy_(torch.where(_mine(lengths, table, page), to[table.clamp(min=0).long()].int(), -1))
    refs_out.zero_().index_add_(0, to, torch.where(live, refs, 0))
    return moves, count.int().reshape(1)


def run(state):
    op, st, page = state["case"]["op"], state, state["page"]
    if own:
        import flashattention_backward_gb300 as fa

        if op == "decode":
            return fa.attention_decode(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lengths"], st["scale"])
        if op == "append":
            fa.cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["start"], st["counts"])
            return st["k_pages"], st["v_pages"]
        if op == "fork":
            moves = fa.pages_fork(st["table"], st["lengths"], st["refs"], st["src"], st["dst"], page)
            fa.cache_copy_pages(st["k_pages"], st["v_pages"], moves)
            start = fa.pages_extend(st["table"], st["lengths"], st["refs"], st["new"], page)
            fa.cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], start, st["new"])
            fa.pages_free(st["table"], st["lengths"], st["refs"], st["dst"], page)
        else:
            moves, count = fa.pages_compact(st["table"], st["lengths"], st["refs"], page,
                                            out=(st["table_out"], st["refs_out"]))
            fa.cache_copy_pages(st["k_pages"], st["v_pages"], moves, count)
    else:
        if op == "decode":
            return _decode(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lengths"], st["scale"])
        if op == "append":
            _append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["start"], st["counts"], page)
            return st["k_pages"], st["v_pages"]
        if op == "fork":
            moves = _fork(st["table"], st["lengths"], st["refs"], st["src"], st["dst"], page)
            _copy(st["k_pages"], st["v_pages"], moves)
            start = _extend_by_one(st["table"], st["lengths"], st["refs"], st["new"], page)
            live = st["case"]["live"]
            _append(st["k"][live:], st["v"][live:], st["k_pages"], st["v_pages"], st["table"][live:], start[live:],
                    st["new"][live:], page)
            _free(st["table"], st["lengths"], st["refs"], st["dst"], page)
        else:
            moves, count = _compact(st["table"], st["lengths"], st["refs"], st["table_out"], st["refs_out"], page)
            _copy(st["k_pages"], st["v_pages"], moves)
    if op == "fork":
        return moves, start, st["table"], st["lengths"], st["refs"], st["k_pages"], st["v_pages"]
    return moves, count, st["table_out"], st["refs_out"], st["k_pages"], st["v_pages"]


def exact(case, seed):
    """The attention of one token, sequence by sequence in 64 bits.  The other operators move values and compute none."""
    if case["op"] != "decode":
        return None
    st = prepare(case, seed)
    page, group = case["page"], case["heads"] // case["kv_heads"]
    out = torch.zeros(case["batch"], case["heads"], 1, case["dim"], dtype=torch.float64, device=_DEV)
    lse = torch.full((case["batch"], case["heads"], 1), math.inf, dtype=torch.float64, device=_DEV)
    for b, n in enumerate(st["lengths"].tolist()):
        if n == 0:
            continue
        ids = st["table"][b, : -(-n // page)].long()
        for g in range(case["kv_heads"]):
            keys = st["k_pages"][ids, g].reshape(-1, case["dim"])[:n].double()
            values = st["v_pages"][ids, g].reshape(-1, case["dim"])[:n].double()
            mine = slice(g * group, (g + 1) * group)
            scores = torch.einsum("hd,nd->hn", st["q"][b, mine, 0].double(), keys) * st["scale"]
            lse[b, mine, 0] = torch.logsumexp(scores, 1)
            weights = torch.exp(scores - lse[b, mine])
            out[b, mine, 0] = torch.einsum("hn,nd->hd", weights, values)
    return out, lse
