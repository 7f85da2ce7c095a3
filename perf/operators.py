"""Workloads of the paged-cache operators: what is called, on what inputs, and what it has to do.

The operators carry one decode step of sparse attention next to the prefill logits: new key and value
rows are quantised into paged e4m3 caches (``cache_write``), packed back for a prompt chunk
(``cache_read``), scored for the newest tokens straight from the pages (``logits_paged``) and attended
to, all of them or the selected ones (``attention_paged``).

``own`` false computes an operator from elementary torch operations in 32 bits, rounded once at the end;
``own`` true calls the library.  Both take the same state from ``prepare``.

A paged cache is ``data [pages, page, heads, dim]`` with, for e4m3, ``scale [pages, page, heads]``: a row's
values are data * scale.  ``table[b, i]`` is the page that holds positions [i * page, (i + 1) * page) of
sequence b; an id outside [0, pages) is a page that is not there.
"""
import math

import torch

own = False

INDEX_HEADS = 32   # the indexer's heads and width, as the prefill logits have them
INDEX_DIM = 128
E4M3_MAX = 448.0
TINY = 1e-30       # the least row maximum that a scale is made from
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": F8}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 32 running requests: a key and a value row of 8 heads each, sliced out of
        # the fused projection's output; some slots are the padding of a captured batch
        {"name": "write_step", "op": "write", "tokens": 32, "heads": 8, "q_heads": 32, "dim": 128, "page": 64,
         "dtype": "bf16", "pair": True, "fused": True, "step": True},
        # a whole prompt chunk entering the same caches
        {"name": "write_prompt", "op": "write", "tokens": 16384, "heads": 8, "q_heads": 32, "dim": 128, "page": 64,
         "dtype": "bf16", "pair": True, "fused": True, "step": False},
        # the indexer's keys of four requests, packed as the prefill logits take them (e4m3 and scales)
        {"name": "read_keys", "op": "read", "rows": 4, "heads": 1, "dim": 128, "page": 64, "lo": 7001, "hi": 8192,
         "empty": 0, "out": "e4m3"},
        # cached keys of an eight-head layer, read back in 16 bits for a chunk's own attention
        {"name": "read_values", "op": "read", "rows": 9, "heads": 8, "dim": 128, "page": 64, "lo": 513, "hi": 16385,
         "empty": 1, "out": "bf16"},
        # a chat turn: one request, a short cache, where latency is all
        {"name": "logits_short", "op": "logits", "rows": 1, "tokens": 1, "page": 64, "lo": 4096, "hi": 4096, "empty": 0},
        # one request at the long-context workload's length
        {"name": "logits_long", "op": "logits", "rows": 1, "tokens": 1, "page": 64, "lo": 131072, "hi": 131072, "empty": 0},
        # a serving batch with a second, drafted token for each request; ragged and odd lengths
        {"name": "logits_batch", "op": "logits", "rows": 64, "tokens": 2, "page": 64, "lo": 129, "hi": 32767, "empty": 1},
        # one request, grouped heads, an odd short cache: latency again
        {"name": "attend_short", "op": "attend", "rows": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "lo": 1021, "hi": 1021, "empty": 0, "select": 0, "cache": "e4m3", "dtype": "bf16", "joint": False, "shared": False},
        # one request at the long-context length, one shared key head: all the parallelism is in the cache's length
        {"name": "attend_long", "op": "attend", "rows": 1, "q_heads": 32, "kv_heads": 1, "dim": 128, "page": 64,
         "lo": 131072, "hi": 131072, "empty": 0, "select": 0, "cache": "e4m3", "dtype": "bf16", "joint": False, "shared": False},
        # a full serving batch of ragged requests over the quantised cache: the largest
        {"name": "attend_batch", "op": "attend", "rows": 64, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "lo": 257, "hi": 20001, "empty": 1, "select": 0, "cache": "e4m3", "dtype": "bf16", "joint": False, "shared": False},
        # the same kind of batch over a 16-bit cache that keeps keys and values in one tensor, odd page size
        {"name": "attend_16bit", "op": "attend", "rows": 16, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 48,
         "lo": 1000, "hi": 16385, "empty": 0, "select": 0, "cache": "bf16", "dtype": "bf16", "joint": True, "shared": False},
        # sparse attention: every request attends to the 2048 entries that its top-k selected out of 32768
        {"name": "attend_selected", "op": "attend", "rows": 64, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 64,
         "lo": 32768, "hi": 32768, "empty": 0, "select": 2048, "cache": "e4m3", "dtype": "bf16", "joint": False,
         "shared": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """A size spread over its logarithm; most are no round number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.75 or n < 64 else n // 64 * 64


def draw(rng):
    op = rng.choice(["write", "read", "logits", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 48, 64, 64, 64, 100, 128])
    dim = rng.choice([64, 128, 128])
    if op == "write":
        heads = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _odd(rng, 1, 16384), "heads": heads, "q_heads": heads * rng.choice([1, 4, 8]), "dim": dim,
                "page": page, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "pair": rng.random() < 0.7,
                "fused": rng.random() < 0.7, "step": rng.random() < 0.4}
    if op == "read":
        rows = _log(rng, 1, 64)
        hi = _odd(rng, 1, max(1, min(32768, 131072 // rows)))
        return {"op": op, "rows": rows, "heads": rng.choice([1, 1, 2, 4, 8]), "dim": dim, "page": page,
                "lo": rng.randint(1, hi), "hi": hi, "empty": rng.choice([0, 0, 1]) if rows > 1 else 0,
                "out": rng.choice(["e4m3", "bf16", "f16", "f32"])}
    if op == "logits":
        rows, tokens = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4])
        hi = _odd(rng, 64, max(64, min(131072, (1 << 22) // (rows * tokens))))
        return {"op": op, "rows": rows, "tokens": tokens, "page": page, "lo": rng.randint(max(1, hi // 8), hi), "hi": hi,
                "empty": rng.choice([0, 0, 1]) if rows > 1 else 0}
    rows, kv_heads, group = _log(rng, 1, 128), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 4, 8, 8, 16, 32])
    cache = rng.choice(["e4m3", "e4m3", "e4m3", "bf16", "f16"])
    select = rng.choice([0, 0, 512, 2048, _log(rng, 17, 2048)])
    # at most about a gigabyte of cache
    most = (1 << 30) // (rows * kv_heads * 2 * (dim * SIZES[cache] + (4 if cache == "e4m3" else 0)))
    hi = _odd(rng, 1, max(1, min(131072, most)))
    return {"op": op, "rows": rows, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page,
            "lo": rng.randint(max(1, hi // 16), hi), "hi": hi, "empty": rng.choice([0, 0, 1]) if rows > 1 else 0,
            "select": select, "cache": cache, "dtype": cache if cache != "e4m3" else rng.choice(["bf16", "bf16", "f16"]),
            "joint": rng.random() < 0.3, "shared": select > 0 and rng.random() < 0.4}


def _lens(case):
    """The sequences' lengths: an even spread of [lo, hi], and the empty ones."""
    n = case["rows"]
    if case.get("shared"):
        return [case["hi"]] * n
    lens = [case["hi"] - (case["hi"] - case["lo"]) * i // max(1, n - 1) for i in range(n)]
    for i in range(case["empty"]):
        lens[-1 - i] = 0
    return lens


# ------------------------------------------------------------------------------------ inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _cache(g, pages, page, heads, dim, kind):
    """A filled cache: rows of unequal size, channels of unequal spread, as keys and values have them."""
    spread = torch.exp(0.5 * _randn(g, dim)).to(torch.bfloat16)
    x = _randn(g, pages, page, heads, dim, dtype=torch.bfloat16) * spread
    if kind != "e4m3":
        return x.to(TYPES[kind]), None
    amax = x.abs().amax(-1).float().clamp_(min=TINY)
    data = x.mul_((E4M3_MAX / amax).to(torch.bfloat16).unsqueeze(-1)).clamp_(-E4M3_MAX, E4M3_MAX).to(F8)
    return data, amax * torch.exp(0.3 * _randn(g, pages, page, heads)) / E4M3_MAX


def _pages(g, case):
    """(table [rows, most pages] int32, lens [rows] int32, pages): every sequence's pages lie anywhere in the pool."""
    page, rows = case["page"], case["rows"]
    if case.get("shared"):
        need = -(-case["hi"] // page)
        one = torch.randperm(need + 3, generator=g, device="cuda")[:need].to(torch.int32)
        lens = torch.full((rows,), case["hi"], dtype=torch.int32, device="cuda")
        return one.unsqueeze(0).expand(rows, need), lens, need + 3
    lens = torch.tensor(_lens(case), device="cuda")[torch.randperm(rows, generator=g, device="cuda")]
    need = (lens + page - 1) // page
    pages = sum(-(-n // page) for n in _lens(case)) + 3
    pool = torch.randperm(pages, generator=g, device="cuda")
    col = torch.arange(-(-case["hi"] // page), device="cuda")
    at = (need.cumsum(0) - need).unsqueeze(1) + col
    table = torch.where(col < need.unsqueeze(1), pool[at.clamp(max=pages - 1)], -1)
    return table.to(torch.int32), lens.to(torch.int32), pages


def prepare(case, seed):
    g = _rng(seed)
    s = {"case": case}
    if case["op"] == "write":
        T, H, D, page = case["tokens"], case["heads"], case["dim"], case["page"]
        pages = -(-T // page) + 5 if not case["step"] else T + 5
        dtype = TYPES[case["dtype"]]
        width = case["q_heads"] if case["fused"] else 0
        qkv = (_randn(g, T, width + 2 * H, D) * torch.exp(0.3 * _randn(g, T, 1, 1))).to(dtype)
        s["k"] = qkv[:, width:width + H]
        s["k_data"], s["k_scale"] = _cache(g, pages, page, H, D, "e4m3")
        if case["pair"]:
            s["v"] = qkv[:, width + H:]
            s["v_data"], s["v_scale"] = _cache(g, pages, page, H, D, "e4m3")
        pool = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        if case["step"]:  # one new row in a page of each request; every 16th slot is padding
            slots = pool[t] * page + torch.randint(page, (T,), generator=g, device="cuda")
            slots = torch.where(t % 16 == 15, -1, slots)
        else:
            slots = pool[t // page] * page + t % page
        s["slots"] = slots.to(torch.int32)
        return s
    s["table"], s["lens"], pages = _pages(g, case)
    if case["op"] == "read":
        s["data"], s["scale"] = _cache(g, pages, case["page"], case["heads"], case["dim"], "e4m3")
        s["starts"] = torch.nn.functional.pad(s["lens"].cumsum(0), (1, 0)).to(torch.int32)
        s["total"] = sum(_lens(case))
    elif case["op"] == "logits":
        B, T = case["rows"], case["tokens"]
        s["data"], s["scale"] = _cache(g, pages, case["page"], 1, INDEX_DIM, "e4m3")
        s["q"] = _randn(g, B, T, INDEX_HEADS, INDEX_DIM).to(F8)
        s["w"] = _randn(g, B, T, INDEX_HEADS) / math.sqrt(INDEX_HEADS * INDEX_DIM)
    else:
        B, D, H = case["rows"], case["dim"], case["kv_heads"]
        s["q"] = _randn(g, B, case["q_heads"], D).to(TYPES[case["dtype"]])
        if case["joint"]:  # keys and values of a page side by side in one tensor
            kv, sc = _cache(g, 2 * pages, case["page"], H, D, case["cache"])
            kv = kv.view(pages, 2, case["page"], H, D)
            s["k_data"], s["v_data"] = kv[:, 0], kv[:, 1]
            sc = sc.view(pages, 2, case["page"], H) if sc is not None else None
            s["k_scale"], s["v_scale"] = (sc[:, 0], sc[:, 1]) if sc is not None else (None, None)
        else:
            s["k_data"], s["k_scale"] = _cache(g, pages, case["page"], H, D, case["cache"])
            s["v_data"], s["v_scale"] = _cache(g, pages, case["page"], H, D, case["cache"])
        s["sm_scale"] = 1.0 / math.sqrt(D)
        s["indices"] = None
        if case["select"]:  # distinct positions in any order, as an unsorted top-k returns them; -1 pads
            n, L = case["select"], s["table"].shape[1] * case["page"]
            x = torch.rand((B, max(n, L)), generator=g, device="cuda")
            x = x.masked_fill_(torch.arange(max(n, L), device="cuda") >= s["lens"].unsqueeze(1), -1.0)
            val, idx = x.topk(n, dim=1, sorted=False)
            s["indices"] = torch.where(val >= 0, idx, -1).to(torch.int32)
    return s


# ------------------------------------------------------------------------------------ plain forms

def _quantise(x):
    """Rows of x as e4m3 values and one scale each, in 32 bits."""
    x = x.float()
    amax = x.abs().amax(-1).clamp(min=TINY)
    y = (x * (torch.full_like(amax, E4M3_MAX) / amax).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(F8), amax * (1.0 / E4M3_MAX)


def _store(slots, x, data, scale):
    pages, page, heads, dim = data.shape
    values, scales = _quantise(x)
    there = (slots >= 0) & (slots < pages * page)
    at = slots[there].long()
    data.view(torch.uint8).view(pages * page, heads, dim)[at] = values.view(torch.uint8)[there]
    scale.view(pages * page, heads)[at] = scales[there]


def _fetch(data, scale, ids, offsets):
    """Rows of a cache at (page, offset), in 32 bits."""
    if scale is None:
        return data[ids, offsets].float()
    return data.view(torch.uint8)[ids, offsets].view(F8).float() * scale[ids, offsets].unsqueeze(-1)


def _locate(table, position, valid, pages, page):
    """(valid, page, offset) of each sequence's positions [rows, n]; what is not there points at the first row."""
    position = torch.where(valid, position, 0)
    ids = table.long().gather(1, position // page)
    valid = valid & (ids >= 0) & (ids < pages)
    return valid, torch.where(valid, ids, 0), torch.where(valid, position % page, 0)


def _read(s):
    data, scale, table, starts, total = s["data"], s["scale"], s["table"], s["starts"], s["total"]
    pages, page, _, _ = data.shape
    row = torch.arange(total, device=data.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    position = row - starts[seq]
    ids = table[seq, position // page].long()
    offsets = position % page
    if s["case"]["out"] == "e4m3":
        return data.view(torch.uint8)[ids, offsets].view(F8), scale[ids, offsets]
    return _fetch(data, scale, ids, offsets).to(TYPES[s["case"]["out"]])


def _logits(s):
    q, w, lens, table = s["q"].float(), s["w"], s["lens"].long(), s["table"]
    B, T, H, D = q.shape
    pages, page, _, _ = s["data"].shape
    L = s["case"]["hi"]
    position = torch.arange(L, device=q.device).expand(B, L)
    valid, ids, offsets = _locate(table, position, position < lens.unsqueeze(1), pages, page)
    keys = s["data"].view(torch.uint8)[ids, offsets, 0].view(F8).float()                       # [B, L, D]
    dots = torch.matmul(q.view(B, T * H, D), keys.transpose(1, 2)).view(B, T, H, L)
    out = (dots.relu_() * w.unsqueeze(-1)).sum(2) * s["scale"][ids, offsets, 0].unsqueeze(1)
    # token t is the (T - t)th newest: it sees the cache up to itself
    end = lens.view(B, 1, 1) - (T - 1 - torch.arange(T, device=q.device).view(1, T, 1))
    seen = (position.unsqueeze(1) < end) & valid.unsqueeze(1)
    return torch.where(seen, out, -math.inf).view(B * T, L)


def _attend(s):
    q, lens, table = s["q"], s["lens"].long(), s["table"]
    B, Hq, D = q.shape
    pages, page, Hk, _ = s["k_data"].shape
    if s["indices"] is None:
        position = torch.arange(table.shape[1] * page, device=q.device).expand(B, -1)
    else:
        position = s["indices"].long()
    valid, ids, offsets = _locate(table, position, (position >= 0) & (position < lens.unsqueeze(1)), pages, page)
    k = _fetch(s["k_data"], s["k_scale"], ids, offsets).permute(0, 2, 3, 1)                     # [B, Hk, D, n]
    x = torch.matmul(q.float().view(B, Hk, Hq // Hk, D), k) * s["sm_scale"]
    del k
    x = x.masked_fill_(~valid.view(B, 1, 1, -1), -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = _fetch(s["v_data"], s["v_scale"], ids, offsets).permute(0, 2, 1, 3)                     # [B, Hk, n, D]
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = top + torch.log(total)
    return out.view(B, Hq, D).to(q.dtype), torch.where(total > 0, lse, -math.inf).view(B, Hq)


# ------------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        import fp8_mqa_logits_02_gb300 as fm
    if case["op"] == "write":
        pair = case["pair"]
        if own:
            if pair:
                fm.cache_write(s["slots"], s["k"], s["k_data"], s["k_scale"], s["v"], s["v_data"], s["v_scale"])
            else:
                fm.cache_write(s["slots"], s["k"], s["k_data"], s["k_scale"])
        else:
            _store(s["slots"], s["k"], s["k_data"], s["k_scale"])
            if pair:
                _store(s["slots"], s["v"], s["v_data"], s["v_scale"])
        out = {"k": s["k_data"], "k_scale": s["k_scale"]}
        return out | ({"v": s["v_data"], "v_scale": s["v_scale"]} if pair else {})
    if case["op"] == "read":
        if own:
            return fm.cache_read(s["data"], s["scale"], s["table"], s["starts"], s["total"], dtype=TYPES[case["out"]])
        return _read(s)
    if case["op"] == "logits":
        if own:
            return fm.logits_paged(s["q"], s["data"], s["scale"], s["w"], s["table"], s["lens"], max_len=case["hi"])
        return _logits(s)
    if own:
        return fm.attention_paged(s["q"], s["k_data"], s["v_data"], s["table"], s["lens"], s["sm_scale"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"], indices=s["indices"], return_lse=True)
    return _attend(s)


def work(case):
    if case["op"] == "write":
        rows = case["tokens"] * case["heads"] * (2 if case["pair"] else 1)
        return {"bytes": rows * (case["dim"] * (SIZES[case["dtype"]] + 1) + 4) + 4 * case["tokens"],
                "flops": 3 * rows * case["dim"]}
    lens = _lens(case)
    total, cols = sum(lens), -(-case["hi"] // case["page"])
    if case["op"] == "read":
        rows = total * case["heads"]
        back = case["dim"] * SIZES[case["out"]] + (4 if case["out"] == "e4m3" else 0)
        return {"bytes": rows * (case["dim"] + 4 + back) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": rows * case["dim"]}
    if case["op"] == "logits":
        rows = case["rows"] * case["tokens"]
        return {"bytes": total * (INDEX_DIM + 4) + rows * (case["hi"] * 4 + INDEX_HEADS * (INDEX_DIM + 4)),
                "flops": 2 * INDEX_HEADS * INDEX_DIM * total * case["tokens"]}
    size, D = SIZES[case["cache"]], case["dim"]
    row = 2 * (D * size + (4 if case["cache"] == "e4m3" else 0)) * case["kv_heads"]
    if case["select"]:
        total = sum(min(n, case["select"]) for n in lens)
    read = min(total, case["hi"]) if case["shared"] else total
    return {"bytes": read * row + case["rows"] * (2 * case["q_heads"] * D * SIZES[case["dtype"]] + 4 * case["q_heads"]
                                                  + 4 * (case["select"] or cols)),
            "flops": 4 * case["q_heads"] * D * total}


# ------------------------------------------------------------------------------------ 64 bits

def _e4m3_64(y):
    """y rounded to the nearest e4m3 value, ties to even, in 64 bits."""
    _, e = torch.frexp(y)                       # |y| in [2^(e-1), 2^e): spacing 2^(e-4), subnormals 2^-9
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(y / step) * step


def _rows_64(data, scale, ids, offsets):
    x = data[ids, offsets].to(torch.float32).double()
    return x if scale is None else x * scale[ids, offsets].double().unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        out = {}
        for name in ("k", "v") if case["pair"] else ("k",):
            data, scale = s[name + "_data"].float().double(), s[name + "_scale"].double()
            pages, page, heads, dim = data.shape
            x = s[name].double()
            amax = x.abs().amax(-1).clamp(min=TINY)
            rows, scales = _e4m3_64(x * E4M3_MAX / amax.unsqueeze(-1)), amax / E4M3_MAX
            keep = torch.nonzero(s["slots"] >= 0).view(-1)
            at = s["slots"][keep].long()
            data.view(-1, heads, dim)[at] = rows[keep]
            scale.view(-1, heads)[at] = scales[keep]
            out[name], out[name + "_scale"] = data, scale
        return out
    lens, table, page = s["lens"].tolist(), s["table"].long(), case["page"]
    if case["op"] == "read":
        rows, scales = [], []
        for b, n in enumerate(lens):
            p = torch.arange(n, device="cuda")
            ids, off = table[b, p // page], p % page
            rows.append(_rows_64(s["data"], None if case["out"] == "e4m3" else s["scale"], ids, off))
            scales.append(s["scale"][ids, off].double())
        return (torch.cat(rows), torch.cat(scales)) if case["out"] == "e4m3" else torch.cat(rows)
    if case["op"] == "logits":
        T, L = case["tokens"], case["hi"]
        out = torch.full((case["rows"], T, L), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            p = torch.arange(n, device="cuda")
            keys = s["data"][table[b, p // page], p % page, 0].float().double()
            by = s["scale"][table[b, p // page], p % page, 0].double()
            for t in range(T):
                end = max(0, n - (T - 1 - t))
                dots = s["q"][b, t].float().double() @ keys[:end].T
                out[b, t, :end] = (dots.clamp(min=0) * s["w"][b, t].double().unsqueeze(1)).sum(0) * by[:end]
        return out.view(case["rows"] * T, L)
    B, Hq, D = s["q"].shape
    Hk = case["kv_heads"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        if s["indices"] is not None:
            p = s["indices"][b].long()
            p = p[p >= 0]
        if not p.numel():
            continue
        ids, off = table[b, p // page], p % page
        k, v = _rows_64(s["k_data"], s["k_scale"], ids, off), _rows_64(s["v_data"], s["v_scale"], ids, off)
        x = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(Hk, Hq // Hk, D), k) * s["sm_scale"]
        lse[b] = torch.logsumexp(x, -1).view(Hq)
        out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(Hq, D)
    return out, lse
