"""Workloads of a serving step's other operators: what is called, on what inputs, and what it has to do.

They stand around the paged caches of ``perf/operators.py``: page tables, slots and positions of a step are made
on the GPU (``pages_update``), queries and keys are normed and rotated head by head (``norm_rotate``), keys and
values go into caches of 4 bits and come back in 16 (``cache_write``, ``cache_read``), and a new token attends to
such a cache (``attention_paged``).

``own`` false computes an operator from elementary torch operations in 32 bits (angles in 64), rounded once at the
end; ``own`` true calls the library.  Both take the same state from ``prepare``.

A 4-bit cache is ``data [pages, page, heads, dim / 2]``, two e2m1 values a byte (the first one low), ``groups
[pages, page, heads, dim / 16]``, an e4m3 scale for each 16 values, and ``scale [pages, page, heads]``: a row's
values are data * group * scale.  ``table[b, i]`` is the page that holds positions [i * page, (i + 1) * page) of
sequence b; an id outside [0, pages) is a page that is not there.
"""
import math

import torch

own = False

TINY = 1e-30       # the least row maximum that a scale is made from
E4M3_MAX, E2M1_MAX = 448.0, 6.0
GROUP = 16
F8, F4 = torch.float8_e4m3fn, torch.float4_e2m1fn_x2
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": F8}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of 256 running requests with a drafted token each; now and then one ends or begins
        {"name": "pages_step", "op": "pages", "rows": 256, "new": 2, "page": 64, "cols": 512, "lo": 257, "hi": 20001},
        # a step that takes in prompts: ragged chunks of 64 requests, 16 thousand tokens
        {"name": "pages_prompt", "op": "pages", "rows": 64, "new": 511, "page": 64, "cols": 512, "lo": 0, "hi": 20001},
        # one decode step of 32 requests: 32 query and 8 key heads, sliced out of the fused projection's output
        {"name": "rotate_step", "op": "rotate", "tokens": 32, "q_heads": 32, "k_heads": 8, "dim": 128, "rotated": 128,
         "dtype": "bf16", "out": "bf16", "norm": True, "interleaved": False, "step": True},
        # a whole prompt chunk through the same layer
        {"name": "rotate_prompt", "op": "rotate", "tokens": 16384, "q_heads": 32, "k_heads": 8, "dim": 128, "rotated": 128,
         "dtype": "bf16", "out": "bf16", "norm": True, "interleaved": False, "step": False},
        # the indexer's queries of a chunk, half of each head rotated, as the prefill logits take them (e4m3 and scales)
        {"name": "rotate_index", "op": "rotate", "tokens": 8192, "q_heads": 32, "k_heads": 0, "dim": 128, "rotated": 64,
         "dtype": "bf16", "out": "e4m3", "norm": True, "interleaved": True, "step": False},
        # four short prompts written into 4-bit caches and read back for their own attention: latency
        {"name": "store_short", "op": "store", "rows": 4, "heads": 8, "dim": 128, "page": 64, "lo": 7, "hi": 33,
         "dtype": "bf16", "out": "bf16"},
        # a chunk of long prompts through the same caches
        {"name": "store_prompt", "op": "store", "rows": 5, "heads": 8, "dim": 128, "page": 64, "lo": 513, "hi": 6001,
         "dtype": "bf16", "out": "bf16"},
        # cached keys of an eight-head layer, read back in 16 bits for a chunk's own attention
        {"name": "read_values", "op": "read", "rows": 9, "heads": 8, "dim": 128, "page": 64, "lo": 513, "hi": 16385,
         "empty": 1, "out": "bf16"},
        # one request, grouped heads, an odd short 4-bit cache: latency again
        {"name": "attend_short", "op": "attend", "rows": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "lo": 1021, "hi": 1021, "empty": 0, "select": 0, "dtype": "bf16", "shared": False},
        # one request at the long-context length, one shared key head: all the parallelism is in the cache's length
        {"name": "attend_long", "op": "attend", "rows": 1, "q_heads": 32, "kv_heads": 1, "dim": 128, "page": 64,
         "lo": 131072, "hi": 131072, "empty": 0, "select": 0, "dtype": "bf16", "shared": False},
        # a full serving batch of ragged requests: the largest
        {"name": "attend_batch", "op": "attend", "rows": 64, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "lo": 257, "hi": 20001, "empty": 1, "select": 0, "dtype": "bf16", "shared": False},
        # sparse attention: every request attends to the 2048 entries that its top-k selected out of 32768
        {"name": "attend_selected", "op": "attend", "rows": 64, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 64,
         "lo": 32768, "hi": 32768, "empty": 0, "select": 2048, "dtype": "bf16", "shared": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """A size spread over its logarithm; most are no round number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.75 or n < 64 else n // 64 * 64


def draw(rng):
    op = rng.choice(["pages", "rotate", "rotate", "store", "read", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 48, 64, 64, 64, 100, 128])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "pages":
        rows = _log(rng, 1, 2048)
        new = rng.choice([1, 1, 2, 4, _odd(rng, 5, max(6, min(4096, 32768 // rows)))])
        cols = _odd(rng, 40, max(41, min(2048, (1 << 18) // rows)))
        hi = rng.randint(0, cols * page - new)
        return {"op": op, "rows": rows, "new": new, "page": page, "cols": cols, "lo": rng.randint(0, hi), "hi": hi}
    if op == "rotate":
        heads = rng.choice([1, 2, 4, 8])
        q_heads = rng.choice([heads, 4 * heads, 8 * heads])
        norm = rng.random() < 0.7
        return {"op": op, "tokens": _odd(rng, 1, 16384 * 40 // (q_heads + heads) if q_heads + heads > 40 else 16384),
                "q_heads": q_heads, "k_heads": rng.choice([0, heads, heads, heads]), "dim": dim,
                "rotated": rng.choice([dim, dim, dim // 2, 32, 48]), "dtype": rng.choice([dtype, dtype, "f32"]),
                "out": "e4m3" if rng.random() < 0.3 else "same", "norm": norm, "interleaved": rng.random() < 0.4,
                "step": rng.random() < 0.4}
    if op == "store":
        rows = _log(rng, 1, 64)
        hi = _odd(rng, 1, max(1, 16384 // rows))
        return {"op": op, "rows": rows, "heads": rng.choice([1, 2, 4, 8]), "dim": dim, "page": page, "lo": rng.randint(1, hi),
                "hi": hi, "dtype": rng.choice([dtype, dtype, "f32"]), "out": dtype}
    if op == "read":
        rows = _log(rng, 1, 64)
        hi = _odd(rng, 1, max(1, min(32768, 131072 // rows)))
        return {"op": op, "rows": rows, "heads": rng.choice([1, 1, 2, 4, 8]), "dim": dim, "page": page,
                "lo": rng.randint(1, hi), "hi": hi, "empty": rng.choice([0, 0, 1]) if rows > 1 else 0,
                "out": rng.choice(["bf16", "f16", "f32"])}
    rows, kv_heads, group = _log(rng, 1, 128), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 4, 8, 8, 16, 32])
    select = rng.choice([0, 0, 512, 2048, _log(rng, 17, 2048)])
    # at most about what the largest listed case reads
    most = (700 << 20) // (rows * kv_heads * 2 * (dim // 2 + dim // GROUP + 4))
    hi = _odd(rng, 1, max(1, min(131072, most)))
    return {"op": op, "rows": rows, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page,
            "lo": rng.randint(max(1, hi // 16), hi), "hi": hi, "empty": rng.choice([0, 0, 1]) if rows > 1 else 0,
            "select": select, "dtype": dtype, "shared": select > 0 and rng.random() < 0.4}


def _lens(case):
    """The sequences' lengths: an even spread of [lo, hi], and the empty ones."""
    n = case["rows"]
    if case.get("shared"):
        return [case["hi"]] * n
    lens = [case["hi"] - (case["hi"] - case["lo"]) * i // max(1, n - 1) for i in range(n)]
    for i in range(case.get("empty", 0)):
        lens[-1 - i] = 0
    return lens


def _news(case):
    """(lengths, change of each): every 16th request ends, every 16th begins with a short prompt, the others get
    new tokens, all of them in a step and a ragged number of a prompt's."""
    lens, news = _lens(case), []
    for i in range(case["rows"]):
        if i % 16 == 5:
            news.append(-lens[i])
        elif i % 16 == 11:
            lens[i] = 0
            news.append(min(33 + i, case["cols"] * case["page"]))
        else:
            news.append(case["new"] if case["new"] < 5 else 1 + (i * 7919 + 13) % (2 * case["new"] - 1))
        news[i] = min(news[i], case["cols"] * case["page"] - lens[i])
    return lens, news


# ------------------------------------------------------------------------------------ inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _cache(g, pages, page, heads, dim):
    """A filled 4-bit cache (data, groups, scale): codes as values about a maximum of 6 have them."""
    # e2m1 codes of a normal spread: magnitudes 0 .. 6 fall off towards the top, signs are even
    codes = torch.randint(0, 256, (pages, page, heads, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
    fewer = torch.randint(0, 256, (pages, page, heads, dim // 2), generator=g, device="cuda", dtype=torch.uint8) | 0xBB
    spread = torch.exp(0.5 * _randn(g, dim // GROUP))
    groups = (100.0 * spread * torch.exp(0.4 * _randn(g, pages, page, heads, dim // GROUP))).clamp_(0, E4M3_MAX).to(F8)
    scale = torch.exp(0.3 * _randn(g, pages, page, heads)) / 256
    return (codes & fewer).view(F4), groups, scale


def _pages_of(g, case):
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
    if case["op"] == "pages":
        page, rows, cols = case["page"], case["rows"], case["cols"]
        lens, news = _news(case)
        mix = torch.randperm(rows, generator=g, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[mix].contiguous()
        s["new"] = torch.tensor(news, dtype=torch.int32, device="cuda")[mix].contiguous()
        s["back"] = -s["new"]
        s["total"] = sum(max(0, n) for n in news) + 3          # three rows of padding
        s["back_total"] = sum(max(0, -n) for n in news)
        have = (s["lens"].long() + page - 1) // page
        pages = sum(-(-n // page) for n in lens)
        grow = sum(-(-max(0, n + m) // page) for n, m in zip(lens, news)) + rows
        pool = torch.randperm(pages + grow, generator=g, device="cuda").to(torch.int32)
        col = torch.arange(cols, device="cuda")
        at = (have.cumsum(0) - have).unsqueeze(1) + col
        s["table"] = torch.where(col < have.unsqueeze(1), pool[at.clamp(max=pages + grow - 1)], -1)
        s["free"] = torch.cat([pool[pages:], torch.full((pages,), -1, dtype=torch.int32, device="cuda")])
        s["n_free"] = torch.full((1,), grow, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "rotate":
        T, Hq, Hk, D = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        dtype = TYPES[case["dtype"]]
        qkv = (_randn(g, T, Hq + 2 * Hk, D) * torch.exp(0.3 * _randn(g, T, 1, 1))).to(dtype)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk] if Hk else None
        first = torch.randint(0, 100000, (T if case["step"] else 1,), generator=g, device="cuda")
        s["positions"] = (first if case["step"] else first + torch.arange(T, device="cuda")).to(torch.int32)
        R = case["rotated"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)).float()
        weight = lambda: torch.exp(0.2 * _randn(g, D)).to(dtype) if case["norm"] else None  # noqa: E731
        s["q_weight"], s["k_weight"] = weight(), weight() if Hk else None
        s["dtype"] = dtype if case["out"] in ("same", case["dtype"]) else TYPES[case["out"]]
        return s
    s["table"], s["lens"], pages = _pages_of(g, case)
    if case["op"] in ("store", "read"):
        H, D, page = case["heads"], case["dim"], case["page"]
        s["starts"] = torch.nn.functional.pad(s["lens"].cumsum(0), (1, 0)).to(torch.int32)
        s["total"] = sum(_lens(case))
        s["k_data"], s["k_groups"], s["k_scale"] = _cache(g, pages, page, H, D)
        if case["op"] == "store":
            s["v_data"], s["v_groups"], s["v_scale"] = _cache(g, pages, page, H, D)
            spread = torch.exp(0.5 * _randn(g, 2 * H, D))
            kv = (_randn(g, s["total"], 2 * H, D) * spread).to(TYPES[case["dtype"]])
            s["k"], s["v"] = kv[:, :H], kv[:, H:]
            row = torch.arange(s["total"], device="cuda")
            seq = torch.searchsorted(s["starts"], row, right=True) - 1
            position = row - s["starts"][seq]
            s["slots"] = (s["table"][seq, position // page] * page + position % page).to(torch.int32)
    else:
        B, D, H = case["rows"], case["dim"], case["kv_heads"]
        s["q"] = _randn(g, B, case["q_heads"], D).to(TYPES[case["dtype"]])
        s["k_data"], s["k_groups"], s["k_scale"] = _cache(g, pages, case["page"], H, D)
        s["v_data"], s["v_groups"], s["v_scale"] = _cache(g, pages, case["page"], H, D)
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

def _update(s, new, total):
    """One step of the page tables: shrinking requests give pages back, then growing ones take theirs."""
    table, lens, free, n_free = s["table"], s["lens"].long(), s["free"], s["n_free"].long()
    new, page = new.long(), s["case"]["page"]
    B, cols = table.shape
    have = (lens + page - 1) // page
    to = (lens + new).clamp(min=0)
    need = (to + page - 1) // page
    fits = to <= cols * page
    take = torch.where((new > 0) & fits, need - have, 0)
    give = torch.where(new < 0, have - need, 0)
    taken, given = torch.nn.functional.pad(take.cumsum(0), (1, 0)), torch.nn.functional.pad(give.cumsum(0), (1, 0))
    most = n_free + given[-1]
    ok = fits & ((take == 0) | (taken[1:] <= most))
    col = torch.arange(cols, device=table.device)
    # the stack of free pages, with what was given back on top
    stack = torch.nn.functional.pad(free, (0, 1))
    back = (col >= need.unsqueeze(1)) & (col < have.unsqueeze(1)) & (new < 0).unsqueeze(1)
    number = n_free + given[:-1].unsqueeze(1) + col - need.unsqueeze(1)
    stack.scatter_(0, torch.where(back, number, free.numel()).view(-1), table.reshape(-1))
    fresh = (col >= have.unsqueeze(1)) & (col < need.unsqueeze(1)) & (ok & (new > 0)).unsqueeze(1)
    number = most - 1 - (taken[:-1].unsqueeze(1) + col - have.unsqueeze(1))
    table.copy_(torch.where(fresh, stack[torch.where(fresh, number, 0)], table))
    left = most - torch.where(ok, take, 0).sum()
    at = torch.arange(free.numel(), device=table.device)
    free.copy_(torch.where((at >= n_free) & (at < left), stack[:-1], free))
    # the new tokens
    starts = torch.nn.functional.pad(new.clamp(min=0).cumsum(0), (1, 0))
    token = torch.arange(total, device=table.device)
    there = token < starts[-1]
    row = torch.where(there, torch.searchsorted(starts, token, right=True) - 1, 0)
    position = torch.where(there, lens[row] + token - starts[row], 0)
    where = torch.where(there & ok[row], table[row, (position // page).clamp(max=cols - 1)].long(), -1)
    slots = torch.where(where >= 0, where * page + position % page, -1)
    s["lens"].copy_(torch.where(ok, to, lens))
    s["n_free"].copy_(left)
    change = torch.where(ok, to - lens, 0)
    return [x.to(torch.int32) for x in (slots, position, row, starts, change)]


def _round_e2m1(y):
    """Magnitudes as e2m1 codes without the sign: to the nearest, ties to the even code, 6 at most."""
    return ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))


def _quantise(x):
    """Rows of x in 4 bits: (bytes, groups, scale), in 32 bits."""
    x = x.float()
    amax = x.abs().amax(-1).clamp(min=TINY)
    parts = x.unflatten(-1, (-1, GROUP))
    top = parts.abs().amax(-1)
    groups = (top * 0.875 / (amax * 2.0 ** -9).unsqueeze(-1)).to(F8)
    by = (groups.float() * (amax * 2.0 ** -12).unsqueeze(-1)).unsqueeze(-1)
    y = torch.where(by > 0, parts.abs() * (2688.0 / 4096.0) / by, 0.0).flatten(-2)
    code = _round_e2m1(y) | torch.signbit(x).to(torch.uint8) << 3
    pairs = code.unflatten(-1, (-1, 2))
    return pairs[..., 0] | pairs[..., 1] << 4, groups, amax * (1.0 / 2688.0)


def _store(slots, x, data, groups, scale):
    pages, page, heads, _ = data.shape
    values, parts, scales = _quantise(x)
    there = (slots >= 0) & (slots < pages * page)
    at = slots[there].long()
    data.view(torch.uint8).view(pages * page, heads, -1)[at] = values[there]
    groups.view(torch.uint8).view(pages * page, heads, -1)[at] = parts.view(torch.uint8)[there]
    scale.view(pages * page, heads)[at] = scales[there]


def _fetch(data, groups, scale, ids, offsets):
    """Rows of a cache at (page, offset), in 32 bits."""
    codes = data.view(torch.uint8)[ids, offsets]
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=data.device)
    x = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1).flatten(-2)
    by = groups.view(torch.uint8)[ids, offsets].view(F8).float()
    x.unflatten(-1, (-1, GROUP)).mul_(by.unsqueeze(-1))
    return x.mul_(scale[ids, offsets].unsqueeze(-1))


def _read(s, which):
    row = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["starts"], row, right=True) - 1
    position, page = row - s["starts"][seq], s["k_data"].shape[1]
    ids = s["table"][seq, position // page].long()
    x = _fetch(s[which + "_data"], s[which + "_groups"], s[which + "_scale"], ids, position % page)
    return x.to(TYPES[s["case"]["out"]])


def _rotate(s, x, weight):
    """Rows of x [T, H, D] normed (where there is a weight), then rotated by their token's position."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["case"].get("eps", 1e-6)) * weight.float()
    angle = s["positions"].double().unsqueeze(1) * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    R = 2 * s["inv_freq"].numel()
    if s["case"]["interleaved"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    y = torch.cat([turned, y[..., R:]], -1)
    if s["dtype"] != F8:
        return y.to(s["dtype"])
    amax = y.abs().amax(-1).clamp(min=TINY)
    return (y * (E4M3_MAX / amax).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(F8), amax * (1.0 / E4M3_MAX)


def _attend(s):
    q, lens, table = s["q"], s["lens"].long(), s["table"]
    B, Hq, D = q.shape
    pages, page, Hk, _ = s["k_data"].shape
    if s["indices"] is None:
        position = torch.arange(table.shape[1] * page, device=q.device).expand(B, -1)
    else:
        position = s["indices"].long()
    valid = (position >= 0) & (position < lens.unsqueeze(1))
    position = torch.where(valid, position, 0)
    ids = table.long().gather(1, position // page)
    valid = valid & (ids >= 0) & (ids < pages)
    ids, offsets = torch.where(valid, ids, 0), torch.where(valid, position % page, 0)
    k = _fetch(s["k_data"], s["k_groups"], s["k_scale"], ids, offsets).permute(0, 2, 3, 1)       # [B, Hk, D, n]
    x = torch.matmul(q.float().view(B, Hk, Hq // Hk, D), k) * s["sm_scale"]
    del k
    x = x.masked_fill_(~valid.view(B, 1, 1, -1), -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = _fetch(s["v_data"], s["v_groups"], s["v_scale"], ids, offsets).permute(0, 2, 1, 3)       # [B, Hk, n, D]
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = top + torch.log(total)
    return out.view(B, Hq, D).to(q.dtype), torch.where(total > 0, lse, -math.inf).view(B, Hq)


# ------------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        import fp8_mqa_logits_02_gb300 as fm
    if case["op"] == "pages":
        # the step's pages, and all of it given back, so that a state can take the same step again
        if own:
            step = fm.pages_update(s["table"], s["lens"], s["new"], s["free"], s["n_free"], case["page"], s["total"])
            undo = fm.pages_update(s["table"], s["lens"], s["back"], s["free"], s["n_free"], case["page"], s["back_total"])
        else:
            step, undo = _update(s, s["new"], s["total"]), _update(s, s["back"], s["back_total"])
        return {"step": list(step), "undo": list(undo), "table": s["table"], "lens": s["lens"], "free": s["free"],
                "n_free": s["n_free"]}
    if case["op"] == "rotate":
        if own:
            return fm.norm_rotate(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], interleaved=case["interleaved"], dtype=s["dtype"])
        return _rotate(s, s["q"], s["q_weight"]), _rotate(s, s["k"], s["k_weight"]) if s["k"] is not None else None
    if case["op"] == "store":
        if own:
            fm.cache_write(s["slots"], s["k"], s["k_data"], s["k_scale"], s["v"], s["v_data"], s["v_scale"],
                           k_groups=s["k_groups"], v_groups=s["v_groups"])
        else:
            _store(s["slots"], s["k"], s["k_data"], s["k_groups"], s["k_scale"])
            _store(s["slots"], s["v"], s["v_data"], s["v_groups"], s["v_scale"])
    if case["op"] in ("store", "read"):
        if own:
            back = [fm.cache_read(s[w + "_data"], s[w + "_scale"], s["table"], s["starts"], s["total"],
                                  dtype=TYPES[case["out"]], groups=s[w + "_groups"])
                    for w in ("kv" if case["op"] == "store" else "k")]
        else:
            back = [_read(s, w) for w in ("kv" if case["op"] == "store" else "k")]
        if case["op"] == "read":
            return back
        return back + [s["k_groups"], s["k_scale"], s["v_groups"], s["v_scale"]]
    if own:
        return fm.attention_paged(s["q"], s["k_data"], s["v_data"], s["table"], s["lens"], s["sm_scale"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"], indices=s["indices"], return_lse=True,
                                  k_groups=s["k_groups"], v_groups=s["v_groups"])
    return _attend(s)


def work(case):
    if case["op"] == "pages":
        lens, news = _news(case)
        page = case["page"]
        moved = sum(abs(-(-max(0, n + m) // page) - -(-n // page)) for n, m in zip(lens, news))
        tokens = sum(abs(m) for m in news) + 3
        # both calls: lengths, changes and starts of each request, 12 bytes a token, each page that moves twice
        return {"bytes": 2 * (20 * case["rows"] + 8 * moved + 8) + 12 * tokens, "flops": 4 * tokens}
    if case["op"] == "rotate":
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        size = SIZES[case["dtype"]]
        to = size if case["out"] in ("same", case["dtype"]) else SIZES[case["out"]]
        scales = 4 if case["out"] == "e4m3" else 0
        return {"bytes": rows * (case["dim"] * (size + to) + scales) + 4 * case["tokens"],
                "flops": rows * (4 * case["dim"] + 3 * case["rotated"])}
    lens = _lens(case)
    total, cols = sum(lens), -(-case["hi"] // case["page"])
    held = case["dim"] // 2 + case["dim"] // GROUP + 4  # bytes of a row in 4 bits
    if case["op"] == "store":
        rows = 2 * total * case["heads"]
        return {"bytes": rows * (case["dim"] * (SIZES[case["dtype"]] + SIZES[case["out"]]) + 2 * held) + 4 * total,
                "flops": 6 * rows * case["dim"]}
    if case["op"] == "read":
        rows = total * case["heads"]
        return {"bytes": rows * (held + case["dim"] * SIZES[case["out"]]) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 2 * rows * case["dim"]}
    if case["select"]:
        total = sum(min(n, case["select"]) for n in lens)
    read = min(total, case["hi"]) if case["shared"] else total
    D = case["dim"]
    return {"bytes": read * 2 * held * case["kv_heads"]
            + case["rows"] * (2 * case["q_heads"] * D * SIZES[case["dtype"]] + 4 * case["q_heads"] + 4 * (case["select"] or cols)),
            "flops": 4 * case["q_heads"] * D * total}


# ------------------------------------------------------------------------------------ 64 bits

def _nearest(y, mantissa, lowest, most):
    """y rounded to the nearest value of a small float format, ties to even, in 64 bits."""
    y = y.clamp(-most, most)
    _, e = torch.frexp(y)                       # |y| in [2^(e-1), 2^e): spacing 2^(e-1-mantissa)
    step = torch.exp2((e - 1 - mantissa).clamp(min=lowest).double())
    return torch.round(y / step) * step


def _rows_64(data, groups, scale, ids, offsets):
    c = data.view(torch.uint8)[ids, offsets]
    c = torch.stack([c % 16, c // 16], -1).flatten(-2).double()
    m = c % 8
    x = torch.where(m < 2, m / 2, torch.exp2(torch.floor(m / 2) - 1) * (1 + (m % 2) / 2)) * torch.where(c >= 8, -1.0, 1.0)
    by = groups[ids, offsets].float().double().repeat_interleave(GROUP, -1)
    return x * by * scale[ids, offsets].double().unsqueeze(-1)


def _exact_rotate(s, x, weight):
    x, R = x.double(), s["case"]["rotated"]
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.double()
    out = x.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + R // 2)
        angle = (s["positions"].double() * s["inv_freq"][i].double()).unsqueeze(1)
        out[..., a] = x[..., a] * torch.cos(angle) - x[..., b] * torch.sin(angle)
        out[..., b] = x[..., b] * torch.cos(angle) + x[..., a] * torch.sin(angle)
    if s["dtype"] != F8:
        return out
    amax = out.abs().amax(-1).clamp(min=TINY)
    return _nearest(out * E4M3_MAX / amax.unsqueeze(-1), 3, -9, E4M3_MAX), amax / E4M3_MAX


def exact(case, seed):
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return (_exact_rotate(s, s["q"], s["q_weight"]),
                _exact_rotate(s, s["k"], s["k_weight"]) if s["k"] is not None else None)
    lens, table, page = s["lens"].tolist(), s["table"].long(), case["page"]
    if case["op"] in ("store", "read"):
        ids = torch.cat([table[b, torch.arange(n, device="cuda") // page] for b, n in enumerate(lens)])
        off = torch.cat([torch.arange(n, device="cuda") % page for n in lens])
        if case["op"] == "read":
            return [_rows_64(s["k_data"], s["k_groups"], s["k_scale"], ids, off)]
        back, held = [], []
        for w in "kv":
            x = s[w].double()
            amax = x.abs().amax(-1).clamp(min=TINY)
            top = x.unflatten(-1, (-1, GROUP)).abs().amax(-1)
            groups = _nearest(top * E4M3_MAX / amax.unsqueeze(-1), 3, -9, E4M3_MAX)
            by = (groups * amax.unsqueeze(-1) / (E4M3_MAX * E2M1_MAX)).repeat_interleave(GROUP, -1)
            values = torch.where(by > 0, _nearest(x / by.clamp(min=1e-300), 1, -1, E2M1_MAX), 0.0)
            back.append(values * by)
            all_groups, all_scale = s[w + "_groups"].float().double(), s[w + "_scale"].double()
            all_groups[ids, off] = groups
            all_scale[ids, off] = amax / (E4M3_MAX * E2M1_MAX)
            held += [all_groups, all_scale]
        return back + held
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
        k = _rows_64(s["k_data"], s["k_groups"], s["k_scale"], ids, off)
        v = _rows_64(s["v_data"], s["v_groups"], s["v_scale"], ids, off)
        x = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(Hk, Hq // Hk, D), k) * s["sm_scale"]
        lse[b] = torch.logsumexp(x, -1).view(Hq)
        out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(Hq, D)
    return out, lse
