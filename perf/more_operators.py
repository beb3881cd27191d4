"""Cases of generation with several beams over the paged MX key/value cache: the
choice of the next beams, and the cache's pages between two steps: forked, freed,
moved together and copied.

``run`` computes a case either with elementary torch operations (scores in 64 bits,
as two near candidates differ by little), or, where ``own`` is true, through the
library's entry points.  A pool of pages has a count of holders for every page
(``refs``, 0: free); a row of the page table lists the pages of a sequence.  The
cache holds MXFP8 codes in blocks of 32 along the head dimension with one E8M0 scale
each, codes [pages][heads][page][dim] and scales [pages][heads][page][dim / 32], one
such set for every layer.  Codes are returned as float8 and scales as E8M0 tensors.
"""

import math

import torch

own = False


def listed():
    kv = {"kv_heads": 8, "dim": 128}
    beams = {"kind": "beams", "new": 1, "spread": 0.5}
    return [
        # one request's step with four beams: launch latency
        {"name": "select 1x4 32k", "op": "select", "requests": 1, "beams": 4, "width": 4, "vocab": 32768, "pad": 0,
         "dtype": "f32", "done": 0.0, "banned": 0.0, "cols": 128},
        # a batch over an odd vocabulary in a padded projection's output, some beams finished, some tokens banned
        {"name": "select 32x4 50k odd", "op": "select", "requests": 32, "beams": 4, "width": 8, "vocab": 50001,
         "pad": 63, "dtype": "f16", "done": 0.2, "banned": 0.01, "cols": 1000},
        # a large batch of eight beams over a large vocabulary
        {"name": "select 256x8 128k", "op": "select", "requests": 256, "beams": 8, "width": 8, "vocab": 131072,
         "pad": 0, "dtype": "bf16", "done": 0.0, "banned": 0.0, "cols": 2048},
        # four beams of one request, reordered: launch latency
        {"name": "fork 1x4", "op": "fork", "requests": 1, "ctx": 1021, "page": 64, "layers": 2, "slack": 64, "beams": 4,
         **kv, **beams},
        # beams of many requests, reordered, partly filled pages copied in eight layers
        {"name": "fork 64x4", "op": "fork", "requests": 64, "ctx": 2048, "page": 16, "layers": 8, "slack": 1024,
         "beams": 4, **kv, **beams},
        # chunks of prompts entering a large pool of small pages
        {"name": "grow 512 by 1024", "op": "fork", "kind": "grow", "requests": 512, "beams": 1, "ctx": 4000, "page": 16,
         "layers": 1, "slack": 65536, "kv_heads": 1, "dim": 64, "new": 1024, "spread": 0.5},
        # two of eight sequences end, one goes back by a few tokens: launch latency
        {"name": "free 8 rows", "op": "free", "requests": 8, "beams": 1, "ctx": 2048, "page": 64, "slack": 64,
         "spread": 0.5},
        # the rows of a large batch, each ended, cut or kept, over a pool of two million pages
        {"name": "free 4096 rows", "op": "free", "requests": 1024, "beams": 4, "ctx": 16384, "page": 16,
         "slack": 65536, "spread": 0.5},
        # a small pool, half in use
        {"name": "compact small", "op": "compact", "requests": 6, "beams": 1, "ctx": 500, "page": 64, "layers": 1,
         "fill": 0.5, "spread": 0.5, **kv},
        # the pool of one layer of a large batch, half in use
        {"name": "compact 12k pages", "op": "compact", "requests": 64, "beams": 2, "ctx": 8192, "page": 64, "layers": 1,
         "fill": 0.5, "spread": 0.5, **kv},
        # a few pages of a shared prefix copied within the pool, two layers
        {"name": "copy 5 pages", "op": "copy", "count": 5, "room": 64, "within": True, "page": 64, "layers": 2, **kv},
        # sequences swapped out to another pool, four layers
        {"name": "copy 1024x4", "op": "copy", "count": 1024, "room": 1536, "within": False, "page": 64, "layers": 4,
         **kv},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "fork", "free", "compact", "copy"])
    if op == "select":
        vocab, beams = _log(rng, 64, 262144), rng.randint(1, 16)
        return {"op": op, "requests": _log(rng, 1, max(1, min(256, 2 ** 27 // (vocab * beams)))), "beams": beams,
                "width": rng.choice([beams, min(64, 2 * beams)]), "vocab": vocab, "pad": rng.choice([0, 0, 1, 32]),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "done": rng.choice([0.0, 0.3]),
                "banned": rng.choice([0.0, 0.3]), "cols": _log(rng, 1, 2048)}
    shape = {"page": rng.choice([16, 32, 48, 64, 128]), "kv_heads": rng.choice([1, 2, 4, 8]),
             "dim": rng.choice([64, 96, 128, 192, 256]), "layers": _log(rng, 1, 8)}
    per_page = 2 * shape["page"] * shape["kv_heads"] * shape["dim"] * shape["layers"]
    if op == "copy":
        n = _log(rng, 1, max(1, min(4096, 2 ** 28 // per_page)))
        return {"op": op, "count": n, "room": 2 * n + rng.randint(0, 40), "within": rng.random() < 0.5, **shape}
    if op == "free":
        shape = {"page": shape["page"]}
        per_page = 256
    ctx, beams = _log(rng, 1, 8192), rng.choice([1, 2, 3, 4, 8])
    row = beams * (-(-ctx // shape["page"]) + 1)
    while op != "free" and row * per_page > 2 ** 29 and shape["layers"] > 1:
        shape["layers"] -= 1
        per_page = per_page * shape["layers"] // (shape["layers"] + 1)
    case = {"op": op, "requests": _log(rng, 1, max(1, min(512, 2 ** 29 // per_page // row))), "beams": beams, "ctx": ctx,
            "spread": rng.choice([0.0, 0.5, 0.95]), **shape}
    if op == "compact":
        return {**case, "fill": rng.choice([0.2, 0.5, 0.9])}
    case["slack"] = _log(rng, 16, 4096)
    if op == "free":
        return case
    kind = rng.choice(["beams", "branch", "grow"])
    return {**case, "kind": kind, "new": _log(rng, 1, 256) if kind == "grow" else 1}


# ------------------------------------------------------------------ sizes that a case stands for
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _lengths(c):
    """Cached tokens of each request."""
    return [max(1, int(c["ctx"] * (1.0 - c["spread"] * ((b * 0.6180339887) % 1.0)))) for b in range(c["requests"])]


def _new_tokens(c):
    """New tokens of the rows of a case that grows, in some order: from none to the most."""
    return [int((c["new"] + 1) * ((b * 0.6180339887) % 1.0)) for b in range(c["requests"] * c["beams"])]


def _page_bytes(c):
    """Bytes of a page in all layers."""
    n = c["page"] * c["kv_heads"] * c["dim"]
    return 2 * (n + n // 32) * c["layers"]


def _pages_used(c):
    """Pages of all sequences: three quarters of a request are common to its beams."""
    p, b = c["page"], c["beams"]
    return sum(s + b * (-(-n // p) - s) for n in _lengths(c) for s in [n * 3 // 4 // p])


def work(c):
    if c["op"] == "select":
        n = int(c["requests"] * c["beams"] * (1.0 - c["done"])) * c["vocab"]      # finished beams' logits need no look
        out = c["requests"] * c["width"]
        return {"bytes": n * _DT[c["dtype"]].itemsize + 9 * c["requests"] * c["beams"] + out * (17 + 8 * c["cols"]),
                "flops": 5 * n}
    if c["op"] == "copy":
        return {"bytes": 2 * c["count"] * _page_bytes(c) + 8 * c["count"], "flops": 0}
    p, b, used = c["page"], c["beams"], _pages_used(c)
    held = [-(-n // p) for n in _lengths(c)]
    if c["op"] == "free":
        # a quarter of the rows end: their entries are read, and the counts of their pages read and written
        return {"bytes": sum(held) * b + 2 * used + 4 * c["requests"] * b * 3, "flops": sum(held) * b // 4}
    if c["op"] == "compact":
        pages = int(used / c["fill"])
        moved = used * (1.0 - used / pages)
        return {"bytes": 2 * moved * _page_bytes(c) + 8 * pages + 8 * sum(held) * b, "flops": 0}
    n = c["requests"] * b
    new = sum(_new_tokens(c)) if c["kind"] == "grow" else n
    again = b * (1.0 - 1.0 / b) ** b if c["kind"] == "beams" else float(b) if c["kind"] == "branch" else 0.0
    tails = sum(again * -(-(m % p) // 16) * 16 / p for m in _lengths(c))
    return {"bytes": 2 * tails * _page_bytes(c) + 8 * (used + c["slack"]) + 8 * sum(held) * b + 8 * new + 16 * n,
            "flops": n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _cache(c, pages, g):
    """Codes and scales of a pool's pages, one set for every layer."""
    sets = []
    for _ in range(c["layers"]):
        one = []
        for n in (c["dim"], c["dim"] // 32) * 2:
            shape = (pages, c["kv_heads"], c["page"], n)
            lo, hi = (0, 126) if n == c["dim"] else (120, 135)
            one.append(torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8))
        sets.append(tuple(one))
    return sets


def _sequences(c, pages, g):
    """Counts, page table and lengths of beams that share the first three quarters of their request."""
    p, b = c["page"], c["beams"]
    lens = torch.tensor(_lengths(c), dtype=torch.int64)
    held = (lens + p - 1) // p
    both = lens * 3 // 4 // p
    total = both + b * (held - both)
    start = (total.cumsum(0) - total)[:, None, None]
    j = torch.arange(int(held.max()) + -(-c.get("new", 0) // p))
    beam = torch.arange(b)[None, :, None]
    both, held = both[:, None, None], held[:, None, None]
    at = torch.where(j < both, start + j, start + both + beam * (held - both) + j - both)
    at = torch.where(j < held, at, 0).flatten(0, 1).cuda()
    real = (j < held).expand(-1, b, -1).flatten(0, 1).cuda()
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.where(real, order[at], -1)
    refs = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    refs.index_add_(0, torch.where(real, table, pages).flatten(), torch.ones_like(table).flatten())
    return refs[:pages].int(), table.int(), lens.repeat_interleave(b).int().cuda()


def prepare(c, seed):
    g = _gen(seed)
    rand = lambda *n: torch.rand(n, generator=g, device="cuda")  # noqa: E731
    if c["op"] == "select":
        r, b, v = c["requests"], c["beams"], c["vocab"]
        x = torch.empty((r, b, v + c["pad"]), dtype=_DT[c["dtype"]], device="cuda")
        for i in range(0, r, 16):
            y = torch.randn((min(16, r - i), b, v + c["pad"]), generator=g, device="cuda") * 2.5
            if c["banned"]:
                y[rand(*y.shape) < c["banned"]] = -math.inf
            x[i:i + 16] = y
        return {"c": c, "logits": x[:, :, :v], "scores": rand(r, b) * -20.0, "finished": rand(r, b) < c["done"],
                "eos": int(v * 0.37), "lens": torch.randint(0, c["cols"] + 1, (r, b), generator=g, device="cuda").int(),
                "history": torch.randint(0, v, (r, b, c["cols"]), generator=g, device="cuda").int()}
    if c["op"] == "copy":
        pool = _cache(c, c["room"], g)
        order = torch.randperm(c["room"], generator=g, device="cuda").int()
        n = c["count"]
        return {"c": c, "src": pool, "dst": pool if c["within"] else _cache(c, c["room"], g),
                "from": order[:n].contiguous(), "to": order[c["room"] - n:].contiguous()}
    used = _pages_used(c)
    if c["op"] == "compact":
        pages = int(used / c["fill"])
        refs, table, lens = _sequences(c, pages, g)
        return {"c": c, "refs": refs, "table": table, "lens": lens, "cache": _cache(c, pages, g)}
    refs, table, lens = _sequences(c, used + c["slack"], g)
    n = lens.numel()
    if c["op"] == "free":
        # a quarter of the rows end, a quarter go back by up to two pages, the others stay
        fate = rand(n)
        back = torch.randint(0, 2 * c["page"], (n,), generator=g, device="cuda")
        keep = torch.where(fate < 0.25, 0, torch.where(fate < 0.5, (lens - back).clamp_min(0), lens)).int()
        return {"c": c, "refs": refs, "table": table, "lens": lens, "keep": keep}
    if c["kind"] == "grow":
        parents = None
        new = torch.tensor(_new_tokens(c), device="cuda")[torch.randperm(n, generator=g, device="cuda")]
    else:
        b = c["beams"]
        pick = torch.arange(b, device="cuda").repeat(c["requests"])
        if c["kind"] == "beams":
            pick = torch.randint(0, b, (n,), generator=g, device="cuda")
        parents = (torch.arange(n, device="cuda") // b * b + pick).int()
        new = torch.ones(n, dtype=torch.int64, device="cuda")
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
    return {"c": c, "refs": refs, "table": table, "lens": lens, "parents": parents, "cu": cu, "tokens": int(cu[-1]),
            "cache": _cache(c, used + c["slack"], g)}


# ------------------------------------------------------------------ plain forms
def _as_values(sets):
    return [[t.view(torch.float8_e8m0fnu if i & 1 else torch.float8_e4m3fn) for i, t in enumerate(s)] for s in sets]


def _ordered(x):
    """Whole numbers in the order of float32 values."""
    i = x.view(torch.int32).long()
    return torch.where(i < 0, -(i & 0x7FFFFFFF), i)


def _plain_select(s):
    c, x = s["c"], s["logits"].float()
    r, b, v, w = c["requests"], c["beams"], c["vocab"], c["width"]
    k = min(w, v)
    # the k best of each beam: equal logits in the order of their tokens
    key = _ordered(x) * (1 << 31) + (v - 1 - torch.arange(v, device="cuda"))
    token = v - 1 - (key.topk(k, -1).values & ((1 << 31) - 1))
    top = x.amax(-1, keepdim=True)
    lse = top.double() + (x - top).exp().sum(-1, keepdim=True, dtype=torch.float64).log()
    score = s["scores"].double()[..., None] + (x.gather(-1, token).double() - lse)
    first = torch.arange(k, device="cuda") == 0
    done = s["finished"][..., None]
    score = torch.where(done, torch.where(first, s["scores"].double()[..., None], -math.inf), score)
    score = torch.where(torch.isfinite(score), score, -math.inf)
    token = torch.where(done, 0, token)
    # candidates of all beams, the better first, of equal ones the lower beam's
    score, at = torch.nn.functional.pad(score.flatten(1), (0, max(0, w - b * k)), value=-math.inf).sort(
        dim=-1, descending=True, stable=True)
    score, at = score[:, :w], at[:, :w].clamp_max(b * k - 1)
    real = score > -math.inf
    beam = torch.where(real, at // k, 0)
    token = torch.where(real, token.flatten(1).gather(1, at), 0)
    was = s["finished"].gather(1, beam) & real
    live = real & ~was
    lens = s["lens"].gather(1, beam)
    history = s["history"].gather(1, beam[..., None].expand(-1, -1, c["cols"]))
    put = live[..., None] & (torch.arange(c["cols"], device="cuda") == lens[..., None])
    history = torch.where(put, token[..., None].int(), history)
    lens = torch.where(live, (lens + 1).clamp_max(c["cols"]), lens)
    row = torch.arange(r, device="cuda")[:, None] * b + beam
    return [score.float(), row.int(), token.int(), was | (live & (token == s["eos"])), history, lens.int()]


def _counted(refs, table, held, weight):
    """refs plus weight for every page that the table's rows hold."""
    real = (torch.arange(table.shape[1], device="cuda") < held[:, None]) & (table >= 0)
    return refs.index_add(0, table[real], weight[real])


def _copied(sets, src, dst, tokens):
    """Tokens [0, tokens) of pages dst of every layer become those of pages src."""
    for one in sets:
        for t in one:
            keep = torch.arange(t.shape[2], device="cuda") >= tokens[:, None]
            t[dst] = torch.where(keep[:, None, :, None], t[dst], t[src])


def _plain_fork(s):
    c, refs, table, p = s["c"], s["refs"].long(), s["table"].long(), s["c"]["page"]
    rows, cols = table.shape
    release = c["kind"] != "branch"
    parent = torch.arange(rows, device="cuda") if s["parents"] is None else s["parents"].long()
    n = parent.numel()
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    lens = s["lens"].long()
    had, held = lens[parent], (lens + p - 1) // p
    out = table[parent]
    count = _counted(refs, out, held[parent], torch.ones_like(out))
    if release:
        count = _counted(count, table, held, torch.full_like(table, -1))
    # the page that is partly filled stays with the first child that writes where only such children hold it
    writes = (new > 0) & (had % p > 0)
    i = torch.arange(n, device="cuda")
    writers = torch.zeros_like(lens).index_add(0, parent, writes.long())
    first = torch.full_like(lens, n).scatter_reduce(0, parent, torch.where(writes, i, n), "amin")
    tail = out.gather(1, (held[parent] - 1).clamp_min(0)[:, None])[:, 0]
    copies = writes & ~((count[tail] == writers[parent]) & (first[parent] == i))
    after = (had + new + p - 1) // p
    need = copies.long() + after - held[parent]
    end = need.cumsum(0)
    free = torch.argsort((count != 0).long(), stable=True)
    fits = (new > 0) & ((end <= (count == 0).sum()) | (need == 0)) & (after <= cols)
    copies = copies & fits
    # column j of a child: its parent's page, or a new one
    j = torch.arange(cols, device="cuda")
    nth = j - held[parent][:, None] + copies[:, None].long()
    fresh = fits[:, None] & (nth >= 0) & (j < after[:, None])
    page = free[((end - need)[:, None] + nth).clamp(0, free.numel() - 1)]
    out = torch.where(fresh, page, torch.where(j < held[parent][:, None], out, -1))
    count = count.index_add(0, tail, -copies.long())
    count[page[fresh]] = 1
    token = torch.arange(s["tokens"], device="cuda")
    child = torch.searchsorted(s["cu"].long(), token, right=True) - 1
    at = had[child] + token - s["cu"].long()[child]
    slots = out[child, (at // p).clamp_max(cols - 1)] * p + at % p
    slots = torch.where(fits[child], slots, -1)
    _copied(s["cache"], tail[copies], free[(end - need)[copies]], ((had % p + 15) // 16 * 16)[copies])
    return [count.int(), out.int(), torch.where(fits, had + new, had).int(), slots, _as_values(s["cache"])]


def _plain_free(s):
    p, lens, keep = s["c"]["page"], s["lens"].long(), s["keep"].long()
    left = torch.minimum(lens, keep.clamp_min(0))
    j = torch.arange(s["table"].shape[1], device="cuda")
    gone = (j >= ((left + p - 1) // p)[:, None]) & (j < ((lens + p - 1) // p)[:, None])
    page = s["table"][gone].long()
    return [s["refs"].index_add(0, page, torch.full_like(page, -1, dtype=torch.int32)), left.int()]


def _plain_compact(s):
    p, refs = s["c"]["page"], s["refs"]
    pages = refs.numel()
    page = torch.arange(pages, device="cuda")
    live = refs != 0
    used = live.sum()
    before = live.long().cumsum(0) - live.long()
    # the nth free page below `used` takes the nth used one from the top
    hole, mover = ~live & (page < used), live & (page >= used)
    nth = torch.where(hole, page - before, torch.where(mover, used - 1 - before, 0))
    to = torch.zeros(pages + 1, dtype=torch.int64, device="cuda").index_put((torch.where(hole, nth, pages),), page)
    goes = torch.where(mover, to[nth], page)
    j = torch.arange(s["table"].shape[1], device="cuda")
    real = j < ((s["lens"].long() + p - 1) // p)[:, None]
    table = torch.where(real, goes[torch.where(real, s["table"], 0).long()], s["table"].long()).int()
    moved = torch.zeros_like(refs).index_add(0, goes, torch.where(live, refs, 0))
    moved = torch.where(page < used, moved, 0)
    src, dst = page[mover], goes[mover]
    for one in s["cache"]:
        for t in one:
            t[dst] = t[src]
    return [moved, table, used.int().reshape(1), _as_values(s["cache"])]


def _plain_copy(s):
    src, dst = s["from"].long(), s["to"].long()
    for a, b in zip(s["src"], s["dst"]):
        for x, y in zip(a, b):
            y[dst] = x[src]
    return _as_values(s["dst"])


# ------------------------------------------------------------------ the library's calls
def _own_run(s):
    import mx_block_scaled_quantize_amd as mxa
    c = s["c"]
    if c["op"] == "select":
        return list(mxa.mx_beam_select(s["logits"], s["scores"], c["width"], finished=s["finished"], eos=s["eos"],
                                       history=s["history"], lens=s["lens"]))
    if c["op"] == "copy":
        src, dst = ([mxa.KVCache(*one) for one in s[k]] for k in ("src", "dst"))
        mxa.mx_kv_copy(src, s["from"], dst, s["to"])
        return _as_values(s["dst"])
    if c["op"] == "free":
        return list(mxa.mx_kv_free(s["refs"], s["table"], s["lens"], c["page"], keep=s["keep"]))
    cache = [mxa.KVCache(*one) for one in s["cache"]]
    if c["op"] == "compact":
        return [*mxa.mx_kv_compact(cache, s["refs"], s["table"], s["lens"]), _as_values(s["cache"])]
    return [*mxa.mx_kv_fork(cache, s["refs"], s["table"], s["lens"], s["cu"], parents=s["parents"],
                            release=c["kind"] != "branch", tokens=s["tokens"]), _as_values(s["cache"])]


def run(s):
    if own:
        return _own_run(s)
    op = s["c"]["op"]
    if op == "select":
        return _plain_select(s)
    if op == "fork":
        return _plain_fork(s)
    if op == "free":
        return _plain_free(s)
    return _plain_compact(s) if op == "compact" else _plain_copy(s)


# ------------------------------------------------------------------ from the definitions, 64 bits
def _exact_select(s):
    c = s["c"]
    out = [[] for _ in range(6)]
    v, w = c["vocab"], c["width"]
    for r in range(c["requests"]):
        x = s["logits"][r].double()
        score = s["scores"][r].double()[:, None] + torch.log_softmax(x, -1)
        score = torch.where(torch.isfinite(score), score, -math.inf)
        for b in s["finished"][r].nonzero().flatten().tolist():
            score[b] = -math.inf
            score[b, 0] = s["scores"][r, b].double()
        order = torch.sort(score.flatten(), descending=True, stable=True)
        found = [(z, a // v, a % v) for z, a in zip(order.values[:w].tolist(), order.indices[:w].tolist())]
        found += [(-math.inf, 0, 0)] * (w - len(found))
        finished, lens = s["finished"][r].tolist(), s["lens"][r].tolist()
        history = s["history"][r].tolist() if c["cols"] else None
        for z, b, t in found:
            if z == -math.inf:
                b, t = 0, 0
            live = z > -math.inf and not finished[b]
            row, n = list(history[b]), lens[b]
            if live and n < c["cols"]:
                row[n] = t
                n += 1
            for at, y in enumerate((z, r * c["beams"] + b, t, z > -math.inf and (finished[b] or t == s["eos"]), row, n)):
                out[at].append(y)
    shape = (c["requests"], w)
    kind = (torch.float64, torch.int32, torch.int32, torch.bool, torch.int32, torch.int32)
    return [torch.tensor(o, dtype=k).view(*shape, *((c["cols"],) if i == 4 else ()))
            for i, (o, k) in enumerate(zip(out, kind))]


def _decoded(sets):
    """What codes and scales stand for, from the formats' definitions."""
    code = torch.arange(256, dtype=torch.float64)
    sign, e, m = 1 - 2 * (code // 128), code // 8 % 16, code % 8
    value = sign * torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    value[127] = value[255] = math.nan
    scale = torch.exp2(code - 127)
    scale[255] = math.nan
    return [[(scale if i & 1 else value)[t.int().cpu()] for i, t in enumerate(one)] for one in sets]


def _exact_fork(s):
    """Child after child, with lists."""
    c, p = s["c"], s["c"]["page"]
    refs, table, lens, cu = (s[k].tolist() for k in ("refs", "table", "lens", "cu"))
    rows = [row[: -(-n // p)] for row, n in zip(table, lens)]
    parents = list(range(len(rows))) if s["parents"] is None else s["parents"].tolist()
    for i in parents:
        for q in rows[i]:
            refs[q] += 1
    if c["kind"] != "branch":
        for row in rows:
            for q in row:
                refs[q] -= 1
    free = [q for q, n in enumerate(refs) if n == 0]
    writers = {}
    for child, i in enumerate(parents):
        if cu[child + 1] > cu[child] and lens[i] % p:
            writers.setdefault(i, []).append(child)
    shared = list(refs)
    out, new_lens, slots, copies, at = [], [], [], [], 0
    for child, i in enumerate(parents):
        row, n, new = list(rows[i]), lens[i], cu[child + 1] - cu[child]
        mine = writers.get(i, ())
        copy = child in mine and not (shared[row[-1]] == len(mine) and mine[0] == child)
        need = copy + -(-(n + new) // p) - len(row)
        at += need
        if new and (at <= len(free) or not need) and -(-(n + new) // p) <= len(table[0]):
            pages = free[at - need:at]
            if copy:
                copies.append((row[-1], pages[0], -(-(n % p) // 16) * 16))
                refs[row[-1]] -= 1
                row[-1] = pages.pop(0)
                refs[row[-1]] += 1
            for q in pages:
                row.append(q)
                refs[q] += 1
            slots += [row[t // p] * p + t % p for t in range(n, n + new)]
            n += new
        else:
            slots += [-1] * new
        out.append(row + [-1] * (len(table[0]) - len(row)))
        new_lens.append(n)
    cache = [[t.clone() for t in one] for one in s["cache"]]
    for src, dst, n in copies:
        for one in cache:
            for t in one:
                t[dst, :, :n] = t[src, :, :n]
    as_int = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return [as_int(refs), as_int(out), as_int(new_lens), torch.tensor(slots), _decoded(cache)]


def _exact_compact(s):
    p = s["c"]["page"]
    refs, table, lens = (s[k].tolist() for k in ("refs", "table", "lens"))
    live = [q for q, n in enumerate(refs) if n]
    used, goes = len(live), {}
    for q in range(used):
        if refs[q] == 0:
            goes[live.pop()] = q
    for src, dst in goes.items():
        refs[dst], refs[src] = refs[src], 0
    out = [[goes.get(q, q) if j < -(-n // p) else q for j, q in enumerate(row)] for row, n in zip(table, lens)]
    cache = [[t.clone() for t in one] for one in s["cache"]]
    for src, dst in goes.items():
        for one in cache:
            for t in one:
                t[dst] = t[src]
    return [torch.tensor(refs, dtype=torch.int32), torch.tensor(out, dtype=torch.int32),
            torch.tensor([used], dtype=torch.int32), _decoded(cache)]


def exact(c, seed):
    if c["op"] == "free":
        return None                      # whole numbers only
    if c["op"] == "select":
        return _exact_select(prepare(c, seed)) if c["requests"] * c["width"] * c["cols"] <= 2 ** 23 else None
    pool = c["room"] if c["op"] == "copy" else _pages_used(c) / c.get("fill", 1.0) + c.get("slack", 0)
    if pool * _page_bytes(c) > 2 ** 27 or c.get("requests", 1) * c.get("beams", 1) > 2 ** 10:
        return None                      # lists and 8 bytes a code: small pools
    s = prepare(c, seed)
    if c["op"] == "copy":
        dst = [[t.clone() for t in one] for one in s["dst"]]
        for a, b in zip(s["from"].tolist(), s["to"].tolist()):
            for x, y in zip(s["src"], dst):
                for t, u in zip(x, y):
                    u[b] = t[a]
        return _decoded(dst)
    return _exact_fork(s) if c["op"] == "fork" else _exact_compact(s)
