"""The paged 8-bit key/value cache: its operators' cases, their plain forms and their 64-bit definition.

Three operators of a serving step, in the order in which a step uses them:

* ``plan``: block tables and slot maps from request lengths. One pass is a speculative step that is
  rejected: every request grows by its draft, then drops it again, which leaves the state as it was.
* ``append``: new keys and values quantised into the cache (one scale for each page and head), then the
  touched pages read back as the values they stand for.
* ``attention``: queries of each request over its pages: single tokens, drafts, prompts, chunks of prompts.

The cache holds unsigned codes u and one fp32 scale for each page and head: value = (u - 128) * scale.
"""
import math
import random

import torch

own = False

FLOOR = 2.0 ** -100        # smallest scale of a block
DEV = "cuda"


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a few requests of an interactive server, five drafted tokens each: latency alone
        {"name": "plan 4 drafts", "op": "plan", "batch": 4, "new": 5, "kv": 700, "page": 16, "lens": 1},
        # a full server taking in a 64 Ki-token step of prompts and chunks, tables of 2048 positions and more
        {"name": "plan 512 prompts", "op": "plan", "batch": 512, "new": 128, "kv": 1900, "page": 16, "lens": 2},
        # one token of each of 16 requests, heads of the 7B-shaped block
        {"name": "append 16 tokens", "op": "append", "batch": 16, "new": 1, "kv_heads": 32, "dim": 128, "page": 16,
         "lens": 3},
        # a batch of prompts with odd lengths, grouped heads, larger pages
        {"name": "append ragged prompts", "op": "append", "batch": 7, "new": 391, "kv_heads": 8, "dim": 64, "page": 64,
         "lens": 4},
        # a long prompt, heads of the 7B-shaped block
        {"name": "append 8192 prompt", "op": "append", "batch": 1, "new": 8192, "kv_heads": 32, "dim": 128, "page": 64,
         "lens": 5},
        # one request that has just begun to answer: latency alone
        {"name": "attend 1 short", "op": "attention", "batch": 1, "new": 1, "kv": 130, "heads": 32, "kv_heads": 32,
         "dim": 128, "page": 16, "causal": True, "window": 0, "lens": 6},
        # ordinary decoding at the pages' sequence length of 2048, heads of the 7B-shaped block
        {"name": "attend 16 decode", "op": "attention", "batch": 16, "new": 1, "kv": 2048, "heads": 32, "kv_heads": 32,
         "dim": 128, "page": 16, "causal": True, "window": 0, "lens": 7},
        # a large batch with grouped heads, ragged lengths
        {"name": "attend 128 grouped", "op": "attention", "batch": 128, "new": 1, "kv": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "causal": True, "window": 0, "lens": 8},
        # one request with a very long context
        {"name": "attend 1 long", "op": "attention", "batch": 1, "new": 1, "kv": 131072, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "causal": True, "window": 0, "lens": 9},
        # drafts being verified, heads of 64, a sliding window
        {"name": "attend 32 drafts", "op": "attention", "batch": 32, "new": 5, "kv": 1500, "heads": 16, "kv_heads": 16,
         "dim": 64, "page": 32, "causal": True, "window": 1024, "lens": 10},
        # a whole prompt of 2048, heads of the 7B-shaped block
        {"name": "attend 2048 prompt", "op": "attention", "batch": 1, "new": 2048, "kv": 2048, "heads": 32,
         "kv_heads": 32, "dim": 128, "page": 16, "causal": True, "window": 0, "lens": 11},
        # chunks of long prompts over what is cached already, grouped heads
        {"name": "attend 4 chunks", "op": "attention", "batch": 4, "new": 2048, "kv": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 128, "causal": True, "window": 0, "lens": 12},
    ]


def log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "attention", "attention"))
    page = rng.choice((16, 32, 64, 128))
    lens = rng.randrange(1, 1 << 20)
    if op == "plan":
        batch = log_uniform(rng, 1, 512)
        return {"op": op, "batch": batch, "new": log_uniform(rng, 1, min(4096, 65536 // batch)),
                "kv": log_uniform(rng, 16, 2048), "page": page, "lens": lens}
    dim = rng.choice((64, 128))
    if op == "append":
        kv_heads = rng.choice((1, 2, 8, 16, 32))
        batch = log_uniform(rng, 1, 256)
        most = max(1, min(65536, 8192 * 32 * 128 // (kv_heads * dim)) // batch)
        return {"op": op, "batch": batch, "new": rng.choice((1, log_uniform(rng, 1, min(8192, most)))),
                "kv_heads": kv_heads, "dim": dim, "page": page, "lens": lens}
    kv_heads = rng.choice((1, 2, 4, 8, 16, 32))
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 8, 16) if g * kv_heads <= 64])
    new = rng.choice((1, 1, rng.randrange(2, 9), log_uniform(rng, 9, 4096)))
    batch = log_uniform(rng, 1, 128 if new < 9 else 8)
    # no more bytes and products than the largest listed cases
    most_kv = min(131072, (1 << 29) // (batch * kv_heads * dim), 4 * 32 * 2048 * 8192 * 128 // (batch * heads * new * dim))
    kv = max(log_uniform(rng, 1, max(1, most_kv)), new)
    while batch * heads * new * kv > 4 * 32 * 2048 * 8192:
        new, kv = max(1, new // 2), max(1, kv // 2)
    return {"op": op, "batch": batch, "new": new, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "causal": rng.random() < 0.85, "window": 0, "lens": lens} | (
                {"causal": True, "window": log_uniform(rng, 1, kv)} if rng.random() < 0.2 else {})


def lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request: they follow from the case."""
    rng = random.Random(case["lens"])
    news, kvs = [], []
    for b in range(case["batch"]):
        new = case["new"] if b == 0 or case["new"] < 9 else rng.randint(max(1, case["new"] // 2), case["new"])
        if case["op"] == "append":
            kv = new + rng.randint(0, 2 * case["page"])        # what the request has in the cache already
        else:
            kv = case["kv"] if b == 0 else rng.randint(max(1, case["kv"] // 2), case["kv"])
            kv = max(kv, new) if case["op"] == "attention" else kv
        news.append(new)
        kvs.append(kv)
    return news, kvs


def pages_of(n, page):
    return -(-n // page)


# ----------------------------------------------------------------------------- inputs
def table_of(g, counts, width, spare):
    """Block tables whose pages lie anywhere in the cache: (table, number of pages, a permutation of all pages)."""
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device=DEV, dtype=torch.int32)
    used = torch.tensor(counts, device=DEV)
    first = torch.cumsum(used, 0) - used
    col = torch.arange(width, device=DEV)
    at = first[:, None] + col
    return torch.where(col < used[:, None], order[at.clamp(max=total - 1)], torch.zeros((), dtype=torch.int32, device=DEV)), total, order


def random_cache(g, pages, kv_heads, page, dim):
    """Codes of roughly normal values and scales that differ from block to block."""
    def codes():
        c = torch.empty(pages, kv_heads, page, dim, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (kv_heads * page * dim))
        for p in range(0, pages, step):
            x = torch.randn(c[p:p + step].shape, generator=g, device=DEV, dtype=torch.float16)
            c[p:p + step] = (x * 32).round().clamp(-127, 127).add(128).to(torch.uint8)
        return c

    def scales():
        return torch.exp(torch.randn(pages, kv_heads, generator=g, device=DEV) * 0.3) * (4.0 / 127)

    return {"kcodes": codes(), "vcodes": codes(), "kscale": scales(), "vscale": scales()}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    news, kvs = lengths(case)
    page, batch = case["page"], case["batch"]
    s = {"case": case, "new": torch.tensor(news, dtype=torch.int32, device=DEV), "tokens": sum(news)}
    if case["op"] == "plan":
        width = max(pages_of(n + k, page) for n, k in zip(news, kvs))
        extra = sum(pages_of(n + k, page) - pages_of(k, page) for n, k in zip(news, kvs))
        table, total, order = table_of(g, [pages_of(k, page) for k in kvs], width, extra + 3)
        live = total - extra - 3
        free = torch.zeros(total, dtype=torch.int32, device=DEV)
        free[:extra + 3] = order[live:]
        return s | {"kv": torch.tensor(kvs, dtype=torch.int32, device=DEV), "drop": -s["new"], "table": table,
                    "free": free, "count": torch.tensor([extra + 3], dtype=torch.int32, device=DEV)}
    table, total, _ = table_of(g, [pages_of(k, page) for k in kvs], max(pages_of(k, page) for k in kvs), 2)
    kv_heads, dim = case["kv_heads"], case["dim"]
    kv = torch.tensor(kvs, dtype=torch.int64, device=DEV)
    new = s["new"].long()
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    s |= {"table": table, "kv": kv.int(), "cu": cu} | random_cache(g, total, kv_heads, page, dim)
    if case["op"] == "append":
        # keys and values as one projection's output holds them, side by side, with a few loud channels
        x = torch.randn(s["tokens"], 2 * kv_heads * dim, generator=g, device=DEV)
        x[:, torch.randperm(x.shape[1], generator=g, device=DEV)[:max(1, x.shape[1] // 100)]] *= 8
        x = x.to(torch.bfloat16)
        s["K"] = x[:, :kv_heads * dim].unflatten(1, (kv_heads, dim))
        s["V"] = x[:, kv_heads * dim:].unflatten(1, (kv_heads, dim))
        row = torch.repeat_interleave(torch.arange(batch, device=DEV), new)
        pos = torch.arange(s["tokens"], device=DEV) - cu[row] + (kv - new)[row]
        s["slots"] = (table[row, pos // page].long() * page + pos % page).int()
        # every token of the touched pages, to be read back
        start = (kv - new) // page * page
        count = kv - start
        row = torch.repeat_interleave(torch.arange(batch, device=DEV), count)
        pos = torch.arange(int(count.sum()), device=DEV) - (torch.cumsum(count, 0) - count)[row] + start[row]
        s["back"] = (table[row, pos // page].long() * page + pos % page).int()
        return s
    s["Q"] = (torch.randn(s["tokens"], case["heads"], dim, generator=g, device=DEV) * 3).to(torch.bfloat16)
    s["max_q"], s["max_kv"] = max(news), max(kvs)
    return s


# ----------------------------------------------------------------------------- plain forms
def plain_plan(new, kv, table, free, count, page, tokens):
    """One step of the page table, in place: (slots, row starts, refused)."""
    batch, width = table.shape
    n, q = kv.long(), new.long()
    after, grow = (n + q).clamp(min=0), q.clamp(min=0)
    ends = torch.cumsum(grow, 0)
    starts = ends - grow
    have, want = (n + page - 1) // page, (after + page - 1) // page
    wide = (want > width) | (ends > tokens) & (grow > 0)
    need = torch.where(wide, 0, (want - have).clamp(min=0))
    gone = (have - want).clamp(min=0)
    taken, given = torch.cumsum(need, 0), torch.cumsum(gone, 0)
    stock = count.long()
    back = given[-1]
    refused = wide | (taken > stock + back) & (need > 0)
    # the pages given back, in order, then the stack from its top
    col = torch.arange(width, device=kv.device)
    leaving = (col >= want[:, None]) & (col < have[:, None])
    at = torch.arange(free.numel(), device=kv.device)
    index = (given - gone)[:, None] + col - want[:, None]
    released = torch.zeros(free.numel() + 1, dtype=torch.int32, device=kv.device)
    released.scatter_(0, torch.where(leaving, index, free.numel()).reshape(-1), table.reshape(-1))
    pool = torch.where(at < back, released[:-1], free[(stock - 1 - (at - back)).clamp(0, free.numel() - 1)])
    fresh = (col >= have[:, None]) & (col < want[:, None]) & ~refused[:, None]
    index = (taken - need)[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, pool[index.clamp(0, free.numel() - 1)], table))
    used = torch.where(refused | (need == 0), 0, taken).amax()
    top = stock + back - 1 - at                       # which released page stays at this place of the stack
    stays = (at >= stock) & (at < stock + back - used)
    free.copy_(torch.where(stays, released[:-1][top.clamp(0, free.numel() - 1)], free))
    count.copy_((stock + back - used).int())
    cu = torch.cat([torch.zeros_like(ends[:1]), ends]).clamp(max=tokens)
    t = torch.arange(tokens, device=kv.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=batch - 1)
    pos = n[b] + t - cu[b]
    slot = table[b, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    slots = torch.where((t < cu[-1]) & ~refused[b], slot, -1).int()
    kv.copy_(torch.where(refused, n, after).int())
    return slots, cu.int(), refused.int()


def plain_append(x, slots, codes, scale, page):
    """Keys (or values) of the tokens quantised into their blocks, in place."""
    pages, heads = scale.shape
    at, off = slots.long() // page, slots.long() % page
    peak = x.float().abs().amax(2)
    gamma = torch.zeros_like(scale).index_reduce_(0, at, peak, "amax")
    first = torch.full((pages,), page, device=x.device).index_reduce_(0, at, off, "amin")
    touched = (first < page)[:, None]
    before = torch.where(first[:, None] > 0, scale, 0.0)
    after = torch.where(touched, torch.maximum(before, (gamma / 127).clamp(min=FLOOR)), scale)
    # what a page held before the first of its new tokens, in the new scale
    held = (codes.float() - 128) * before[:, :, None, None]
    again = torch.round(held.double() / after[:, :, None, None].double())
    keeps = touched[:, :, None, None] & (torch.arange(page, device=x.device)[:, None] < first[:, None, None, None])
    codes.copy_(torch.where(keeps, again + 128, codes.double()).to(torch.uint8))
    code = torch.round(x.double() / after[at].double()[:, :, None])
    codes[at, :, off] = (code + 128).to(torch.uint8)
    scale.copy_(after)


def plain_read(slots, codes, scale, page):
    at, off = slots.long() // page, slots.long() % page
    return ((codes[at, :, off].float() - 128) * scale[at][:, :, None]).to(torch.bfloat16)


def plain_attention(s):
    case = s["case"]
    kcodes, vcodes, kscale, vscale, table, cu = (s[k] for k in ("kcodes", "vcodes", "kscale", "vscale", "table", "cu"))
    batch, heads, kv_heads, dim = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    group, most = heads // kv_heads, s["max_q"]
    at = table.long()

    def dense(codes, scale):                          # [batch, kv head, position, channel]
        x = (codes[at].float() - 128) * scale[at][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(batch, kv_heads, -1, dim)

    row = (cu[:-1, None].long() + torch.arange(most, device=cu.device)).clamp(max=s["tokens"] - 1)
    q = s["Q"].float()[row]                           # [batch, query, head, channel]
    q = q.reshape(batch, most, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv_heads, group * most, dim)
    score = torch.matmul(q, dense(kcodes, kscale).transpose(2, 3)) * (1.0 / math.sqrt(dim))
    key = torch.arange(score.shape[-1], device=cu.device)
    kv, new = s["kv"].long()[:, None, None], (cu[1:] - cu[:-1]).long()[:, None, None]
    position = kv - new + torch.arange(most, device=cu.device)[:, None]
    seen = (key < kv).expand(batch, most, -1)
    if case["causal"]:
        seen = seen & (key <= position)
    if case["window"]:
        seen = seen & (key > position - case["window"])
    score = score.reshape(batch, kv_heads, group, most, -1)
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    peak = score.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = torch.exp_(score - peak)
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.reshape(batch, kv_heads, group * most, -1), dense(vcodes, vscale))
    out = out.reshape(batch, kv_heads, group, most, dim) / total.clamp(min=1e-30)
    lse = (peak + torch.log(total)).squeeze(-1)
    i = torch.arange(s["tokens"], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), i.int(), right=True)
    i = i - cu[b]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, most, heads, dim)[b, i]
    return out.to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(batch, most, heads)[b, i]


# ----------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    page = case["page"]
    if own:
        from hadamard_bit_quant_b200 import layer
        if case["op"] == "plan":
            pages = layer.KVPages(s["kv"], s["table"], s["free"], s["count"], page)
            step = pages.plan(s["new"], s["tokens"])
            table = s["table"].clone()
            pages.plan(s["drop"], 0)
            return step.slots, step.cu_q, step.refused, table, s["kv"], s["free"], s["count"]
        cache = layer.KVCache(s["kcodes"], s["vcodes"], s["kscale"], s["vscale"])
        if case["op"] == "append":
            cache.append(s["K"], s["V"], s["slots"])
            return (*cache.read(s["back"]), s["kscale"], s["vscale"])
        return cache.attention(s["Q"], s["cu"], s["kv"], s["table"], max_q=s["max_q"], max_kv=s["max_kv"],
                               causal=case["causal"], window=case["window"], return_lse=True)
    if case["op"] == "plan":
        state = s["kv"], s["table"], s["free"], s["count"], page
        step = plain_plan(s["new"], *state, s["tokens"])
        table = s["table"].clone()
        plain_plan(s["drop"], *state, 0)
        return *step, table, s["kv"], s["free"], s["count"]
    if case["op"] == "append":
        plain_append(s["K"], s["slots"], s["kcodes"], s["kscale"], page)
        plain_append(s["V"], s["slots"], s["vcodes"], s["vscale"], page)
        return (plain_read(s["back"], s["kcodes"], s["kscale"], page),
                plain_read(s["back"], s["vcodes"], s["vscale"], page), s["kscale"], s["vscale"])
    return plain_attention(s)


def work(case):
    news, kvs = lengths(case)
    page, new = case["page"], sum(news)
    if case["op"] == "plan":
        grown = sum(pages_of(n + k, page) - pages_of(k, page) for n, k in zip(news, kvs))
        # a step reads and writes each request's lengths and what it takes or gives back, and writes the slots;
        # the table that comes back is read and written once
        width = max(pages_of(n + k, page) for n, k in zip(news, kvs))
        return {"bytes": 4 * (2 * 5 * len(news) + 4 * grown + new + 2 * len(news) * width), "flops": 0}
    heads, dim = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        back = sum(k - (k - n) // page * page for n, k in zip(news, kvs))
        blocks = sum(pages_of(k, page) - (k - n) // page for n, k in zip(news, kvs))
        # bf16 in and codes out, then the touched tokens read as codes and written as bf16
        return {"bytes": 2 * heads * (dim * (3 * new + 3 * back) + 8 * blocks) + 4 * (new + back), "flops": 0}
    attended, cached = 0, 0
    for n, k in zip(news, kvs):
        w = case["window"] or k
        if case["causal"]:                            # the last query sees min(k, w) keys, the one before it one fewer, ...
            full = max(0, min(n, k - w + 1))          # queries whose window is full
            attended += full * w + sum(range(k - n + 1, k - full + 1)) if full < n else full * w
            cached += min(k, w + n - 1)
        else:
            attended += n * k
            cached += k
    blocks = sum(pages_of(k, page) for k in kvs)
    return {"bytes": 2 * heads * (cached * dim + 4 * blocks) + 4 * blocks + new * case["heads"] * (4 * dim + 4),
            "flops": 4 * dim * case["heads"] * attended}


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "plan":                          # whole numbers throughout, request by request
        news, kvs = lengths(case)
        table, stack = s["table"].tolist(), s["free"].tolist()
        top, slots, cu = int(s["count"]), [], [0]
        for b, (n, k) in enumerate(zip(news, kvs)):
            for pos in range(k, k + n):
                if pos % page == 0:
                    top -= 1
                    table[b][pos // page] = stack[top]
                slots.append(table[b][pos // page] * page + pos % page)
            cu.append(len(slots))
        whole = [torch.tensor(x, dtype=torch.int32) for x in (slots, cu, [0] * len(news), table)]
        return (*whole, s["kv"], s["free"], s["count"])
    if case["op"] == "append":
        values, scales = [], []
        for x, codes, scale in ((s["K"], s["kcodes"], s["kscale"]), (s["V"], s["vcodes"], s["vscale"])):
            x, scale = x.double(), scale.clone()
            value = (codes.double() - 128) * scale.double()[:, :, None, None]
            news, kvs = lengths(case)
            t, table = 0, s["table"].tolist()
            for b, (n, k) in enumerate(zip(news, kvs)):
                pos = k - n
                while pos < k:                        # one page at a time
                    p, off = table[b][pos // page], pos % page
                    m = min(page - off, k - pos)
                    part = x[t:t + m].transpose(0, 1)
                    most = (part.abs().amax((1, 2)) / 127).clamp(min=FLOOR).float()   # a scale is held in 32 bits
                    step = torch.maximum(most, scale[p]) if off else most
                    scale[p] = step
                    step = step.double()[:, None, None]
                    value[p, :, :off] = torch.round(value[p, :, :off].float().double() / step) * step
                    value[p, :, off:off + m] = torch.round(part / step) * step
                    pos, t = pos + m, t + m
            at, off = s["back"].long() // page, s["back"].long() % page
            values.append(value[at, :, off])
            scales.append(scale.double())
        return (*values, *scales)
    news, kvs = lengths(case)
    group, dim = case["heads"] // case["kv_heads"], case["dim"]
    outs, lses, t = [], [], 0
    for b, (n, k) in enumerate(zip(news, kvs)):
        at = s["table"][b, :pages_of(k, page)].long()
        q = s["Q"][t:t + n].double()
        t += n
        i = torch.arange(n, device=DEV)[:, None] + k - n
        j = torch.arange(k, device=DEV)
        hidden = (j > i) if case["causal"] else torch.zeros(n, k, dtype=torch.bool, device=DEV)
        if case["window"]:
            hidden = hidden | (j <= i - case["window"])
        out = torch.empty(n, case["heads"], dim, dtype=torch.float64, device=DEV)
        lse = torch.empty(n, case["heads"], dtype=torch.float64, device=DEV)
        for h in range(case["kv_heads"]):
            key, val = (((c[at, h].double() - 128) * z[at, h].double()[:, None, None]).reshape(-1, dim)[:k]
                        for c, z in ((s["kcodes"], s["kscale"]), (s["vcodes"], s["vscale"])))
            for m in range(h * group, (h + 1) * group):
                a = (q[:, m] @ key.T / math.sqrt(dim)).masked_fill(hidden, -math.inf)
                lse[:, m] = torch.logsumexp(a, 1)
                out[:, m] = torch.exp(a - lse[:, m:m + 1]) @ val
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
