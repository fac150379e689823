"""Plain CPU oracle of the paged 8-bit key/value cache (test infrastructure only).

The definitions of include/hbl.h, request by request and token by token, in
fp64 (scales are held in fp32, as the cache holds them). It shares no code
with the product path. Codes are unsigned; a block of one page and head
stands for (u - 128) * s.
"""
from __future__ import annotations

import math

import numpy as np

KV_SCALE_FLOOR = 2.0 ** -100
BF16_MAX = float(np.float32((2 - 2 ** -7) * 2.0 ** 127))


def kv_plan(new_lens, kv_lens, table, free_pages, free_count, page, tokens):
    """One step of the page table. Returns new copies of the state and what the step writes, as a dict."""
    table, stack = np.array(table), [int(x) for x in free_pages[:free_count]]
    B, width = table.shape
    pages = lambda n: -(-n // page)  # noqa: E731
    after = [max(0, int(n) + int(q)) for n, q in zip(kv_lens, new_lens)]
    cu = [0]
    for q in new_lens:
        cu.append(cu[-1] + max(0, int(q)))
    given = []
    for b in range(B):
        given += [int(table[b, j]) for j in range(pages(after[b]), pages(int(kv_lens[b])))]
    pool = given + stack[::-1]
    taken, used, refused = 0, 0, []
    slots = np.full(tokens, -1, dtype=np.int64)
    lens = [int(n) for n in kv_lens]
    for b in range(B):
        n, q = int(kv_lens[b]), int(new_lens[b])
        if q > 0 and (after[b] > width * page or cu[b + 1] > tokens):
            refused.append(1)
            continue
        need = max(0, pages(after[b]) - pages(n))
        start, taken = taken, taken + need
        if need and taken > len(pool):
            refused.append(1)
            continue
        refused.append(0)
        used = max(used, taken if need else 0)
        table[b, pages(n):pages(n) + need] = pool[start:taken]
        lens[b] = after[b]
        for i in range(max(0, q)):
            pos = n + i
            slots[cu[b] + i] = int(table[b, pos // page]) * page + pos % page
    left = stack[:len(stack) - max(0, used - len(given))] + given[used:][::-1]
    out = np.array(free_pages)
    out[:len(left)] = left
    return {"kv_lens": np.array(lens), "table": table, "free_pages": out, "free_count": len(left),
            "cu_q": np.minimum(np.array(cu), tokens), "slots": slots, "refused": np.array(refused)}


def kv_append(x, slots, codes, scale, page):
    """Tokens x (T, heads, D) into (codes, scale) of shape (pages, heads, page, D) and (pages, heads): new copies."""
    x = np.array(x, dtype=np.float64)
    x = np.where(np.isnan(x), 0.0, np.clip(x, -BF16_MAX, BF16_MAX))
    codes, scale = np.array(codes), np.array(scale, dtype=np.float32)
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        end = t + 1
        while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % page:
            end += 1
        p, off = int(slots[t]) // page, int(slots[t]) % page
        for h in range(scale.shape[1]):
            gamma = np.max(np.abs(x[t:end, h]))
            before = scale[p, h] if off else np.float32(0)
            s = max(before, np.float32(gamma / 127.0), np.float32(KV_SCALE_FLOOR))
            for j in range(off if s != before else 0):       # c * s / s is c, also where c * s is no float
                held = np.float32((codes[p, h, j].astype(np.float64) - 128.0) * np.float64(before))
                codes[p, h, j] = (np.rint(held.astype(np.float64) / np.float64(s)) + 128).astype(np.uint8)
            codes[p, h, off:off + end - t] = (np.rint(x[t:end, h] / np.float64(s)) + 128).astype(np.uint8)
            scale[p, h] = s
        t = end
    return codes, scale


def kv_read(slots, codes, scale, page):
    """Values of the named slots, fp64 (T, heads, D); zeros for a negative slot."""
    out = np.zeros((len(slots), codes.shape[1], codes.shape[3]))
    for t, s in enumerate(slots):
        if s >= 0:
            out[t] = (codes[s // page, :, s % page].astype(np.float64) - 128.0) * scale[s // page].astype(np.float64)[:, None]
    return out


def kv_attention(Q, cu_q, kv_lens, table, kcodes, vcodes, kscale, vscale, page, softmax_scale, causal=True, window=0):
    """(out, lse, magnitude, spread) in fp64 for Q (T, heads, D).

    magnitude: the same sums with |v|; spread: softmax_scale * max over the keys seen of sum |q||k|. Both
    serve error bounds. Rows that see nothing: zeros and -inf; rows of no request: NaN.
    """
    Q = np.asarray(Q, dtype=np.float64)
    T, heads, D = Q.shape
    kv_heads = kscale.shape[1]
    out = np.full((T, heads, D), np.nan)
    mag = np.full((T, heads, D), np.nan)
    lse, spread = np.full((T, heads), np.nan), np.zeros((T, heads))
    for b in range(len(kv_lens)):
        q0, q1, kv = int(cu_q[b]), int(cu_q[b + 1]), int(kv_lens[b])
        slots = [int(table[b, j // page]) * page + j % page for j in range(kv)]
        ok = np.array([0 <= s < kcodes.shape[0] * page for s in slots], dtype=bool)
        at = np.where(ok, slots, -1).astype(np.int64) if kv else np.zeros(0, dtype=np.int64)
        K, V = kv_read(at, kcodes, kscale, page), kv_read(at, vcodes, vscale, page)
        j = np.arange(kv)
        for t in range(q0, q1):
            pos = kv - (q1 - q0) + (t - q0)
            seen = ok.copy()
            if causal:
                seen &= j <= pos
            if window:
                seen &= j > pos - window
            for i in range(heads):
                h = i // (heads // kv_heads)
                if not seen.any():
                    out[t, i], mag[t, i], lse[t, i] = 0.0, 0.0, -math.inf
                    continue
                k, v = K[seen, h], V[seen, h]
                a = softmax_scale * (k @ Q[t, i])
                m = a.max()
                p = np.exp(a - m)
                l = p.sum()
                out[t, i], mag[t, i] = p @ v / l, p @ np.abs(v) / l
                lse[t, i] = m + math.log(l)
                spread[t, i] = softmax_scale * np.max(np.abs(k) @ np.abs(Q[t, i]))
    return out, lse, mag, spread
