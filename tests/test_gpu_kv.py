"""The paged 8-bit key/value cache on the GPU against the 64-bit oracle: page planning, appending, reading
back, attention, and the four together as a serving loop uses them."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from hadamard_bit_quant_b200 import build, hbl, layer
    build.build()
    assert torch.cuda.is_available()
    hbl.lib()
    yield layer
    assert hbl.hbl_get_device_error() == 0


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def np64(x):
    return x.double().cpu().numpy()


# ----------------------------------------------------------------------------- plan
def random_state(rng, B, page, max_pages, spare):
    """Lengths, a table and a stack of free pages, all pages somewhere."""
    kv = rng.integers(0, max_pages * page + 1, B)
    kv[rng.random(B) < 0.2] = 0
    held = -(-kv // page)
    num = int(held.sum()) + spare
    order = rng.permutation(num)
    table = rng.integers(0, num, (B, max_pages))
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(num, -7)
    free[:spare] = order[at:]
    return kv, table, free, spare, num


@pytest.mark.parametrize("B,page,max_pages,spare,most,T", [
    (1, 16, 1, 1, 5, 5), (1, 128, 4, 3, 200, 512), (3, 16, 5, 0, 20, 64), (9, 32, 7, 6, 64, 300),
    (40, 16, 9, 30, 40, 700), (33, 64, 3, 2, 90, 100), (257, 16, 12, 500, 60, 9000), (1500, 16, 4, 900, 9, 8000),
    (8192, 16, 2, 4000, 3, 20000)])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan(L, B, page, max_pages, spare, most, T, seed):
    rng = np.random.default_rng(1000 * seed + B)
    kv, table, free, count, num = random_state(rng, B, page, max_pages, spare)
    pages = L.KVPages(i32(kv), i32(table), i32(free), i32([count]), page)
    for step in range(3):
        new = rng.integers(-most, most + 1, B)
        new[rng.random(B) < 0.15] = 0
        new[rng.random(B) < 0.05] = -2 ** 31
        want = oracle.kv_plan(new, kv, table, free, count, page, T)
        got = pages.plan(i32(new), T)
        assert np.array_equal(got.cu_q.cpu(), want["cu_q"])
        assert np.array_equal(got.refused.cpu(), want["refused"])
        assert np.array_equal(got.slots.cpu(), want["slots"])
        assert np.array_equal(pages.kv_lens.cpu(), want["kv_lens"])
        assert np.array_equal(pages.block_table.cpu(), want["table"])
        assert int(pages.free_count) == want["free_count"]
        assert np.array_equal(pages.free_pages[:want["free_count"]].cpu(), want["free_pages"][:want["free_count"]])
        kv, table, count = want["kv_lens"], want["table"], want["free_count"]
        free = pages.free_pages.cpu().numpy()


def test_plan_survives_any_state(L):
    """Lengths, counts and page numbers that no step could have left: nothing out of bounds, what is bad is recorded."""
    from hadamard_bit_quant_b200 import hbl
    rng = np.random.default_rng(5)
    B, width, num = 50, 4, 30
    huge = rng.integers(-2 ** 31, 2 ** 31, 5 * B)
    guard = torch.full((num + 64,), 77, dtype=torch.int32, device="cuda")       # what lies behind the stack stays
    guard[:num] = i32(rng.integers(-2 ** 31, 2 ** 31, num))
    for new in (huge[:B], np.full(B, 3), np.full(B, -2 ** 31), rng.integers(-70, 70, B)):
        table = i32(rng.integers(-2 ** 31, 2 ** 31, (B, width)))
        pages = L.KVPages(i32(huge[B:2 * B]), table, guard[:num], i32([2 ** 31 - 1]), 16)
        step = pages.plan(i32(new), 200)
        slots = step.slots.cpu().numpy()
        assert np.all((slots >= -1) & (slots < num * 16))
        assert 0 <= int(pages.free_count) <= num and bool((guard[num:] == 77).all())
        lens = pages.kv_lens.cpu().numpy()
        assert np.all((lens >= 0) & (lens <= width * 16))
        cu = step.cu_q.cpu().numpy()
        assert cu[0] == 0 and np.all(np.diff(cu) >= 0) and cu[-1] <= 200
    assert hbl.hbl_get_device_error() == 1


def test_plan_dropping_a_step_restores_the_stack(L):
    rng = np.random.default_rng(3)
    kv, table, free, count, num = random_state(rng, 20, 16, 10, 40)
    pages = L.KVPages(i32(kv), i32(table), i32(free), i32([count]), 16)
    new = np.minimum(rng.integers(0, 30, 20), 160 - kv)
    step = pages.plan(i32(new), 600)
    assert int(step.refused.sum()) == 0
    pages.plan(i32(-new), 0)
    assert np.array_equal(pages.kv_lens.cpu(), kv) and int(pages.free_count) == count
    assert np.array_equal(pages.free_pages.cpu(), free)


# ----------------------------------------------------------------------------- append and read
def random_tokens(rng, T, H, D, kind):
    x = rng.standard_normal((T, H, D))
    if kind == "loud":
        x[:, :, rng.integers(0, D, 3)] *= 60
    elif kind == "ties":                 # halves of the absmax and of its steps: exact ties of x / s
        x = rng.integers(-254, 255, (T, H, D)) * 0.5
        x[:, :, 0] = 127
    elif kind == "tiny":
        x *= 1e-37
    elif kind == "zero":
        x[:] = 0
    elif kind == "odd":                  # NaN, infinities, the largest and the smallest values
        x[rng.random(x.shape) < 0.02] = np.nan
        x[rng.random(x.shape) < 0.01] = np.inf
        x[rng.random(x.shape) < 0.01] = -np.inf
        x[rng.random(x.shape) < 0.05] = 3.38e38
        x[rng.random(x.shape) < 0.05] = 1e-40
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def fresh_cache(L, rng, pages, H, page, D):
    """A cache whose memory holds anything: random codes, scales from tiny to NaN."""
    cache = L.KVCache.empty(pages, H, page, D)
    for c in (cache.kcodes, cache.vcodes):
        c.copy_(torch.tensor(rng.integers(0, 256, c.shape), dtype=torch.uint8))
    for s in (cache.kscale, cache.vscale):
        s.copy_(torch.tensor(rng.choice([0.0, 1e-3, 0.5, 40.0], s.shape), dtype=torch.float32))
    return cache


@pytest.mark.parametrize("H,D,page", [(1, 64, 16), (3, 128, 16), (5, 64, 128), (32, 128, 64), (8, 128, 32)])
@pytest.mark.parametrize("kind", ["plain", "loud", "ties", "tiny", "zero", "odd"])
def test_append_and_read(L, H, D, page, kind):
    rng = np.random.default_rng(H + D + page)
    num = 12
    cache = fresh_cache(L, rng, num, H, page, D)
    ref = [(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))]
    order = rng.permutation(num)
    # runs: (page, offset, tokens), page boundaries and skipped rows among them
    steps = [[(0, 0, 1), (1, 0, page), (2, 0, page - 3), (3, 0, 2)],
             [(0, 1, 1), (2, page - 3, 3), (4, 0, page), (3, 2, page - 5)],
             [(0, 2, page - 2), (3, page - 3, 1), (5, 0, 7)]]
    for i, runs in enumerate(steps):
        slots = []
        for p, off, n in runs:
            slots += [int(order[p]) * page + off + k for k in range(n)] + ([-1] if i == 1 else [])
        T = len(slots)
        x = random_tokens(rng, T, 2 * H, D, kind) * (4.0 if i == 1 and kind == "plain" else 1.0)
        xg = x.cuda()
        K, V = xg[:, :H], xg[:, H:]                      # parts of one tensor: tokens lie apart
        cache.append(K, V, i32(slots))
        for j, (part, (codes, scale)) in enumerate(((K, ref[0]), (V, ref[1]))):
            ref[j] = oracle.kv_append(np64(part), slots, codes, scale, page)
    for (codes, scale), (c, s) in zip(ref, ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))):
        assert np.array_equal(s.cpu().numpy(), scale)
        assert np.array_equal(c.cpu().numpy(), codes)    # exact quotients: every code, and every byte not named
    back = [-1] + [int(order[p]) * page + k for p in (0, 1, 2, 3, 4) for k in range(page)]
    for got, (codes, scale) in zip(cache.read(i32(back)), ref):
        want = torch.tensor(oracle.kv_read(back, codes, scale, page)).float().to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)


def test_append_many_requests_of_one_token(L):
    """Single tokens of 300 requests: every run is one token long, offsets of all kinds."""
    rng = np.random.default_rng(8)
    H, D, page, B = 2, 128, 16, 300
    cache = fresh_cache(L, rng, B, H, page, D)
    off = rng.integers(0, page, B)
    slots = rng.permutation(B) * page + off
    x = random_tokens(rng, B, 2 * H, D, "loud").cuda()
    want = [oracle.kv_append(np64(p), slots, c.cpu().numpy(), s.cpu().numpy(), page)
            for p, c, s in ((x[:, :H], cache.kcodes, cache.kscale), (x[:, H:], cache.vcodes, cache.vscale))]
    cache.append(x[:, :H], x[:, H:], i32(slots))
    for (codes, scale), (c, s) in zip(want, ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))):
        assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(c.cpu().numpy(), codes)


def test_append_a_prompt(L):
    """One long prompt that begins inside a page; consecutive pages follow each other in the cache (one row of
    slots without a gap must still be cut at the page ends)."""
    rng = np.random.default_rng(9)
    H, D, page, T = 3, 64, 32, 1000
    cache = fresh_cache(L, rng, 40, H, page, D)
    slots = np.arange(T) + 5 * page + 11
    x = random_tokens(rng, T, 2 * H, D, "plain").cuda()
    want = [oracle.kv_append(np64(p), slots, c.cpu().numpy(), s.cpu().numpy(), page)
            for p, c, s in ((x[:, :H], cache.kcodes, cache.kscale), (x[:, H:], cache.vcodes, cache.vscale))]
    cache.append(x[:, :H], x[:, H:], i32(slots))
    for (codes, scale), (c, s) in zip(want, ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))):
        assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(c.cpu().numpy(), codes)


# ----------------------------------------------------------------------------- attention
def close(got, lse, want, vmax, keys):
    """Error bounds of one attention call, by element.

    delta: a score is a sum of D products of exact fp16 values in fp32: D + 2 roundings of 2^-23 (the tensor
    cores may truncate), relative to sum |q||k|; then a product and a difference in fp32. A probability is
    off by that (twice, for the sum it is divided by), by 2^-11 for its rounding to fp16 and by 2^-25 at most
    below fp16's normal range, where it is relative to the largest: that much of 127 vmax for each key, over a
    sum of at least 1. The result is rounded to bf16, half a step.
    """
    out, ref_lse, mag, spread = want
    D = out.shape[2]
    got, lse = np64(got), np64(lse)
    rows = ~np.isnan(ref_lse)
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse[rows]), empty[rows])
    finite = rows & ~empty
    delta = spread * (D + 6) * 2.0 ** -23 + 2.0 ** -20
    assert np.all(np.abs(lse[finite] - ref_lse[finite]) <= (delta + np.abs(np.where(finite, ref_lse, 0)) * 2.0 ** -21)[finite])
    bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -10 + 4 * delta[..., None]) * mag + 2.0 ** -25 * 127 * vmax * keys
    err = np.abs(got - out)
    assert np.all(err[rows] <= bound[rows]), float(np.nanmax((err - bound)[rows]))
    assert np.all(got[empty] == 0)


def make_case(L, seed, qs, kvs, Hq, Hkv, D, page, spare_rows=0, width=None, scale_spread=0.3):
    rng = np.random.default_rng(seed)
    B = len(qs)
    counts = [-(-k // page) for k in kvs]
    width = width or max(1, max(counts) + 1)
    num = sum(counts) + 2
    order = rng.permutation(num)
    table = rng.integers(0, num, (B, width))
    at = 0
    for b in range(B):
        table[b, :counts[b]] = order[at:at + counts[b]]
        at += counts[b]
    cache = L.KVCache.empty(num, Hkv, page, D)
    for c in (cache.kcodes, cache.vcodes):
        c.copy_(torch.tensor(np.clip(np.rint(rng.standard_normal(c.shape) * 32), -127, 127) + 128, dtype=torch.uint8))
    for s in (cache.kscale, cache.vscale):
        s.copy_(torch.tensor(np.exp(rng.standard_normal(s.shape) * scale_spread) * 0.03, dtype=torch.float32))
    T = sum(qs) + spare_rows
    cu = np.concatenate([[0], np.cumsum(qs)])
    Q = torch.tensor(rng.standard_normal((T, Hq, D)) * 2, dtype=torch.float32).to(torch.bfloat16).cuda()
    return cache, Q, cu, np.array(kvs), table


def reference(cache, Q, cu, kvs, table, **kw):
    return oracle.kv_attention(np64(Q), cu, kvs, table, cache.kcodes.cpu().numpy(), cache.vcodes.cpu().numpy(),
                               cache.kscale.cpu().numpy(), cache.vscale.cpu().numpy(), cache.page,
                               kw.pop("scale", cache.head_dim ** -0.5), **kw)


def check(L, case, **kw):
    cache, Q, cu, kvs, table = case
    want = reference(*case, **kw)
    out = torch.full_like(Q, 7.0)
    lse = torch.full(Q.shape[:2], 7.0, device="cuda")
    got, glse = cache.attention(Q, i32(cu), i32(kvs), i32(table), out=out, lse=lse, return_lse=True, **kw)
    assert got is out and glse is lse
    close(got, glse, want, float(cache.vscale.max()), int(np.max(kvs, initial=1)))
    behind = np.isnan(want[1])
    assert np.all(np64(got)[behind] == 7) and np.all(np64(glse)[behind] == 7)       # rows of no request: as they were
    return got, glse


# Batches of up to 6144 rows of all heads go to the kernel that streams the keys, whatever their requests; more (rows
# behind the last request count too) send a request of more than 32 rows a head to the tensor-core kernel.
BOTH = pytest.mark.parametrize("many", [False, True])


def spare(many, heads, least=0):
    return 6144 // heads + 1 if many else least


HEADS = [(4, 4, 128, 16), (8, 1, 64, 32), (6, 2, 128, 64), (16, 1, 128, 128), (3, 3, 64, 16), (40, 2, 64, 64)]


@pytest.mark.parametrize("Hq,Hkv,D,page", HEADS)
def test_attention_single_tokens(L, Hq, Hkv, D, page):
    kvs = [1, 2, page - 1, page, page + 1, 31, 32, 33, 257, 0, 700]
    check(L, make_case(L, 1, [1] * len(kvs), kvs, Hq, Hkv, D, page))


@pytest.mark.parametrize("Hq,Hkv,D,page", HEADS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40)])
@BOTH
def test_attention_ragged_rows(L, Hq, Hkv, D, page, causal, window, many):
    qs = [3, 0, 1, 17, 40, 5, 2, 8]
    kvs = [3, 9, 300, 17, 90, 2, 0, 140]      # 5 rows over 2 keys and 2 over none: rows that see nothing
    check(L, make_case(L, 2, qs, kvs, Hq, Hkv, D, page, spare_rows=spare(many, Hq, 3)), causal=causal, window=window)


@pytest.mark.parametrize("kv,Hq,Hkv,D,page", [(20011, 4, 1, 128, 16), (40000, 2, 2, 64, 64), (9973, 16, 1, 128, 128)])
def test_attention_long_context_is_split(L, kv, Hq, Hkv, D, page):
    check(L, make_case(L, 3, [1], [kv], Hq, Hkv, D, page))
    check(L, make_case(L, 4, [2, 1], [kv // 2, 5], Hq, Hkv, D, page), window=kv // 3)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 4, 128, 16), (4, 2, 64, 128), (8, 2, 128, 64), (5, 1, 128, 32)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
@BOTH
def test_attention_prompts(L, Hq, Hkv, D, page, causal, window, many):
    check(L, make_case(L, 5, [200, 333, 1, 64], [200, 500, 77, 70], Hq, Hkv, D, page, spare_rows=spare(many, Hq, 2)),
          causal=causal, window=window)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(2, 1, 128, 16), (2, 2, 64, 32), (3, 1, 64, 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 300)])
@BOTH
def test_attention_long_prompts(L, Hq, Hkv, D, page, causal, window, many):
    """More keys than any ring holds, more rows than a tile, block scales that keep outgrowing what came before."""
    case = make_case(L, 15, [450, 130], [1500, 2049], Hq, Hkv, D, page, spare(many, Hq), scale_spread=1.5)
    check(L, case, causal=causal, window=window)
    cache, Q, cu, kvs, table = case
    grow = torch.arange(table.shape[1], device="cuda", dtype=torch.float32)
    for b in range(2):                                       # louder from page to page, keys and values
        at = torch.tensor(table[b], device="cuda").long()[:-(-int(kvs[b]) // page)]
        cache.kscale[at] = (0.002 * 1.05 ** grow[:len(at)])[:, None].clamp(max=0.1)
        cache.vscale[at] = (1e-6 * 1.5 ** grow[:len(at)])[:, None].clamp(max=1e3)
    check(L, case, causal=causal, window=window)


@BOTH
def test_attention_prompts_of_all_scales(L, many):
    """Zero scales, and first tiles that a row does not see at all."""
    case = make_case(L, 16, [300, 100, 90], [300, 60, 0], 2, 1, 128, 32, spare(many, 2))      # the last has no key at all
    check(L, case)
    case[0].vscale[:] = 0
    check(L, case)
    case[0].vscale[::2] = 0.5
    case[0].kscale[::3] = 0
    check(L, case)


def test_attention_rows_beyond_the_bound_are_left(L):
    from hadamard_bit_quant_b200 import hbl
    case = make_case(L, 17, [2, 300], [50, 400], 4, 2, 64, 16)
    cache, Q, cu, kvs, table = case
    out = torch.full_like(Q, 7.0)
    cache.attention(Q, i32(cu), i32(kvs), i32(table), max_q=2, out=out)
    assert hbl.hbl_get_device_error() == 1
    assert bool((out[2:] == 7).all())
    assert torch.equal(out[:2], cache.attention(Q, i32(cu), i32(kvs), i32(table))[:2])


@BOTH
def test_attention_widest_window_and_rows(L, many):
    """A window as wide as an int and more rows than keys: no limit of the kernels' own shows."""
    case = make_case(L, 18, [5, 300], [2, 100], 2, 1, 64, 16, spare(many, 2))
    cache, Q, cu, kvs, table = case
    want = check(L, case)
    got = cache.attention(Q, i32(cu), i32(kvs), i32(table), window=2 ** 31 - 1, return_lse=True)
    assert torch.equal(want[0][:305], got[0][:305]) and torch.equal(want[1][:305], got[1][:305])


@pytest.mark.parametrize("kvs", [[130], [512, 1, 0], [513, 40, 33]])
def test_attention_short_and_split_agree(L, kvs):
    """The same rows by one block each (short contexts) and split between blocks."""
    case = make_case(L, 19, [1] * len(kvs), kvs, 8, 4, 128, 32, width=20)
    cache, Q, cu, kv, table = case
    want = reference(*case)
    for kw in ({"max_q": 1, "max_kv": max(kvs)}, {"max_q": 1}, {"max_q": 1, "max_kv": 5}):
        out, lse = cache.attention(Q, i32(cu), i32(kv), i32(table), return_lse=True, **kw)
        close(out, lse, want, float(cache.vscale.max()), max(kvs))


def test_layer_refuses(L):
    case = make_case(L, 20, [1, 1], [40, 30], 4, 2, 64, 16)
    cache, Q, cu, kvs, table = case
    cu, kvs, table = i32(cu), i32(kvs), i32(table)
    for bad in (lambda: cache.attention(Q.float(), cu, kvs, table), lambda: cache.attention(Q, cu.long(), kvs, table),
                lambda: cache.attention(Q, cu[:-1], kvs, table), lambda: cache.attention(Q.cpu(), cu, kvs, table),
                lambda: cache.attention(Q, cu.cpu(), kvs, table), lambda: cache.attention(Q[..., :32], cu, kvs, table),
                lambda: cache.attention(Q, cu, kvs, table[:1]), lambda: cache.attention(Q, cu, kvs, table, out=Q.float()),
                lambda: cache.append(Q, Q, kvs), lambda: cache.append(Q[:, :2], Q[:1, :2], kvs),
                lambda: cache.read(kvs.float()), lambda: L.KVCache(cache.kcodes, cache.vcodes[:1], cache.kscale, cache.vscale),
                lambda: L.KVCache(cache.kcodes.cpu(), cache.vcodes, cache.kscale, cache.vscale),
                lambda: L.KVPages(kvs, table.t(), kvs, kvs[:1], 16)):
        with pytest.raises((AssertionError, ValueError)):
            bad()
    from hadamard_bit_quant_b200.hbl import HblError
    for bad in (lambda: cache.attention(Q, cu, kvs, table, window=-1), lambda: cache.attention(Q, cu, kvs, table, scale=0.0),
                lambda: cache.attention(Q, cu, kvs, table, causal=False, window=3),
                lambda: cache.attention(Q[:, :3].contiguous(), cu, kvs, table),
                lambda: cache.attention(Q, cu, kvs, table, ws=torch.empty(256, dtype=torch.uint8, device="cuda")),
                lambda: L.KVPages(kvs, table, kvs, kvs[:1], 20).plan(kvs, 4)):
        with pytest.raises(HblError):
            bad()


@BOTH
def test_attention_hints_do_not_change_results(L, many):
    case = make_case(L, 6, [1, 4, 150], [100, 900, 400], 8, 2, 128, 32, spare(many, 8))
    got = [check(L, case, **kw) if not kw else case[0].attention(case[1], i32(case[2]), i32(case[3]), i32(case[4]),
                                                                 return_lse=True, **kw)
           for kw in ({}, {"max_q": 150, "max_kv": 900})]
    want = reference(*case)
    for o, l in got:
        close(o, l, want, float(case[0].vscale.max()), 900)


def test_attention_many_requests(L):
    rng = np.random.default_rng(11)
    kvs = rng.integers(0, 40, 700)
    check(L, make_case(L, 7, rng.integers(0, 3, 700), kvs, 2, 1, 64, 16))


@BOTH
def test_attention_scales_of_all_sizes(L, many):
    """Block scales from 2^-60 to 2^40 side by side, queries from 1e-30 to 3e38."""
    case = make_case(L, 8, [40, 1] if many else [1, 1], [500, 90], 4, 2, 128, 16, spare(many, 4))
    cache, Q = case[0], case[1]
    rng = np.random.default_rng(5)
    cache.vscale.copy_(torch.tensor(2.0 ** rng.integers(-60, 40, cache.vscale.shape), dtype=torch.float32))
    check(L, case)
    cache.vscale.fill_(0.03)
    cache.kscale.mul_(1e30)
    Q.copy_((Q.float() * 1e-30).to(torch.bfloat16))
    check(L, case)
    cache.kscale.mul_(1e-35)
    cache.kscale.mul_(1e-25)
    Q.copy_((Q.float() * 1e30).to(torch.bfloat16))
    Q.mul_(1e30)
    check(L, case)
    Q.mul_(3e7).clamp_(-3e38, 3e38)
    Q[0, 0, :40] = 3e38
    check(L, case, scale=2.0 ** -27)


def test_cache_beyond_32_bit_offsets(L):
    """Pages more than 4 GiB into the cache: the same bits as in a small cache."""
    H, D, page, T = 8, 128, 64, 300
    far = L.KVCache(*(torch.empty(66000, H, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)),
                    *(torch.zeros(66000, H, device="cuda") for _ in range(2)))
    near = L.KVCache.empty(8, H, page, D)
    ids = [65999, 3, 65700, 65536, 65998]
    pos = np.arange(T)
    slots = [i32(np.array(p)[pos // page] * page + pos % page) for p in (ids, [0, 1, 2, 3, 4])]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    Q = torch.randn(T, 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    outs = []
    for cache, s, p in ((far, slots[0], ids), (near, slots[1], [0, 1, 2, 3, 4])):
        cache.append(x[:250, :H], x[:250, H:], s[:250])
        cache.append(x[250:, :H], x[250:, H:], s[250:])       # rescales what the page holds
        table = i32([p])
        outs.append((*cache.read(s), *cache.attention(Q, i32([0, T]), i32([T]), table, return_lse=True),
                     cache.attention(Q[:1], i32([0, 1]), i32([T]), table)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(far.kcodes[65999], near.kcodes[0]) and torch.equal(far.vscale[ids], near.vscale[:5])


def test_attention_what_is_masked_has_no_influence(L):
    """NaN and infinite scales of pages that no row sees, and rows behind the last key of a page."""
    case = make_case(L, 9, [1, 2], [100, 300], 4, 2, 128, 16)
    cache, Q, cu, kvs, table = case
    first = [c.clone() for c in check(L, case, window=50)]
    used = set()
    for b, (lo, hi) in enumerate(((50, 100), (249, 300))):
        used |= {int(table[b, j]) for j in range(lo // 16, -(-hi // 16))}
    for p in range(cache.num_pages):
        if p not in used:
            cache.kscale[p], cache.vscale[p] = float("nan"), float("inf")
            cache.kcodes[p], cache.vcodes[p] = 0, 255
    again = cache.attention(Q, i32(cu), i32(kvs), i32(table), window=50, return_lse=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("rows", [4, 80])      # 80 of them, and padding: the tensor-core kernel
def test_attention_odd_queries(L, rows):
    """A NaN or an infinity in one row stays in that row; a row of zeros averages the values."""
    case = make_case(L, 10, [rows], [200], 2, 1, 64, 32, spare(rows > 32, 2))
    cache, Q, cu, kvs, table = case
    Q[1, 0, 3] = float("nan")
    Q[2, 1, 5] = float("inf")
    Q[3, 0] = 0
    out, lse = cache.attention(Q, i32(cu), i32(kvs), i32(table), return_lse=True)
    bad = torch.zeros(len(Q), 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    good = ~bad & (torch.arange(len(Q), device="cuda") < rows)[:, None]
    assert out[good].isfinite().all() and lse[good].isfinite().all()
    assert out[1, 0].isnan().all() and lse[1, 0].isnan()
    clean = Q.clone()
    clean[1, 0, 3] = 0
    clean[2, 1, 5] = 0
    want = reference(cache, clean, cu, kvs, table)
    want[1][bad.cpu().numpy()] = np.nan                      # not compared
    close(out, lse, want, float(cache.vscale.max()), 200)


def test_attention_query_as_part_of_a_projection(L):
    case = make_case(L, 12, [3, 1], [60, 200], 4, 2, 64, 16)
    cache, Q, cu, kvs, table = case
    wide = torch.randn(4, 4 + 2 + 2, 64, device="cuda").to(torch.bfloat16)
    wide[:, :4] = Q
    want = cache.attention(Q, i32(cu), i32(kvs), i32(table), return_lse=True)
    got = cache.attention(wide[:, :4], i32(cu), i32(kvs), i32(table), return_lse=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_bad_pages_and_slots_are_skipped_and_recorded(L):
    from hadamard_bit_quant_b200 import hbl
    assert hbl.hbl_get_device_error() == 0
    for rows, pad in ((2, 0), (90, 1600)):                    # the streaming kernel, the tensor-core kernel
        case = make_case(L, 13, [1, rows], [100, 200], 4, 2, 128, 16, pad)
        cache, Q, cu, kvs, table = case
        table[0, 2], table[1, 5], table[1, 0] = -1, cache.num_pages, 2 ** 31 - 1
        check(L, case)
        assert hbl.hbl_get_device_error() == 1
        assert hbl.hbl_get_device_error() == 0
    before = [x.clone() for x in (cache.kcodes, cache.vcodes, cache.kscale, cache.vscale)]
    x = torch.randn(2, 2, 128, device="cuda").to(torch.bfloat16)
    cache.append(x, x, i32([cache.num_pages * 16, 2 ** 31 - 1]))
    assert hbl.hbl_get_device_error() == 1
    for a, b in zip(before, (cache.kcodes, cache.vcodes, cache.kscale, cache.vscale)):
        assert torch.equal(a, b)
    K, _ = cache.read(i32([cache.num_pages * 16, 3]))
    assert hbl.hbl_get_device_error() == 1
    assert bool((K[0] == 0).all())
    # lengths beyond the table and rows beyond the queries are cut
    out = cache.attention(Q, i32([0, 1, 9000]), i32([2 ** 30, -5]), i32(np.abs(table) % cache.num_pages))
    assert out[0].isfinite().all() and bool((out[1:] == 0).all())


# ----------------------------------------------------------------------------- together
def test_serving_loop(L):
    """Requests arrive, decode, draft, are rejected and released; after every step the cache and the attention
    over it are those of the oracle."""
    rng = np.random.default_rng(21)
    B, Hq, Hkv, D, page, num, width = 5, 4, 2, 64, 16, 24, 8
    pages = L.KVPages.empty(B, width, num, page)
    cache = L.KVCache.empty(num, Hkv, page, D)
    ref = {"kv": np.zeros(B, int), "table": np.zeros((B, width), int), "free": np.arange(num)[::-1].copy(), "count": num}
    codes = [(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))]
    plans = [[40, 17, 0, 0, 1], [1, 1, 30, 0, 1], [1, 4, 1, 50, 1], [1, -3, 1, 1, -1], [-41, 1, 1, 1, 1],
             [100, 4, 4, 4, 4], [-2 ** 31, 1, -33, 1, 1], [70, 1, 16, 1, 1]]
    for new in plans:
        T = sum(max(0, n) for n in new) + 2
        step = pages.plan(i32(new), T)
        want = oracle.kv_plan(np.array(new), ref["kv"], ref["table"], ref["free"], ref["count"], page, T)
        ref = {"kv": want["kv_lens"], "table": want["table"], "free": want["free_pages"], "count": want["free_count"]}
        assert np.array_equal(step.slots.cpu(), want["slots"]) and int(pages.free_count) == want["free_count"]
        assert int(step.refused.sum()) == 0
        qkv = torch.tensor(rng.standard_normal((T, Hq + 2 * Hkv, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
        Q, K, V = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        cache.append(K, V, step.slots)
        codes = [oracle.kv_append(np64(x), want["slots"], c, s, page) for x, (c, s) in zip((K, V), codes)]
        out, lse = cache.attention(Q, step.cu_q, pages.kv_lens, pages.block_table, return_lse=True)
        for (c, s), (gc, gs) in zip(codes, ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))):
            assert np.array_equal(gc.cpu().numpy(), c) and np.array_equal(gs.cpu().numpy(), s)
        close(out, lse, oracle.kv_attention(np64(Q), want["cu_q"], ref["kv"], ref["table"], codes[0][0], codes[1][0],
                                            codes[0][1], codes[1][1], page, D ** -0.5), float(cache.vscale.max()),
              int(max(1, ref["kv"].max())))


def test_captured_step_replays_with_new_lengths(L):
    """One decode step (plan, append, attention) captured once and replayed: lengths live on the GPU, so each replay
    adds a token to every request."""
    B, Hq, Hkv, D, page, num, width = 3, 8, 4, 128, 16, 40, 8

    def make():
        pages = L.KVPages.empty(B, width, num, page)
        cache = L.KVCache.empty(num, Hkv, page, D)
        g = torch.Generator(device="cuda").manual_seed(4)
        x = torch.randn(40, 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        step = pages.plan(i32([13, 20, 7]), 40)
        cache.append(x[:, :Hkv], x[:, Hkv:], step.slots)
        return pages, cache, g

    one, qkv = i32([1] * B), torch.empty(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")

    def decode(pages, cache, ws, out):
        step = pages.plan(one, B)
        cache.append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], step.slots)
        return cache.attention(qkv[:, :Hq], step.cu_q, pages.kv_lens, pages.block_table, max_q=1, out=out, ws=ws)

    pages, cache, g = make()
    ws, out = cache.workspace(B), torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    qkv.normal_(generator=g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                            # a call on another stream than the tensors' own
        decode(pages, cache, ws, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(pages, cache, ws, out)
    outs = []
    pages2, cache2, g2 = make()
    g.manual_seed(99)
    for i in range(20):
        if i:
            qkv.normal_(generator=g)
        else:
            # the eager copy takes the step that was run before the capture
            g2.manual_seed(4)
            torch.randn(40, 2 * Hkv, D, generator=g2, device="cuda")
            keep = qkv.clone()
            qkv.normal_(generator=g2)
            decode(pages2, cache2, cache2.workspace(B), torch.empty_like(out))
            qkv.copy_(keep)
        graph.replay()
        outs.append(out.clone())
        eager = decode(pages2, cache2, cache2.workspace(B), torch.empty_like(out))
        assert torch.equal(outs[-1], eager)
    assert np.array_equal(pages.kv_lens.cpu(), [13 + 21, 20 + 21, 7 + 21])
    assert torch.equal(cache.kcodes[pages.block_table[0, 0].item()], cache2.kcodes[pages2.block_table[0, 0].item()])


def test_two_streams_with_workspaces_of_their_own(L):
    case = make_case(L, 14, [1] * 4, [3000, 200, 5000, 1], 8, 2, 128, 64)
    cache, Q, cu, kvs, table = case
    args = i32(cu), i32(kvs), i32(table)
    want = cache.attention(Q, *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for r in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(cache.attention(Q, *args, ws=cache.workspace(4)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("handle", [False, True])
def test_allocations_belong_to_the_stream_of_the_call(L, monkeypatch, handle):
    """A call on another stream than the current one frees its workspace when it returns: that memory must stay with its
    stream."""
    case = make_case(L, 15, [1] * 4, [3000, 200, 5000, 1], 8, 2, 128, 64)
    cache, Q, cu, kvs, table = case
    args = i32(cu), i32(kvs), i32(table)
    want = cache.attention(Q, *args, return_lse=True)
    slots = torch.arange(100, dtype=torch.int32, device="cuda")
    values = cache.read(slots)
    seen, call = [], L.hbl.hbl_kv_attention
    monkeypatch.setattr(L.hbl, "hbl_kv_attention", lambda *a: seen.append(a[-3].data_ptr()) or call(*a))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = s.cuda_stream if handle else s
    got = cache.attention(Q, *args, return_lse=True, stream=on)
    again = cache.workspace(4)
    assert seen and again.data_ptr() != seen[0]
    read = cache.read(slots, stream=on)
    pages, new = L.KVPages.empty(3, 4, 12, 16), i32([5, 0, 17])
    torch.cuda.synchronize()
    step = pages.plan(new, 22, stream=on)
    s.synchronize()
    assert all(torch.equal(g, w) for g, w in zip((*got, *read), (*want, *values)))
    assert step.cu_q.tolist() == [0, 5, 5, 22] and step.slots.tolist()[:6] == [0, 1, 2, 3, 4, 16]


def test_a_batch_has_a_request(L):
    with pytest.raises(AssertionError):
        L.KVPages.empty(0, 4, 8, 16)


@pytest.mark.parametrize("B,Hkv,rows", [(24, 1, 17), (3, 8, 40), (1, 2, 1)])
def test_attention_any_bound_on_the_rows(L, B, Hkv, rows):
    """A bound beyond all rows, up to the widest int, is no bound: the same bits, over short contexts too."""
    case = make_case(L, 22, [rows] * B, [512] * B, 2 * Hkv, Hkv, 64, 16, spare_rows=2)
    cache, Q, cu, kvs, table = case
    args, ref = (Q, i32(cu), i32(kvs), i32(table)), reference(*case)
    for kw in ({}, {"max_kv": 512}):
        want = cache.attention(*args, return_lse=True, **kw)
        close(*want, ref, float(cache.vscale.max()), 512)
        for max_q in (len(Q) - 1, len(Q), len(Q) + 1, 2 ** 27, 2 ** 31 - 1):
            got = cache.attention(*args, return_lse=True, max_q=max_q, **kw)
            if max_q < len(Q):                               # fewer row tiles: other parts, not other results
                close(*got, ref, float(cache.vscale.max()), 512)
            else:
                assert all(torch.equal(g[:rows * B], w[:rows * B]) for g, w in zip(got, want))


@pytest.mark.parametrize("B", [3054, 3055, 3071, 8192])
def test_plan_in_a_fresh_process(B):
    """Batches about the size where the kernel's shared memory passes 48 KB, with no larger one before them."""
    import os
    import subprocess
    import sys
    code = f"""
import torch
from hadamard_bit_quant_b200 import layer
pages = layer.KVPages.empty({B}, 1, {B}, 16)
step = pages.plan(torch.ones({B}, dtype=torch.int32, device="cuda"), {B})
assert int(step.refused.sum()) == 0 and int(pages.free_count) == 0
assert torch.equal(step.slots.cpu(), 16 * torch.arange({B}, dtype=torch.int32))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_plan_of_the_most_rows(L):
    """As many rows as an int counts: each of them is written, and nothing but them."""
    T = 2 ** 31 - 1
    buf = torch.full((T + 64,), 7, dtype=torch.int32, device="cuda")
    pages = L.KVPages.empty(2, 4, 8, 16)
    step = L.KVStep(buf[:T], i32([0] * 3), i32([0] * 2))
    pages.plan(i32([20, 3]), T, out=step)
    assert step.cu_q.tolist() == [0, 20, 23] and step.refused.tolist() == [0, 0]
    assert step.slots[:23].tolist() == list(range(20)) + [32, 33, 34]
    assert bool((buf[T:] == 7).all())
    for part in buf[23:T].split(2 ** 28):
        assert int(part.max()) == int(part.min()) == -1


@pytest.mark.parametrize("q", [5, 10])
@pytest.mark.parametrize("kv,kw", [(300, {}), (300, {"max_kv": 512}), (20000, {})])
@BOTH
def test_attention_few_rows_beyond_the_bound_are_left(L, q, kv, kw, many):
    """Rows beyond the bound that a kernel of few rows could take: left all the same, the other requests' are written."""
    from hadamard_bit_quant_b200 import hbl
    case = make_case(L, 23, [2, q, 1], [50, kv, 40], 4, 2, 64, 16, spare(many, 4), width=32 if kv < 500 else None)
    cache, Q, cu, kvs, table = case
    out, lse = torch.full_like(Q, 7.0), torch.full(Q.shape[:2], 7.0, device="cuda")
    cache.attention(Q, i32(cu), i32(kvs), i32(table), max_q=2, out=out, lse=lse, return_lse=True, **kw)
    assert hbl.hbl_get_device_error() == 1
    left = slice(2, 2 + q)
    assert bool((out[left] == 7).all()) and bool((lse[left] == 7).all())
    kvs = kvs.copy()
    kvs[1] = 0                                               # not compared, and quick
    want = reference(cache, Q, cu, kvs, table)
    want[1][left] = np.nan
    close(out, lse, want, float(cache.vscale.max()), 50)


# ----------------------------------------------------------------------------- a row and the keys that it sees
def own_bounds(case, scale=None, causal=True, window=0, lag=0):
    """(out, lse, bound, lse bound) of each row from the keys that it sees alone, and nothing of other rows, heads or
    requests; NaN where a row belongs to no request.

    A weight is w = p s, of the key's probability and value scale. It is rounded to fp16 relative to a reference that is
    never above 2^lag of the row's largest weight: by 2^-11 of itself, or by 2^-25 of the reference where that is more,
    times a code of at most 127. Scales below 2^-110, but for 0, count as that much. delta is ``close``'s, but that the log2 of a scale is added to the exponent: up to 2^8,
    off by 2^-17 once for the weight and once for the sum. bf16's least values are 2^-133 apart.
    """
    cache, Q, cu, kvs, table = case
    Q, page, D = np64(Q), cache.page, cache.head_dim
    scale = D ** -0.5 if scale is None else scale
    codes = [c.cpu().numpy().astype(np.float64) - 128 for c in (cache.kcodes, cache.vcodes)]
    ks, vs = (s.double().cpu().numpy() for s in (cache.kscale, cache.vscale))
    T, heads, _ = Q.shape
    out, bound = np.full((2, T, heads, D), np.nan)
    lse, off = np.full((2, T, heads), np.nan)
    for b, kv in enumerate(int(k) for k in kvs):
        rows = np.arange(cu[b], cu[b + 1])
        j = np.arange(kv)
        pos = kv - len(rows) + np.arange(len(rows))[:, None]
        seen = np.ones((len(rows), kv), bool) if not causal else j <= pos
        if window:
            seen = seen & (j > pos - window)
        at, o = table[b, j // page], j % page
        for i in range(heads):
            h = i // (heads // cache.kv_heads)
            k, v, s = codes[0][at, h, o] * ks[at, h][:, None], codes[1][at, h, o], vs[at, h]
            a = np.where(seen, scale * (Q[rows, i] @ k.T), -np.inf)
            spread = scale * np.max(np.where(seen, np.abs(Q[rows, i]) @ np.abs(k).T, 0), axis=1, initial=0)
            m = np.max(a, axis=1, initial=-np.inf, keepdims=True)
            p = np.exp(a - np.where(np.isneginf(m), 0, m))
            l = p.sum(1)
            w = p * s
            delta = spread * (D + 6) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -16
            with np.errstate(divide="ignore", invalid="ignore"):
                lse[rows, i] = m[:, 0] + np.log(l)
                inv = np.where(l > 0, 1 / l, 0)
            out[rows, i] = (w @ v) * inv[:, None]
            mag = (w @ np.abs(v)) * inv[:, None]
            tiny = 2.0 ** (lag - 25) * 127 * w.max(1, initial=0) * inv * seen.sum(1)
            bound[rows, i] = 2.0 ** -134 + 2.0 ** -8 * np.abs(out[rows, i]) + (2.0 ** -11 + 4 * delta[:, None]) * mag + tiny[:, None]
            off[rows, i] = delta + np.abs(np.where(l > 0, lse[rows, i], 0)) * 2.0 ** -21
    return out, lse, bound, off


def check_rows(case, **kw):
    cache, Q, cu, kvs, table = case
    out, lse, bound, off = own_bounds(case, **kw)
    kw.pop("lag", None)
    got, glse = (np64(x) for x in cache.attention(Q, i32(cu), i32(kvs), i32(table), return_lse=True, **kw))
    rows = ~np.isnan(lse)
    some = rows & np.isfinite(lse)
    assert np.array_equal(np.isneginf(glse[rows]), np.isneginf(lse[rows]))
    assert np.all(np.abs(glse[some] - lse[some]) <= off[some])
    worst = np.abs(got - out) - bound
    assert np.all(worst[rows] <= 0), (float(np.max(worst[rows])), np.argwhere(rows)[np.argmax(worst.max(2)[rows])])


# rows of a request, query heads, key/value heads: 8 rows a tile, 16 rows, and more, which `many` sends to the tensor cores
SHAPES = pytest.mark.parametrize("q,Hq,Hkv,D,page,many", [
    (6, 2, 2, 128, 16, False), (6, 2, 2, 64, 16, False), (20, 2, 2, 128, 16, False), (15, 4, 2, 64, 32, False),
    (60, 2, 1, 128, 16, True), (300, 2, 2, 64, 16, True), (150, 4, 1, 128, 64, True)])


@SHAPES
@pytest.mark.parametrize("louder", [14, 20, 28, 40, 110])
def test_attention_later_keys_do_not_round_a_row(L, q, Hq, Hkv, D, page, many, louder):
    """Values that only later rows see are louder by far; a row's result is as exact as without them."""
    for kv in (q, q + 2 * page + 3):
        case = make_case(L, 24, [q, 3], [kv, 2 * page], Hq, Hkv, D, page, spare(many, Hq))
        cache, _, _, _, table = case
        first = max(kv - q // 2, page) // page               # pages from here on are loud
        at = torch.tensor(table[0, first:-(-kv // page)], device="cuda").long()
        cache.vscale[at] *= 2.0 ** louder
        check_rows(case)


@SHAPES
@pytest.mark.parametrize("louder", [20, 40])
def test_attention_keys_before_the_window_do_not_round_a_row(L, q, Hq, Hkv, D, page, many, louder):
    """Loud values in front of a row's window, which earlier rows see."""
    kv = q + 4 * page + 5
    case = make_case(L, 25, [q], [kv], Hq, Hkv, D, page, spare(many, Hq))
    cache, _, _, _, table = case
    window = 5
    last = (kv - q + 1) // page                              # the first rows' keys and all before them
    cache.vscale[torch.tensor(table[0, :last + 1], device="cuda").long()] *= 2.0 ** louder
    check_rows(case, window=window)


@SHAPES
def test_attention_largest_and_smallest_values_side_by_side(L, q, Hq, Hkv, D, page, many):
    """What appending makes of an infinity, of zeros and of ordinary values, over all that a row sees: the largest stay
    finite, and the smallest count in the sum."""
    kv = max(q, 12 * page)
    case = make_case(L, 26, [q], [kv], Hq, Hkv, D, page, spare(many, Hq))
    cache, Q, cu, kvs, table = case
    top = float(torch.tensor((2 - 2 ** -7) * 2.0 ** 127 / 127, dtype=torch.float32))
    pages = torch.tensor(table[0, :-(-kv // page)], device="cuda").long()
    for scales in ((top,), (2.0 ** -100,), (top, 2.0 ** -100), (2.0 ** -100, 0.01), (2.0 ** -100, 0.01, top, 0.3), (0.0, top),
                   (0.0, 2.0 ** -100), (0.0,), (2.0 ** 20, 2.0 ** -100, 2.0 ** -60)):
        for n, p in enumerate(pages):
            cache.vscale[p] = scales[n % len(scales)]
        check_rows(case)
    cache.vscale[pages] = top
    cache.vcodes[pages] = 255
    check_rows(case)
    out = cache.attention(Q, i32(cu), i32(kvs), i32(table))[:q]
    assert out.isfinite().all()


@BOTH
def test_attention_masked_pages_of_prompts_have_no_influence(L, many):
    """NaN and infinite scales of pages that no row of the request sees."""
    case = make_case(L, 27, [80], [400], 4, 2, 128, 16, spare(many, 4))
    cache, Q, cu, kvs, table = case
    args = i32(cu), i32(kvs), i32(table)
    want = [x[:80].clone() for x in cache.attention(Q, *args, window=50, return_lse=True)]
    used = {int(table[0, j]) for j in range((400 - 80 + 1 - 50) // 16, 25)}
    for p in range(cache.num_pages):
        if p not in used:
            cache.kscale[p], cache.vscale[p] = float("nan"), float("inf")
    again = cache.attention(Q, *args, window=50, return_lse=True)
    assert torch.equal(want[0], again[0][:80]) and torch.equal(want[1], again[1][:80])


@SHAPES
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_attention_scores_against_value_scales(L, q, Hq, Hkv, D, page, many, seed):
    """Scores about a hundred powers of two apart and value scales as far: the keys with the largest weights are not those
    with the largest probabilities."""
    kv = max(q, 9 * page + 5)
    case = make_case(L, 28 + seed, [q, 1], [kv, 5 * page], Hq, Hkv, D, page, spare(many, Hq))
    cache = case[0]
    rng = np.random.default_rng(seed)
    cache.kscale.copy_(torch.tensor(2.0 ** rng.uniform(-6, 0, cache.kscale.shape), dtype=torch.float32))
    cache.vscale.copy_(torch.tensor(2.0 ** rng.uniform(-100, 110, cache.vscale.shape), dtype=torch.float32))
    check_rows(case)
    check_rows(case, causal=False)
    check_rows(case, window=3 * page)


@pytest.mark.parametrize("q,Hq,Hkv,D,page,many", [(1, 2, 2, 128, 16, False), (1, 8, 1, 64, 64, False), (12, 2, 1, 128, 32, False),
                                                  (40, 2, 1, 128, 16, True), (300, 1, 1, 64, 32, True)])
@pytest.mark.parametrize("below", [24.0, 25.2, 27.3])
def test_attention_many_keys_of_small_weight(L, q, Hq, Hkv, D, page, many, below):
    """One key that takes nearly all of the probability and has no value, beside thousands 2^-25 as probable: they are
    the whole output, and rounded relative to 2^-7 of the largest weight."""
    kv = 20000 if q == 1 else 3000
    case = make_case(L, 31, [q], [kv], Hq, Hkv, D, page, spare(many, Hq))
    cache, Q, cu, kvs, table = case
    Q.fill_(1.0)
    cache.kcodes.fill_(128)
    cache.vcodes.copy_(cache.vcodes.clamp(min=150))
    cache.vscale.fill_(0.25)
    cache.kscale.fill_(below * np.log(2) / (D ** 0.5 * 100))
    first = int(table[0, 1])                                 # not the first key: the reference is raised on the way
    cache.kcodes[first, :, 3] = 228
    cache.vcodes[first, :, 3] = 128
    check_rows(case, lag=-7)
    check_rows(case, lag=-7, causal=False)


def test_a_workspace_is_whole(L):
    """A strided view has bytes between its own that are not the call's to write."""
    case = make_case(L, 32, [1, 1], [40, 30], 4, 2, 64, 16)
    cache, Q, cu, kvs, table = case
    need = cache.workspace(2).numel()
    wide = torch.zeros(need, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(AssertionError):
        cache.attention(Q, i32(cu), i32(kvs), i32(table), ws=wide[:, 0])
    assert bool((wide == 0).all())


@pytest.mark.parametrize("kw", [{"max_q": 2 ** 32 + 1}, {"max_kv": 2 ** 31}, {"window": 2 ** 32 + 3}, {"window": 3 - 2 ** 32}])
def test_numbers_wider_than_an_int_are_refused(L, kw):
    """Cut to 32 bits they would be other numbers: a window of 3, a bound of one row."""
    case = make_case(L, 33, [5, 1], [40, 30], 4, 2, 64, 16)
    cache, Q, cu, kvs, table = case
    with pytest.raises(AssertionError):
        cache.attention(Q, i32(cu), i32(kvs), i32(table), **kw)


@pytest.mark.parametrize("H,D,page", [(2, 64, 16), (3, 128, 64)])
def test_append_to_blocks_of_odd_scales(L, H, D, page):
    """Scales that no append has left: of no matter where a run begins the page, and 0 elsewhere if negative or not finite."""
    rng = np.random.default_rng(41)
    odd = [np.nan, np.inf, -np.inf, -1.0, -0.0, 3.4025e38, 1e-45, 2.0 ** -110, 1e30]
    runs = [(p, off) for off in (0, 5) for p in range(len(odd))]
    cache = fresh_cache(L, rng, len(runs), H, page, D)
    slots = []
    for n, (p, off) in enumerate(runs):
        for s in (cache.kscale, cache.vscale):
            s[n] = float(np.float32(odd[p]))
        slots += [n * page + off + k for k in range(3)] + [-1]
    x = random_tokens(rng, len(slots), 2 * H, D, "plain").cuda()
    want = []
    for part, c, s in ((x[:, :H], cache.kcodes, cache.kscale), (x[:, H:], cache.vcodes, cache.vscale)):
        scale = s.cpu().numpy()
        want.append(oracle.kv_append(np64(part), slots, c.cpu().numpy(),
                                     np.where(np.isfinite(scale) & (scale >= 0), scale, np.float32(0)), page))
    cache.append(x[:, :H], x[:, H:], i32(slots))
    for (codes, scale), (c, s) in zip(want, ((cache.kcodes, cache.kscale), (cache.vcodes, cache.vscale))):
        assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(c.cpu().numpy(), codes)


@pytest.mark.parametrize("q,Hq,Hkv,D,page,many", [(6, 2, 2, 128, 16, False), (20, 2, 2, 64, 16, False), (60, 2, 1, 128, 16, True),
                                                  (300, 2, 2, 64, 16, True)])
@pytest.mark.parametrize("below", [60, 100, 115])
def test_attention_output_of_one_faint_key(L, q, Hq, Hkv, D, page, many, below):
    """Keys with all of the probability and no value beside a block 2^-60 to 2^-115 as probable: it is the output."""
    kv = max(q, 100)
    case = make_case(L, 42, [q], [kv], Hq, Hkv, D, page, spare(many, Hq))
    cache, Q, cu, kvs, table = case
    Q.fill_(1.0)
    cache.kcodes.fill_(28)                                   # -100: scores `below` under those of the first page
    cache.kscale.fill_(below * np.log(2) / (D ** 0.5 * 100))
    cache.vscale.fill_(0)
    cache.vscale[int(table[0, 1])] = 0.02
    cache.kcodes[int(table[0, 0])] = 128
    check_rows(case, lag=-7)
    check_rows(case, lag=-7, causal=False)


def test_dropped_tokens_leave_their_scale(L):
    """A rejected draft: lengths and pages go back, the block it was in keeps the scale that it was raised to."""
    H, D, page = 2, 64, 16
    pages, cache = L.KVPages.empty(1, 2, 4, page), L.KVCache.empty(4, H, page, D)
    x = random_tokens(np.random.default_rng(43), 12, H, D, "plain").cuda()
    step = pages.plan(i32([6]), 6)
    cache.append(x[:6], x[:6], step.slots)
    codes, scale = (c.clone() for c in (cache.kcodes, cache.kscale))
    step = pages.plan(i32([3]), 3)
    cache.append(x[6:9] * 50, x[6:9] * 50, step.slots)
    pages.plan(i32([-3]), 0)
    assert pages.kv_lens.tolist() == [6] and pages.free_count.tolist() == [3]
    want, raised = oracle.kv_append(np64(x[6:9] * 50), [6, 7, 8], codes.cpu().numpy(), scale.cpu().numpy(), page)
    assert np.array_equal(cache.kcodes[0, :, :6].cpu().numpy(), want[0, :, :6]) and np.array_equal(cache.kscale.cpu().numpy(), raised)
    assert bool((cache.kscale[0] > 10 * scale[0]).all())
