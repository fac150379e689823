"""Pins for the oracle of the paged 8-bit key/value cache: hand-worked values, invariants and facts that do
not come from its own formulas; and the host-side refusals of the cache's entry points."""
import math

import numpy as np
import pytest

import oracle
from hadamard_bit_quant_b200 import build as hbuild


def test_plan_by_hand():
    # pages of 16, table of 3: request 0 grows inside its page, request 1 needs two pages, request 2 gives one
    # back, request 3 would need four pages of three, request 4 leaves
    table = np.array([[5, 0, 0], [6, 0, 0], [7, 8, 0], [9, 0, 0], [1, 2, 0]])
    r = oracle.kv_plan([2, 20, -10, 60, -99], [3, 16, 20, 4, 32], table, np.array([3, 4, 0, 0, 0, 0, 0, 0, 0, 0]), 2, 16, 90)
    assert list(r["refused"]) == [0, 0, 0, 1, 0]
    assert list(r["kv_lens"]) == [5, 36, 10, 4, 0]
    # given back: 8 (request 2), then 1 and 2 (request 4); request 1 takes 8 and 1, 2 stays on the stack
    assert list(r["table"][1]) == [6, 8, 1]
    assert r["free_count"] == 3 and list(r["free_pages"][:3]) == [3, 4, 2]
    assert list(r["cu_q"]) == [0, 2, 22, 22, 82, 82]
    assert list(r["slots"][:6]) == [5 * 16 + 3, 5 * 16 + 4, 8 * 16, 8 * 16 + 1, 8 * 16 + 2, 8 * 16 + 3]
    assert list(r["slots"][18:24]) == [16, 17, 18, 19, -1, -1] and list(r["slots"][82:]) == [-1] * 8


def test_plan_runs_out_of_pages_in_order():
    r = oracle.kv_plan([16, 32, 16, 1], [0, 0, 0, 3], np.array([[0, 0], [0, 0], [0, 0], [9, 0]]), np.array([4, 5]), 2, 16, 70)
    # the second wants two of the one page left, the third would fit but comes after it, the fourth needs none
    assert list(r["refused"]) == [0, 1, 1, 0]
    assert r["free_count"] == 1 and r["table"][0, 0] == 5 and list(r["kv_lens"]) == [16, 0, 0, 4]


@pytest.mark.parametrize("seed", range(6))
def test_plan_never_loses_or_doubles_a_page(seed):
    rng = np.random.default_rng(seed)
    B, page, width, num = 7, 16, 5, 20
    kv, table, free, count = np.zeros(B, int), np.zeros((B, width), int), np.arange(num), num
    for _ in range(30):
        r = oracle.kv_plan(rng.integers(-30, 40, B), kv, table, free, count, page, 150)
        kv, table, free, count = r["kv_lens"], r["table"], r["free_pages"], r["free_count"]
        held = [int(table[b, j]) for b in range(B) for j in range(-(-int(kv[b]) // page))]
        assert sorted(held + list(free[:count])) == list(range(num))
        live = r["slots"][r["slots"] >= 0]
        assert len(set(live.tolist())) == len(live)


def test_append_by_hand():
    codes, scale = np.zeros((2, 1, 16, 64), np.uint8), np.full((2, 1), 9.0, np.float32)
    x = np.zeros((2, 1, 64))
    x[0, 0, :3] = [127, 0.5, 1.5]            # scale 1: 0.5 and 1.5 are ties, to 0 and 2
    x[1, 0, 0] = -63.5
    c, s = oracle.kv_append(x, [16, 17], codes, scale, 16)
    assert s[1, 0] == 1 and s[0, 0] == 9
    assert list(c[1, 0, 0, :4]) == [255, 128, 130, 128] and c[1, 0, 1, 0] == 64        # -63.5: a tie, to -64
    y = np.zeros((1, 1, 64))
    y[0, 0, 5] = 254                          # twice as loud: what is there is rescaled
    c, s = oracle.kv_append(y, [18], c, s, 16)
    assert s[1, 0] == 2 and c[1, 0, 2, 5] == 255
    assert list(c[1, 0, 0, :4]) == [192, 128, 129, 128] and c[1, 0, 1, 0] == 96        # 63.5 -> 64, 1, and -32
    c, s = oracle.kv_append(np.zeros((1, 1, 64)), [32 - 16], c, s, 16)                 # a new first token: a new scale
    assert s[1, 0] == np.float32(2.0 ** -100) and np.all(c[1, 0, 0] == 128)


def test_append_error_is_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((16, 3, 64)) * np.exp(rng.standard_normal((16, 3, 1)))
    codes, scale = oracle.kv_append(x, np.arange(16), np.zeros((1, 3, 16, 64), np.uint8), np.zeros((1, 3), np.float32), 16)
    y = oracle.kv_read(np.arange(16), codes, scale, 16)
    assert np.all(np.abs(y - x) <= scale[0].astype(float)[:, None] * 0.5000001)
    assert np.all(np.abs(np.abs(x).max((0, 2)) / 127 / scale[0] - 1) < 1e-6)
    odd = np.array([np.nan, np.inf, -np.inf, 0.0] * 16).reshape(1, 1, 64)
    codes, scale = oracle.kv_append(odd, [0], np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32), 16)
    assert list(codes[0, 0, 0, :4]) == [128, 255, 1, 128] and np.isfinite(scale).all()


def test_attention_facts():
    rng = np.random.default_rng(1)
    pages, H, P, D = 6, 2, 16, 64
    kc, vc = (rng.integers(0, 256, (pages, H, P, D)) for _ in range(2))
    ks, vs = (rng.random((pages, H)).astype(np.float32) * 0.02 for _ in range(2))
    table, kv = np.array([[4, 1, 3], [0, 5, 2]]), [40, 3]
    Q = rng.standard_normal((6, 4, D))
    args = Q, [0, 2, 5], kv, table, kc, vc, ks, vs, P, 0.125
    out, lse, mag, _ = oracle.kv_attention(*args)
    assert np.isnan(out[5]).all() and not np.isnan(out[:5]).any()
    V = oracle.kv_read([0 * 16], vc, vs, P)
    assert np.allclose(out[2, 0], V[0, 0]) and np.allclose(out[2, 3], V[0, 1])       # one key: its value
    # zero queries average the values; the lse is the log of the number of keys
    out0, lse0, _, _ = oracle.kv_attention(np.zeros_like(Q), *args[1:])
    slots = [int(table[0, j // P]) * P + j % P for j in range(40)]
    assert np.allclose(out0[1, 2], oracle.kv_read(slots, vc, vs, P)[:, 1].mean(0))
    assert np.allclose(lse0[:2, 0], [math.log(39), math.log(40)]) and np.allclose(lse0[4], math.log(3))
    # a window of one sees one key; no causal mask: the rows of a request see the same keys
    out1 = oracle.kv_attention(*args, causal=True, window=1)[0]
    assert np.allclose(out1[1, 1], oracle.kv_read(slots[39:], vc, vs, P)[0, 0])
    assert np.allclose(oracle.kv_attention(*args, causal=False)[1][:2], oracle.kv_attention(*args, causal=False)[1][:2])
    # rows before the first key see nothing
    few = oracle.kv_attention(Q, [0, 4, 4], [2, 0], table, kc, vc, ks, vs, P, 0.125)
    assert np.isneginf(few[1][:2]).all() and np.all(few[0][:2] == 0) and np.isfinite(few[1][2:4]).all()
    # parts of the keys join by their lse
    a = oracle.kv_attention(Q, [0, 2, 2], [16, 0], table, kc, vc, ks, vs, P, 0.125, causal=False)
    b = oracle.kv_attention(Q, [0, 2, 2], [24, 0], table[:, 1:], kc, vc, ks, vs, P, 0.125, causal=False)
    c = oracle.kv_attention(Q, [0, 2, 2], [40, 0], table, kc, vc, ks, vs, P, 0.125, causal=False)
    w = np.exp(a[1][:2] - c[1][:2])[..., None]
    assert np.allclose(a[0][:2] * w + b[0][:2] * (1 - w), c[0][:2])


# ----------------------------------------------------------------------------- refusals, on the host
@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    from hadamard_bit_quant_b200 import hbl
    return hbl.lib()


A = 0x1000   # never dereferenced: every call below is rejected before any launch


def plan_args(**kw):
    d = dict(new_lens=A, B=2, page=16, num_pages=8, max_pages=4, T=3, kv_lens=A, block_table=A, free_pages=A,
             free_count=A, cu_q=A, slots=A, refused=A) | kw
    return (*d.values(), None)


def append_args(**kw):
    d = dict(K=A, V=A, T=3, Hkv=2, D=64, ks=128, vs=128, slots=A, page=16, num_pages=8, kcodes=A, vcodes=A, kscale=A,
             vscale=A) | kw
    return (*d.values(), None)


def read_args(**kw):
    d = dict(slots=A, T=3, Hkv=2, D=64, page=16, num_pages=8, kcodes=A, vcodes=A, kscale=A, vscale=A, K=A, V=A) | kw
    return (*d.values(), None)


def attention_args(**kw):
    d = dict(Q=A, T=3, Hq=4, Hkv=2, D=64, qs=256, cu_q=A, kv_lens=A, B=2, max_q=0, max_kv=0, table=A, max_pages=4,
             page=16, num_pages=8, kcodes=A, vcodes=A, kscale=A, vscale=A, scale=0.125, causal=1, window=0, O=A, lse=A,
             ws=A, ws_bytes=1 << 40) | kw
    return (*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    ({"page": 8}, 2), ({"page": 48}, 2), ({"page": 256}, 2), ({"num_pages": 0}, 2), ({"num_pages": 1 << 27}, 2),
    ({"B": -1}, 2), ({"B": 8193}, 2), ({"T": -1}, 2), ({"max_pages": 0}, 2), ({"max_pages": 1 << 30}, 2),
    ({"max_pages": (1 << 26) + 1}, 2), ({"B": 8192, "max_pages": 1 << 18}, 2), ({"new_lens": None}, 1), ({"kv_lens": None}, 1), ({"block_table": None}, 1), ({"free_pages": None}, 1),
    ({"free_count": None}, 1), ({"cu_q": None}, 1), ({"slots": None}, 1), ({"refused": None}, 1), ({"slots": A + 2}, 1),
    ({"B": 0, "kv_lens": None}, 0)])
def test_plan_refusals(lib, kw, status):
    assert lib.hbl_kv_plan(*plan_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({"page": 17}, 2), ({"D": 32}, 2), ({"D": 96}, 2), ({"D": 256}, 2), ({"Hkv": 0}, 2), ({"T": -1}, 2),
    ({"Hkv": 65536}, 2), ({"T": 1 << 30, "Hkv": 2, "ks": 1 << 20, "vs": 1 << 20}, 2), ({"ks": 120}, 2), ({"vs": 129}, 2),
    ({"ks": -128}, 2), ({"K": None}, 1), ({"V": None}, 1), ({"slots": None}, 1), ({"kcodes": None}, 1),
    ({"vcodes": None}, 1), ({"kscale": None}, 1), ({"vscale": None}, 1), ({"K": A + 8}, 1), ({"vcodes": A + 4}, 1),
    ({"slots": A + 1}, 1), ({"kscale": A + 2}, 1), ({"T": 0, "K": None}, 0)])
def test_append_refusals(lib, kw, status):
    assert lib.hbl_kv_append(*append_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({"page": 0}, 2), ({"D": 72}, 2), ({"slots": None}, 1), ({"kcodes": None}, 1), ({"vscale": None}, 1), ({"K": A + 2}, 1),
    ({"T": 0}, 0), ({"K": None, "V": None}, 0)])
def test_read_refusals(lib, kw, status):
    assert lib.hbl_kv_read(*read_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({"page": 20}, 2), ({"D": 80}, 2), ({"Hq": 5}, 2), ({"Hq": 0}, 2), ({"Hkv": 0}, 2), ({"qs": 255}, 2), ({"qs": 260}, 2),
    ({"B": 8193}, 2), ({"B": -1}, 2), ({"T": -1}, 2), ({"max_pages": 0}, 2), ({"max_pages": (1 << 26) + 1}, 2), ({"T": 1 << 28}, 2), ({"max_q": -1}, 2), ({"max_kv": -1}, 2),
    ({"causal": 2}, 1), ({"window": -1}, 1), ({"causal": 0, "window": 4}, 1), ({"scale": 0.0}, 1), ({"scale": -1.0}, 1),
    ({"scale": math.inf}, 1), ({"scale": math.nan}, 1), ({"Q": None}, 1), ({"cu_q": None}, 1), ({"kv_lens": None}, 1),
    ({"table": None}, 1), ({"kcodes": None}, 1), ({"vscale": None}, 1), ({"O": None}, 1), ({"O": A + 8}, 1),
    ({"lse": A + 1}, 1), ({"ws": None}, 7), ({"ws_bytes": 4096}, 7), ({"ws": A + 16}, 1), ({"T": 0, "Q": None}, 0),
    ({"B": 0, "cu_q": None}, 0)])
def test_attention_refusals(lib, kw, status):
    assert lib.hbl_kv_attention(*attention_args(**kw)) == status


def test_workspace_query(lib):
    assert lib.hbl_kv_attention_workspace_bytes(1, 64) % 256 == 0
    assert 0 < lib.hbl_kv_attention_workspace_bytes(1, 64) < lib.hbl_kv_attention_workspace_bytes(8192, 128) < 16 << 20
    assert lib.hbl_kv_attention_workspace_bytes(-1, 64) == 0 and lib.hbl_kv_attention_workspace_bytes(4, 100) == 0
