"""The C-ABI library: it builds, loads, exports every declared symbol, and its
host-side argument checks answer without touching a GPU."""
import ctypes
import os
import re

import pytest

from hadamard_bit_quant_b200 import build as hbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hbl.h")


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    from hadamard_bit_quant_b200 import hbl
    return hbl.lib()


def declared_functions():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(hbl_[a-z0-9_]+)\s*\(", src, flags=re.M)
    return sorted(set(names))


def test_header_declares_the_boundary():
    names = declared_functions()
    for want in ("hbl_pack_weights", "hbl_forward", "hbl_forward_ws", "hbl_workspace_bytes",
                 "hbl_hadamard_f32", "hbl_quantize", "hbl_gemm_codes", "hbl_unpack_weights",
                 "hbl_packed_bytes", "hbl_status_string", "hbl_get_device_error", "hbl_version"):
        assert want in names


def test_library_exports_every_declared_symbol(lib):
    for name in declared_functions():
        assert hasattr(lib, name), name


def test_binding_covers_every_declared_symbol():
    from hadamard_bit_quant_b200 import hbl
    bound = {n for n, _, _ in hbl.SIGNATURES}
    assert set(declared_functions()) <= bound
    for n in bound:
        assert callable(getattr(hbl, n))


def test_host_side_queries(lib):
    from hadamard_bit_quant_b200 import hbl
    assert hbl.hbl_version() == 1
    assert hbl.hbl_packed_bytes(4096, 4096) == 4096 * 4096 // 4
    assert hbl.hbl_packed_bytes(0, 4096) == 0
    assert hbl.hbl_status_string(0) == "HBL_OK"
    assert hbl.hbl_status_string(2) == "HBL_ERR_SHAPE"
    assert hbl.hbl_status_string(99) == "HBL_ERR_UNKNOWN"
    w = hbl.hbl_workspace_bytes(16, 4096, 4096)
    assert w >= 16 * 4096 + 16 * 4 * 2 and w % 256 == 0
    assert hbl.hbl_workspace_bytes(0, 4096, 4096) >= 0


def test_gemm_path_selector_bounds(lib):
    # host-side only: the selector is a library global, checked before it is stored
    from hadamard_bit_quant_b200 import hbl
    raw = hbl.lib()
    try:
        for p in range(7):
            assert raw.hbl_set_gemm_path(p) == 0
        assert raw.hbl_set_gemm_path(-1) == 1
        assert raw.hbl_set_gemm_path(7) == 1
    finally:
        assert raw.hbl_set_gemm_path(0) == 0


BAD = 0x1000  # never dereferenced: every call below is rejected before any launch


@pytest.mark.parametrize("args,status", [
    # act_bits / use_hadamard
    ((BAD, 4, 4096, 4096, BAD, BAD, 3, 1, BAD), 1),
    ((BAD, 4, 4096, 4096, BAD, BAD, 4, 2, BAD), 1),
    # K not a power of two with the Hadamard on, K too small, K too large
    ((BAD, 4, 768, 4096, BAD, BAD, 4, 1, BAD), 2),
    ((BAD, 4, 128, 4096, BAD, BAD, 4, 0, BAD), 2),
    ((BAD, 4, 65536, 4096, BAD, BAD, 4, 1, BAD), 2),
    # N not a multiple of 16, K not a multiple of 256
    ((BAD, 4, 4096, 4100, BAD, BAD, 4, 1, BAD), 2),
    ((BAD, 4, 1000, 4096, BAD, BAD, 8, 0, BAD), 2),
    # negative M, null pointers
    ((BAD, -1, 4096, 4096, BAD, BAD, 4, 1, BAD), 2),
    ((None, 4, 4096, 4096, BAD, BAD, 4, 1, BAD), 1),
    ((BAD, 4, 4096, 4096, None, BAD, 4, 1, BAD), 1),
    ((BAD, 4, 4096, 4096, BAD, BAD, 4, 1, None), 1),
])
def test_forward_argument_checks(lib, args, status):
    st = lib.hbl_forward(*args, None)
    assert st == status
    st = lib.hbl_forward_ws(*args, BAD, 1 << 20, None)
    assert st == status
    st = lib.hbl_forward_noalloc(*args, None)
    assert st == status


def test_empty_batch_is_a_noop(lib):
    # M == 0: nothing to do, nothing launched, HBL_OK even with null buffers
    assert lib.hbl_forward(None, 0, 4096, 4096, None, None, 4, 1, None, None) == 0
    assert lib.hbl_forward_noalloc(None, 0, 4096, 4096, None, None, 4, 1, None, None) == 0
    assert lib.hbl_forward_ws(None, 0, 4096, 4096, None, None, 4, 1, None, None, 0, None) == 0
    assert lib.hbl_quantize(None, 0, 4096, 4, 1, None, None, None, None) == 0
    assert lib.hbl_gemm_codes(None, 0, 4096, 4096, None, None, None) == 0


def test_pack_argument_checks(lib):
    assert lib.hbl_pack_weights(BAD, 4096, 1000, BAD, BAD, None) == 2
    assert lib.hbl_pack_weights(BAD, 4095, 4096, BAD, BAD, None) == 2
    assert lib.hbl_pack_weights(None, 4096, 4096, BAD, BAD, None) == 1
    assert lib.hbl_pack_weights(BAD, 4096, 4096, BAD + 1, BAD, None) == 1   # Wpk not 16-byte aligned
    assert lib.hbl_unpack_weights(BAD, 16, 100, BAD, None) == 2


def test_quantize_and_hadamard_argument_checks(lib):
    assert lib.hbl_quantize(BAD, 2, 4096, 5, 1, BAD, BAD, None, None) == 1
    assert lib.hbl_quantize(BAD, 2, 3000, 4, 1, BAD, BAD, None, None) == 2
    assert lib.hbl_hadamard_f32(BAD, 2, 3000, BAD, None) == 2
    assert lib.hbl_hadamard_f32(None, 2, 4096, BAD, None) == 1


def test_noalloc_rejects_sizes_beyond_its_array(lib):
    # the fixed 8 MiB array: a size whose workspace exceeds it is refused before
    # any device work (HBL_ERR_WORKSPACE), one that fits passes the size check
    from hadamard_bit_quant_b200 import hbl
    assert hbl.hbl_workspace_bytes(4096, 16384, 256) > 8 << 20
    assert lib.hbl_forward_noalloc(BAD, 4096, 16384, 256, BAD, BAD, 4, 1, BAD, None) == 7
    assert hbl.hbl_workspace_bytes(16, 4096, 4096) <= 8 << 20
    # still refused on its arguments first
    assert lib.hbl_forward_noalloc(BAD, 4096, 16384, 256, BAD, BAD, 5, 1, BAD, None) == 1


def kv_attention_args(**kw):
    """Arguments of a call that would be launched, some of them changed."""
    a = dict(Q=BAD, T=4, Hq=8, Hkv=2, D=128, q_stride=1024, cu_q=BAD, kv_lens=BAD, B=2, max_q=0, max_kv=0, block_table=BAD,
             max_pages=8, page=16, num_pages=20, kcodes=BAD, vcodes=BAD, kscale=BAD, vscale=BAD, scale=0.1, causal=1, window=0,
             O=BAD, lse=None, ws=BAD, ws_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    return list({**a, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(scale=3e38), 1),                       # times log2(e) no longer a float
    (dict(causal=2), 1), (dict(window=-1), 1), (dict(causal=0, window=4), 1),
    (dict(page=20), 2), (dict(page=256), 2), (dict(num_pages=0), 2), (dict(num_pages=1 << 27), 2), (dict(D=96), 2),
    (dict(T=-1), 2), (dict(T=1 << 27), 2), (dict(Hq=7), 2), (dict(q_stride=1016), 2), (dict(q_stride=1028), 2),
    (dict(B=-1), 2), (dict(B=8193), 2), (dict(max_pages=0), 2), (dict(max_pages=1 << 28), 2), (dict(max_q=-1), 2),
    (dict(max_kv=-1), 2), (dict(Q=None), 1), (dict(O=None), 1), (dict(vscale=None), 1), (dict(Q=BAD + 2), 1),
    (dict(lse=BAD + 2), 1), (dict(ws=None), 7), (dict(ws_bytes=1000), 7), (dict(ws=BAD + 16), 1),
    (dict(T=0, Q=None, O=None), 0), (dict(B=0, cu_q=None), 0),
])
def test_kv_attention_argument_checks(lib, kw, status):
    assert lib.hbl_kv_attention(*kv_attention_args(**kw)) == status


def test_kv_cache_argument_checks(lib):
    plan = lambda new=BAD, B=2, page=16, num=20, width=8, T=4, state=BAD, slots=BAD: lib.hbl_kv_plan(   # noqa: E731
        new, B, page, num, width, T, state, BAD, BAD, BAD, BAD, slots, BAD, None)
    assert plan(page=24) == plan(num=0) == plan(num=1 << 27) == plan(B=8193) == plan(B=-1) == plan(T=-1) == 2
    assert plan(width=0) == plan(width=1 << 28) == plan(B=8192, width=1 << 18) == 2
    assert plan(new=None) == plan(state=None) == plan(slots=None) == plan(new=BAD + 1) == plan(slots=BAD + 2) == 1
    assert plan(B=0, new=None) == 0
    append = lambda K=BAD, T=4, H=2, D=64, stride=256, slots=BAD, page=16, num=20, codes=BAD, scale=BAD: lib.hbl_kv_append(  # noqa: E731
        K, BAD, T, H, D, stride, 256, slots, page, num, codes, BAD, scale, BAD, None)
    assert append(page=8) == append(D=32) == append(H=0) == append(H=65536) == append(T=-1) == append(T=1 << 30) == 2
    assert append(stride=120) == append(stride=260) == append(num=-1) == 2
    assert append(K=None) == append(slots=None) == append(codes=None) == append(scale=None) == 1
    assert append(K=BAD + 8) == append(slots=BAD + 1) == append(codes=BAD + 4) == append(scale=BAD + 2) == 1
    assert append(T=0, K=None, slots=None) == 0
    read = lambda slots=BAD, T=4, D=64, K=BAD, V=BAD, codes=BAD, scale=BAD: lib.hbl_kv_read(            # noqa: E731
        slots, T, 2, D, 16, 20, codes, BAD, scale, BAD, K, V, None)
    assert read(D=80) == read(T=-1) == 2
    assert read(slots=None) == read(codes=None) == read(scale=None) == read(K=BAD + 8) == read(V=BAD + 2) == 1
    assert read(T=0) == read(K=None, V=None) == 0
