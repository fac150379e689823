"""Tensor-level helpers over the C ABI: pack a weight matrix, run the forward.

These only allocate outputs with torch and call the binding; the arithmetic
is in libhbl's kernels.
"""
from __future__ import annotations

from contextlib import nullcontext
from functools import lru_cache
from typing import NamedTuple

import torch

from . import hbl


def pack_weights(W: torch.Tensor, stream=None):
    """Ternarise and pack an N x K fp32 CUDA tensor. Returns (Wpk uint8 [N*K/4], wscale fp32 [1])."""
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.is_contiguous()
    N, K = W.shape
    Wpk = torch.empty(hbl.hbl_packed_bytes(N, K), dtype=torch.uint8, device=W.device)
    wscale = torch.empty(1, dtype=torch.float32, device=W.device)
    hbl.hbl_pack_weights(W, N, K, Wpk, wscale, stream)
    return Wpk, wscale


def unpack_weights(Wpk: torch.Tensor, N: int, K: int, stream=None) -> torch.Tensor:
    T = torch.empty(N, K, dtype=torch.int8, device=Wpk.device)
    hbl.hbl_unpack_weights(Wpk, N, K, T, stream)
    return T


def workspace(M: int, K: int, N: int, device) -> torch.Tensor:
    return torch.empty(max(1, hbl.hbl_workspace_bytes(M, K, N)), dtype=torch.uint8, device=device)


def forward(X: torch.Tensor, Wpk: torch.Tensor, wscale: torch.Tensor, N: int, act_bits: int = 4,
            use_hadamard: int = 1, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Y = H-BitLinear(X) for bf16 X (M x K). Uses ``ws`` (caller workspace) when given."""
    assert X.is_cuda and X.dtype == torch.bfloat16 and X.dim() == 2 and X.is_contiguous()
    M, K = X.shape
    Y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
    if ws is None:
        hbl.hbl_forward(X, M, K, N, Wpk, wscale, act_bits, use_hadamard, Y, stream)
    else:
        hbl.hbl_forward_ws(X, M, K, N, Wpk, wscale, act_bits, use_hadamard, Y, ws, ws.numel(), stream)
    return Y


def hadamard_f32(X: torch.Tensor, stream=None) -> torch.Tensor:
    M, K = X.shape
    Xr = torch.empty(M, K, dtype=torch.float32, device=X.device)
    hbl.hbl_hadamard_f32(X, M, K, Xr, stream)
    return Xr


def quantize(X: torch.Tensor, act_bits: int, use_hadamard: int, stream=None):
    M, K = X.shape
    codes = torch.empty(M, K, dtype=torch.int8, device=X.device)
    scales = torch.empty(M, dtype=torch.float32, device=X.device)
    csum = torch.empty(M, dtype=torch.int32, device=X.device)
    hbl.hbl_quantize(X, M, K, act_bits, use_hadamard, codes, scales, csum, stream)
    return codes, scales, csum


def gemm_codes(codes: torch.Tensor, Wpk: torch.Tensor, N: int, stream=None) -> torch.Tensor:
    M, K = codes.shape
    acc = torch.empty(M, N, dtype=torch.int32, device=codes.device)
    hbl.hbl_gemm_codes(codes, M, K, N, Wpk, acc, stream)
    return acc


class HBitLinear:
    """One H-BitLinear (or plain BitLinear with use_hadamard=0) layer with packed weights."""

    def __init__(self, W: torch.Tensor, act_bits: int = 4, use_hadamard: int = 1):
        self.N, self.K = W.shape
        self.act_bits = act_bits
        self.use_hadamard = use_hadamard
        self.Wpk, self.wscale = pack_weights(W)

    def __call__(self, X: torch.Tensor, out=None, ws=None, stream=None) -> torch.Tensor:
        return forward(X, self.Wpk, self.wscale, self.N, self.act_bits, self.use_hadamard, out, ws, stream)


class KVStep(NamedTuple):
    """What one step of ``KVPages.plan`` wrote: a slot for each row, the requests' rows, who could not grow."""
    slots: torch.Tensor
    cu_q: torch.Tensor
    refused: torch.Tensor


def _index(*tensors):
    """Index arrays: contiguous int32 on the current device, where the kernels are launched."""
    dev = torch._C._cuda_getDevice()
    for x in tensors:
        assert x.get_device() == dev and x.dtype is torch.int32 and x.is_contiguous()


def _allocating(stream):
    """Context in which a call's own tensors are allocated: on the stream that it runs on, so that memory which it frees
    at its end (a workspace) is not handed to another stream before it is through."""
    if stream is None:
        return nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class KVPages:
    """Lengths, block table and free pages of a batch, shared by the caches of all layers.

    kv_lens: int32 [B]; block_table: int32 [B, max_pages]; free_pages: int32 [num_pages], a stack whose first
    free_count[0] entries are free. ``plan`` changes them in place.
    """

    def __init__(self, kv_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                 free_count: torch.Tensor, page: int):
        _index(kv_lens, block_table, free_pages, free_count)
        assert block_table.dim() == 2 and block_table.shape[0] == kv_lens.numel() > 0 and free_count.numel() == 1
        self.kv_lens, self.block_table = kv_lens, block_table
        self.free_pages, self.free_count, self.page = free_pages, free_count, page

    @classmethod
    def empty(cls, requests: int, max_pages: int, num_pages: int, page: int, device="cuda") -> "KVPages":
        """No tokens, every page free (page 0 is handed out first)."""
        def full(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)
        stack = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        return cls(full(requests), full(requests, max_pages), stack, full(1) + num_pages, page)

    def plan(self, new_lens: torch.Tensor, tokens: int, out: KVStep | None = None, stream=None) -> KVStep:
        """Grow each request by new_lens[b] tokens (or drop -new_lens[b] of them): rows for ``tokens`` new ones."""
        _index(new_lens, self.kv_lens)
        B, max_pages = self.block_table.shape
        assert new_lens.numel() == B
        if out is None:
            with _allocating(stream):
                out = KVStep(*new_lens.new_empty(tokens + 2 * B + 1).split_with_sizes((tokens, B + 1, B)))
        else:
            _index(*out)
            assert out.slots.numel() == tokens and out.cu_q.numel() == B + 1 and out.refused.numel() == B
        hbl.hbl_kv_plan(new_lens, B, self.page, self.free_pages.numel(), max_pages, tokens, self.kv_lens,
                        self.block_table, self.free_pages, self.free_count, out.cu_q, out.slots, out.refused, stream)
        return out


@lru_cache(maxsize=256)
def _attention_bytes(requests: int, head_dim: int) -> int:
    return hbl.hbl_kv_attention_workspace_bytes(requests, head_dim)


class KVCache:
    """One layer's paged 8-bit key/value cache.

    kcodes, vcodes: uint8 [num_pages, kv_heads, page, head_dim]; kscale, vscale: fp32 [num_pages, kv_heads]. A
    block stands for (codes - 128) * scale.
    """

    def __init__(self, kcodes: torch.Tensor, vcodes: torch.Tensor, kscale: torch.Tensor, vscale: torch.Tensor):
        shape, dev = kcodes.shape, kcodes.get_device()
        assert len(shape) == 4 and vcodes.shape == shape and kscale.shape == vscale.shape == shape[:2]
        assert kcodes.dtype is vcodes.dtype is torch.uint8 and kscale.dtype is vscale.dtype is torch.float32
        for x in (kcodes, vcodes, kscale, vscale):
            assert x.is_contiguous() and x.get_device() == dev >= 0
        self.kcodes, self.vcodes, self.kscale, self.vscale = kcodes, vcodes, kscale, vscale
        self.num_pages, self.kv_heads, self.page, self.head_dim = shape

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page: int, head_dim: int, device="cuda") -> "KVCache":
        shape = (num_pages, kv_heads, page, head_dim)
        codes = [torch.full(shape, 128, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)

    def _rows(self, x: torch.Tensor, heads: int | None = None) -> int:
        """Elements from token to token of a [tokens, heads, head_dim] tensor whose tokens may lie apart."""
        assert x.dtype is torch.bfloat16 and x.get_device() == self.kcodes.get_device()
        T, H, D = x.shape
        st, sh, sd = x.stride()
        assert D == self.head_dim and H == (heads or H) and sd == 1 and (H == 1 or sh == D)
        return st if T > 1 else H * D

    def append(self, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """Quantise K and V (bf16 [T, kv_heads, head_dim], e.g. parts of one projection's output) into their slots.

        A louder token raises its block's scale for good, also where ``KVPages.plan`` drops it again.
        """
        _index(slots)
        assert slots.get_device() == self.kcodes.get_device()
        ks, vs = self._rows(K, self.kv_heads), self._rows(V, self.kv_heads)
        T = K.shape[0]
        assert V.shape[0] == T and slots.numel() == T
        hbl.hbl_kv_append(K, V, T, self.kv_heads, self.head_dim, ks, vs, slots, self.page, self.num_pages,
                          self.kcodes, self.vcodes, self.kscale, self.vscale, stream)

    def read(self, slots: torch.Tensor, stream=None):
        """The values in the given slots: (K, V), bf16 [T, kv_heads, head_dim]."""
        _index(slots)
        assert slots.get_device() == self.kcodes.get_device()
        T = slots.numel()
        with _allocating(stream):
            K, V = self.kcodes.new_empty((2, T, self.kv_heads, self.head_dim), dtype=torch.bfloat16)
        hbl.hbl_kv_read(slots, T, self.kv_heads, self.head_dim, self.page, self.num_pages, self.kcodes, self.vcodes,
                        self.kscale, self.vscale, K, V, stream)
        return K, V

    def workspace(self, requests: int) -> torch.Tensor:
        """Workspace of ``attention`` for a batch of that many requests."""
        return self.kcodes.new_empty(_attention_bytes(requests, self.head_dim))

    def attention(self, Q: torch.Tensor, cu_q: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                  max_q: int = 0, max_kv: int = 0, scale: float | None = None, causal: bool = True, window: int = 0,
                  out: torch.Tensor | None = None, return_lse: bool = False, lse: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None):
        """Attention of Q (bf16 [T, heads, head_dim]) over the cache: out, or (out, lse) with ``return_lse``.

        Request b's rows are cu_q[b] .. cu_q[b + 1], its cache kv_lens[b] tokens in the pages block_table[b].
        scale: 1 / sqrt(head_dim) unless given. Rows of no request, and of one with more than max_q, are not written: what
        ``out`` and ``lse`` held, or anything where they are not given.
        """
        _index(cu_q, kv_lens, block_table)
        stride = self._rows(Q)
        T, Hq, D = Q.shape
        B, max_pages = block_table.shape
        assert kv_lens.numel() == B and cu_q.numel() == B + 1 and kv_lens.get_device() == self.kcodes.get_device()
        assert max(max_q, max_kv, window) < 1 << 31 and min(max_q, max_kv, window) >= -1 << 31     # ctypes would cut them
        if out is not None:
            assert out.shape == Q.shape and out.is_contiguous() and self._rows(out) == Hq * D
        if lse is not None:
            assert lse.shape == (T, Hq) and lse.dtype is torch.float32 and lse.is_contiguous()
            assert lse.get_device() == Q.get_device()
        if ws is not None:
            assert ws.dtype is torch.uint8 and ws.is_contiguous() and ws.get_device() == Q.get_device()
        with _allocating(stream):
            if out is None:
                out = Q.new_empty(T, Hq, D)
            if lse is None and return_lse:
                lse = self.kscale.new_empty(T, Hq)
            if ws is None:
                ws = self.workspace(B)
        hbl.hbl_kv_attention(Q, T, Hq, self.kv_heads, D, stride, cu_q, kv_lens, B, max_q, max_kv, block_table,
                             max_pages, self.page, self.num_pages, self.kcodes, self.vcodes, self.kscale, self.vscale,
                             D ** -0.5 if scale is None else scale, int(causal), window, out, lse, ws,
                             ws.numel(), stream)
        return (out, lse) if return_lse else out
