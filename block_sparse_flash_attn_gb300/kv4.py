"""A paged key/value cache in 4 bits, and attention over it token by token.

    cache = bsattn.Kv4Cache(pages, kv_heads, head_dim)
    bsattn.kv4_append(cache, k, v, block_table, lengths)       # new tokens, prompts or single ones
    lengths += k.shape[2]
    pages = bsattn.kv4_select(cache, q, block_table, lengths, keep=64)  # optional
    o, lse = bsattn.kv4_attn(cache, q, block_table, lengths, pages)
    bsattn.kv4_status(cache)                                   # raises if a table named a bad page
    k, v = bsattn.kv4_read(cache, block_table, start, tokens)  # cached tokens as bf16
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

import block_sparse_flash_attn_gb300 as _bs

from ._args import launch_on, output, pointer, tensor

_I32, _BF16 = torch.int32, torch.bfloat16


class _CacheStruct(ctypes.Structure):  # bsattn_kv4_cache
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales",
                                               "k_means", "status")] + \
               [(n, ctypes.c_int) for n in ("pages", "kv_heads", "page_size", "head_dim", "group")]


class Kv4Cache:
    """The cache's tensors (all CUDA, one device), zero at first, to be changed in
    place only:

    k_codes, v_codes    uint8 [pages, kv_heads, page_size, head_dim/2], even channel in the low bits
    k_scales, v_scales  bf16 [pages, kv_heads, page_size, head_dim/group, 2]: (step, least)
    k_means             bf16 [pages, kv_heads, head_dim]: the rounded mean key of a full page

    A channel stands for step * code + least.  page_size: 16, 32, 64, 128 or 256
    tokens; group (channels that share a step): 32, 64 or 128, default head_dim."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                 group: int | None = None, device=None):
        group = head_dim if group is None else group
        if pages <= 0 or kv_heads <= 0:
            raise ValueError("pages and kv_heads must be positive")
        if head_dim not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256")
        if group not in (32, 64, 128) or group > head_dim:
            raise ValueError("group must be 32, 64 or 128, at most head_dim")
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise TypeError("device must be a CUDA device")
        self.pages, self.kv_heads, self.head_dim = int(pages), int(kv_heads), int(head_dim)
        self.page_size, self.group = int(page_size), int(group)

        def zeros(*shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=device)

        rows = (pages, kv_heads, page_size)
        self.k_codes, self.v_codes = (zeros(*rows, head_dim // 2, dtype=torch.uint8) for _ in "kv")
        self.k_scales, self.v_scales = (zeros(*rows, head_dim // group, 2, dtype=_BF16) for _ in "kv")
        self.k_means = zeros(pages, kv_heads, head_dim, dtype=_BF16)
        self.status = zeros(1, dtype=_I32)
        self.device = self.k_codes.device
        self._struct = _CacheStruct(*(t.data_ptr() for t in (
            self.k_codes, self.v_codes, self.k_scales, self.v_scales, self.k_means, self.status)),
            self.pages, self.kv_heads, self.page_size, self.head_dim, self.group)
        self._ref = ctypes.byref(self._struct)


@functools.lru_cache(maxsize=256)
def _attn_workspace(device, *sizes):  # a function of the sizes and the (current) device
    return _bs.load().bsattn_kv4_attn_workspace(*sizes)


@functools.lru_cache(maxsize=256)
def _select_workspace(device, *sizes):
    return _bs.load().bsattn_kv4_select_workspace(*sizes)


def _cache(cache) -> Kv4Cache:
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    return cache


def _table(cache, block_table, lengths, counts=None, name="lengths"):
    """Checks the shared index tensors; returns (B, row stride, columns)."""
    tensor("block_table", block_table, (_I32,), device=cache.device, contiguous=False)
    if block_table.dim() != 2 or block_table.shape[1] == 0 or \
            (block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("block_table must be [B, pages a sequence], rows contiguous")
    B, columns = block_table.shape
    tensor(name, lengths, (_I32,), (B,), cache.device)
    if counts is not None:
        tensor("counts", counts, (_I32,), (B,), cache.device)
    return B, block_table.stride(0), columns


def _queries(cache, q, B):
    tensor("q", q, (_BF16,), device=cache.device)
    if q.dim() != 4 or q.shape[0] != B or q.shape[3] != cache.head_dim or not q.shape[2] \
            or not q.shape[1] or q.shape[1] % cache.kv_heads:
        raise ValueError("q must be [B, H, T, head_dim] with H a multiple of the cache's kv_heads")
    H, T = q.shape[1:3]
    if H // cache.kv_heads * T > 128:
        raise ValueError("at most 128 query rows a key/value head (H / kv_heads * T)")
    return H, T


def _rows(name, t, cache, B, T):
    """Checks new keys or values; returns their strides of batch, head and token."""
    tensor(name, t, (_BF16,), (B, cache.kv_heads, T, cache.head_dim), cache.device, False)
    sb, sh, st, sd = t.stride()
    if (sb | sh | st) % 8:  # a stride along a single entry does not matter
        sb, sh, st = (s if n > 1 else 0 for s, n in zip((sb, sh, st), t.shape))
    if t.numel() and (sd != 1 or (sb | sh | st) % 8 or t.data_ptr() % 16):
        raise ValueError(f"{name}: channels must be contiguous, other strides multiples of 8 "
                         "elements, the data 16-byte aligned")
    return sb, sh, st


def kv4_append(cache: Kv4Cache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
               lengths: torch.Tensor, counts: torch.Tensor | None = None, stream=None) -> None:
    """Write new tokens: k, v CUDA bf16 [B, kv_heads, T, head_dim] (channels
    contiguous, other strides multiples of 8), token t of sequence b at position
    lengths[b] + t for t < counts[b] (default T).  block_table: int32 [B, pages
    a sequence]; lengths, counts: int32 [B].  lengths is not changed."""
    _cache(cache)
    B, stride, columns = _table(cache, block_table, lengths, counts)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k, v must be [B, kv_heads, T, head_dim]")
    T = k.shape[2]
    k_strides, v_strides = _rows("k", k, cache, B, T), _rows("v", v, cache, B, T)
    if B * T == 0:
        return
    with launch_on(cache.device, stream) as on:
        _bs._check(_bs.load().bsattn_kv4_append(
            cache._ref, k.data_ptr(), *k_strides, v.data_ptr(), *v_strides, B, T,
            block_table.data_ptr(), stride, columns, lengths.data_ptr(), pointer(counts),
            on), "bsattn_kv4_append")


def kv4_read(cache: Kv4Cache, block_table: torch.Tensor, start: torch.Tensor, tokens: int,
             counts: torch.Tensor | None = None, k: torch.Tensor | None = None,
             v: torch.Tensor | None = None, stream=None):
    """k, v (CUDA bf16 [B, kv_heads, tokens, head_dim]): positions start[b] .. start[b] +
    tokens - 1 of every sequence; rows from counts[b] on are zero."""
    _cache(cache)
    B, stride, columns = _table(cache, block_table, start, counts, "start")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    shape = (B, cache.kv_heads, tokens, cache.head_dim)
    with launch_on(cache.device, stream) as on:
        k = output("k", k, _BF16, shape, cache.device)
        v = output("v", v, _BF16, shape, cache.device)
        if B * tokens:
            _bs._check(_bs.load().bsattn_kv4_read(
                cache._ref, B, tokens, block_table.data_ptr(), stride, columns, start.data_ptr(),
                pointer(counts), k.data_ptr(), v.data_ptr(), on),
                "bsattn_kv4_read")
    return k, v


def kv4_select(cache: Kv4Cache, q: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor,
               keep: int, sink: int = 1, recent: int = 1, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """int32 [B, kv_heads, keep]: the pages (position // page_size), ascending and
    then -1, that the queries q [B, H, T, head_dim] agree best with by their mean
    keys: the first `sink` and last `recent` pages always, then the best.
    lengths counts the T new tokens too."""
    _cache(cache)
    B, stride, columns = _table(cache, block_table, lengths)
    H, T = _queries(cache, q, B)
    if sink < 0 or recent < 1 or keep < sink + recent:
        raise ValueError("sink must not be negative, recent at least 1, keep at least sink + recent")
    with launch_on(cache.device, stream) as on:
        out = output("out", out, _I32, (B, cache.kv_heads, keep), cache.device)
        if B:
            lib = _bs.load()
            nbytes = _select_workspace(cache.device.index, B, cache.kv_heads, columns)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device) if nbytes else None
            _bs._check(lib.bsattn_kv4_select(
                cache._ref, q.data_ptr(), B, H, T, block_table.data_ptr(), stride, columns,
                lengths.data_ptr(), keep, sink, recent, out.data_ptr(), pointer(ws), nbytes,
                on), "bsattn_kv4_select")
    return out


def kv4_attn(cache: Kv4Cache, q: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor,
             selected: torch.Tensor | None = None, scale: float | None = None,
             out_f32: bool = False, out: torch.Tensor | None = None,
             lse: torch.Tensor | None = None, stream=None):
    """O [B, H, T, head_dim] (bf16, or fp32 with out_f32), LSE fp32 [B, H, T] of the
    last T tokens of every sequence against the cache.

    q: CUDA bf16 [B, H, T, head_dim]; query t of T sits at position lengths[b] - T + t
    and sees the cached tokens up to there (lengths counts the T new tokens
    too).  selected: kv4_select's pages (int32 [B, kv_heads, n], strictly
    ascending, then -1); default: all.  scale: default 1/sqrt(head_dim)."""
    _cache(cache)
    B, stride, columns = _table(cache, block_table, lengths)
    H, T = _queries(cache, q, B)
    n_selected = 0
    if selected is not None:
        tensor("selected", selected, (_I32,), device=cache.device)
        if selected.dim() != 3 or selected.shape[:2] != (B, cache.kv_heads) or not selected.shape[2]:
            raise ValueError("selected must be [B, kv_heads, pages]")
        n_selected = selected.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(cache.head_dim)
    odt = torch.float32 if out_f32 else _BF16
    with launch_on(cache.device, stream) as on:
        out = output("out", out, odt, q.shape, cache.device)
        lse = output("lse", lse, torch.float32, q.shape[:3], cache.device)
        if B:
            lib = _bs.load()
            nbytes = _attn_workspace(cache.device.index, B, H, cache.kv_heads, T, cache.head_dim,
                                     cache.page_size, columns, n_selected)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device) if nbytes else None
            _bs._check(lib.bsattn_kv4_attn(
                cache._ref, q.data_ptr(), B, H, T, block_table.data_ptr(), stride, columns,
                lengths.data_ptr(), pointer(selected), n_selected, float(scale),
                _bs.OUT_F32 if out_f32 else 0, out.data_ptr(), lse.data_ptr(), pointer(ws),
                nbytes, on), "bsattn_kv4_attn")
    return out, lse


def kv4_status(cache: Kv4Cache, stream=None) -> None:
    """Wait for the stream; raise if a call met a bad page or page list since the last check."""
    _cache(cache)
    with launch_on(cache.device, stream) as on:
        _bs._check(_bs.load().bsattn_kv4_status(cache._ref, on),
                   "kv4 status")
