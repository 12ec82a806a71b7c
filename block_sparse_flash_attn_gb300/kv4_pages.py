"""The pages of a 4-bit cache: given to sequences that grow, shared by sequences
that fork, copied, and moved together.

    refs = torch.zeros(cache.pages, dtype=torch.int32, device="cuda")   # holders of each page
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    table, refs = bsattn.kv4_reserve(cache, refs, table, lengths, counts)    # before kv4_append
    table, lengths, refs = bsattn.kv4_fork(cache, refs, table, lengths, parents)
    table, refs, page_map = bsattn.kv4_compact(cache, refs, table)
    bsattn.kv4_copy(cache, src, dst, to=other)
    bsattn.kv4_status(cache)                       # raises if pages ran out or a page was bad

refs counts the table's rows that hold a page; one that none holds is free.  A page
that is not full belongs to one row (so a row that becomes shorter does not end inside
a page that it shares).
Where rows did become shorter than pages were reserved for (drafts that were refused),
the next call that takes `held` needs it, or those pages are lost:

    table, refs = bsattn.kv4_reserve(cache, refs, table, lengths, counts, held=held)
    held = lengths + counts                        # what the rows have pages for
    lengths += accepted                            # at most counts

The lowest free page is given out first, in the order of rows and columns.  Results
are new tensors, or those of `out`, which may be the arguments themselves where that
is said.  At most 16384 rows.
"""
from __future__ import annotations

import functools

import torch

import block_sparse_flash_attn_gb300 as _bs

from ._args import launch_on, output, pointer, tensor
from .kv4 import Kv4Cache, _cache, _table

_I32 = torch.int32


@functools.lru_cache(maxsize=256)
def _fork_workspace(n):
    return _bs.load().bsattn_kv4_fork_workspace(n)


@functools.lru_cache(maxsize=256)
def _compact_workspace(pages):
    return _bs.load().bsattn_kv4_compact_workspace(pages)


def _refs(cache, refs):
    return tensor("refs", refs, (_I32,), (cache.pages,), cache.device)


def _outputs(out, names):
    if out is None:
        return (None,) * len(names)
    if not isinstance(out, (tuple, list)) or len(out) != len(names):
        raise ValueError(f"out must be ({', '.join(names)})")
    return tuple(out)


def _table_out(name, t, block_table):
    """t, checked, or a new table: rows contiguous, of any stride where it is given."""
    if t is None:
        return torch.empty(block_table.shape, dtype=_I32, device=block_table.device)
    tensor(name, t, (_I32,), block_table.shape, block_table.device, False)
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t


def _release(cache, refs, block_table, stride, columns, lengths, held, table, new_refs, on):
    """Pages behind the lengths, up to those of `held` tokens, lose their rows (table: None, or for the rows
    without them)."""
    _bs._check(_bs.load().bsattn_kv4_release(
        cache._ref, refs.data_ptr(), block_table.data_ptr(), stride, columns, lengths.data_ptr(),
        held.data_ptr(), block_table.shape[0], pointer(table), 0 if table is None else table.stride(0),
        new_refs.data_ptr(), on), "bsattn_kv4_release")


def kv4_copy(cache: Kv4Cache, src: torch.Tensor, dst: torch.Tensor, to: Kv4Cache | None = None,
             stream=None) -> None:
    """Copy pages src[i] of the cache to pages dst[i] of `to` (default: the same cache; another
    one has the same sizes but for its number of pages).  src, dst: CUDA int32 [n]; a pair
    with a negative page is no move.  A page must not be written twice in one call, nor be
    read where it is written.  A page that is not there is reported by both caches."""
    to = _cache(cache) if to is None else _cache(to)
    tensor("src", src, (_I32,), device=cache.device)
    if src.dim() != 1:
        raise ValueError("src, dst must be [n]")
    tensor("dst", dst, (_I32,), src.shape, cache.device)
    if to.device != cache.device:
        raise TypeError(f"to must be on {cache.device}")
    if (to.kv_heads, to.page_size, to.head_dim, to.group) != (cache.kv_heads, cache.page_size,
                                                              cache.head_dim, cache.group):
        raise ValueError("to must have the cache's kv_heads, page_size, head_dim and group")
    if src.numel() == 0:
        return
    with launch_on(cache.device, stream) as on:
        _bs._check(_bs.load().bsattn_kv4_copy(cache._ref, to._ref, src.data_ptr(), dst.data_ptr(),
                                              src.numel(), on), "bsattn_kv4_copy")


def kv4_fork(cache: Kv4Cache, refs: torch.Tensor, block_table: torch.Tensor,
             lengths: torch.Tensor, parents: torch.Tensor, out=None, stream=None,
             held: torch.Tensor | None = None):
    """(block_table [n, columns], lengths [n], refs): new row i continues row parents[i] of the
    old table; a row that none continues ends, and row i is empty where parents[i] is
    negative.  So samples fork, beams change places, and ended sequences give their pages
    back in one call.  Full pages are shared; of a last page that is not full the first
    child keeps the parent's, the others get copies (pages of ended rows among those given
    out).

    refs: int32 [pages], block_table [B, columns] and lengths [B]: all rows that refs
    counts; parents: CUDA int32 [n].  out: (block_table, lengths, refs), of which refs may
    be the argument itself.  held: int32 [B], the tokens that the old rows have pages for,
    where that is more than lengths: those behind the lengths are given back."""
    _cache(cache)
    B, stride, columns = _table(cache, block_table, lengths)
    _refs(cache, refs)
    tensor("parents", parents, (_I32,), device=cache.device)
    if parents.dim() != 1:
        raise ValueError("parents must be [n]")
    if held is not None:
        tensor("held", held, (_I32,), (B,), cache.device)
    n = parents.numel()
    table, new_lengths, new_refs = _outputs(out, ("block_table", "lengths", "refs"))
    with launch_on(cache.device, stream) as on:
        table = output("block_table", table, _I32, (n, columns), cache.device)
        new_lengths = output("lengths", new_lengths, _I32, (n,), cache.device)
        new_refs = output("refs", new_refs, _I32, (cache.pages,), cache.device)
        if B == 0 or n == 0:
            raise ValueError("there must be rows")
        if held is not None:
            _release(cache, refs, block_table, stride, columns, lengths, held, None, new_refs, on)
            refs = new_refs
        nbytes = _fork_workspace(n)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        _bs._check(_bs.load().bsattn_kv4_fork(
            cache._ref, refs.data_ptr(), block_table.data_ptr(), stride, columns,
            lengths.data_ptr(), B, parents.data_ptr(), n, table.data_ptr(), new_lengths.data_ptr(),
            new_refs.data_ptr(), ws.data_ptr(), nbytes, on), "bsattn_kv4_fork")
    return table, new_lengths, new_refs


def kv4_reserve(cache: Kv4Cache, refs: torch.Tensor, block_table: torch.Tensor,
                lengths: torch.Tensor, counts: torch.Tensor | int, out=None, stream=None,
                held: torch.Tensor | None = None):
    """(block_table, refs) with pages for counts[b] (int32 [B], or one number) more tokens of
    every row: the columns behind those of lengths[b] tokens get new pages, whatever they
    held.  Where pages run out the last ones are -1.  out: (block_table, refs), which may be
    the arguments themselves.

    held: int32 [B], the tokens that the rows have pages for already, where that is more than
    lengths: lengths + counts of the call before, if drafts were refused since, or of this very
    call, if it ran out of pages and is tried again in place.  Those pages are given back
    first, so that refs counts what the table holds behind the call."""
    _cache(cache)
    T = 0
    if isinstance(counts, int):
        T, counts = counts, None
        if not 0 <= T < 1 << 31:
            raise ValueError("counts must not be negative")
    elif not isinstance(counts, torch.Tensor):
        raise TypeError("counts must be a tensor or an int")
    B, stride, columns = _table(cache, block_table, lengths, counts)
    _refs(cache, refs)
    if held is not None:
        tensor("held", held, (_I32,), (B,), cache.device)
    table, new_refs = _outputs(out, ("block_table", "refs"))
    if B == 0:
        raise ValueError("there must be rows")
    with launch_on(cache.device, stream) as on:
        table = _table_out("block_table", table, block_table)
        new_refs = output("refs", new_refs, _I32, (cache.pages,), cache.device)
        if held is not None:
            _release(cache, refs, block_table, stride, columns, lengths, held, table, new_refs, on)
            refs, block_table, stride = new_refs, table, table.stride(0)
        _bs._check(_bs.load().bsattn_kv4_reserve(
            cache._ref, refs.data_ptr(), block_table.data_ptr(), stride, columns,
            lengths.data_ptr(), pointer(counts), T, B, table.data_ptr(), table.stride(0),
            new_refs.data_ptr(), on), "bsattn_kv4_reserve")
    return table, new_refs


def kv4_compact(cache: Kv4Cache, refs: torch.Tensor, block_table: torch.Tensor, out=None,
                stream=None):
    """(block_table, refs, page_map): the n pages in use are brought to places 0 .. n - 1,
    those at n and above moving to the free ones below, both in ascending order.
    page_map: int32 [pages], the new place of each page (-1: free), for tables that the call
    does not see.  out: (block_table, refs, page_map), of which the first two may be the
    arguments themselves."""
    _cache(cache)
    tensor("block_table", block_table, (_I32,), device=cache.device, contiguous=False)
    if block_table.dim() != 2 or not block_table.numel() or \
            (block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("block_table must be [B, pages a sequence], rows contiguous")
    _refs(cache, refs)
    B, columns = block_table.shape
    table, new_refs, page_map = _outputs(out, ("block_table", "refs", "page_map"))
    with launch_on(cache.device, stream) as on:
        table = _table_out("block_table", table, block_table)
        new_refs = output("refs", new_refs, _I32, (cache.pages,), cache.device)
        page_map = output("page_map", page_map, _I32, (cache.pages,), cache.device)
        nbytes = _compact_workspace(cache.pages)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        _bs._check(_bs.load().bsattn_kv4_compact(
            cache._ref, refs.data_ptr(), block_table.data_ptr(), block_table.stride(0), columns, B,
            table.data_ptr(), table.stride(0), new_refs.data_ptr(), page_map.data_ptr(),
            ws.data_ptr(), nbytes, on), "bsattn_kv4_compact")
    return table, new_refs, page_map
