"""Block masks chosen by a cheap score (block means), for plan().

    mask = bsattn.select_blocks(q, k, keep=51, causal=True, sink=1, local=2)
    plan = bsattn.plan(mask, causal=True)
"""
from __future__ import annotations

import functools

import torch

import block_sparse_flash_attn_gb300 as _bs

from ._args import launch_on, output, pointer, tensor


@functools.lru_cache(maxsize=256)
def _workspace(*sizes):  # a function of the sizes
    return _bs.load().bsattn_select_blocks_workspace(*sizes)


def select_blocks(q: torch.Tensor, k: torch.Tensor, keep: int, causal: bool = False,
                  key_block: int = 128, sink: int = 0, local: int = 1,
                  allow: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """uint8 [B, H, S/128, S/key_block]: of every 128-query block the `keep` key
    blocks that its mean query agrees best with.

    q: CUDA bf16 [B, H, S, D], k: [B, Hkv, S, D] (H % Hkv == 0).  Block means are
    rounded to 7 bits beside their largest entry, so scores are exact and the
    mask depends on the inputs alone; equal scores go to the lower index.  The
    first `sink` key blocks and those of the 128-token blocks fewer than `local`
    away are kept first (all of them, even if they are more than `keep`);
    causal rules out what lies behind the query block; allow (uint8
    [B, H or 1, S/128, S/key_block]) rules out blocks by hand.  A query block with
    nothing allowed keeps nothing (fwd gives O = 0, LSE = -inf there)."""
    bf16 = torch.bfloat16
    tensor("q", q, (bf16,))
    if q.dim() != 4:
        raise ValueError("q must be [B, H, S, D]")
    B, H, S, D = q.shape
    tensor("k", k, (bf16,), device=q.device)
    if k.dim() != 4 or k.shape[0] != B or k.shape[2:] != q.shape[2:] or not k.shape[1] \
            or H % k.shape[1]:
        raise ValueError("k must be [B, Hkv, S, D] with H % Hkv == 0")
    if S == 0 or S % 128 or D not in (64, 128):
        raise ValueError("S must be a positive multiple of 128, D 64 or 128")
    if key_block not in (64, 128):
        raise ValueError("key_block must be 128 or 64")
    if keep <= 0 or sink < 0 or local < 0:
        raise ValueError("keep must be positive, sink and local not negative")
    Hkv, nb, nk = k.shape[1], S // 128, S // key_block
    keep, sink, local = min(keep, nk), min(sink, nk), min(local, nb)  # (C ints)
    allow_heads = 0
    if allow is not None:
        tensor("allow", allow, (torch.uint8,), device=q.device)
        if allow.dim() != 4 or allow.shape[1] not in (1, H) or \
                (allow.shape[0], *allow.shape[2:]) != (B, nb, nk):
            raise ValueError(f"allow must be [B, H or 1, S/128, S/{key_block}]")
        allow_heads = allow.shape[1]
    flags = (_bs.CAUSAL if causal else 0) | (_bs.KEY_BLOCK_64 if key_block == 64 else 0)
    with launch_on(q.device, stream) as on:
        out = output("out", out, torch.uint8, (B, H, nb, nk), q.device)
        if B * H:
            lib = _bs.load()
            nbytes = _workspace(B, H, Hkv, S, D, flags)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            _bs._check(lib.bsattn_select_blocks(
                q.data_ptr(), k.data_ptr(), B, H, Hkv, S, D, keep, sink, local, flags,
                pointer(allow), allow_heads, out.data_ptr(), ws.data_ptr(), nbytes, on),
                "bsattn_select_blocks")
    return out
