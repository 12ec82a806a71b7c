"""Q, K, V from a projection: per-head RMS norm, rotation by position and the
head-major layout of the forward pass in one kernel, and its gradient.

    table = bsattn.rope_table(max_positions, rotary_dim)           # once
    q, k, v = bsattn.qk_norm_rope(x, H, Hkv, wq, wk, table)        # x: [B, S, H + 2 Hkv, D]
    o, lse = bsattn.fwd(q, k, v, plan)
    dq, dk, dv = bsattn.bwd(q, k, v, o, lse, dout, plan)
    dx, dwq, dwk = bsattn.qk_norm_rope_bwd(x, dq, dk, dv, wq, wk, table)
"""
from __future__ import annotations

import functools

import torch

import block_sparse_flash_attn_gb300 as _bs

from ._args import launch_on, output, pointer, tensor

ROPE_INTERLEAVED, WEIGHT_F32 = 1, 2

_F32, _BF16 = torch.float32, torch.bfloat16


def rope_table(positions: int, rotary_dim: int, theta: float = 10000.0,
               inv_freq: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """cos and sin of every position's angles, CUDA fp32 [positions, rotary_dim/2, 2].

    Angle i of position p is p * inv_freq[i] (default theta^(-2i/rotary_dim)),
    evaluated in 64 bits.  rotary_dim: a multiple of 16, at most 128."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise TypeError("device must be a CUDA device")
    if positions <= 0 or rotary_dim <= 0 or rotary_dim % 16 or rotary_dim > 128:
        raise ValueError("positions must be positive, rotary_dim a multiple of 16 up to 128")
    if inv_freq is None:
        inv_freq = float(theta) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.shape != (rotary_dim // 2,):
        raise ValueError("inv_freq must be a tensor of rotary_dim / 2 frequencies")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with launch_on(device, stream) as on:
        inv = inv_freq.to(device=device, dtype=torch.float64).contiguous()
        table = torch.empty((positions, rotary_dim // 2, 2), dtype=_F32, device=device)
        _bs._check(_bs.load().bsattn_rope_table(inv.data_ptr(), positions, rotary_dim,
                                                table.data_ptr(), on),
                   "bsattn_rope_table")
    return table


@functools.lru_cache(maxsize=256)
def _workspace(device, *sizes):  # a function of the sizes and the (current) device
    return _bs.load().bsattn_qk_norm_rope_bwd_workspace(*sizes)


def _common(x, heads, kv_heads, q_weight, k_weight, table, positions, interleaved):
    """The checks of both directions; returns the C call's shared arguments."""
    tensor("x", x, (_BF16,), contiguous=False)
    if heads <= 0 or kv_heads <= 0 or heads % kv_heads:
        raise ValueError("heads must be a positive multiple of kv_heads")
    if x.dim() != 4 or x.shape[2] != heads + 2 * kv_heads:
        raise ValueError("x must be [B, S, heads + 2 * kv_heads, D]")
    B, S, _, D = x.shape
    if D not in (64, 128):
        raise ValueError("D must be 64 or 128")
    sb, ss, sh, sd = x.stride()
    if sd != 1 or sh != D or (ss % 8 and S > 1) or (sb % 8 and B > 1) or x.data_ptr() % 16:
        raise ValueError("the rows of a token must be contiguous, tokens and batch entries a "
                         "multiple of 8 elements apart, x 16-byte aligned")
    flags = ROPE_INTERLEAVED if interleaved else 0
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight come together")
    if q_weight is not None:
        tensor("q_weight", q_weight, (_BF16, _F32), (D,), x.device)
        tensor("k_weight", k_weight, (q_weight.dtype,), (D,), x.device)
        if q_weight.dtype == _F32:
            flags |= WEIGHT_F32
    n_pos = rotary = 0
    if table is not None:
        tensor("table", table, (_F32,), device=x.device)
        if table.dim() != 3 or table.shape[2] != 2 or table.shape[1] % 8 or table.shape[1] * 2 > D \
                or table.numel() == 0:
            raise ValueError("table must be rope_table's: [positions, rotary_dim / 2, 2], "
                             "rotary_dim a multiple of 16 up to D")
        n_pos, rotary = table.shape[0], 2 * table.shape[1]
        if positions is None and S > n_pos:
            raise ValueError(f"the table has {n_pos} positions, x {S} tokens")
    elif positions is not None:
        raise ValueError("positions need a table")
    if positions is not None:
        tensor("positions", positions, (torch.int32,), (B, S), x.device)
    return B, S, D, n_pos, rotary, flags, sb if B > 1 else 0, ss if S > 1 else 0


def qk_norm_rope(x: torch.Tensor, heads: int, kv_heads: int, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, table: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, q: torch.Tensor | None = None,
                 k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """q [B, heads, S, D], k, v [B, kv_heads, S, D] (CUDA bf16) from a projection
    x: CUDA bf16 [B, S, heads + 2 * kv_heads, D] (heads of Q, of K, of V; the rows
    of a token contiguous).

    Rows of Q and K: x / sqrt(mean(x^2) + eps) * weight (without weights: x),
    then the first rotary_dim channels turned by the token's angles in `table`
    (rope_table; without: not turned), in pairs (i, i + rotary_dim/2), or
    (2i, 2i + 1) with interleaved.  positions: CUDA int32 [B, S] (default 0 .. S-1); one
    outside the table gives NaN.  Weights: bf16 or fp32 [D].  S need not be a
    multiple of 128 here."""
    B, S, D, n_pos, rotary, flags, sb, ss = _common(x, heads, kv_heads, q_weight, k_weight, table,
                                                    positions, interleaved)
    with launch_on(x.device, stream) as on:
        q = output("q", q, _BF16, (B, heads, S, D), x.device)
        k = output("k", k, _BF16, (B, kv_heads, S, D), x.device)
        v = output("v", v, _BF16, (B, kv_heads, S, D), x.device)
        if B * S:
            _bs._check(_bs.load().bsattn_qk_norm_rope(
                x.data_ptr(), sb, ss, B, S, heads, kv_heads, D,
                pointer(q_weight), pointer(k_weight), pointer(table), n_pos, rotary,
                pointer(positions), float(eps), flags, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                on), "bsattn_qk_norm_rope")
    return q, k, v


def qk_norm_rope_bwd(x: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                     table: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                     eps: float = 1e-6, interleaved: bool = False,
                     dx: torch.Tensor | None = None, stream=None):
    """dx (bf16, like x), dq_weight, dk_weight (fp32 [D]; None without weights):
    the gradient of qk_norm_rope, from dq [B, H, S, D], dk, dv [B, Hkv, S, D]
    (CUDA fp32, as bwd returns them) and the forward call's other arguments.
    dx may be x itself, but must not overlap it otherwise.  Repeated calls give the
    same bits."""
    for name, t in (("dq", dq), ("dk", dk)):
        if not isinstance(t, torch.Tensor) or t.dtype != _F32:
            raise TypeError(f"{name} must be a tensor of {_F32}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, H, S, D]")
    heads, kv_heads = dq.shape[1], dk.shape[1]
    B, S, D, n_pos, rotary, flags, sb, ss = _common(x, heads, kv_heads, q_weight, k_weight, table,
                                                    positions, interleaved)
    for name, t, h in (("dq", dq, heads), ("dk", dk, kv_heads), ("dv", dv, kv_heads)):
        tensor(name, t, (_F32,), (B, h, S, D), x.device)
    with launch_on(x.device, stream) as on:
        dx = output("dx", dx, _BF16, x.shape, x.device)
        dwq = dwk = ws = None
        row = x.shape[2] * D  # dx is contiguous (the strides of its axes of one entry may be anything)
        lib = _bs.load()
        if q_weight is not None:
            dwq = torch.empty(D, dtype=_F32, device=x.device)
            dwk = torch.empty(D, dtype=_F32, device=x.device)
            if B * S == 0:
                dwq.zero_(), dwk.zero_()
        if B * S:
            nbytes = 0
            if q_weight is not None:
                nbytes = _workspace(x.device.index, B, S, heads, kv_heads, D)
                ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
            _bs._check(lib.bsattn_qk_norm_rope_bwd(
                x.data_ptr(), sb, ss, dq.data_ptr(), dk.data_ptr(),
                dv.data_ptr(), B, S, heads, kv_heads, D, pointer(q_weight), pointer(k_weight),
                pointer(table), n_pos, rotary, pointer(positions), float(eps), flags,
                dx.data_ptr(), S * row, row, pointer(dwq), pointer(dwk),
                pointer(ws), nbytes, on), "bsattn_qk_norm_rope_bwd")
    return dx, dwq, dwk
