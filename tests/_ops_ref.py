"""Plain 64-bit restatements of the operators around the attention (torch on
any device), for the tests of those operators."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
UBF = 2.0 ** -8    # half a step of bf16


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


# ------------------------------------------------------------- norm + rotation

def pair_index(D, rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(table, positions, B, S, D, interleaved):
    """cos, sin [B, S, 1, D] (1, 0 on channels that are not rotated) and the partner of every
    channel with its sign: y = n cos + sign * n[partner] sin."""
    dev = table.device
    rot = 2 * table.shape[1]
    pos = torch.arange(S, device=dev).expand(B, S) if positions is None else positions.long()
    bad = (pos < 0) | (pos >= table.shape[0])
    t = table.double()[pos.clamp(0, table.shape[0] - 1)]
    t[bad] = float("nan")
    a, b = pair_index(D, rot, interleaved)
    cos = torch.ones(B, S, D, dtype=torch.float64, device=dev)
    sin = torch.zeros_like(cos)
    cos[..., a] = cos[..., b] = t[..., 0]
    sin[..., a] = sin[..., b] = t[..., 1]
    partner, sign = torch.arange(D), torch.ones(D, dtype=torch.float64)
    partner[a], partner[b] = b, a
    sign[a] = -1.0
    return cos[:, :, None], sin[:, :, None], partner.to(dev), sign.to(dev)


def rotate(n, rot):
    if rot is None:
        return n
    cos, sin, partner, sign = rot
    return n * cos + sign * n[..., partner] * sin


def rotate_back(g, rot):
    if rot is None:
        return g
    cos, sin, partner, sign = rot
    return g * cos - sign * g[..., partner] * sin


def norm_rope(x, w, eps, rot):
    """[B, S, h, D] in, y in 64 bits and the scale of its 32-bit errors."""
    x = x.double()
    n = x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    size = n.abs()
    if rot is not None:
        cos, sin, partner, _ = rot
        size = size * cos.abs() + size[..., partner] * sin.abs()
    return rotate(n, rot), size


def norm_rope_bwd(x, dy, w, eps, rot):
    """dx, dw and the scales of their 32-bit errors; dy [B, S, h, D]."""
    x, dy = x.double(), dy.double()
    g = rotate_back(dy, rot)
    gs = dy.abs()
    if rot is not None:
        cos, sin, partner, _ = rot
        gs = gs * cos.abs() + gs[..., partner] * sin.abs()
    if w is None:
        return g, None, gs, None
    w = w.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    u = g * w
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
    size = r * (gs * w.abs() + x.abs() * r * r * (gs * w.abs() * x.abs()).mean(-1, keepdim=True))
    return dx, (g * x * r).flatten(0, 2).sum(0), size, (gs * x.abs() * r).flatten(0, 2).sum(0)


# ------------------------------------------------------------- block choice

def round7(m):
    """(whole numbers, exponent) of m [..., D]: t = rint(m 2^(6 - E)), E = floor(log2 max |m|)."""
    m = torch.where(m.isfinite(), m, 0.0)
    top = m.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 1, 0).double()
    return torch.round(m * torch.exp2(6 - e)), e - 6


def select_blocks(q, k, keep, causal=False, key_block=128, sink=0, local=1, allow=None):
    B, H, S, D = q.shape
    Hkv, nb, kd = k.shape[1], S // 128, 128 // key_block
    nk = nb * kd
    tq, _ = round7(q.double().view(B, H, nb, 128, D).mean(3))
    tk, ek = round7(k.double().view(B, Hkv, nk, key_block, D).mean(3))
    mk = (tk * torch.exp2(ek)).repeat_interleave(H // Hkv, 1)
    score = tq @ mk.transpose(-1, -2)
    row = torch.arange(nb, device=q.device)[:, None]
    blk = torch.arange(nk, device=q.device)[None]
    ok = (blk // kd <= row) if causal else torch.ones(nb, nk, dtype=torch.bool, device=q.device)
    ok = ok.expand(B, H, nb, nk)
    if allow is not None:
        ok = ok & (allow != 0)
    must = ok & ((blk < sink) | ((blk // kd - row).abs() < local))
    score = score.masked_fill(must, float("inf")).masked_fill(~ok, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order)
    rank.scatter_(-1, order, torch.arange(nk, device=q.device).expand_as(order).contiguous())
    most = must.sum(-1, keepdim=True).clamp(min=keep)
    return ((rank < most) & ok).to(torch.uint8)


# ------------------------------------------------------------- the 4-bit cache

def quantise(x, group):
    """codes [..., D] and (step, least) [..., D / group, 2], 64-bit values of the bf16 scales."""
    xg = x.double().unflatten(-1, (x.shape[-1] // group, group))
    least = xg.amin(-1, keepdim=True)
    top = xg.amax(-1, keepdim=True)
    bad = ~xg.isfinite().all(-1, keepdim=True) | ((top - least) > torch.finfo(torch.float32).max)
    step = ((top - least).float() / 15).bfloat16().double()
    step = torch.where(step < 2.0 ** -100, 0.0, step)
    code = torch.where(step > 0, torch.round((xg - least) / torch.where(step > 0, step, 1.0)), 0.0)
    code = torch.where(bad, 0.0, code.clamp(0, 15))
    nan = float("nan")
    scales = torch.cat([torch.where(bad, nan, step), torch.where(bad, nan, least)], -1)
    return code.flatten(-2).to(torch.uint8), scales


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def values(packed, scales):
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).double()
    s = scales.double().repeat_interleave(code.shape[-1] // scales.shape[-2], -2)
    return code * s[..., 0] + s[..., 1]


def fill(cache, seed, spread=1.0):
    """Random tokens in every slot of a Kv4Cache (and the means that go with them)."""
    g = gen(seed)
    shape = (cache.pages, cache.kv_heads, cache.page_size, cache.head_dim)
    for name in "kv":
        x = (torch.randn(shape, generator=g, device="cuda") * spread).bfloat16()
        if name == "k":  # pages apart from one another
            x += torch.randn(shape[0], shape[1], 1, shape[3], generator=g, device="cuda").bfloat16()
        code, scales = quantise(x, cache.group)
        getattr(cache, name + "_codes").copy_(pack(code))
        getattr(cache, name + "_scales").copy_(scales)
    means(cache)


def means(cache, pages=slice(None)):
    v = values(cache.k_codes[pages], cache.k_scales[pages]).float().double()
    t, e = round7(v.mean(-2))
    cache.k_means[pages] = (t * torch.exp2(e)).bfloat16()


def table(cache, lengths, columns, seed):
    """A block table over scattered pages of the cache, -1 where a sequence has none."""
    order = torch.randperm(cache.pages, generator=gen(seed, "cpu")).to(torch.int32)
    t = torch.full((len(lengths), columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lengths):
        need = -(-n // cache.page_size)
        t[b, :need] = order[at:at + need]
        at += need
    assert at <= cache.pages
    return t.cuda()


def select_pages(cache, q, block_table, lengths, keep, sink, recent):
    B, H, T, D = q.shape
    Hkv, page = cache.kv_heads, cache.page_size
    out = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=q.device)
    for b, n in enumerate(lengths):
        n = -(-max(n, 0) // page)
        if n == 0:
            continue
        mean = cache.k_means[block_table[b, :n].long()].double()
        for h in range(Hkv):
            rows = q[b, h * H // Hkv:(h + 1) * H // Hkv].double().reshape(-1)
            t = round7(rows)[0].view(-1, D)
            s = (t @ mean[:, h].T).amax(0)
            s[:sink] = float("inf")
            s[max(0, n - recent):] = float("inf")
            best = torch.sort(s, descending=True, stable=True)[1][:keep].sort()[0]
            out[b, h, :best.numel()] = best.to(torch.int32)
    return out


def attn(cache, q, block_table, lengths, selected=None, scale=None):
    """O, LSE in 64 bits, and per sequence the bounds (on O, on LSE) of 32-bit arithmetic."""
    B, H, T, D = q.shape
    Hkv, page, dev = cache.kv_heads, cache.page_size, q.device
    G = H // Hkv
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, H, T, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=dev)
    tol_o, tol_l = torch.zeros_like(lse), torch.zeros_like(lse)
    for b, n in enumerate(lengths):
        for h in range(Hkv):
            lp = torch.arange(-(-max(n, 0) // page), device=dev) if selected is None else selected[b, h]
            lp = lp[(lp >= 0) & (lp * page < n)].long()
            if lp.numel() == 0:
                continue
            pg = block_table[b, lp].long()
            k = values(cache.k_codes[pg, h], cache.k_scales[pg, h]).reshape(-1, D)
            v = values(cache.v_codes[pg, h], cache.v_scales[pg, h]).reshape(-1, D)
            pos = (lp[:, None] * page + torch.arange(page, device=dev)).reshape(-1)
            k, v, pos = k[pos < n], v[pos < n], pos[pos < n]
            ks, vs = ((getattr(cache, m + "_scales")[pg, h].double().reshape(-1, D // cache.group, 2)) for m in "kv")
            ks, vs = ks[:pos.numel()], vs[:pos.numel()]
            kbig = (15 * ks[..., 0] + ks[..., 1].abs()).amax()
            vbig = (15 * vs[..., 0] + vs[..., 1].abs()).amax()
            for t in range(T):
                see = pos <= n - T + t
                if not bool(see.any()):
                    continue
                qq = q[b, h * G:(h + 1) * G, t].double()
                s = qq @ k[see].T * scale
                lse[b, h * G:(h + 1) * G, t] = torch.logsumexp(s, -1)
                out[b, h * G:(h + 1) * G, t] = torch.softmax(s, -1) @ v[see]
                # a score is a sum of D products, step and least apart: at most (D + 8) roundings
                # of terms below |q| (15 step + |least|)
                m = int(see.sum())
                ds = (D + 8) * U32 * abs(scale) * qq.abs().sum(-1) * kbig
                # exp2 of a 32-bit argument (2 ulp and the argument's own rounding), weights held
                # in 21 bits or more, sums of m terms
                dp = ds + 2.0 ** -20 + (m + 8) * U32 + s.abs().amax() * 4 * U32
                tol_l[b, h * G:(h + 1) * G, t] = dp
                tol_o[b, h * G:(h + 1) * G, t] = 2 * dp * vbig
    return out, lse, tol_o, tol_l
