"""Workloads of the operators around block-sparse attention, for measuring.

Six kinds of pass, each in two forms on the same inputs: the plain form
(elementary torch operations in 32 bits, 64 where 32 lose what matters) and,
with ``own = True``, the calls that a user makes of this package.

    rope       per-head RMS norm of Q and K, rotation by position, head-major layout
    rope_grad  its gradient: the projection's and the two norm weights'
    select     block masks chosen by block means (prompts)
    append     new keys and values into the paged 4-bit cache, read back
    attn       attention of new tokens over the 4-bit cache
    sparse     pages chosen by page means, then attention over those pages
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 64 sequences: latency counts
        dict(name="rope-step", op="rope", B=64, S=1, H=32, Hkv=8, D=128, rot=128,
             interleaved=False, norm=True, given=True),
        # a prompt of two sequences at S = 16384
        dict(name="rope-prompt", op="rope", B=2, S=16384, H=32, Hkv=8, D=128, rot=128,
             interleaved=False, norm=True, given=False),
        # a small ragged training batch: odd length, half of the channels rotated, pairs side by side
        dict(name="rope-grad-odd", op="rope_grad", B=3, S=1021, H=16, Hkv=4, D=64, rot=32,
             interleaved=True, norm=True, given=True),
        # a training step at the size of the causal S = 4096 workload, one K/V head per query head
        dict(name="rope-grad-train", op="rope_grad", B=4, S=4096, H=16, Hkv=16, D=128, rot=128,
             interleaved=False, norm=True, given=False),
        # a short prompt at 64-key blocks with some blocks ruled out (padding, other documents)
        dict(name="select-short", op="select", B=1, S=1664, H=6, Hkv=2, D=64, key_block=64,
             keep=7, sink=1, local=1, causal=False, allow=True),
        # a long causal prompt, a tenth of the blocks kept
        dict(name="select-long", op="select", B=1, S=65536, H=32, Hkv=8, D=128, key_block=128,
             keep=51, sink=1, local=2, causal=True, allow=False),
        # one new token for each of 64 sequences
        dict(name="append-step", op="append", B=64, T=1, Hkv=8, D=128, page=64, group=128, longest=8192),
        # ragged prompts written behind what the cache holds already
        dict(name="append-prompt", op="append", B=8, T=4096, Hkv=8, D=128, page=64, group=32, longest=1000),
        # one sequence, a short context, small pages
        dict(name="attn-short", op="attn", B=1, T=1, H=16, Hkv=2, D=64, page=16, group=64, longest=777),
        # a serving batch of long contexts, lengths apart
        dict(name="attn-long", op="attn", B=32, T=1, H=32, Hkv=8, D=128, page=64, group=128, longest=65536),
        # drafted tokens checked together, a few pages of each sequence
        dict(name="sparse-draft", op="sparse", B=3, T=4, H=16, Hkv=4, D=128, page=32, group=32,
             longest=5000, keep=24, sink=1, recent=2),
        # long contexts of which every step reads one page in sixteen
        dict(name="sparse-long", op="sparse", B=16, T=1, H=32, Hkv=8, D=128, page=64, group=128,
             longest=65536, keep=64, sink=1, recent=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "select", "append", "attn", "sparse"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("rope", "rope_grad"):
        rows = _log(rng, 1, 1 << 20)  # (token, head) rows
        B = _log(rng, 1, 16)
        S = max(1, rows // (B * (H + 2 * Hkv)))
        return dict(op=op, B=B, S=S, H=H, Hkv=Hkv, D=D, rot=rng.choice([32, 64, D]),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, given=rng.random() < 0.5)
    if op == "select":
        nb = _log(rng, 12, 256)
        key_block = rng.choice([64, 128])
        sink, local = rng.choice([0, 1, 3]), rng.choice([0, 1, 2])
        forced = sink + max(0, 2 * local - 1) * 128 // key_block
        return dict(op=op, B=rng.choice([1, 2]) if nb < 100 else 1, S=128 * nb, H=min(H, 16), Hkv=1 if H > 16 else Hkv,
                    D=D, key_block=key_block, keep=forced + _log(rng, 1, nb // 3), sink=sink, local=local,
                    causal=rng.random() < 0.6, allow=rng.random() < 0.3)
    page = rng.choice([16, 32, 64, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= D])
    B = _log(rng, 1, 64)
    if op == "append":
        return dict(op=op, B=B, T=1 if rng.random() < 0.4 else _log(rng, 1, max(2, 30000 // B)), Hkv=Hkv, D=D,
                    page=page, group=group, longest=_log(rng, 1, 8192))
    T = rng.choice([1, 1, 1, 2, 3, 5])
    longest = _log(rng, 1, min(65536, (1 << 21) // (B * Hkv)))
    case = dict(op=op, B=B, T=T, H=H, Hkv=Hkv, D=D, page=page, group=group, longest=longest)
    if op == "sparse":
        sink, recent = rng.choice([0, 1]), rng.choice([1, 2])
        case.update(keep=sink + recent + _log(rng, 1, 64), sink=sink, recent=recent)
    return case


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV)


def _heads_spread(g, *shape):
    """Keys as models have them: a few channels of every head much wider than the rest."""
    return _randn(g, *shape) * (1.0 + 4.0 * (torch.rand(shape[-1], generator=g, device=DEV) < 0.04))


def _lengths(g, case, least):
    """Context lengths between half the longest and the longest, the first one the longest."""
    n = _randint(g, (case["longest"] + 1) // 2, case["longest"] + 1, (case["B"],))
    n[0] = case["longest"]
    return n.clamp(min=least).to(torch.int32)


def _pages(g, lengths, page, most):
    """A block table over scattered pages of a cache with room for `most` tokens a sequence:
    (table [B, pages a sequence], pages in all)."""
    need = ((lengths + page - 1) // page).tolist()
    most = -(-most // page)
    order = torch.randperm(len(need) * most + 3, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(need), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order.numel()


def _quantise(x, group):
    """4-bit codes [..., D] and (step, minimum) [..., D / group, 2] of x [..., D]."""
    xg = x.float().unflatten(-1, (x.shape[-1] // group, group))
    least = xg.amin(-1, keepdim=True)
    step = ((xg.amax(-1, keepdim=True) - least) / 15).bfloat16().float()
    code = ((xg - least).double() / torch.where(step > 0, step, torch.inf).double()).round_().clamp_(0, 15)
    return code.reshape(x.shape).to(torch.uint8), torch.cat([step, least], -1).bfloat16()


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(packed, scales):
    """What the cache stands for, 32 bits: step * code + minimum."""
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float()
    s = scales.float()
    code = code.unflatten(-1, (s.shape[-2], code.shape[-1] // s.shape[-2]))
    return (code * s[..., 0:1] + s[..., 1:2]).flatten(-2)


def _cache(case, g, pages):
    Hkv, D, page, group = case["Hkv"], case["D"], case["page"], case["group"]
    if own:
        import block_sparse_flash_attn_gb300 as bs
        cache = bs.Kv4Cache(pages, Hkv, D, page_size=page, group=group)
        t = dict(k_codes=cache.k_codes, v_codes=cache.v_codes, k_scales=cache.k_scales,
                 v_scales=cache.v_scales, k_means=cache.k_means, handle=cache)
    else:
        t = {}
        for n in "kv":
            t[n + "_codes"] = torch.zeros(pages, Hkv, page, D // 2, dtype=torch.uint8, device=DEV)
            t[n + "_scales"] = torch.zeros(pages, Hkv, page, D // group, 2, dtype=torch.bfloat16, device=DEV)
        t["k_means"] = torch.zeros(pages, Hkv, D, dtype=torch.bfloat16, device=DEV)
    part = max(1, (1 << 26) // (Hkv * page * D))
    for p in range(0, pages, part):
        n = min(part, pages - p)
        # keys of a page resemble one another, more on some pages than on others
        k = _heads_spread(g, n, Hkv, page, D) + _randn(g, n, Hkv, 1, D) * torch.rand(n, 1, 1, 1, generator=g, device=DEV)
        for name, x in (("k", k), ("v", _randn(g, n, Hkv, page, D))):
            code, scales = _quantise(x.bfloat16(), group)
            t[name + "_codes"][p:p + n] = _pack(code)
            t[name + "_scales"][p:p + n] = scales
        t["k_means"][p:p + n] = _round7(_values(t["k_codes"][p:p + n], t["k_scales"][p:p + n]).double().mean(2)).bfloat16()
    return t


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("rope", "rope_grad"):
        B, S, H, Hkv, D, rot = (case[n] for n in ("B", "S", "H", "Hkv", "D", "rot"))
        far = 0 if not case["given"] else 100000
        st = dict(x=_randn(g, B, S, H + 2 * Hkv, D).mul_(1 + torch.rand(D, generator=g, device=DEV)).bfloat16(),
                  wq=None, wk=None, positions=None)
        if case["norm"]:
            st["wq"] = (1 + 0.1 * _randn(g, D)).bfloat16()
            st["wk"] = (1 + 0.1 * _randn(g, D)).bfloat16()
        if case["given"]:
            st["positions"] = (_randint(g, 0, far, (B, 1)) + torch.arange(S, device=DEV)).to(torch.int32)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(far + S, dtype=torch.float64, device=DEV)[:, None] * freq
        st["table"] = torch.stack([angle.cos(), angle.sin()], -1).float()
        if op == "rope_grad":
            for n, h in (("dq", H), ("dk", Hkv), ("dv", Hkv)):
                st[n] = _randn(g, B, h, S, D) * 0.05
    elif op == "select":
        B, S, H, Hkv, D = (case[n] for n in ("B", "S", "H", "Hkv", "D"))
        nb, kd = S // 128, 128 // case["key_block"]

        def by_topic(h):  # neighbouring tokens resemble one another
            x = _randn(g, B, h, S, D)
            x.view(B, h, nb, 128, D).add_(_randn(g, B, h, nb, 1, D), alpha=0.5)
            return x.bfloat16()

        st = dict(q=by_topic(H), k=by_topic(Hkv), allow=None)
        if case["allow"]:
            st["allow"] = (torch.rand(B, H, nb, nb * kd, generator=g, device=DEV) < 0.7).to(torch.uint8)
            st["allow"][:, :, nb // 2] = 0  # a query block of padding
    elif op == "append":
        B, T, Hkv, D, page = (case[n] for n in ("B", "T", "Hkv", "D", "page"))
        lengths = _randint(g, 0, case["longest"] + 1, (B,)).to(torch.int32)
        counts = _randint(g, (T + 1) // 2, T + 1, (B,)).to(torch.int32)
        counts[0] = T
        table, pages = _pages(g, lengths + counts, page, case["longest"] + T)
        st = _cache(case, g, pages)
        st.update(lengths=lengths, counts=counts, table=table, k=_heads_spread(g, B, Hkv, T, D).bfloat16(),
                  v=_randn(g, B, Hkv, T, D).bfloat16())
    else:
        B, T, H, D, page = (case[n] for n in ("B", "T", "H", "D", "page"))
        lengths = _lengths(g, case, T)
        table, pages = _pages(g, lengths, page, max(case["longest"], T))
        st = _cache(case, g, pages)
        st.update(lengths=lengths, table=table, q=_randn(g, B, H, T, D).bfloat16())
    if "lengths" in st:
        st["host_lengths"] = st["lengths"].tolist()  # a server counts its tokens on the host too
    st["case"] = case
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    return (_run_own if own else _PLAIN[op])(st)


def _run_own(st):
    import block_sparse_flash_attn_gb300 as bs
    c = st["case"]
    op = c["op"]
    if op == "rope":
        return bs.qk_norm_rope(st["x"], c["H"], c["Hkv"], st["wq"], st["wk"], st["table"], st["positions"],
                               interleaved=c["interleaved"])
    if op == "rope_grad":
        return bs.qk_norm_rope_bwd(st["x"], st["dq"], st["dk"], st["dv"], st["wq"], st["wk"], st["table"],
                                   st["positions"], interleaved=c["interleaved"])
    if op == "select":
        return bs.select_blocks(st["q"], st["k"], c["keep"], causal=c["causal"], key_block=c["key_block"],
                                sink=c["sink"], local=c["local"], allow=st["allow"])
    cache = st["handle"]
    if op == "append":
        bs.kv4_append(cache, st["k"], st["v"], st["table"], st["lengths"], st["counts"])
        k, v = bs.kv4_read(cache, st["table"], st["lengths"], c["T"], st["counts"])
        return k, v, cache.k_means
    if op == "attn":
        return bs.kv4_attn(cache, st["q"], st["table"], st["lengths"])
    chosen = bs.kv4_select(cache, st["q"], st["table"], st["lengths"], c["keep"], sink=c["sink"], recent=c["recent"])
    return (chosen,) + tuple(bs.kv4_attn(cache, st["q"], st["table"], st["lengths"], chosen))


def _angles(st):
    """cos, sin [B or 1, S, 1, rot / 2] of every token's position."""
    S = st["x"].shape[1]
    t = st["table"][:S][None] if st["positions"] is None else st["table"][st["positions"].long()]
    return t[:, :, None, :, 0], t[:, :, None, :, 1]


def _pairs(x, rot, interleaved):
    """The two halves of the rotated channels, and the channels left alone."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, interleaved):
    ab = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([ab, rest], -1)


def _plain_rope(st):
    c = st["case"]
    H, Hkv = c["H"], c["Hkv"]
    cos, sin = _angles(st)
    out = []
    for x, w in ((st["x"][:, :, :H], st["wq"]), (st["x"][:, :, H:H + Hkv], st["wk"])):
        y = x.float()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b, rest = _pairs(y, c["rot"], c["interleaved"])
        y = _join(a * cos - b * sin, b * cos + a * sin, rest, c["interleaved"])
        out.append(y.to(x.dtype).transpose(1, 2).contiguous())
    return out[0], out[1], st["x"][:, :, H + Hkv:].transpose(1, 2).contiguous()


def _plain_rope_grad(st):
    c = st["case"]
    H, Hkv = c["H"], c["Hkv"]
    cos, sin = _angles(st)
    dx = torch.empty(st["x"].shape, dtype=st["x"].dtype, device=DEV)
    dw = []
    for lo, hi, dy, w in ((0, H, st["dq"], st["wq"]), (H, H + Hkv, st["dk"], st["wk"])):
        a, b, rest = _pairs(dy.transpose(1, 2), c["rot"], c["interleaved"])
        g = _join(a * cos + b * sin, b * cos - a * sin, rest, c["interleaved"])
        if w is None:
            dw.append(None)
        else:
            x = st["x"][:, :, lo:hi].float()
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            n = x * r
            dw.append((g * n).sum((0, 1, 2), dtype=torch.float64).float())
            u = g * w.float()
            g = r * (u - n * (u * n).mean(-1, keepdim=True))
        dx[:, :, lo:hi] = g
    dx[:, :, H + Hkv:] = st["dv"].transpose(1, 2)
    return dx, dw[0], dw[1]


def _round7(m):
    """Means rounded to 7 bits beside the largest of the last axis; 64 bits in and out."""
    m = torch.where(m.isfinite(), m, 0.0)
    top = torch.frexp(m.abs().amax(-1, keepdim=True))[1] - 1
    return torch.ldexp(torch.ldexp(m, 6 - top).round(), top - 6)


def _plain_select(st):
    c = st["case"]
    q, k = st["q"], st["k"]
    B, H, S, D = q.shape
    nb, kd = S // 128, 128 // c["key_block"]
    nk = nb * kd
    mask = torch.empty(B, H, nb, nk, dtype=torch.uint8, device=DEV)
    rows, cols = torch.arange(nb, device=DEV)[:, None], torch.arange(nk, device=DEV)[None]
    reach = cols // kd <= rows if c["causal"] else torch.ones(nb, nk, dtype=torch.bool, device=DEV)
    forced = reach & ((cols < c["sink"]) | ((cols // kd - rows).abs() < c["local"]))
    for b in range(B):
        for h in range(H):
            mq = _round7(q[b, h].view(nb, 128, D).double().mean(1))
            mk = _round7(k[b, h * c["Hkv"] // H].view(nk, c["key_block"], D).double().mean(1))
            score = (mq / 2.0 ** 6) @ mk.T
            can = reach if st["allow"] is None else reach & st["allow"][b, h].bool()
            must = can & forced
            score = torch.where(must, torch.inf, torch.where(can, score, -torch.inf))
            n = torch.minimum(must.sum(-1, keepdim=True).clamp(min=c["keep"]), can.sum(-1, keepdim=True))
            border = score.sort(-1, descending=True)[0].gather(-1, (n - 1).clamp(min=0))
            above, at = score > border, score == border
            at &= (at.cumsum(-1) <= n - above.sum(-1, keepdim=True))
            mask[b, h] = ((above | at) & (n > 0)).to(torch.uint8)
    return mask


def _slots(st, first, T):
    """(b, t, page, place) of the tokens that each sequence has among T."""
    t = torch.arange(T, device=DEV)[None]
    b, t = torch.nonzero(t < st["counts"][:, None], as_tuple=True)
    pos = first[b].long() + t
    page = st["case"]["page"]
    return b, t, st["table"][b, pos // page].long(), pos % page


def _plain_append(st):
    c = st["case"]
    b, t, page, place = _slots(st, st["lengths"], c["T"])
    read = []
    for n in "kv":
        code, scales = _quantise(st[n][b, :, t], c["group"])
        st[n + "_codes"][page, :, place] = _pack(code)
        st[n + "_scales"][page, :, place] = scales
    full = page[place == c["page"] - 1]
    st["k_means"][full] = _round7(_values(st["k_codes"][full], st["k_scales"][full]).double().mean(2)).bfloat16()
    for n in "kv":
        x = torch.zeros_like(st[n])
        x[b, :, t] = _values(st[n + "_codes"][page, :, place], st[n + "_scales"][page, :, place]).to(x.dtype)
        read.append(x)
    return read[0], read[1], st["k_means"]


def _plain_attn(st, chosen=None):
    c = st["case"]
    q = st["q"]
    B, H, T, D = q.shape
    Hkv, page = c["Hkv"], c["page"]
    out = torch.zeros_like(q)
    lse = torch.full((B, H, T), -torch.inf, device=DEV)
    for b in range(B):
        n = st["host_lengths"][b]
        at = torch.arange((n + page - 1) // page, device=DEV).expand(Hkv, -1) if chosen is None else chosen[b].long()
        ok = (at >= 0)[:, :, None].expand(-1, -1, page).reshape(Hkv, 1, -1)
        pos = (at[:, :, None] * page + torch.arange(page, device=DEV)).view(Hkv, 1, -1)
        p = st["table"][b, at.clamp(min=0)].long()
        head = torch.arange(Hkv, device=DEV)[:, None]
        k = _values(st["k_codes"][p, head], st["k_scales"][p, head]).flatten(1, 2)
        qb = q[b].float().reshape(Hkv, -1, D)
        s = qb @ k.transpose(1, 2) * D ** -0.5
        last = (n - T + torch.arange(T, device=DEV)).repeat(H // Hkv)[None, :, None]
        s = torch.where(ok & (pos <= last), s, -torch.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-1e30)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        v = _values(st["v_codes"][p, head], st["v_scales"][p, head]).flatten(1, 2)
        o = e @ v / torch.where(z > 0, z, 1.0)
        out[b] = o.reshape(H, T, D).to(q.dtype)
        lse[b] = (m + torch.log(z)).reshape(H, T)
    return out, lse


def _plain_sparse(st):
    c = st["case"]
    q, page, keep = st["q"], c["page"], c["keep"]
    B, H, T, D = q.shape
    chosen = torch.full((B, c["Hkv"], keep), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        n = (st["host_lengths"][b] + page - 1) // page
        mean = st["k_means"][st["table"][b, :n].long()].double().transpose(0, 1)  # [Hkv, n, D]
        rows = q[b].double().reshape(c["Hkv"], -1, D)
        rows = _round7(rows.flatten(1)).view_as(rows)
        score = (rows @ mean.transpose(1, 2)).amax(1)
        score[:, :c["sink"]] = torch.inf
        score[:, max(n - c["recent"], 0):] = torch.inf
        take = min(keep, n)
        best = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, :take]
        chosen[b, :, :take] = best.sort(-1)[0].to(torch.int32)
    return (chosen,) + _plain_attn(st, chosen)


_PLAIN = dict(rope=_plain_rope, rope_grad=_plain_rope_grad, select=_plain_select, append=_plain_append,
              attn=_plain_attn, sparse=_plain_sparse)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, D = case["op"], case["D"]
    if op in ("rope", "rope_grad"):
        heads, tokens = case["H"] + 2 * case["Hkv"], case["B"] * case["S"]
        n = tokens * heads * D
        table = min(tokens, case["S"] if not case["given"] else tokens) * case["rot"] * 4
        return dict(bytes=n * (4 if op == "rope" else 8) + table, flops=n * (10 if op == "rope" else 25))
    if op == "select":
        B, S, H, Hkv = (case[n] for n in ("B", "S", "H", "Hkv"))
        nb, nk = S // 128, S // case["key_block"]
        cells = B * H * nb * nk
        return dict(bytes=B * S * D * 2 * (H + Hkv) + cells * (2 if case["allow"] else 1),
                    flops=B * S * D * (H + Hkv) + cells * D * (1 if case["causal"] else 2))
    row = D // 2 + 4 * (D // case["group"])
    if op == "append":
        tokens = case["B"] * case["T"] * 0.75
        return dict(bytes=int(tokens * case["Hkv"] * 2 * (4 * D + 2 * row)), flops=int(tokens * case["Hkv"] * 2 * D * 8))
    tokens = case["B"] * case["longest"] * 0.75
    qo = case["B"] * case["H"] * case["T"] * (4 * D + 4)
    if op == "attn":
        return dict(bytes=int(tokens * case["Hkv"] * 2 * row + qo), flops=int(tokens * case["H"] * case["T"] * 4 * D))
    read = min(tokens, case["B"] * case["keep"] * case["page"])
    means = tokens / case["page"] * case["Hkv"] * D * 2
    return dict(bytes=int(read * case["Hkv"] * 2 * row + means + qo),
                flops=int((read * 4 + tokens / case["page"] * 2) * case["H"] * case["T"] * D))


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """What run returns for these inputs, from the definitions, in 64 bits."""
    st = prepare(case, seed)
    return _EXACT[case["op"]](st)


def _turn(x, table, positions, interleaved, sign):
    """x [B, S, h, D] as complex numbers turned by the table's angles (sign -1: turned back)."""
    rot = 2 * table.shape[1]
    at = torch.arange(x.shape[1], device=DEV)[None] if positions is None else positions.long()
    turn = torch.complex(table[at, :, 0].double(), sign * table[at, :, 1].double())[:, :, None]
    i = torch.arange(rot // 2, device=DEV)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(x[..., re], x[..., im]) * turn
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_rope(st):
    c = st["case"]
    outs = []
    for h, x in enumerate(st["x"].double().split([c["H"], c["Hkv"], c["Hkv"]], 2)):
        if h < 2:
            w = (st["wq"], st["wk"])[h]
            if w is not None:
                x = x * (x.square().sum(-1, keepdim=True) / c["D"] + 1e-6).rsqrt() * w.double()
            x = _turn(x, st["table"], st["positions"], c["interleaved"], 1.0)
        outs.append(x.permute(0, 2, 1, 3))
    return tuple(outs)


def _exact_rope_grad(st):
    c = st["case"]
    dx, dw = [], []
    for h, x in enumerate(st["x"].double().split([c["H"], c["Hkv"], c["Hkv"]], 2)):
        g = (st["dq"], st["dk"], st["dv"])[h].double().permute(0, 2, 1, 3)
        if h < 2:
            w = (st["wq"], st["wk"])[h]
            g = _turn(g, st["table"], st["positions"], c["interleaved"], -1.0)
            if w is None:
                dw.append(None)
            else:
                ms = x.square().sum(-1, keepdim=True) / c["D"] + 1e-6
                dw.append((g * x * ms.rsqrt()).flatten(0, 2).sum(0))
                u = g * w.double()
                g = u * ms.rsqrt() - x * ms.pow(-1.5) * (u * x).sum(-1, keepdim=True) / c["D"]
        dx.append(g)
    return torch.cat(dx, 2), dw[0], dw[1]


def _whole7(m):
    """(whole numbers up to 128, exponent) of means m [..., D]."""
    m = m.nan_to_num(0.0, 0.0, 0.0)
    e = torch.floor(torch.log2(m.abs().max(-1, keepdim=True)[0].clamp(min=1e-300)))
    return torch.round(m * torch.exp2(6 - e)), e - 6


def _exact_select(st):
    c = st["case"]
    B, H, S, D = st["q"].shape
    nb, kb = S // 128, c["key_block"]
    nk = S // kb
    i, j = torch.meshgrid(torch.arange(nb, device=DEV), torch.arange(nk, device=DEV) * kb // 128, indexing="ij")
    near = (i - j).abs() < c["local"]
    near[:, :c["sink"]] = True
    masks = []
    for b in range(B):
        for h in range(H):
            a, _ = _whole7(st["q"][b, h].double().unflatten(0, (nb, 128)).sum(1) / 128)
            w, e = _whole7(st["k"][b, h // (H // c["Hkv"])].double().unflatten(0, (nk, kb)).sum(1) / kb)
            s = torch.einsum("id,jd->ij", a, w) * torch.exp2(e).T
            ok = torch.ones(nb, nk, dtype=torch.bool, device=DEV)
            if c["causal"]:
                ok &= j <= i
            if st["allow"] is not None:
                ok &= st["allow"][b, h] != 0
            s[near] = 1e200
            s[~ok] = -1e200
            rank = torch.empty_like(s, dtype=torch.int64)
            rank.scatter_(1, torch.argsort(-s, dim=1, stable=True), torch.arange(nk, device=DEV).expand(nb, -1).contiguous())
            most = (near & ok).sum(1, keepdim=True).clamp(min=c["keep"])
            masks.append((rank < most) & ok)
    return torch.stack(masks).view(B, H, nb, nk).to(torch.uint8)


def _exact_append(st):
    c = st["case"]
    B, Hkv, T, D = st["k"].shape
    page, g = c["page"], c["group"]
    behind = (torch.arange(T, device=DEV)[None] >= st["counts"][:, None])[:, None, :, None]
    new = []
    for n in "kv":
        x = st[n].double().view(B, Hkv, T, D // g, g)
        lo, hi = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
        step = ((hi - lo).float() / 15).to(torch.bfloat16).double()
        y = lo + step * torch.where(step > 0, torch.round((x - lo) / step.clamp(min=1e-300)), 0.0).clamp(0, 15)
        new.append(y.view(B, Hkv, T, D).masked_fill(behind, 0.0))
    means = st["k_means"].double()
    for b, (n0, count) in enumerate(zip(st["host_lengths"], st["counts"].tolist())):
        for p in range(n0 // page, (n0 + count) // page):  # the pages that this call fills
            at = int(st["table"][b, p])
            tokens = _decoded(st, "k", at, slice(None))
            pos = p * page + torch.arange(page, device=DEV)
            tokens[:, pos >= n0] = new[0][b][:, pos[pos >= n0] - n0]
            whole, e = _whole7(tokens.sum(1) / page)
            means[at] = whole * torch.exp2(e)
    return new[0], new[1], means


def _decoded(st, n, pages, head):
    b = st[n + "_codes"][pages, head]
    x = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = (b % 16).double(), torch.div(b, 16, rounding_mode="floor").double()
    sc = st[n + "_scales"][pages, head].double().repeat_interleave(st["case"]["group"], -2)
    return x * sc[..., 0] + sc[..., 1]


def _exact_attn(st, chosen=None):
    c = st["case"]
    B, H, T, D = st["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    out = torch.zeros(B, H, T, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, T), -torch.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = st["host_lengths"][b]
        for h in range(Hkv):
            lp = torch.arange(-(-n // page), device=DEV)
            if chosen is not None:
                lp = chosen[b, h][chosen[b, h] >= 0].long()
            k, v = (_decoded(st, m, st["table"][b, lp].long(), h).reshape(-1, D) for m in "kv")
            pos = (lp[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)
            for t in range(T):
                see = pos <= n - T + t
                rows = slice(h * H // Hkv, (h + 1) * H // Hkv)
                if not bool(see.any()):
                    continue
                s = st["q"][b, rows, t].double() @ k[see].T / math.sqrt(D)
                lse[b, rows, t] = torch.logsumexp(s, -1)
                out[b, rows, t] = torch.softmax(s, -1) @ v[see]
    return out, lse


def _exact_sparse(st):
    c = st["case"]
    B, H, T, D = st["q"].shape
    Hkv = c["Hkv"]
    chosen = torch.full((B, Hkv, c["keep"]), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        n = -(-st["host_lengths"][b] // c["page"])
        for h in range(Hkv):
            a, _ = _whole7(st["q"][b, h * H // Hkv:(h + 1) * H // Hkv].double().reshape(1, -1))
            s = torch.einsum("rd,pd->rp", a.view(-1, D), st["k_means"][st["table"][b, :n].long(), h].double())
            s = s.max(0)[0]
            s[:c["sink"]] = 1e200
            s[max(0, n - c["recent"]):] = 1e200
            take = torch.argsort(-s, stable=True)[:c["keep"]].sort()[0]
            chosen[b, h, :take.numel()] = take.to(torch.int32)
    return (chosen,) + _exact_attn(st, chosen)


_EXACT = dict(rope=_exact_rope, rope_grad=_exact_rope_grad, select=_exact_select, append=_exact_append,
              attn=_exact_attn, sparse=_exact_sparse)
