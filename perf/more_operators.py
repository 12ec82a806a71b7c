"""Workloads of serving over the paged 4-bit cache, for measuring.

Five kinds of pass, each in two forms on the same inputs: the plain form
(elementary torch operations in 32 bits, 64 where 32 lose what matters) and,
with ``own = True``, the calls that a user makes of this package.

    chunk    attention of a chunk of new tokens over the cache
    scored   the same with capped scores, a bias that depends on distance, or both
    fork     sequences copied, reordered and ended, then pages for their new tokens
    compact  the pages in use moved to the lowest places
    copy     pages copied from one cache to another
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the first chunks of eight ragged prompts, nothing cached before them
        dict(name="chunk-prompts", op="chunk", B=8, T=2048, H=32, Hkv=8, D=128, page=64, group=128,
             longest=2048, prefix=False),
        # one chunk of a very long prompt
        dict(name="chunk-long", op="chunk", B=1, T=4096, H=32, Hkv=8, D=128, page=128, group=32,
             longest=65536, prefix=False),
        # a few new tokens a sequence, small pages, three query heads a key/value head; the first
        # part of each sequence is seen by all of its tokens
        dict(name="chunk-odd", op="chunk", B=3, T=37, H=6, Hkv=2, D=64, page=16, group=32,
             longest=1000, prefix=True),
        # one decoding step of 64 sequences, scores capped
        dict(name="scored-step", op="scored", B=64, T=1, H=32, Hkv=8, D=128, page=64, group=128,
             longest=8192, prefix=False, cap=50.0, slopes=False),
        # drafted tokens checked together over long contexts, a bias by distance
        dict(name="scored-draft", op="scored", B=5, T=5, H=16, Hkv=2, D=64, page=32, group=64,
             longest=30000, prefix=False, cap=0.0, slopes=True),
        # a chunk of two prompts with both
        dict(name="scored-prompt", op="scored", B=2, T=1999, H=16, Hkv=4, D=128, page=64, group=64,
             longest=12345, prefix=True, cap=30.0, slopes=True),
        # a step of a beam search: latency counts
        dict(name="fork-step", op="fork", requests=4, beams=4, Hkv=2, D=64, page=16, group=64,
             longest=700, T=1),
        # many requests whose samples begin to differ behind their prompts
        dict(name="fork-many", op="fork", requests=64, beams=8, Hkv=8, D=128, page=128, group=128,
             longest=8000, T=3),
        # a small cache after some of its sequences have ended
        dict(name="compact-small", op="compact", pages=500, B=7, Hkv=2, D=64, page=16, group=32),
        # a large one, half of its pages free
        dict(name="compact-large", op="compact", pages=16384, B=64, Hkv=8, D=128, page=64, group=128),
        # a few pages of one sequence
        dict(name="copy-few", op="copy", pages=100, n=11, Hkv=4, D=64, page=32, group=64),
        # sequences handed over to another cache
        dict(name="copy-many", op="copy", pages=20000, n=12000, Hkv=8, D=128, page=64, group=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "scored", "fork", "compact", "copy"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    case = dict(op=op, Hkv=Hkv, D=D, page=page, group=rng.choice([g for g in (32, 64, 128) if g <= D]))
    if op in ("chunk", "scored"):
        B = _log(rng, 1, 64)
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
        pairs = (1 << 31) // (B * H)  # of a query and a key, at most, a sequence and head
        T = 1 if op == "scored" and rng.random() < 0.4 else _log(rng, 1, int(min(16384 // B, pairs ** 0.5)))
        most = min(65536, pairs // T, (1 << 24) // (B * Hkv))
        case.update(B=B, T=T, H=H, longest=_log(rng, T, max(T, most)), prefix=rng.random() < 0.3)
        if op == "scored":
            kind = rng.choice([1, 2, 3])
            case.update(cap=rng.choice([20.0, 30.0, 50.0]) if kind & 1 else 0.0, slopes=kind >= 2)
        return case
    if op == "fork":
        requests, beams = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 8])
        longest = _log(rng, 1, min(16384, (1 << 23) // (requests * beams * Hkv)))
        case.update(requests=requests, beams=beams, longest=longest, T=_log(rng, 1, 200))
        return case
    room = max(8, min(16384, (1 << 23) // (page * Hkv)))
    pages = _log(rng, 7, room)
    if op == "compact":
        case.update(pages=pages, B=_log(rng, 1, max(1, min(64, pages // 4))))
    else:
        case.update(pages=pages, n=_log(rng, 1, pages))
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


def _quantise(x, group):
    """4-bit codes [..., D / 2] and (step, minimum) [..., D / group, 2] of x [..., D]."""
    xg = x.float().unflatten(-1, (x.shape[-1] // group, group))
    least = xg.amin(-1, keepdim=True)
    step = ((xg.amax(-1, keepdim=True) - least) / 15).bfloat16().float()
    code = ((xg - least) / torch.where(step > 0, step, torch.inf)).round_().clamp_(0, 15)
    code = code.reshape(x.shape).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([step, least], -1).bfloat16()


BUFFERS = ("k_codes", "v_codes", "k_scales", "v_scales", "k_means")


def _empty_cache(case, pages):
    """The cache's tensors (with the package: its cache, a user's program keeps it)."""
    Hkv, D, page, group = case["Hkv"], case["D"], case["page"], case["group"]
    if own:
        import block_sparse_flash_attn_gb300 as bs
        cache = bs.Kv4Cache(pages, Hkv, D, page_size=page, group=group)
        return dict({n: getattr(cache, n) for n in BUFFERS}, handle=cache)
    t = {}
    for n in "kv":
        t[n + "_codes"] = torch.zeros(pages, Hkv, page, D // 2, dtype=torch.uint8, device=DEV)
        t[n + "_scales"] = torch.zeros(pages, Hkv, page, D // group, 2, dtype=torch.bfloat16, device=DEV)
    t["k_means"] = torch.zeros(pages, Hkv, D, dtype=torch.bfloat16, device=DEV)
    return t


def _cache(case, g, pages):
    """A cache filled with keys and values, every page of it."""
    t = _empty_cache(case, pages)
    Hkv, D, page, group = case["Hkv"], case["D"], case["page"], case["group"]
    part = max(1, (1 << 26) // (Hkv * page * D))
    for p in range(0, pages, part):
        n = min(part, pages - p)
        k = _heads_spread(g, n, Hkv, page, D)
        t["k_means"][p:p + n] = k.mean(2).bfloat16()
        for name, x in (("k", k), ("v", _randn(g, n, Hkv, page, D))):
            t[name + "_codes"][p:p + n], t[name + "_scales"][p:p + n] = _quantise(x.bfloat16(), group)
    return t


def _table(g, need, columns, spare):
    """Scattered pages for sequences that need so many: (table [B, columns], pages in all)."""
    order = torch.randperm(int(need.sum()) + spare, generator=g, device=DEV).to(torch.int32)
    there = torch.arange(columns, device=DEV)[None] < need[:, None]
    at = (there.flatten().cumsum(0) - 1).clamp(min=0).view(there.shape)
    return torch.where(there, order[at], -1), order.numel()


def prepare(case, seed):
    g = _gen(seed)
    op, page = case["op"], case["page"]
    if op in ("chunk", "scored"):
        B, T, H, D = (case[n] for n in ("B", "T", "H", "D"))
        counts = _randint(g, (T + 1) // 2, T + 1, (B,)).to(torch.int32)
        counts[0] = T
        before = _randint(g, (case["longest"] - T) // 2, case["longest"] - T + 1, (B,)).to(torch.int32)
        before[0] = case["longest"] - T
        lengths = before + counts
        table, pages = _table(g, (lengths + page - 1) // page, -(-case["longest"] // page), 3)
        st = _cache(case, g, pages)
        st.update(q=_randn(g, B, H, T, D).bfloat16(), lengths=lengths, counts=counts, table=table,
                  prefix=None, cap=case.get("cap") or None, slopes=None)
        if case["prefix"]:  # the first part of the prompt, now and then more than what was cached before
            st["prefix"] = (lengths * torch.rand(B, generator=g, device=DEV)).to(torch.int32)
        if case.get("slopes"):
            st["slopes"] = 0.5 ** (8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)
    elif op == "fork":
        R, W = case["requests"], case["beams"]
        # a request's beams share the full pages of its prompt; behind it each has its own
        n = _randint(g, (case["longest"] + 1) // 2, case["longest"] + 1, (R, 1)).expand(R, W)
        shared = (n[:, :1] * (0.8 + 0.2 * torch.rand(R, 1, generator=g, device=DEV))).long() // page
        columns = -(-(case["longest"] + case["T"]) // page)
        need = (n + page - 1) // page
        mine = torch.where(torch.arange(W, device=DEV)[None] == 0, need, need - shared)
        full = -(-case["longest"] // page)  # a cache with room for any such requests
        pages = R * (full + (W - 1) * (full // 5 + 2)) + 2 * R * W * (2 + case["T"] // page)
        places, pages = _table(g, mine.flatten(), columns, pages - int(mine.sum()))
        places = places.view(R, W, columns)
        column = torch.arange(columns, device=DEV)
        first = places[:, :1].expand(R, W, columns)
        rest = places.gather(2, (column - shared[:, :, None]).clamp(min=0).expand(R, W, columns))
        own_rows = torch.where(column < need[:, :, None], rest, -1)
        table = torch.where(column < shared[:, :, None], first, own_rows)
        table[:, 0] = places[:, 0]
        table = table.reshape(R * W, columns).contiguous()
        refs = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
        refs.index_add_(0, torch.where(table >= 0, table, pages).flatten().long(),
                        torch.ones(table.numel(), dtype=torch.int32, device=DEV))
        parents = torch.arange(R, device=DEV)[:, None] * W + _randint(g, 0, W, (R, W))
        parents = torch.where(torch.rand(R, W, generator=g, device=DEV) < 0.05, -1, parents)  # some end
        st = _cache(case, g, pages)
        st.update(table=table, refs=refs[:pages].contiguous(), lengths=n.flatten().to(torch.int32).contiguous(),
                  parents=parents.flatten().to(torch.int32).contiguous())
        st["counts"] = torch.where(st["parents"] >= 0, _randint(g, 0, case["T"] + 1, (R * W,)), 0).to(torch.int32)
        # where each row's last page begins, and the tokens there
        left = torch.where(st["parents"] >= 0, st["lengths"][st["parents"].clamp(min=0).long()], 0)
        st["start"] = ((left - 1).clamp(min=0) // page * page).to(torch.int32)
        st["tail"] = (left - st["start"]).to(torch.int32)
    elif op == "compact":
        B, pages = case["B"], case["pages"]
        half = max(1, pages // 2 // B)
        need = _randint(g, max(1, half // 2), half + 1, (B,))
        table, n = _table(g, need, half, pages - int(need.sum()))
        refs = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        refs.index_add_(0, torch.where(table >= 0, table, n).flatten().long(),
                        torch.ones(table.numel(), dtype=torch.int32, device=DEV))
        st = _cache(case, g, n)
        st.update(table=table, refs=refs[:n].contiguous())
    else:
        n, pages = case["n"], case["pages"]
        st = _cache(case, g, pages)
        st["to"] = _empty_cache(case, pages)
        st["src"] = torch.randperm(pages, generator=g, device=DEV)[:n].to(torch.int32)
        st["dst"] = torch.randperm(pages, generator=g, device=DEV)[:n].to(torch.int32)
    st["case"] = case
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    return (_run_own if own else _PLAIN[op])(st)


def _run_own(st):
    import block_sparse_flash_attn_gb300 as bs
    op, cache = st["case"]["op"], st["handle"]
    if op == "chunk":
        return bs.kv4_attn_chunk(cache, st["q"], st["table"], st["lengths"], st["counts"], prefix=st["prefix"])
    if op == "scored":
        return bs.kv4_attn_chunk(cache, st["q"], st["table"], st["lengths"], st["counts"], prefix=st["prefix"],
                                 cap=st["cap"], slopes=st["slopes"])
    if op == "fork":
        table, lengths, refs = bs.kv4_fork(cache, st["refs"], st["table"], st["lengths"], st["parents"])
        table, refs = bs.kv4_reserve(cache, refs, table, lengths, st["counts"])
        k, v = bs.kv4_read(cache, table, st["start"], st["case"]["page"], st["tail"])
        return table, lengths, refs, k, v
    if op == "compact":
        table, refs, moved = bs.kv4_compact(cache, st["refs"], st["table"])
        return (table, refs, moved) + tuple(st[n] for n in BUFFERS)
    bs.kv4_copy(cache, st["src"], st["dst"], to=st["to"]["handle"])
    return tuple(st["to"][n] for n in BUFFERS)


def _values(packed, scales):
    """What the cache stands for, 32 bits: step * code + minimum."""
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float()
    s = scales.float()
    code = code.unflatten(-1, (s.shape[-2], code.shape[-1] // s.shape[-2]))
    return (code * s[..., 0:1] + s[..., 1:2]).flatten(-2)


def _tokens(st, n, table, columns):
    """[B, Hkv, columns * page, D] in 32 bits of the sequences' first pages."""
    p = table[:, :columns].clamp(min=0).long()
    return _values(st[n + "_codes"][p], st[n + "_scales"][p]).transpose(1, 2).flatten(2, 3)


def _plain_chunk(st):
    c = st["case"]
    q, lengths, counts = st["q"], st["lengths"].long(), st["counts"].long()
    B, H, T, D = q.shape
    columns = st["table"].shape[1]
    k, v = _tokens(st, "k", st["table"], columns), _tokens(st, "v", st["table"], columns)
    n = k.shape[2]
    t = torch.arange(T, device=DEV)
    at = (lengths - counts)[:, None] + t                      # a query's position
    last = at if st["prefix"] is None else torch.maximum(at, st["prefix"].long()[:, None] - 1)
    last = torch.where(t < counts[:, None], torch.minimum(last, lengths[:, None] - 1), -1)
    pos = torch.arange(n, device=DEV)
    hidden = pos > last[:, :, None]                           # [B, T, n]
    # a key/value head's query heads and tokens as the rows of one product
    s = (q.float() * D ** -0.5).reshape(B, c["Hkv"], -1, D) @ k.transpose(2, 3)
    s = s.view(B, H, T, n)
    if st["cap"]:
        s = s.div_(st["cap"]).tanh_().mul_(st["cap"])
    if st["slopes"] is not None:
        far = (pos - at[:, :, None]).abs().float()
        s = s.addcmul_(st["slopes"][:, None, None], far[:, None], value=-1.0)
    s.masked_fill_(hidden[:, None], -torch.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    e = s.sub_(m).exp_()
    z = e.sum(-1, keepdim=True)
    o = (e.view(B, c["Hkv"], -1, n) @ v).view(B, H, T, D) / torch.where(z > 0, z, 1.0)
    return o.to(q.dtype), (m + torch.log(z)).squeeze(-1)


def _free_after(refs, n):
    """The n-th free page for every n (the lowest first), -1 where there are no more."""
    free = torch.nonzero(refs == 0).flatten()
    return torch.where(n < free.numel(), free[n.clamp(max=free.numel() - 1)], -1).to(torch.int32)


def _count(refs, table, sign):
    there = table >= 0
    at = torch.where(there, table, 0).flatten().long()
    return refs.index_add(0, at, there.flatten().to(torch.int32) * sign)


def _plain_fork(st):
    c, parents, page = st["case"], st["parents"].long(), st["case"]["page"]
    rows = parents.clamp(min=0)
    lengths = torch.where(parents >= 0, st["lengths"][rows], 0)
    column = torch.arange(st["table"].shape[1], device=DEV)
    there = (parents >= 0)[:, None] & (column < ((lengths + page - 1) // page)[:, None])
    old = torch.where(column < ((st["lengths"] + page - 1) // page)[:, None], st["table"], -1)
    table = torch.where(there, st["table"][rows], -1)
    refs = _count(_count(st["refs"], old, -1), table, 1)
    # a page that is not full goes to its first child; the others get copies
    first = torch.full_like(parents, parents.numel())
    index = torch.arange(parents.numel(), device=DEV)
    first = first.scatter_reduce(0, rows, torch.where(parents >= 0, index, parents.numel()), "amin")
    copies = torch.nonzero((parents >= 0) & (lengths % page != 0) & (first[rows] != index)).flatten()
    last = (lengths // page)[copies].long()
    src = table[copies, last].long()
    dst = _free_after(refs, torch.arange(copies.numel(), device=DEV))
    got = dst >= 0
    refs = refs.index_add(0, src, torch.full_like(dst, -1))
    refs = refs.index_add(0, dst.clamp(min=0).long(), got.to(torch.int32))
    table[copies, last] = dst
    src, dst = src[got], dst[got].long()
    token = torch.arange(page, device=DEV)[None, None, :, None] < (lengths[copies] % page)[got][:, None, None, None]
    for n in "kv":
        codes, scales = st[n + "_codes"], st[n + "_scales"]
        codes[dst] = torch.where(token, codes[src], codes[dst])
        scales[dst] = torch.where(token[..., None], scales[src], scales[dst])
    # pages for the new tokens
    have, want = (lengths + page - 1) // page, (lengths + st["counts"] + page - 1) // page
    new = (column >= have[:, None]) & (column < want[:, None])
    place = (new.flatten().cumsum(0) - 1).view(new.shape)
    got = _free_after(refs, place.clamp(min=0))
    table = torch.where(new, got, table)
    refs = _count(refs, torch.where(new, got, -1), 1)
    # the tokens of every row's last page
    p = table[torch.arange(rows.numel(), device=DEV), st["start"].long() // page].clamp(min=0).long()
    token = torch.arange(page, device=DEV)[None, None, :, None] < st["tail"][:, None, None, None]
    k, v = (torch.where(token, _values(st[n + "_codes"][p], st[n + "_scales"][p]), 0.0).bfloat16() for n in "kv")
    return table, lengths, refs, k, v


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    used = refs > 0
    n = used.sum()
    index = torch.arange(refs.numel(), device=DEV)
    src = torch.nonzero(used & (index >= n)).flatten()
    dst = torch.nonzero(~used & (index < n)).flatten()
    moved = torch.where(used, index, -1).to(torch.int32)
    moved[src] = dst.to(torch.int32)
    refs = refs.clone()
    refs[dst] = refs[src]
    refs[src] = 0
    for name in BUFFERS:
        st[name][dst] = st[name][src]
    return (torch.where(table >= 0, moved[table.clamp(min=0).long()], table), refs, moved) + tuple(st[n] for n in BUFFERS)


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for name in BUFFERS:
        st["to"][name][dst] = st[name][src]
    return tuple(st["to"][n] for n in BUFFERS)


_PLAIN = dict(chunk=_plain_chunk, scored=_plain_chunk, fork=_plain_fork, compact=_plain_compact, copy=_plain_copy)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    D, page, Hkv = case["D"], case["page"], case["Hkv"]
    row = D // 2 + 4 * (D // case["group"])  # a token's keys or values in one head
    op = case["op"]
    if op in ("chunk", "scored"):
        B, T, H, before = case["B"], case["T"], case["H"], case["longest"] - case["T"]
        # new tokens: three quarters of T, behind three quarters of what may be cached, but for the first
        new, old = B * 0.75 * T + 0.25 * T, B * 0.75 * before + 0.25 * before
        seen = (0.75 * (B - 1) * T * (0.75 * before + 0.375 * T) if B > 1 else 0.0) + T * (before + 0.5 * T)
        return dict(bytes=int((new + old) * Hkv * 2 * row + new * H * 4 * D + B * T * H * (2 * D + 4)),
                    flops=int(seen * H * 4 * D))
    if op == "fork":
        rows = case["requests"] * case["beams"]
        columns = -(-(case["longest"] + case["T"]) // page)
        copied = rows * (1 - 1 / case["beams"]) * 0.5 * page * Hkv * 2 * row
        read = rows * 0.5 * page * Hkv * 2 * row + rows * page * Hkv * 2 * 2 * D
        return dict(bytes=int(rows * columns * 12 + 2 * copied + read), flops=int(rows * page * Hkv * 4 * D))
    whole = Hkv * (2 * page * row + 2 * D)
    if op == "compact":
        pages = case["pages"]
        used = 0.375 * pages
        return dict(bytes=int(2 * used * (1 - used / pages) * whole + 12 * pages + 8 * 0.5 * pages), flops=pages)
    return dict(bytes=int(2 * case["n"] * whole), flops=case["n"])


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """What run returns for these inputs, from the definitions, in 64 bits."""
    st = prepare(case, seed)
    return _EXACT[case["op"]](st)


def _decoded(st, n, pages, head):
    """[tokens, D] of the listed pages' tokens in one head, in 64 bits."""
    b = st[n + "_codes"][pages, head]
    x = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = (b & 15).double(), (b >> 4).double()
    s = st[n + "_scales"][pages, head].double().repeat_interleave(st["case"]["group"], -2)
    return (x * s[..., 0] + s[..., 1]).reshape(-1, x.shape[-1])


def _exact_chunk(st):
    c = st["case"]
    B, H, T, D = st["q"].shape
    G = H // c["Hkv"]
    out = torch.zeros(B, H, T, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, T), -torch.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n, m = int(st["lengths"][b]), int(st["counts"][b])
        pages = st["table"][b, :-(-n // c["page"])].long()
        j = torch.arange(n, device=DEV)
        i = n - m + torch.arange(m, device=DEV)
        see = j[None] <= i[:, None]
        if st["prefix"] is not None:
            see |= j[None] < int(st["prefix"][b])
        for h in range(H):
            if h % G == 0:
                k, v = (_decoded(st, x, pages, h // G)[:n] for x in "kv")
            for t in range(0, m, 1024):
                rows = slice(t, min(t + 1024, m))
                x = torch.einsum("td,jd->tj", st["q"][b, h, rows].double(), k) / math.sqrt(D)
                if st["cap"]:
                    x = st["cap"] * torch.tanh(x / st["cap"])
                if st["slopes"] is not None:
                    x = x - st["slopes"][h].double() * (i[rows, None] - j[None]).abs()
                x[~see[rows]] = -torch.inf
                lse[b, h, rows] = torch.logsumexp(x, -1)
                out[b, h, rows] = torch.einsum("tj,jd->td", torch.softmax(x, -1), v)
    return out, lse


def _exact_fork(st):
    c, page = st["case"], st["case"]["page"]
    old, length, parents, counts = (st[n].tolist() for n in ("table", "lengths", "parents", "counts"))
    refs = st["refs"].tolist()
    for row, n in zip(old, length):
        for p in row[:-(-n // page)]:
            refs[p] -= 1
    table, lengths = [], []
    for a in parents:
        n = length[a] if a >= 0 else 0
        pages = old[a][:-(-n // page)] if a >= 0 else []
        for p in pages:
            refs[p] += 1
        table.append(pages + [-1] * (len(old[0]) - len(pages)))
        lengths.append(n)
    free = [p for p, r in enumerate(refs) if r == 0]
    kept, held = set(), list(free)
    holds = [list(row) for row in table]  # which page of the old cache each entry's tokens came from
    for row, a, n in zip(table, parents, lengths):
        if a >= 0 and n % page:
            if a in kept:
                refs[row[n // page]] -= 1
                row[n // page] = held.pop(0) if held else -1
                if row[n // page] >= 0:
                    refs[row[n // page]] += 1
            kept.add(a)
    free = [p for p, r in enumerate(refs) if r == 0]
    for row, n, m in zip(table, lengths, counts):
        for at in range(-(-n // page), -(-(n + m) // page)):
            row[at] = free.pop(0) if free else -1
            if row[at] >= 0:
                refs[row[at]] += 1
    values = []
    for name in "kv":
        x = torch.zeros(len(table), c["Hkv"], page, c["D"], dtype=torch.float64, device=DEV)
        for i, (row, start, m) in enumerate(zip(holds, st["start"].tolist(), st["tail"].tolist())):
            for h in range(c["Hkv"] if m > 0 else 0):
                x[i, h, :m] = _decoded(st, name, row[start // page], h)[:m]
        values.append(x)

    def whole(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    return whole(table), whole(lengths), whole(refs), values[0], values[1]


def _exact_compact(st):
    refs = st["refs"].tolist()
    used = [p for p, r in enumerate(refs) if r > 0]
    to = {p: p for p in used if p < len(used)}
    to.update(zip([p for p in used if p >= len(used)], [p for p in range(len(used)) if refs[p] == 0]))
    moved = [to.get(p, -1) for p in range(len(refs))]
    after = [0] * len(refs)
    for p, q in to.items():
        after[q] = refs[p]
    table = [[moved[p] if p >= 0 else p for p in row] for row in st["table"].tolist()]
    order = list(range(len(refs)))
    for p, q in to.items():
        order[q] = p
    order = torch.tensor(order, device=DEV)

    def whole(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    # (scales and means in 64 bits, as all numbers; codes as they are)
    moves = tuple(st[n][order] if st[n].dtype == torch.uint8 else st[n][order].double() for n in BUFFERS)
    return (whole(table), whole(after), whole(moved)) + moves


def _exact_copy(st):
    out = []
    for n in BUFFERS:
        x = torch.zeros_like(st["to"][n])
        x.index_copy_(0, st["dst"].long(), st[n].index_select(0, st["src"].long()))
        out.append(x if x.dtype == torch.uint8 else x.double())
    return tuple(out)


_EXACT = dict(chunk=_exact_chunk, scored=_exact_chunk, fork=_exact_fork, compact=_exact_compact, copy=_exact_copy)
