"""The 4-bit cache: appended codes, scales and page means equal to the 64-bit
restatement; reading back, choosing pages and attention against it.

Tolerances: reading back is one 32-bit and one bf16 rounding.  Attention: the
bounds that _ops_ref.attn derives from 32-bit sums, plus the output's rounding."""
import pytest
import torch

import _ops_ref as ref
from _ops_ref import U32, UBF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_flash_attn_gb300 as bs
    bs.load()
    return bs


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(cache):
    return [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, cache.k_means)]


def _append_ref(cache, state, k, v, table, lengths, counts):
    """What the cache's tensors must hold after the call."""
    kc, vc, ks, vs, km = [t.clone() for t in state]
    page = cache.page_size
    full = []
    for b, (n, c) in enumerate(zip(lengths, counts)):
        for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
            code, sc = ref.quantise(x[b, :, :c], cache.group)
            pos = torch.arange(n, n + c, device="cuda")
            pg, place = table[b, pos // page].long(), pos % page
            codes[pg, :, place] = ref.pack(code).transpose(0, 1)
            scales[pg, :, place] = sc.transpose(0, 1).bfloat16()
        full += [int(table[b, p]) for p in range(n // page, (n + c) // page)]
    if full:
        val = ref.values(kc[full], ks[full]).float().double()
        t, e = ref.round7(val.mean(-2))
        km[full] = (t * torch.exp2(e)).bfloat16()
    return [kc, vc, ks, vs, km]


#        Hkv D    page group T    lengths            counts
APPENDS = [
    (2, 64, 16, 32, 1, [0, 15, 16, 100], None),
    (2, 64, 16, 64, 40, [0, 7, 33], [40, 0, 13]),
    (1, 128, 64, 128, 1, [63, 64, 0], [1, 1, 0]),
    (3, 128, 32, 32, 70, [5, 0], [70, 69]),
    (8, 128, 128, 64, 129, [0, 127], None),
    (1, 64, 256, 64, 600, [1, 255], [600, 513]),
]


@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append_and_read(bs, case):
    Hkv, D, page, group, T, lengths, counts = case
    B = len(lengths)
    done = counts or [T] * B
    ends = [n + c for n, c in zip(lengths, done)]
    columns = max(-(-e // page) for e in ends) + 1
    cache = bs.Kv4Cache(sum(-(-e // page) for e in ends) + 2, Hkv, D, page_size=page, group=group)
    ref.fill(cache, 11)
    table = ref.table(cache, ends, columns, 5)
    g = ref.gen(6)
    k, v = ((torch.randn(B, Hkv, T, D, generator=g, device="cuda") * (1 + i)).bfloat16() for i in range(2))
    before = _state(cache)
    n, c = _i32(lengths), None if counts is None else _i32(counts)
    bs.kv4_append(cache, k, v, table, n, c)
    bs.kv4_status(cache)
    for got, want in zip(_state(cache), _append_ref(cache, before, k, v, table, lengths, done)):
        assert torch.equal(got, want)
    # read back what was written, and what was there before
    rk, rv = bs.kv4_read(cache, table, n, T, c)
    start = [max(x - 20, 0) for x in lengths]
    back = max(e - s for e, s in zip(ends, start))
    rk2, rv2 = bs.kv4_read(cache, table, _i32(start), back, _i32([e - s for e, s in zip(ends, start)]))
    bs.kv4_status(cache)
    for first, width, pairs in ((lengths, T, ((rk, "k"), (rv, "v"))), (start, back, ((rk2, "k"), (rv2, "v")))):
        for got, m in pairs:
            assert got.shape == (B, Hkv, width, D)
            for b in range(B):
                pos = torch.arange(first[b], ends[b], device="cuda")
                pg, place = table[b, pos // page].long(), pos % page
                codes = getattr(cache, m + "_codes")[pg, :, place].transpose(0, 1)
                sc = getattr(cache, m + "_scales")[pg, :, place].transpose(0, 1)
                want = ref.values(codes, sc)
                size = want.abs() + 2 * sc[..., 1].double().abs().repeat_interleave(group, -1)
                err = (got[b, :, :pos.numel()].double() - want).abs()
                assert bool((err <= UBF * want.abs() + 2 * U32 * size).all())
                assert not bool(got[b, :, pos.numel():].any())


def test_append_token_by_token_equals_a_prompt(bs):
    """The same tokens one at a time, in pieces and at once: the same cache, means included."""
    Hkv, D, T, page = 2, 128, 75, 16
    g = ref.gen(3)
    k, v = (torch.randn(2, Hkv, T, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    caches = []
    for pieces in ([1] * T, [T], [13, 3, 16, 43]):
        cache = bs.Kv4Cache(12, Hkv, D, page_size=page, group=32)
        table = ref.table(cache, [T, T], 5, 2)
        at = 0
        for n in pieces:  # (slices of k, v: strided)
            bs.kv4_append(cache, k[:, :, at:at + n], v[:, :, at:at + n], table, _i32([at, at]))
            at += n
        caches.append(_state(cache))
    for other in caches[1:]:
        assert all(torch.equal(a, b) for a, b in zip(caches[0], other))


def test_append_extreme_values(bs):
    """Constant groups, steps on borders, tiny and huge ranges, NaN and infinities."""
    D, page = 64, 16
    k = torch.randn(1, 1, 16, D, generator=ref.gen(1), device="cuda").bfloat16()
    k[0, 0, 0] = 0
    k[0, 0, 1] = -3.25
    k[0, 0, 2] = (torch.arange(D, device="cuda") % 31).bfloat16() / 2    # halves of a step
    k[0, 0, 3] *= 1e-38
    k[0, 0, 4] *= 1e37
    k[0, 0, 5, 7] = float("nan")
    k[0, 0, 6, 40] = float("inf")
    k[0, 0, 7, 3] = float("-inf")
    k[0, 0, 8, 0], k[0, 0, 8, 1] = 3e38, -3e38
    k[0, 0, 9] = torch.tensor([1.0] * 63 + [1.0078125])
    k[0, 0, 10, ::2] = 0.0
    k[0, 0, 10, 1::2] = -0.0
    for group in (32, 64):
        cache = bs.Kv4Cache(2, 1, D, page_size=page, group=group)
        table = _i32([[1]])
        bs.kv4_append(cache, k, k, table, _i32([0]))
        code, scales = ref.quantise(k[0, 0], group)
        for m in "kv":
            assert torch.equal(getattr(cache, m + "_codes")[1, 0], ref.pack(code))
            got = getattr(cache, m + "_scales")[1, 0].double()
            want = scales.bfloat16().double()
            assert torch.equal(got.nan_to_num(1e5), want.nan_to_num(1e5))
        rk, _ = bs.kv4_read(cache, table, _i32([0]), 16)
        assert bool(rk[0, 0, 5, :32].isnan().all()) and not bool(rk[0, 0, 0].any())
        if group == 32:
            assert not bool(rk[0, 0, 5, 32:].isnan().any())


#         Hkv G  D    page group T  lengths
ATTNS = [
    (1, 1, 64, 16, 64, 1, [1]),
    (2, 4, 128, 64, 128, 1, [0, 1, 63, 64, 65, 700]),
    (2, 8, 64, 16, 32, 1, [777, 16, 300]),
    (1, 5, 128, 32, 64, 3, [2, 3, 40, 555]),
    (4, 1, 128, 128, 32, 1, [1000, 129]),
    (2, 16, 128, 64, 128, 1, [333, 128]),
    (1, 8, 64, 256, 64, 5, [1500, 4, 0]),
    (8, 4, 128, 64, 128, 1, [5000]),
    (1, 40, 64, 16, 32, 3, [200, 31]),
    (1, 3, 128, 16, 128, 1, [900] + list(range(60))),
]


def _attn_case(bs, case, seed=21):
    Hkv, G, D, page, group, T, lengths = case
    B = len(lengths)
    columns = max(1, max(-(-n // page) for n in lengths))
    cache = bs.Kv4Cache(sum(-(-n // page) for n in lengths) + 2, Hkv, D, page_size=page, group=group)
    ref.fill(cache, seed)
    table = ref.table(cache, lengths, columns, seed + 1)
    q = (torch.randn(B, Hkv * G, T, D, generator=ref.gen(seed + 2), device="cuda") * 1.5).bfloat16()
    return cache, table, q, _i32(lengths)


def _check_attn(o, lse, want, out_f32):
    o_ref, l_ref, tol_o, tol_l = want
    assert torch.equal(lse.isneginf(), l_ref.isneginf())
    dead = l_ref.isneginf()
    assert not bool(o[dead].any())
    err = (lse.double() - l_ref).abs()[~dead]
    # the LSE's own rounding to 32 bits and log2's 2 ulp: 4 U32 of its size
    assert bool((err <= tol_l[~dead] + 4 * U32 * (1 + l_ref[~dead].abs())).all()), float(err.max())
    tol = tol_o[..., None] + (U32 if out_f32 else UBF) * o_ref.abs()
    err = (o.double() - o_ref).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / (tol + 1e-300)).max()))


@pytest.mark.parametrize("out_f32", [True, False], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", ATTNS, ids=str)
def test_attn(bs, case, out_f32):
    cache, table, q, n = _attn_case(bs, case)
    o, lse = bs.kv4_attn(cache, q, table, n, out_f32=out_f32)
    bs.kv4_status(cache)
    _check_attn(o, lse, ref.attn(cache, q, table, case[-1]), out_f32)
    again = bs.kv4_attn(cache, q, table, n, out_f32=out_f32)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attn_scale(bs, scale):
    case = (2, 4, 64, 16, 32, 1, [150, 31])
    cache, table, q, n = _attn_case(bs, case)
    o, lse = bs.kv4_attn(cache, q, table, n, scale=scale, out_f32=True)
    _check_attn(o, lse, ref.attn(cache, q, table, case[-1], scale=scale), True)


def test_attn_wide_steps(bs):
    """Values of one head far larger than another token's, steps from 2^-40 to 2^20."""
    case = (1, 4, 128, 16, 32, 1, [300])
    cache, table, q, n = _attn_case(bs, case)
    f = torch.exp2(torch.randint(-40, 21, (cache.pages, 1, 16, 1, 1), generator=ref.gen(1), device="cuda").float())
    cache.v_scales.mul_(f.bfloat16())
    o, lse = bs.kv4_attn(cache, q, table, n, out_f32=True)
    _check_attn(o, lse, ref.attn(cache, q, table, case[-1]), True)


@pytest.mark.parametrize("power", [99, 40, -60, -120])
def test_attn_sizes_of_queries(bs, power):
    """Queries far from 1, up to the documented 2^100, and keys that make up for it."""
    for case in ((1, 4, 128, 16, 32, 1, [300]), (2, 8, 64, 16, 64, 2, [100, 37])):
        cache, table, q, n = _attn_case(bs, case)
        q.mul_(2.0 ** (power - 3))
        cache.k_scales.mul_(2.0 ** min(-power, 100))
        o, lse = bs.kv4_attn(cache, q, table, n, out_f32=True)
        _check_attn(o, lse, ref.attn(cache, q, table, case[-1]), True)


@pytest.mark.parametrize("case", [(1, 4, 128, 16, 32, 2, [300]), (1, 2, 64, 16, 64, 2, [9000])], ids=str)
def test_attn_query_that_is_not_finite_spoils_its_own_row_only(bs, case):
    cache, table, q, n = _attn_case(bs, case)
    want = bs.kv4_attn(cache, q, table, n)
    for bad in (float("nan"), float("inf")):
        spoilt = q.clone()
        spoilt[0, 1, 0, 5] = bad
        for got, old in zip(bs.kv4_attn(cache, spoilt, table, n), want):
            same = got == old
            same[0, 1, 0] = True
            assert bool(same.all())


def test_tables_of_one_page_with_any_stride(bs):
    """A single column cut out of a wider table, whatever its stride."""
    cache, table, q, n = _attn_case(bs, (1, 2, 64, 16, 64, 1, [9, 16]))
    wide = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:4] = table
    for got, want in zip(bs.kv4_attn(cache, q, wide[:, 3::3], n), bs.kv4_attn(cache, q, table, n)):
        assert torch.equal(got, want)
    bs.kv4_status(cache)


def test_attn_growing_scores(bs):
    """Scores that rise along the sequence by far more than a running maximum may lag, and fall."""
    case = (1, 2, 64, 16, 64, 1, [400])
    for sign in (1, -1):
        cache, table, q, n = _attn_case(bs, case)
        q[:] = 1.0
        order = table[0].long()
        for i in range(25):
            cache.k_scales[order[i], ..., 1] = sign * (i - 12) * 2.0
        o, lse = bs.kv4_attn(cache, q, table, n, out_f32=True)
        _check_attn(o, lse, ref.attn(cache, q, table, case[-1]), True)


def test_attn_never_reads_what_is_not_there(bs):
    """NaN scales in unused places, pages and heads' other tokens change nothing."""
    case = (2, 4, 128, 64, 128, 2, [70, 0, 1])
    cache, table, q, n = _attn_case(bs, case)
    want = bs.kv4_attn(cache, q, table, n)
    used = torch.zeros(cache.pages, cache.page_size, dtype=torch.bool, device="cuda")
    for b, length in enumerate(case[-1]):
        pos = torch.arange(length, device="cuda")
        used[table[b, pos // 64].long(), pos % 64] = True
    dead = ~used[:, None].expand(-1, 2, -1)
    for t in (cache.k_scales, cache.v_scales):
        t[dead] = float("nan")
    for t in (cache.k_codes, cache.v_codes):
        t[dead] = 255
    got = bs.kv4_attn(cache, q, table, n)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


SELECTED = [
    (2, 4, 128, 64, 128, 1, [700, 65, 1, 0], 4),
    (1, 8, 64, 16, 32, 3, [900, 17], 9),
    (4, 2, 128, 32, 64, 1, [2000], 64),
]


@pytest.mark.parametrize("case", SELECTED, ids=str)
def test_selected_pages(bs, case):
    *rest, keep = case
    cache, table, q, n = _attn_case(bs, tuple(rest))
    lengths = rest[-1]
    sel = bs.kv4_select(cache, q, table, n, keep, sink=1, recent=2)
    assert torch.equal(sel, ref.select_pages(cache, q, table, lengths, keep, 1, 2))
    o, lse = bs.kv4_attn(cache, q, table, n, sel, out_f32=True)
    bs.kv4_status(cache)
    _check_attn(o, lse, ref.attn(cache, q, table, lengths, sel), True)
    # a list of all pages is the whole cache
    most = table.shape[1]
    every = torch.arange(most, dtype=torch.int32, device="cuda").expand(len(lengths), cache.kv_heads, most).contiguous()
    whole = bs.kv4_attn(cache, q, table, n, every, out_f32=True)
    bs.kv4_status(cache)
    _check_attn(*whole, ref.attn(cache, q, table, lengths), True)


@pytest.mark.parametrize("pages", [1, 63, 64, 65, 1030, 4100, 17000])
def test_select_many_pages(bs, pages):
    """Lists on both sides of what a CTA holds in registers; ties among equal means."""
    page, D = 16, 64
    cache = bs.Kv4Cache(64, 1, D, page_size=page, group=64)
    ref.fill(cache, 4)
    g = ref.gen(5)
    table = torch.randint(0, 64, (2, pages), generator=g, device="cuda").to(torch.int32)  # pages repeat: ties
    lengths = [pages * page, max(1, pages * page // 3)]
    q = torch.randn(2, 4, 2, D, generator=g, device="cuda").bfloat16()
    for keep in (3, 40, 700):
        got = bs.kv4_select(cache, q, table, _i32(lengths), keep, sink=1, recent=2)
        assert torch.equal(got, ref.select_pages(cache, q, table, lengths, keep, 1, 2))
    got = bs.kv4_select(cache, q, table, _i32(lengths), 1, sink=0, recent=1)
    assert torch.equal(got, ref.select_pages(cache, q, table, lengths, 1, 0, 1))


@pytest.mark.parametrize("pages", [1500, 2100, 8192, 8200])
def test_select_many_heads(bs, pages):
    """Enough heads for one CTA each, lists on both sides of what that keeps."""
    page, D, B, Hkv = 16, 64, 20, 8
    cache = bs.Kv4Cache(64, Hkv, D, page_size=page, group=64)
    ref.fill(cache, 4)
    g = ref.gen(5)
    table = torch.randint(0, 64, (B, pages), generator=g, device="cuda").to(torch.int32)
    lengths = [max(1, pages * page - 5 * i * page) for i in range(B)]
    q = torch.randn(B, Hkv, 1, D, generator=g, device="cuda").bfloat16()
    got = bs.kv4_select(cache, q, table, _i32(lengths), 33, sink=1, recent=2)
    assert torch.equal(got, ref.select_pages(cache, q, table, lengths, 33, 1, 2))


def test_select_zero_queries(bs):
    cache, table, q, n = _attn_case(bs, (2, 4, 128, 16, 128, 1, [300, 40]))
    q.zero_()
    got = bs.kv4_select(cache, q, table, n, 5)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 18] and got[1, 1].tolist() == [0, 1, 2, -1, -1]


def test_bad_pages_are_skipped_and_reported(bs):
    case = (1, 4, 64, 16, 64, 1, [100])
    cache, table, q, n = _attn_case(bs, case)
    good = bs.kv4_attn(cache, q, table, n, _i32([[[0, 1, 3, 4, 5, 6]]]), out_f32=True)
    bs.kv4_status(cache)
    for bad in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):
        broken = table.clone()
        broken[0, 2] = bad
        got = bs.kv4_attn(cache, q, broken, n, out_f32=True)
        with pytest.raises(bs.BsattnError, match="page"):
            bs.kv4_status(cache)
        bs.kv4_status(cache)  # reported once
        _check_attn(*got, ref.attn(cache, q, table, [100], _i32([[[0, 1, 3, 4, 5, 6]]])), True)
        before = _state(cache)
        k = torch.randn(1, 1, 5, 64, device="cuda").bfloat16()
        bs.kv4_append(cache, k, k, broken, _i32([33]))
        with pytest.raises(bs.BsattnError):
            bs.kv4_status(cache)
        assert all(torch.equal(a, b) for a, b in zip(before, _state(cache)))
        rk, _ = bs.kv4_read(cache, broken, _i32([30]), 20)
        with pytest.raises(bs.BsattnError):
            bs.kv4_status(cache)
        assert bool((rk[0, 0, 2:18] == 0).all()) and bool(rk[0, 0, 18:].any()) and bool(rk[0, 0, :2].any())
        sel = bs.kv4_select(cache, q, broken, n, 7)
        with pytest.raises(bs.BsattnError):
            bs.kv4_status(cache)
        assert sel[0, 0].tolist() == [0, 1, 3, 4, 5, 6, -1]
    # behind the table, negative lengths, lists out of order
    k = torch.randn(1, 1, 5, 64, device="cuda").bfloat16()
    for length in (7 * 16 - 2, -3, 2 ** 31 - 2):
        bs.kv4_append(cache, k, k, table, _i32([length]))
        with pytest.raises(bs.BsattnError):
            bs.kv4_status(cache)
    bs.kv4_read(cache, table, _i32([-3]), 2)
    with pytest.raises(bs.BsattnError):
        bs.kv4_status(cache)
    got = bs.kv4_attn(cache, q, table, n, _i32([[[0, 1, 1, 3, 2, 4, 5, 6]]]), out_f32=True)
    with pytest.raises(bs.BsattnError):
        bs.kv4_status(cache)
    assert bool(torch.isfinite(got[0]).all()) and bool(torch.isfinite(good[0]).all())
    neg = bs.kv4_attn(cache, q, table, _i32([-7]))
    assert not bool(neg[0].any()) and bool(neg[1].isneginf().all())
    bs.kv4_status(cache)


def test_empty_calls(bs):
    cache = bs.Kv4Cache(2, 1, 64)
    table, n = torch.zeros(0, 1, dtype=torch.int32, device="cuda"), _i32([])
    q = torch.zeros(0, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    assert bs.kv4_attn(cache, q, table, n)[0].shape == q.shape
    assert bs.kv4_select(cache, q, table, n, 2).shape == (0, 1, 2)
    bs.kv4_append(cache, q[:, :1], q[:, :1], table, n)
    one, z = _i32([[0]]), torch.zeros(1, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    bs.kv4_append(cache, z, z, one, _i32([0]))
    assert bs.kv4_read(cache, one, _i32([0]), 0)[0].shape == (1, 1, 0, 64)
    bs.kv4_status(cache)


def test_offsets_past_32_bits(bs):
    """A cache whose code arrays pass 2^32 bytes: pages at its far end."""
    Hkv, D, page = 8, 128, 256
    pages = (1 << 32) // (Hkv * page * D // 2) + 40
    cache = bs.Kv4Cache(pages, Hkv, D, page_size=page, group=128)
    table = _i32([[pages - 1, 3, pages - 2]])
    T = 600
    g = ref.gen(2)
    k, v = (torch.randn(1, Hkv, T, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    bs.kv4_append(cache, k, v, table, _i32([0]))
    rk, rv = bs.kv4_read(cache, table, _i32([0]), T)
    for got, x in ((rk, k), (rv, v)):
        code, sc = ref.quantise(x, 128)
        assert float((got.double() - ref.values(ref.pack(code), sc)).abs().max()) < 0.02
    q = torch.randn(1, 32, 1, D, generator=g, device="cuda").bfloat16()
    o, lse = bs.kv4_attn(cache, q, table, _i32([T]), out_f32=True)
    _check_attn(o, lse, ref.attn(cache, q, table, [T]), True)
    bs.kv4_status(cache)


def test_refusals(bs):
    cache = bs.Kv4Cache(4, 2, 64, page_size=16)
    table, n = _i32([[0, 1]]), _i32([3])
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="group"):
        bs.Kv4Cache(4, 2, 64, group=128)
    with pytest.raises(ValueError, match="page_size"):
        bs.Kv4Cache(4, 2, 64, page_size=48)
    with pytest.raises(TypeError, match="Kv4Cache"):
        bs.kv4_attn(None, q, table, n)
    with pytest.raises(TypeError, match="int32"):
        bs.kv4_attn(cache, q, table.long(), n)
    with pytest.raises(ValueError, match="block_table"):
        bs.kv4_attn(cache, q, table[0], n)
    with pytest.raises(ValueError, match="lengths"):
        bs.kv4_attn(cache, q, table, _i32([3, 4]))
    with pytest.raises(ValueError, match="kv_heads"):
        bs.kv4_attn(cache, q[:, :3].contiguous(), table, n)
    with pytest.raises(ValueError, match="128 query rows"):
        bs.kv4_attn(cache, q.expand(1, 4, 65, 64).contiguous(), table, n)
    with pytest.raises(ValueError, match="selected"):
        bs.kv4_attn(cache, q, table, n, _i32([[0]]))
    with pytest.raises(ValueError, match="keep"):
        bs.kv4_select(cache, q, table, n, 1, sink=1, recent=1)
    with pytest.raises(ValueError, match="recent"):
        bs.kv4_select(cache, q, table, n, 3, recent=0)
    with pytest.raises(ValueError, match="k must have shape|k, v"):
        bs.kv4_append(cache, k[..., :32], k, table, n)
    with pytest.raises(ValueError, match="contiguous"):
        wide = torch.zeros(1, 2, 64, 2, dtype=torch.bfloat16, device="cuda").transpose(2, 3)[:, :, :1]
        bs.kv4_append(cache, wide, wide, table, n)
    with pytest.raises(TypeError, match="cuda"):
        bs.kv4_append(cache, k.cpu(), k.cpu(), table, n)
    with pytest.raises(ValueError, match="counts"):
        bs.kv4_read(cache, table, n, 1, _i32([1, 2]))
    with pytest.raises(bs.BsattnError):
        bs.kv4_attn(cache, q, table, n, scale=float("inf"))


def test_workspaces_too_small_are_refused(bs):
    """Long contexts and long page lists need a workspace; without enough of it nothing is launched."""
    cache = bs.Kv4Cache(3000, 1, 64, page_size=16)
    table = torch.arange(3000, dtype=torch.int32, device="cuda").expand(1, -1).repeat(1, 4).contiguous()
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    n, lib = _i32([100]), bs.load()
    out, lse = torch.full_like(q, 7.0), torch.zeros(1, 1, 1, device="cuda")
    sel = torch.full((1, 1, 4), 7, dtype=torch.int32, device="cuda")
    need = lib.bsattn_kv4_attn_workspace(1, 1, 1, 1, 64, 16, 12000, 0)
    pages = lib.bsattn_kv4_select_workspace(1, 1, 12000)
    assert need > 0 and pages == 4 * 12000
    ws = torch.zeros(max(need, pages), dtype=torch.uint8, device="cuda")
    on = torch.cuda.current_stream().cuda_stream
    for ptr, size in ((ws.data_ptr(), need - 1), (None, need), (ws.data_ptr() + 8, need)):
        assert lib.bsattn_kv4_attn(cache._ref, q.data_ptr(), 1, 1, 1, table.data_ptr(), 12000, 12000, n.data_ptr(),
                                   None, 0, 0.1, 0, out.data_ptr(), lse.data_ptr(), ptr, size, on) == bs.ERR_INVALID_ARG
    for ptr, size in ((ws.data_ptr(), pages - 1), (None, pages), (ws.data_ptr() + 8, pages)):
        assert lib.bsattn_kv4_select(cache._ref, q.data_ptr(), 1, 1, 1, table.data_ptr(), 12000, 12000, n.data_ptr(),
                                     4, 1, 1, sel.data_ptr(), ptr, size, on) == bs.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((sel == 7).all())


#          Hkv G  D    page group T  lengths, table columns behind them: on both sides of each split
SPLITS = [
    (1, 4, 128, 64, 128, 1, [20000], 0),             # one head over many CTAs
    (1, 2, 64, 16, 32, 1, [129, 5000, 1, 0, 640], 900),   # a wide table, short sequences
    (8, 8, 128, 16, 128, 1, [300] * 30 + [2500], 0),      # heads more than CTAs, ragged
    (2, 4, 128, 32, 64, 2, [1000, 900], 0),          # clusters of 8
    (8, 1, 64, 64, 64, 1, [700] * 9, 0),             # clusters of 4
    (2, 4, 128, 16, 32, 4, [513, 90], 800),          # 16 rows, ranges
    (37, 2, 64, 64, 64, 1, [1000], 0),               # clusters of 7, 6, 5 and 3
    (22, 4, 128, 64, 128, 1, [1100, 130], 0),
    (25, 1, 64, 16, 32, 1, [900, 17], 0),
    (20, 4, 128, 64, 128, 1, [1000, 500, 0, 3], 0),
    (16, 16, 64, 64, 64, 1, [800], 0),               # 16 rows, clusters of 6 and 4
    (15, 12, 128, 32, 64, 1, [700, 90], 0),
]


#          Hkv G  D    page group T  sequences, longest: more heads than CTAs
GROUPS = [
    (8, 4, 128, 64, 128, 1, 40, 700),      # 4 warps a head
    (8, 4, 64, 16, 32, 1, 100, 150),       # 2 warps
    (8, 8, 128, 64, 32, 1, 260, 100),      # 1 warp
    (16, 2, 64, 16, 64, 1, 48, 2000),      # 8 warps
    (4, 4, 128, 16, 64, 4, 50, 90),        # 16 rows: 4 warps
    (2, 20, 64, 32, 64, 1, 150, 60),       # rows in two tiles: 2 warps
    (8, 1, 128, 16, 128, 2, 301, 17),      # heads that leave a CTA half empty
    (32, 4, 128, 64, 128, 1, 12, 9000),    # ranges
]


@pytest.mark.parametrize("case", GROUPS, ids=str)
def test_more_heads_than_ctas(bs, case):
    """Ragged batches (empty sequences among them): a dozen different ones, each several times."""
    *rest, B, longest = case
    few = torch.randint(0, longest + 1, (min(B, 12),), generator=torch.Generator().manual_seed(1)).tolist()
    few[0], few[1] = longest, 0
    cache, table, q, n = _attn_case(bs, (*rest, few))
    at = torch.arange(B, device="cuda") % len(few)
    want = [x[at] for x in ref.attn(cache, q, table, few)]
    args = cache, q[at], table[at], n[at]
    o, lse = bs.kv4_attn(*args, out_f32=True)
    _check_attn(o, lse, want, True)
    again = bs.kv4_attn(*args, out_f32=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    # every page listed: the same tokens
    every = torch.arange(table.shape[1], dtype=torch.int32, device="cuda").expand(B, rest[0], -1).contiguous()
    _check_attn(*bs.kv4_attn(*args, every, out_f32=True), want, True)
    bs.kv4_status(cache)


@pytest.mark.parametrize("case", SPLITS, ids=str)
def test_splits(bs, case):
    *rest, extra = case
    cache, table, q, n = _attn_case(bs, tuple(rest))
    if extra:
        table = torch.cat([table, torch.full((table.shape[0], extra), -1, dtype=torch.int32, device="cuda")], 1)
    lengths = rest[-1]
    o, lse = bs.kv4_attn(cache, q, table, n, out_f32=True)
    bs.kv4_status(cache)
    _check_attn(o, lse, ref.attn(cache, q, table, lengths), True)


def test_lengths_behind_the_table(bs):
    """A length that the table has no pages for: reported; the queries see all that there is."""
    case = (2, 4, 64, 16, 64, 2, [112, 50])
    cache, table, q, n = _attn_case(bs, case)
    far = _i32([5000, 50])
    sel = bs.kv4_select(cache, q, table, far, 3)
    with pytest.raises(bs.BsattnError):
        bs.kv4_status(cache)
    assert sel[0, :, -1].tolist() == [6, 6] and sel[1].tolist() == bs.kv4_select(cache, q, table, n, 3)[1].tolist()
    o, lse = bs.kv4_attn(cache, q, table, far, out_f32=True)
    with pytest.raises(bs.BsattnError):
        bs.kv4_status(cache)
    # the last query of the right length sees the same tokens
    want, want_l = bs.kv4_attn(cache, q[:, :, 1:].contiguous(), table, n, out_f32=True)
    assert float((o[0, :, 1:] - want[0]).abs().max()) < 1e-5 and float((lse[0, :, 1:] - want_l[0]).abs().max()) < 1e-5
    bs.kv4_status(cache)


def test_many_sequences(bs):
    """The most sequences that one call takes; copies of a few give the same results."""
    B, case = 4096, (1, 4, 64, 16, 32, 1, [37, 0, 140, 16, 1])
    cache, table, q, n = _attn_case(bs, case)
    at = torch.arange(B, device="cuda") % 5
    want = ref.attn(cache, q, table, case[-1])
    _check_attn(*bs.kv4_attn(cache, q, table, n, out_f32=True), want, True)
    # (split otherwise, so sums in another order: both within the bounds that _ops_ref.attn derives)
    _check_attn(*bs.kv4_attn(cache, q[at], table[at], n[at], out_f32=True), [x[at] for x in want], True)
    bs.kv4_status(cache)
    with pytest.raises(bs.BsattnError, match="unsupported"):
        bs.kv4_attn(cache, q[at[:1]].expand(B + 1, -1, -1, -1).contiguous(), table[at[:1]].expand(B + 1, -1).contiguous(),
                    n[at[:1]].expand(B + 1).contiguous())
    sel = bs.kv4_select(cache, q[at], table[at], n[at], 3)
    assert torch.equal(sel, bs.kv4_select(cache, q, table, n, 3)[at])


def test_attn_long_context(bs):
    """Tens of thousands of tokens of equal standing: the output is a hundred times smaller than the
    values it is the mean of, yet its error stays below a quarter of bf16's half step, 2^-10 of it."""
    case = (2, 4, 128, 64, 128, 1, [60000, 30001])
    cache, table, q, n = _attn_case(bs, case)
    q *= 0.05
    o, lse = bs.kv4_attn(cache, q, table, n, out_f32=True)
    o_ref, l_ref, _, _ = ref.attn(cache, q, table, case[-1])
    err = (o.double() - o_ref).square().mean((1, 2, 3)).sqrt() / o_ref.square().mean((1, 2, 3)).sqrt()
    assert float(err.max()) < 2.0 ** -10, err
    assert float((lse.double() - l_ref).abs().max()) < 1e-5


@pytest.mark.parametrize("T", [1, 5, 8, 9])
def test_append_a_few_tokens(bs, T):
    """Decoding steps across page borders, pages that fill and pages that do not exist among them."""
    Hkv, D, page = 3, 64, 16
    lengths = [0, 7, 8, 15, 16, 31, 30, 100, 11]
    cache = bs.Kv4Cache(60, Hkv, D, page_size=page, group=32)
    ref.fill(cache, 4)
    table = ref.table(cache, [n + T for n in lengths], 8, 5)
    g = ref.gen(6)
    k, v = (torch.randn(len(lengths), Hkv, T, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    for counts in (None, [T, 0, T, 1, T - 1, T, T, T, 0]):
        before = _state(cache)
        bs.kv4_append(cache, k, v, table, _i32(lengths), None if counts is None else _i32(counts))
        bs.kv4_status(cache)
        want = _append_ref(cache, before, k, v, table, lengths, counts or [T] * len(lengths))
        assert all(torch.equal(a, b) for a, b in zip(_state(cache), want))
        k, v = v, k
    # a page that is not there: its tokens are skipped, the others written
    before, bad = _state(cache), table.clone()
    bad[3, 0] = -1  # position 15's
    bs.kv4_append(cache, k, v, bad, _i32(lengths))
    with pytest.raises(bs.BsattnError):
        bs.kv4_status(cache)
    rest = [b for b in range(len(lengths)) if b != 3]
    want = _append_ref(cache, before, k[rest], v[rest], table[rest], [lengths[b] for b in rest], [T] * len(rest))
    want = _append_ref(cache, want, k[3:4, :, 1:], v[3:4, :, 1:], table[3:4], [16], [T - 1])
    assert all(torch.equal(a, b) for a, b in zip(_state(cache), want))


@pytest.mark.parametrize("D, G, T, pages", [(128, 4, 1, 40), (128, 8, 4, 40), (128, 8, 5, 40), (64, 16, 4, 300), (128, 1, 1, 1500)])
def test_select_more_heads_than_sms(bs, D, G, T, pages):
    """On both sides of what the small CTAs take: rows, pages."""
    Hkv, page, B = 4, 16, 50
    few = [pages * page, 0, 1, 37, pages * page // 2 + 3]
    cache = bs.Kv4Cache(2 * pages + 8, Hkv, D, page_size=page)
    ref.fill(cache, 9)
    table = ref.table(cache, few, pages, 3)
    q = torch.randn(5, Hkv * G, T, D, generator=ref.gen(5), device="cuda").bfloat16()
    at = torch.arange(B, device="cuda") % 5
    got = bs.kv4_select(cache, q[at], table[at], _i32(few)[at], 7, sink=1, recent=2)
    assert torch.equal(got, ref.select_pages(cache, q, table, few, 7, 1, 2)[at])


#          Hkv G  D    page group T  lengths, table columns behind them, copies of the batch
WEIGHTED = [
    (2, 4, 128, 16, 128, 1, [1024, 300], 0, 1),          # clusters
    (1, 2, 64, 16, 32, 1, [1024], 900, 1),               # ranges
    (2, 8, 128, 32, 32, 1, [1000, 77], 0, 1),            # 8 rows
    (4, 4, 128, 64, 64, 4, [600], 0, 1),                 # 16 rows
    (8, 4, 64, 16, 64, 1, [700, 1024, 0, 33], 0, 60),    # a few warps a head
    (8, 8, 128, 16, 128, 1, [130, 90], 0, 150),
]


class _Weighted:
    """A case whose queries are positive, so that keys of one sign have weight or none."""

    def __init__(self, bs, case):
        *rest, extra, copies = case
        self.cache, self.table, self.q, self.n = _attn_case(bs, tuple(rest))
        self.q.abs_()
        self.lengths, self.copies = rest[-1], copies
        self.table = torch.cat([self.table, torch.full((len(self.lengths), extra), -1, dtype=torch.int32,
                                                       device="cuda")], 1)

    def places(self, first, last=None, step=1):
        """(page, place) of every sequence's tokens first(n), first(n) + step ... below last(n)."""
        page = self.cache.page_size
        for b, n in enumerate(self.lengths):
            for pos in range(first(n), n if last is None else last(n), step):
                yield int(self.table[b, pos // page]), pos % page

    def key(self, at, value):
        self.cache.k_scales[at[0], :, at[1], :, 0] = 0
        self.cache.k_scales[at[0], :, at[1], :, 1] = value

    def call(self, bs):
        at = torch.arange(len(self.lengths) * self.copies, device="cuda") % len(self.lengths)
        got = bs.kv4_attn(self.cache, self.q[at], self.table[at], self.n[at], out_f32=True)
        bs.kv4_status(self.cache)
        return at, *got

    def sizes(self):
        """Per output channel the size of the terms that it is the sum of: sum_i p_i (15 step_i + |least_i|)."""
        cache, (B, H, T, D) = self.cache, self.q.shape
        Hkv, page, G = cache.kv_heads, cache.page_size, H // cache.kv_heads
        out = torch.zeros(B, H, T, D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(self.lengths):
            pg, pos = self.table[b, :-(-n // page)].long(), torch.arange(n, device="cuda")
            for h in range(Hkv if n else 0):
                k = ref.values(cache.k_codes[pg, h], cache.k_scales[pg, h]).reshape(-1, D)[:n]
                vs = cache.v_scales[pg, h].double().reshape(-1, D // cache.group, 2)[:n]
                size = (15 * vs[..., 0] + vs[..., 1].abs()).repeat_interleave(cache.group, -1)
                for t in range(T):
                    s = self.q[b, h * G:(h + 1) * G, t].double() @ k.T * D ** -0.5
                    s = s.masked_fill(pos > n - T + t, float("-inf"))
                    if n - T + t >= 0:
                        out[b, h * G:(h + 1) * G, t] = torch.softmax(s, -1) @ size
        return out

    def check(self, bs):
        """Every term's relative error is within _ops_ref.attn's bound for a weight (twice: of the
        weight, and of the sum of weights), so an output is off by that part of its own terms' sizes.
        (The pair of halves ends at 2^-31 of a row's largest p step: over m tokens less than the
        m U32 that the bound has for the sums.)"""
        o_ref, _, _, dp = ref.attn(self.cache, self.q, self.table, self.lengths)
        tol = 2 * dp[..., None] * self.sizes() + U32 * o_ref.abs()
        at, o, _ = self.call(bs)
        err = (o.double() - o_ref[at]).abs()
        assert bool((err <= tol[at]).all()), float((err / (tol[at] + 1e-300)).max())


@pytest.mark.parametrize("power", [20, 60])
@pytest.mark.parametrize("case", WEIGHTED, ids=str)
def test_attn_wide_values_without_weight(bs, case, power):
    """Tokens that the queries give no weight (exp(-100)), their values 2^power times the others'."""
    w = _Weighted(bs, case)
    for at in w.places(lambda n: 5, step=97):
        w.key(at, -8.0)
        w.cache.v_scales[at[0], :, at[1]] *= 2.0 ** power
    w.check(bs)


@pytest.mark.parametrize("power", [-20, 0, 90])
@pytest.mark.parametrize("case", WEIGHTED, ids=str)
def test_attn_wide_values_whose_weight_vanishes(bs, case, power):
    """The first three quarters of a context weigh nothing once the rest, with values far smaller, is seen."""
    w = _Weighted(bs, case)
    for at in w.places(lambda n: 0, lambda n: 3 * n // 4):
        w.key(at, -8.0 if power < 50 else -16.0)
        w.cache.v_scales[at[0], :, at[1]] *= 2.0 ** power
    for at in w.places(lambda n: 3 * n // 4):
        w.cache.v_scales[at[0], :, at[1]] *= 2.0 ** -40
    w.check(bs)


@pytest.mark.parametrize("case", WEIGHTED, ids=str)
def test_attn_small_weights_beside_a_value_of_zero(bs, case):
    """One token has nearly all the weight, and its value is zero: the others make the output."""
    w = _Weighted(bs, case)
    w.cache.k_scales.mul_(0.1)
    for at in w.places(lambda n: 0, lambda n: min(n, 1)):
        w.key(at, 1.6)
        w.cache.v_scales[at[0], :, at[1]] = 0
    w.check(bs)


@pytest.mark.parametrize("case", [c for c in WEIGHTED if c[4] < c[2]], ids=str)
def test_attn_groups_of_other_sizes(bs, case):
    """Each group of channels 2^-20 times the one before: every output beside its own group."""
    w = _Weighted(bs, case)
    for n in range(w.cache.head_dim // w.cache.group):
        w.cache.v_scales[..., n, :] *= 2.0 ** (-20 * n)
    w.check(bs)


#         Hkv G  D    page group
CUTS = [(1, 4, 128, 16, 128), (2, 8, 64, 16, 32), (1, 8, 128, 64, 64), (2, 16, 128, 16, 32), (1, 2, 64, 32, 64),
        (1, 16, 64, 16, 64), (1, 3, 128, 16, 32)]


@pytest.mark.parametrize("case", CUTS, ids=str)
def test_attn_small_products_beside_a_large_one(bs, case):
    """One token of weight 1 and fifteen of weight 2^-15.5, all with the same step.

    A tensor instruction lines products up and cuts them: at 2^-21 of a code beside the largest
    weight, 16 products.  Beside that some 24 roundings in 32 bits (weight, its halves, sums) of at
    most 15 steps.  (Operands cut at 2^-15 are off by ten times the bound.)"""
    Hkv, G, D, page, group = case
    cache, table, q, n = _attn_case(bs, (Hkv, G, D, page, group, 1, [16]))
    q.fill_(1.0)
    pg = int(table[0, 0])
    cache.k_scales[pg, ..., 0] = 0
    cache.k_scales[pg, :, 0, :, 1] = 0
    cache.k_scales[pg, :, 1:, :, 1] = -10.75 * D ** -0.5
    cache.v_scales[pg, ..., 0] = 1
    cache.v_scales[pg, ..., 1] = 0
    o, _ = bs.kv4_attn(cache, q, table, n, out_f32=True)
    want = ref.attn(cache, q, table, [16])[0]
    assert float((o.double() - want).abs().max()) <= 16 * 2.0 ** -21 + 24 * U32 * 15


@pytest.mark.parametrize("case", CUTS, ids=str)
def test_attn_small_queries_beside_a_large_one(bs, case):
    """A single cached token, whose LSE is the score: one query channel of 1, the others 1.75 2^-19.

    32-bit sums as in _ops_ref.attn, and the cuts of the 16 products that share an instruction with
    the large one, and of their sum: 2^-18 of a step beside the largest query.  (Cut at 2^-15: twice
    the bound.)"""
    Hkv, G, D, page, group = case
    cache, table, q, n = _attn_case(bs, (Hkv, G, D, page, group, 1, [1]))
    q.fill_(1.75 * 2.0 ** -19)
    q[..., 4] = 1.0
    pg = int(table[0, 0])
    cache.k_codes[pg] = 0x99
    cache.k_scales[pg, ..., 0] = 1
    cache.k_scales[pg, ..., 1] = 0
    _, lse = bs.kv4_attn(cache, q, table, n)
    s = q.double().sum(-1) * 9 * D ** -0.5
    assert float((lse - s).abs().max()) <= D ** -0.5 * (
        (D + 8) * U32 * 15 * float(q[0, 0].double().sum()) + 17 * 2.0 ** -18)


@pytest.mark.parametrize("power", [101, 109, 116])
@pytest.mark.parametrize("case", WEIGHTED, ids=str)
def test_attn_large_values(bs, case, power):
    """Values up to the documented 2^104, and beyond where their sums still fit 32 bits."""
    w = _Weighted(bs, case)
    w.cache.v_scales.mul_(2.0 ** power)
    w.check(bs)


@pytest.mark.parametrize("case", WEIGHTED[:3], ids=str)
def test_attn_large_scores(bs, case):
    """Products of queries and keys up to the documented 2^112, one key a little above the others."""
    w = _Weighted(bs, case)
    D, s = w.cache.head_dim, w.cache.head_dim ** -0.5
    w.q.fill_(2.0 ** 99)
    w.cache.k_scales[..., 0] = 2.0
    w.cache.k_scales[..., 1] = 0.0
    for at in w.places(lambda n: n // 2, lambda n: n // 2 + 1):
        w.cache.k_codes[at[0], :, at[1]] = 0xFF
    w.cache.k_codes[w.cache.k_codes != 0xFF] = 0xEE
    at, o, lse = w.call(bs)
    for b, n in enumerate(w.lengths):
        pos = n // 2
        pg, place, group = int(w.table[b, pos // w.cache.page_size]), pos % w.cache.page_size, w.cache.group
        v = ref.values(w.cache.v_codes[pg, :, place], w.cache.v_scales[pg, :, place])
        v = v.repeat_interleave(o.shape[1] // v.shape[0], 0)
        assert float(((o[b, :, 0].double() - v).abs() - 24 * U32 * 15 * w.cache.v_scales[..., 0].max()).max()) <= 0
        assert float((lse[b, :, 0].double() / (2.0 ** 99 * 30 * D * s) - 1).abs().max()) <= (D + 16) * U32


@pytest.mark.parametrize("case", WEIGHTED, ids=str)
def test_attn_very_negative_scores(bs, case):
    """Equal scores of some -2^121: every visible token has the same weight, whatever the scores' size.

    The LSE is that score (the logarithm of the count is far below its last bit): D + 16 roundings of
    equal terms.  The output is a mean: the bound of _Weighted.check with exact scores."""
    w = _Weighted(bs, case)
    D, U = w.cache.head_dim, 2.0 ** 60
    w.q.fill_(U)
    w.cache.k_scales[..., 0] = 0
    w.cache.k_scales[..., 1] = -U / 2
    at, o, lse = w.call(bs)
    page, T = w.cache.page_size, w.q.shape[2]
    for b, n in enumerate(w.lengths):
        pg = w.table[b, :-(-n // page)].long()
        for t in range(T if n else 0):
            m = n - T + t + 1
            v = ref.values(w.cache.v_codes[pg], w.cache.v_scales[pg]).transpose(1, 2).flatten(0, 1)[:m]
            vs = w.cache.v_scales[pg].double().transpose(1, 2).flatten(0, 1)[:m]
            size = (15 * vs[..., 0] + vs[..., 1].abs()).amax((0, 2))[:, None]
            heads = o[b, :, t].unflatten(0, (w.cache.kv_heads, -1)).double()
            assert bool(((heads - v.mean(0)[:, None]).abs() <= 2 * (2.0 ** -20 + (m + 8) * U32) * size[..., None]).all())
            assert float((lse[b, :, t].double() / (-U * U / 2 * D ** 0.5) - 1).abs().max()) <= (D + 16) * U32


@pytest.mark.parametrize("T", [16, 5])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_append_values_of_far_sizes(bs, group, T):
    """Differences x - least that 32 bits round, on borders between two codes: tiny x of both signs
    beside a least value of -(k + 1/2) steps, and x of k + 1/2 steps beside a tiny least value."""
    D = 128
    tiny = 2.0 ** -torch.arange(15, 39, device="cuda").float()
    x = torch.zeros(1, 4, 16, D, device="cuda")
    x[..., :24], x[..., 32:56], x[..., 64:88], x[..., 96:120] = tiny, -tiny, tiny * 1.5, -tiny * 1.25
    border = torch.arange(16, device="cuda") * 0.25 + 0.125
    steps = torch.cat([border[:15], border.new_tensor([3.75])])
    for g in range(0, D, 32):
        x[0, 0, :, g + 24], x[0, 0, :, g + 25] = -border, 3.75 - border          # step 1/4
        x[0, 1, :, g + 24], x[0, 1, :, g + 25] = -border * 3, (3.75 - border) * 3
        x[0, 2, :, g + 8:g + 24] = steps
        x[0, 2, :, g + 24], x[0, 2, :, g:g + 8] = -tiny[4:20], 0                  # the least: tiny, below 0
        x[0, 3, :, g + 8:g + 24] = steps
        x[0, 3, :, g:g + 8], x[0, 3, :, g + 24:g + 32] = tiny[4:20, None], tiny[4:20, None]  # above 0
    x = x.bfloat16()[:, :, :T].contiguous()
    for k, v in ((x, -x), (-x, x)):
        cache = bs.Kv4Cache(2, 4, D, page_size=16, group=group)
        before = _state(cache)
        bs.kv4_append(cache, k, v, _i32([[1]]), _i32([0]))
        want = _append_ref(cache, before, k, v, _i32([[1]]), [0], [T])
        for got, w in zip(_state(cache), want):
            assert torch.equal(got, w), int((got != w).sum())


def test_report_while_the_status_is_asked(bs):
    """A call on another stream that reports at any time around a check is in that check's answer
    or in the next one's."""
    cache, table, q, n = _attn_case(bs, (1, 4, 64, 16, 64, 1, [100]))
    broken, other = torch.full_like(table, -1), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(1500):
        with torch.cuda.stream(other):
            torch.cuda._sleep(30000 + i % 500 * 400)  # some 15 to 115 us, the check a few after the call
            bs.kv4_attn(cache, q, broken, n)
        answers = []
        for wait in (False, True):
            if wait:
                other.synchronize()
            try:
                bs.kv4_status(cache)
                answers.append(bs.OK)
            except bs.BsattnError as e:
                answers.append(e.status)
        assert bs.ERR_PAGE in answers, i
    bs.kv4_status(cache)


@pytest.mark.parametrize("lengths", [[100], [100, 40, 9] * 120], ids=["clusters", "groups"])
def test_pages_behind_a_negative_entry(bs, lengths):
    """A page directly behind a negative entry is skipped and reported, and so not counted twice."""
    cache, table, q, n = _attn_case(bs, (1, 4, 64, 16, 64, 1, lengths))
    B = len(lengths)

    def call(pages):
        return bs.kv4_attn(cache, q, table, n, _i32(pages).expand(B, 1, -1).contiguous(), out_f32=True)

    for pages, same in (([1, -1, 1], [1, -1, -1]), ([0, -1, 2], [0, -1, -1]), ([0, 2, -5, 0], [0, 2, -1, -1]),
                        ([-1, 1], [-1, -1])):
        want = call(same)
        bs.kv4_status(cache)
        got = call(pages)
        with pytest.raises(bs.BsattnError, match="page"):
            bs.kv4_status(cache)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), pages


@pytest.mark.parametrize("case", [(1, 4, 128, 16, 128, 1, [300]), (1, 2, 64, 16, 32, 3, [9000]), (2, 8, 64, 32, 64, 1, [700, 20]),
                                  (1, 16, 128, 16, 32, 1, [200])], ids=str)
def test_attn_rows_do_not_touch_one_another(bs, case):
    """The bits of a query's result are the same whatever the other queries of its head are: scores
    that rise far above their running maximum, or that are infinite, rescale their own row only."""
    cache, table, q, n = _attn_case(bs, case)
    cache.k_scales[..., 1].abs_()  # keys above zero
    cache.k_codes |= 0x11
    G, rows = case[1], [h for h in range(q.shape[1]) if h % case[1]]
    want = bs.kv4_attn(cache, q, table, n, out_f32=True)
    for value in (float("inf"), 2.0 ** 90, 300.0, -300.0, 0.0, float("nan")):
        other = q.clone()
        other[:, ::G] = value
        got = bs.kv4_attn(cache, other, table, n, out_f32=True)
        for a, b in zip(got, want):
            assert torch.equal(a[:, rows], b[:, rows]), value
