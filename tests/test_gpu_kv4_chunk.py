"""Attention of chunks of new tokens over the 4-bit cache (kv4_attn_chunk) against 64 bits.

Tolerances: the bounds that _ops_ref.attn_chunk derives (32-bit scores and sums, values
and weights of 11 bits, of 8 where the values of 32 tokens lie far apart), plus the
output's own rounding."""
import math
import pathlib
import subprocess
import sys
import threading

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


# with a table that has room for so many tokens up to 128 rows are taken as more are
ROOM = 1 << 18


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(bs, Hkv, G, D, page, group, T, lengths, seed=5, columns=None, spread=1.0):
    B = len(lengths)
    need = [-(-max(n, 0) // page) for n in lengths]
    cache = bs.Kv4Cache(sum(need) + 2, Hkv, D, page_size=page, group=group)
    ref.fill(cache, seed, spread)
    table = ref.table(cache, [max(n, 0) for n in lengths], columns or max(1, max(need)), seed + 1)
    q = (torch.randn(B, Hkv * G, T, D, generator=ref.gen(seed + 2), device="cuda") * 1.5).bfloat16()
    return cache, table, q, _i32(lengths)


def _check(got, want, out_f32=False):
    o, lse = got
    o_ref, l_ref, tol_o, tol_l = want
    dead = l_ref.isneginf()
    assert torch.equal(lse.isneginf(), dead)
    assert not bool(o[dead].any())
    err = (lse.double() - l_ref).abs()[~dead]
    tol = tol_l[~dead] + 4 * U32 * (1 + l_ref[~dead].abs())
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol).max()))
    tol = tol_o[..., None] + (U32 if out_f32 else UBF) * o_ref.abs()
    err = (o.double() - o_ref).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / (tol + 1e-300)).max()))


def _slopes(H):
    return 0.5 ** (8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


#  Hkv G  D    page group T   lengths          counts
CHUNKS = [
    (1, 1, 64, 16, 64, 1, [1], None),                       # one token, nothing else
    (2, 4, 128, 64, 128, 1, [0, 1, 63, 64, 65, 700], None),  # single tokens
    (1, 3, 128, 32, 64, 5, [5, 4, 40, 555], [5, 4, 0, 3]),   # few rows, ragged
    (1, 17, 64, 16, 32, 1, [1, 129, 512, 513], None),        # one row more than the few-row form takes
    (2, 4, 128, 64, 128, 5, [5, 260, 1000], [5, 1, 4]),      # 20 rows: both tiles the same rows
    (1, 1, 128, 256, 32, 128, [128, 700], [100, 128]),       # 128 rows
    (1, 1, 128, 16, 128, 129, [129, 600], [129, 7]),         # 129: the second tile has one
    (1, 5, 64, 128, 64, 61, [61, 305], [61, 50]),            # 305 rows, five heads a tile
    (2, 2, 128, 64, 64, 257, [257, 257, 300, 1111], [257, 0, 1, 256]),
    (3, 1, 64, 32, 64, 500, [900], None),
    (1, 8, 128, 64, 32, 33, [2000, 3, 0, 33], [33, 33, 33, 33]),  # fewer cached than counted
    (1, 2, 128, 128, 128, 70, [4000], [69]),                 # split over CTAs
    (4, 1, 64, 16, 32, 300, [300, 290], [300, 290]),
]
OPTIONS = {"plain": {}, "cap": dict(cap=4.0), "slopes": dict(slopes=True), "prefix": dict(prefix=True),
           "all": dict(cap=20.0, slopes=True, prefix=True)}


def _options(name, H, lengths):
    o = dict(OPTIONS[name])
    if o.get("slopes"):
        o["slopes"] = _slopes(H)
    prefix = [(n * 2) // 3 - (b == 1) * 1000 + (b == 2) * 5000 for b, n in enumerate(lengths)] if "prefix" in o else None
    return o, prefix


CASES = [(c, False) for c in CHUNKS] + [(c, True) for c in CHUNKS if 16 < c[1] * c[5] <= 128]


@pytest.mark.parametrize("option", OPTIONS)
@pytest.mark.parametrize("case,room", CASES,
                         ids=lambda c: "room" * c if isinstance(c, bool) else "-".join(str(x) for x in c[:6]))
def test_chunk(bs, case, room, option):
    Hkv, G, D, page, group, T, lengths, counts = case
    cache, table, q, n = _case(bs, *case[:-1], columns=ROOM // page if room else None)
    o, prefix = _options(option, Hkv * G, lengths)
    args = dict(o, prefix=None if prefix is None else _i32(prefix))
    want = ref.attn_chunk(cache, q, table, lengths, counts, prefix, o.get("cap"), o.get("slopes"))
    c = None if counts is None else _i32(counts)
    got = bs.kv4_attn_chunk(cache, q, table, n, c, **args)
    bs.kv4_status(cache)
    _check(got, want)
    # whatever was in the outputs; the same bits again
    out, lse = torch.full_like(got[0], 7.0), torch.full_like(got[1], 7.0)
    again = bs.kv4_attn_chunk(cache, q, table, n, c, out=out, lse=lse, **args)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    o32 = bs.kv4_attn_chunk(cache, q, table, n, c, out_f32=True, **args)
    _check(o32, want, True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("T", [3, 80])
def test_scale(bs, scale, T):
    cache, table, q, n = _case(bs, 2, 2, 64, 32, 32, T, [300, 100])
    for more in ({}, dict(cap=3.0)):
        _check(bs.kv4_attn_chunk(cache, q, table, n, scale=scale, **more),
               ref.attn_chunk(cache, q, table, [300, 100], scale=scale, **more))


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 0.5, 3.0, 1e6, 1e30])
@pytest.mark.parametrize("T", [3, 80])
@pytest.mark.parametrize("size", [1e-12, 1.0])
def test_caps_of_any_size(bs, T, cap, size):
    """All forms of the tanh, and caps that leave scores as they are."""
    cache, table, q, n = _case(bs, 2, 2, 64, 32, 32, T, [300, 100])
    q = (q.float() * size).bfloat16()
    _check(bs.kv4_attn_chunk(cache, q, table, n, cap=cap), ref.attn_chunk(cache, q, table, [300, 100], cap=cap))


def _put(cache, table, name, b, h, token, x):
    """Token `token` of sequence b holds x [D]."""
    code, scales = ref.quantise(x[None].bfloat16(), cache.group)
    page, place = int(table[b, token // cache.page_size]), token % cache.page_size
    getattr(cache, name + "_codes")[page, h, place] = ref.pack(code)[0]
    getattr(cache, name + "_scales")[page, h, place] = scales[0].bfloat16()


@pytest.mark.parametrize("T,group", [(3, 64), (90, 64), (90, 32), (300, 64)])
@pytest.mark.parametrize("down", [False, True], ids=["growing", "falling"])
def test_scores_that_grow(bs, T, group, down):
    """Keys along the queries, larger and larger (or less and less): the reference moves often."""
    n, D = 900, 64
    cache, table, q, lengths = _case(bs, 1, 2, D, 64, group, T, [n])
    q[:] = q[:, :, :1]
    for t in range(0, n, 37):
        x = q[0, t % 2, 0].float() * ((n - t if down else t) / n) * 2.5
        _put(cache, table, "k", 0, 0, t, x)
    for more in ({}, dict(cap=50.0), dict(slopes=_slopes(2))):
        want = ref.attn_chunk(cache, q, table, [n], cap=more.get("cap"), slopes=more.get("slopes"))
        _check(bs.kv4_attn_chunk(cache, q, table, lengths, **more), want)


@pytest.mark.parametrize("T", [3, 90])
@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_large_and_small_scores(bs, T, size):
    cache, table, q, n = _case(bs, 1, 3, 128, 64, 128, T, [400])
    q = (q.float() * size).bfloat16()
    want = ref.attn_chunk(cache, q, table, [400])
    _check(bs.kv4_attn_chunk(cache, q, table, n), want)
    want = ref.attn_chunk(cache, q, table, [400], cap=5.0)
    _check(bs.kv4_attn_chunk(cache, q, table, n, cap=5.0), want)


@pytest.mark.parametrize("T", [3, 90])
@pytest.mark.parametrize("power", [-60, -9, 9, 60])
def test_values_of_other_sizes(bs, T, power):
    """Some tokens' values far from the others' (bf16 for their neighbours), and all of them."""
    n = 400
    cache, table, q, lengths = _case(bs, 1, 2, 64, 32, 32, T, [n])
    g = ref.gen(3)
    for t in range(5, n, 91):
        _put(cache, table, "v", 0, 0, t, torch.randn(64, generator=g, device="cuda") * 2.0 ** power)
    _check(bs.kv4_attn_chunk(cache, q, table, lengths), ref.attn_chunk(cache, q, table, [n], value_bits=8))
    cache.v_scales.mul_(2.0 ** power)
    _check(bs.kv4_attn_chunk(cache, q, table, lengths), ref.attn_chunk(cache, q, table, [n], value_bits=8))


@pytest.mark.parametrize("T", [3, 90])
@pytest.mark.parametrize("power", [-98, -40, 40, 108])
def test_keys_of_other_sizes(bs, T, power):
    """All keys very large or small, and queries the other way."""
    cache, table, q, n = _case(bs, 1, 2, 128, 32, 64, T, [300])
    cache.k_scales.mul_(2.0 ** power)
    q = (q.float() * 2.0 ** -power).bfloat16()
    _check(bs.kv4_attn_chunk(cache, q, table, n), ref.attn_chunk(cache, q, table, [300]))


@pytest.mark.parametrize("T", [2, 100, 200])
def test_values_that_are_not_numbers(bs, T):
    """A group of channels that stands for NaN spoils those channels of the queries that see it."""
    n, D, group = 700, 128, 32
    cache, table, q, lengths = _case(bs, 1, 2, D, 64, group, T, [n])
    clean = bs.kv4_attn_chunk(cache, q, table, lengths)
    token = n - T // 2 - 1
    page, place = int(table[0, token // 64]), token % 64
    cache.v_scales[page, 0, place, 2] = float("nan")
    o, lse = bs.kv4_attn_chunk(cache, q, table, lengths)
    sees = (n - T + torch.arange(T, device="cuda")) >= token
    bad = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    bad[sees, 2 * group:3 * group] = True
    assert torch.equal(o[0, 0].isnan(), bad) and torch.equal(o[0, 1].isnan(), bad)
    assert torch.equal(lse, clean[1])
    # (neighbours of the token may be held otherwise: both are within their bounds of the same)
    far = (o.double() - clean[0].double()).abs()
    assert float(far[~bad.expand_as(far)].max()) < 0.1
    cache.v_scales[page, 0, place, 2] = 0.0
    cache.k_scales[page, 0, place, 0, 1] = float("inf")
    o, lse = bs.kv4_attn_chunk(cache, q, table, lengths)
    assert bool(lse[..., sees].isnan().all()) and not bool(lse[..., ~sees].isnan().any())
    assert bool(o[:, :, sees].isnan().all()) and not bool(o[:, :, ~sees].isnan().any())


@pytest.mark.parametrize("T", [2, 50, 90])
def test_nothing_behind_the_length_is_read(bs, T):
    """Rows of the last page behind the length hold NaN; so do all other pages."""
    n = 333
    cache, table, q, lengths = _case(bs, 2, 2, 64, 64, 32, T, [n], columns=ROOM // 64 if T == 50 else None)
    want = bs.kv4_attn_chunk(cache, q, table, lengths)
    used = table[0, :6].long()
    for name in "kv":
        scales = getattr(cache, name + "_scales")
        keep = scales[used].clone()
        scales.fill_(float("nan"))
        keep[5, :, n % 64:] = float("nan")
        scales[used] = keep
    got = bs.kv4_attn_chunk(cache, q, table, lengths)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [2, 30, 42, 50])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_a_query_spoils_its_own_row_only(bs, T, bad):
    cache, table, q, n = _case(bs, 1, 3, 64, 64, 32, T, [600], columns=ROOM // 64 if T == 42 else None)
    want = bs.kv4_attn_chunk(cache, q, table, n)
    q2 = q.clone()
    q2[0, 1, 1, 5] = bad
    got = bs.kv4_attn_chunk(cache, q2, table, n)
    others = torch.ones(3, T, dtype=torch.bool, device="cuda")
    others[1, 1] = False
    assert torch.equal(got[0][0][others], want[0][0][others])
    assert torch.equal(got[1][0][others], want[1][0][others])


@pytest.mark.parametrize("T", [2, 40, 60, 70])
def test_bad_pages_are_skipped_and_reported(bs, T):
    lengths = [500, 300]
    cache, table, q, n = _case(bs, 1, 2, 64, 16, 32, T, lengths, columns=ROOM // 16 if T == 60 else None)
    for entry in (-1, cache.pages, 1 << 30):
        t = table.clone()
        t[0, 3], t[1, 18] = entry, entry
        got = bs.kv4_attn_chunk(cache, q, t, n)
        with pytest.raises(bs.BsattnError, match="page"):
            bs.kv4_status(cache)
        _check(got, ref.attn_chunk(cache, q, t, lengths))
    # a table that is too short for the first sequence
    short = table[:, :20]
    got = bs.kv4_attn_chunk(cache, q, short, n)
    with pytest.raises(bs.BsattnError, match="page"):
        bs.kv4_status(cache)
    _check(got, ref.attn_chunk(cache, q, short, lengths))
    bs.kv4_status(cache)


@pytest.mark.parametrize("T", [4, 40, 50, 70])
def test_sequences_that_are_empty(bs, T):
    """Lengths of zero and below, counts of zero and below, counts above T and above the length."""
    lengths, counts = [0, -5, 40, 40, 40, 2], [T, T, 0, -3, T + 9, T]
    cache, table, q, n = _case(bs, 1, 2, 64, 16, 64, T, lengths, columns=ROOM // 16 if T == 50 else None)
    _check(bs.kv4_attn_chunk(cache, q, table, n, _i32(counts)), ref.attn_chunk(cache, q, table, lengths, counts))
    bs.kv4_status(cache)


def test_many_sequences(bs):
    lengths = [(b * 37) % 90 for b in range(300)]
    counts = [min(20, b % 23) for b in range(300)]
    cache, table, q, n = _case(bs, 2, 1, 64, 16, 32, 20, lengths)
    want = ref.attn_chunk(cache, q, table, lengths, counts)
    _check(bs.kv4_attn_chunk(cache, q, table, n, _i32(counts)), want)


def test_offsets_past_32_bits(bs):
    """A cache whose code arrays pass 2^32 bytes: pages at its far end."""
    Hkv, D, page = 8, 128, 256
    pages = (1 << 32) // (Hkv * page * D // 2) + 40
    cache = bs.Kv4Cache(pages, Hkv, D, page_size=page, group=128)
    table = _i32([[pages - 1, 3, pages - 2]])
    g = ref.gen(2)
    k, v = (torch.randn(1, Hkv, 600, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    bs.kv4_append(cache, k, v, table, _i32([0]))
    for T in (2, 70):
        q = torch.randn(1, 16, T, D, generator=g, device="cuda").bfloat16()
        _check(bs.kv4_attn_chunk(cache, q, table, _i32([600])), ref.attn_chunk(cache, q, table, [600]))
    bs.kv4_status(cache)


@pytest.mark.parametrize("T", [2, 40, 50, 200])
def test_captured_and_on_other_streams(bs, T):
    """Graphs follow lengths that grow; two of them, each with its workspace, at once."""
    lengths = [600, 900]
    cache, table, q, _ = _case(bs, 1, 2, 64, 32, 64, T, lengths, columns=ROOM // 32 if T == 50 else None)
    n = _i32([500, 301])
    graphs, results = [], []
    side = torch.cuda.Stream()
    for _ in range(2):
        bs.kv4_attn_chunk(cache, q, table, n)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            results.append(bs.kv4_attn_chunk(cache, q, table, n, cap=30.0))
        graphs.append(graph)
    for now in ([500, 301], lengths):
        n.copy_(_i32(now))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        want = ref.attn_chunk(cache, q, table, now, cap=30.0)
        for got in results:
            _check(got, want)
    eager = bs.kv4_attn_chunk(cache, q, table, n, cap=30.0, stream=side)
    side.synchronize()
    assert torch.equal(eager[0], results[0][0]) and torch.equal(eager[1], results[0][1])


def test_tables_with_any_stride(bs):
    cache, table, q, n = _case(bs, 1, 2, 64, 16, 64, 30, [100, 77])
    want = bs.kv4_attn_chunk(cache, q, table, n)
    wide = torch.full((2, 50), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + table.shape[1]] = table
    got = bs.kv4_attn_chunk(cache, q, wide[:, 3:3 + table.shape[1]], n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_same_as_single_tokens(bs):
    """The last token of a chunk, and the same token by itself."""
    lengths = [700, 333]
    cache, table, q, n = _case(bs, 2, 4, 128, 64, 64, 64, lengths)
    many = bs.kv4_attn_chunk(cache, q, table, n, out_f32=True)
    one = bs.kv4_attn(cache, q[:, :, -1:].contiguous(), table, n, out_f32=True)
    want = ref.attn_chunk(cache, q, table, lengths)
    tol = want[2][:, :, -1:, None]
    assert bool(((many[0][:, :, -1:] - one[0]).abs() <= 2 * tol).all())
    assert bool(((many[1][:, :, -1:] - one[1]).abs() <= 2 * want[3][:, :, -1:] + 1e-5).all())


def test_empty_calls(bs):
    cache = bs.Kv4Cache(2, 1, 64)
    q = torch.zeros(0, 2, 9, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    assert bs.kv4_attn_chunk(cache, q, table, _i32([]))[0].shape == q.shape
    q = torch.zeros(1, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    assert bs.kv4_attn_chunk(cache, q, _i32([[0]]), _i32([5]))[1].shape == (1, 2, 0)


def test_refusals(bs):
    cache = bs.Kv4Cache(4, 2, 64, page_size=16)
    table, n = _i32([[0, 1]]), _i32([3])
    q = torch.zeros(1, 4, 30, 64, dtype=torch.bfloat16, device="cuda")
    for match, change in (("kv_heads", dict(q=q[:, :3].contiguous())), ("counts", dict(counts=_i32([1, 2]))),
                          ("prefix", dict(prefix=_i32([1, 2]))), ("slopes", dict(slopes=torch.zeros(3, device="cuda"))),
                          ("cap", dict(cap=0.0)), ("cap", dict(cap=-1.0)), ("cap", dict(cap=math.nan)),
                          ("contiguous", dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))),
                          ("block_table", dict(block_table=table[0])), ("out", dict(out=q[:, :2].contiguous()))):
        args = dict(q=q, block_table=table, lengths=n)
        args.update(change)
        with pytest.raises(ValueError, match=match):
            bs.kv4_attn_chunk(cache, **args)
    for change in (dict(q=q.float()), dict(counts=n.long()), dict(slopes=torch.zeros(4, device="cuda").double()),
                   dict(prefix=n.cpu()), dict(cache=None)):
        args = dict(cache=cache, q=q, block_table=table, lengths=n)
        args.update(change)
        with pytest.raises(TypeError):
            bs.kv4_attn_chunk(**args)
    with pytest.raises(bs.BsattnError):
        bs.kv4_attn_chunk(cache, q, table, n, scale=float("inf"))
    with pytest.raises(bs.BsattnError):
        bs.kv4_attn_chunk(cache, q, table, n, cap=1e35)


@pytest.mark.parametrize("T", [3, 12, 20, 60])
def test_rows_do_not_touch_one_another(bs, T):
    """One row's wide scores leave the others' bits alone, with a cap and without."""
    cache, table, q, n = _case(bs, 1, 4, 64, 64, 32, T, [700], columns=ROOM // 64 if T == 20 else None)
    for more in ({}, dict(cap=10.0), dict(slopes=_slopes(4))):
        want = bs.kv4_attn_chunk(cache, q, table, n, **more)
        q2 = q.clone()
        q2[0, 2, 1] *= 40
        got = bs.kv4_attn_chunk(cache, q2, table, n, **more)
        others = torch.ones(4, T, dtype=torch.bool, device="cuda")
        others[2, 1] = False
        assert torch.equal(got[0][0][others], want[0][0][others])
        assert torch.equal(got[1][0][others], want[1][0][others])


@pytest.mark.parametrize("T", [3, 90])
@pytest.mark.parametrize("prefix", [-2 ** 31, -1, 2 ** 31 - 1])
def test_prefixes_of_any_value(bs, T, prefix):
    cache, table, q, n = _case(bs, 1, 2, 64, 64, 32, T, [200])
    _check(bs.kv4_attn_chunk(cache, q, table, n, prefix=_i32([prefix])),
           ref.attn_chunk(cache, q, table, [200], prefix=[prefix]))


def test_chain(bs):
    """As a server runs: pages reserved, prompts in ragged chunks, samples forked, drafts, ended
    rows, compaction; each answer against 64 bits of what the cache holds."""
    Hkv, H, D, page = 2, 6, 64, 16
    cache = bs.Kv4Cache(96, Hkv, D, page_size=page, group=32)
    refs = torch.zeros(96, dtype=torch.int32, device="cuda")
    table = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    lengths = _i32([0, 0])
    g = ref.gen(11)

    def step(table, lengths, refs, T, counts, **more):
        B = table.shape[0]
        table, refs = bs.kv4_reserve(cache, refs, table, lengths, _i32(counts))
        k, v = (torch.randn(B, Hkv, T, D, generator=g, device="cuda").bfloat16() for _ in "kv")
        bs.kv4_append(cache, k, v, table, lengths, _i32(counts))
        lengths = lengths + _i32(counts)
        q = torch.randn(B, H, T, D, generator=g, device="cuda").bfloat16()
        got = bs.kv4_attn_chunk(cache, q, table, lengths, _i32(counts), **more)
        _check(got, ref.attn_chunk(cache, q, table, lengths.tolist(), counts, cap=more.get("cap"),
                                   slopes=more.get("slopes")))
        return table, lengths, refs

    state = step(table, lengths, refs, 75, [75, 40])
    state = step(*state, 33, [20, 33], cap=20.0)
    table, lengths, refs = bs.kv4_fork(cache, state[2], state[0], state[1], _i32([0, 0, 1, 0, 1]))
    state = step(table, lengths, refs, 1, [1] * 5, slopes=_slopes(H))
    state = step(*state, 4, [4, 3, 0, 1, 2], cap=5.0, slopes=_slopes(H))
    table, lengths, refs = bs.kv4_fork(cache, state[2], state[0], state[1], _i32([4, -1, 1]))
    table, refs, page_map = bs.kv4_compact(cache, refs, table)
    used = int((refs > 0).sum())
    assert bool((refs[:used] > 0).all()) and not bool(refs[used:].any())
    state = step(table, lengths, refs, 2, [2, 2, 1])
    assert ref.count_refs(cache, state[0].tolist(), state[1].tolist()) == state[2].tolist()
    bs.kv4_status(cache)


FIRST_USE = """
import torch
import block_sparse_flash_attn_gb300 as bs
cache, other = (bs.Kv4Cache(200, 2, 64, page_size=32, group=32) for _ in range(2))
refs = torch.zeros(200, dtype=torch.int32, device="cuda")
empty = torch.full((3, 50), -1, dtype=torch.int32, device="cuda")
zero = torch.zeros(3, dtype=torch.int32, device="cuda")
counts = torch.tensor([700, 30, 333], dtype=torch.int32, device="cuda")
parents = torch.tensor([2, 0, 0, -1], dtype=torch.int32, device="cuda")
pages = torch.arange(200, dtype=torch.int32, device="cuda")
k, v = (torch.randn(3, 2, 700, 64, device="cuda").bfloat16() for _ in "kv")
q = torch.randn(3, 4, 700, 64, device="cuda").bfloat16()
slopes = torch.rand(4, device="cuda")


def step():
    table, held = bs.kv4_reserve(cache, refs, empty, zero, counts)
    bs.kv4_append(cache, k, v, table, zero, counts)
    got = []
    for T in (1, 4, 30, 700):
        x = q[:, :, -T:].contiguous()
        got += bs.kv4_attn_chunk(cache, x, table, counts, torch.clamp(counts, max=T))
        got += bs.kv4_attn_chunk(cache, x, table, counts, torch.clamp(counts, max=T), cap=5.0, slopes=slopes)
    table, lengths, held = bs.kv4_fork(cache, held, table, counts, parents)
    table, held, moved = bs.kv4_compact(cache, held, table)
    bs.kv4_copy(cache, pages, pages, to=other)
    return got + [table, lengths, held, moved] + list(bs.kv4_read(other, table, torch.zeros_like(lengths), 700))


graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
bs.kv4_status(cache)
"""


def test_first_use_inside_a_capture(bs):
    """A process whose first calls are captured into a graph."""
    root = pathlib.Path(__file__).resolve().parents[1]
    subprocess.run([sys.executable, "-c", FIRST_USE], cwd=root, check=True, timeout=120)


def test_calls_from_several_threads(bs):
    """Each thread with its stream, one cache, calls of both kernels."""
    cache, table, q, n = _case(bs, 2, 4, 64, 64, 32, 50, [700, 300])
    few = q[:, :, -2:].contiguous()
    want = [bs.kv4_attn_chunk(cache, x, table, n, cap=7.0) for x in (q, few)]
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(10):
            for x, w in zip((q, few), want):
                got = bs.kv4_attn_chunk(cache, x, table, n, cap=7.0, stream=stream)
                stream.synchronize()
                bad.extend(1 for a, b in zip(got, w) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    bs.kv4_status(cache)
