"""Chunk attention over the 4-bit cache where it can go wrong at the ends of its ranges: values that
are not numbers far behind the queries, values of very different sizes together, what one row's
bits depend on, and errors by their norms (closer than bounds for each entry can be)."""
import pytest
import torch

import _ops_ref as ref
from _ops_ref import UBF
from test_gpu_kv4_chunk import ROOM, _case, _check, _i32, _put, bs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True], ids=["exact", "wide"])
@pytest.mark.parametrize("T,B", [(2, 1), (8, 1), (20, 1), (60, 1), (300, 1), (300, 80)])
def test_values_far_away_that_are_not_numbers(bs, T, B, wide):  # noqa: F811
    """A group of channels that stands for NaN spoils those channels of all queries that see it, also
    where a bias by distance leaves it no weight at all, in one range of tokens or in many."""
    n, D, group = 2900, 128, 32
    cache, table, q, lengths = _case(bs, 1, 2, D, 64, group, T, [n], columns=ROOM // 64 if wide else None)
    table, q, lengths = table.expand(B, -1), q.expand(B, -1, -1, -1).contiguous(), lengths.expand(B).contiguous()
    slopes = torch.tensor([0.5, 0.25], device="cuda")
    clean = bs.kv4_attn_chunk(cache, q, table, lengths, slopes=slopes)
    assert bool(clean[0].isfinite().all())
    cache.v_scales[int(table[0, 0]), 0, 3, 2] = float("nan")
    o, lse = bs.kv4_attn_chunk(cache, q, table, lengths, slopes=slopes)
    bad = torch.zeros(D, dtype=torch.bool, device="cuda")
    bad[2 * group:3 * group] = True
    assert torch.equal(o.isnan(), bad.expand_as(o))
    assert torch.equal(lse, clean[1])
    # (the token's neighbours may be held otherwise: both are within their bounds of the same)
    assert float((o - clean[0])[..., ~bad].abs().max()) < 0.1


@pytest.mark.parametrize("T", [3, 5, 8])
@pytest.mark.parametrize("more", [{}, dict(cap=20.0), dict(slopes=True)], ids=["plain", "cap", "slopes"])
def test_few_rows_that_do_not_see_a_value(bs, T, more):  # noqa: F811
    n, D, group = 700, 128, 32
    cache, table, q, lengths = _case(bs, 1, 2, D, 64, group, T, [n])
    if "slopes" in more:
        more = dict(slopes=torch.tensor([0.5, 0.01], device="cuda"))
    clean = bs.kv4_attn_chunk(cache, q, table, lengths, **more)
    token = n - T // 2 - 1
    cache.v_scales[int(table[0, token // 64]), 0, token % 64, 2] = float("nan")
    o, lse = bs.kv4_attn_chunk(cache, q, table, lengths, **more)
    sees = (n - T + torch.arange(T, device="cuda")) >= token
    assert 0 < int(sees.sum()) < T
    bad = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    bad[sees, 2 * group:3 * group] = True
    assert torch.equal(o[0, 0].isnan(), bad) and torch.equal(o[0, 1].isnan(), bad)
    assert torch.equal(lse, clean[1])
    assert float((o[:, :, ~sees].double() - clean[0][:, :, ~sees].double()).abs().max()) < 0.1


@pytest.mark.parametrize("T", [3, 90, 300])
@pytest.mark.parametrize("slopes", [False, True])
def test_one_value_far_above_the_others(bs, T, slopes):  # noqa: F811
    """All values near 2^-60 but one token's near 2^100: the output is that token's.  It is off by the
    rounding of its weight and of the value (2^-8 each), of the output, and by the score's error."""
    n = 400
    cache, table, q, lengths = _case(bs, 1, 2, 64, 32, 32, T, [n])
    cache.v_scales.mul_(2.0 ** -60)
    _put(cache, table, "v", 0, 0, 5, torch.randn(64, generator=ref.gen(3), device="cuda") * 2.0 ** 100)
    s = torch.tensor([0.01, 0.003], device="cuda") if slopes else None
    o, _ = bs.kv4_attn_chunk(cache, q, table, lengths, slopes=s)
    want, _, _, tol_l = ref.attn_chunk(cache, q, table, [n], slopes=s)
    assert bool(o.isfinite().all())
    tol = (2 * 2.0 ** -8 + UBF + 2 * tol_l[..., None]) * want.abs() + 2.0 ** -30 * want.abs().amax(-1, keepdim=True)
    assert bool(((o.double() - want).abs() <= tol).all()), float(((o.double() - want).abs() / tol).max())


@pytest.mark.parametrize("slopes", [False, True])
def test_values_far_below_those_of_later_tokens(bs, slopes):  # noqa: F811
    """Queries that see small values only, beside queries (of the same tiles) that see very large ones."""
    n = 200
    cache, table, q, lengths = _case(bs, 1, 1, 64, 64, 32, n, [n])
    cache.v_scales[table[0, :2].long()] *= 2.0 ** -30
    cache.v_scales[table[0, 2:4].long()] *= 2.0 ** 100
    s = torch.tensor([0.01], device="cuda") if slopes else None
    o, lse = bs.kv4_attn_chunk(cache, q, table, lengths, slopes=s)
    early = slice(0, 128)
    want = ref.attn_chunk(cache, q[:, :, early].contiguous(), table, [128], slopes=s, value_bits=8)
    _check((o[:, :, early], lse[:, :, early]), want)
    want = ref.attn_chunk(cache, q, table, [n], slopes=s, value_bits=8)
    assert bool(((o.double() - want[0]).abs()[:, :, 128:] <= (want[2][..., None] + UBF * want[0].abs())[:, :, 128:]).all())


def test_another_heads_slope_leaves_a_row_alone(bs):  # noqa: F811
    """12 heads: 16 rows in a row are 8 heads of one token and 8 of the next.  The prefix ends
    behind the first of the two tokens, so that only it sees keys behind itself."""
    G, T, B = 12, 12, 8
    lengths = [701 + 3 * b for b in range(B)]
    cache, table, q, n = _case(bs, 1, G, 64, 64, 32, T, lengths)
    prefix = _i32([m - T + 3 for m in lengths])  # token 1 sees token 2, which sees itself
    slopes = torch.tensor([0.37, 0.21, 0.13, 0.09] + [0.0] * 8, device="cuda")
    want = bs.kv4_attn_chunk(cache, q, table, n, prefix=prefix, slopes=slopes, out_f32=True)
    slopes[9] = 0.3
    got = bs.kv4_attn_chunk(cache, q, table, n, prefix=prefix, slopes=slopes, out_f32=True)
    assert not torch.equal(got[0][:, 9], want[0][:, 9])
    others = [h for h in range(G) if h != 9]
    assert torch.equal(got[1][:, others], want[1][:, others])
    assert torch.equal(got[0][:, others], want[0][:, others])


@pytest.mark.parametrize("option", [{}, dict(cap=20.0)], ids=["plain", "cap"])
def test_tables_much_wider_than_their_sequences(bs, option):  # noqa: F811
    lengths = [150, 700, 161]
    cache, table, q, n = _case(bs, 2, 2, 128, 64, 32, 150, lengths, columns=ROOM // 64)
    _check(bs.kv4_attn_chunk(cache, q, table, n, **option), ref.attn_chunk(cache, q, table, lengths, cap=option.get("cap")))


HEADS = [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32)]


@pytest.mark.parametrize("D,group", HEADS)
@pytest.mark.parametrize("n", [150, 2000])
@pytest.mark.parametrize("form", ["steps", "halves"])
def test_errors_by_norm(bs, D, group, n, form):  # noqa: F811
    """Weights and values are rounded to 11 bits each, independently: the root mean square of such a
    rounding is at most 2^-11 / sqrt(3) of the number, 2.8e-4, of both 4.0e-4, and of a sum over tokens with
    it.  (Rounded to 8 bits one of them alone would be 1.6e-3.)  A score sums D products in 9 steps of 32
    bits: off by at most 9 * 2^-23 of sum |q k| scale, here about 10, so by 1.1e-5, and a lse, which is a
    mean of those, by less."""
    cache, table, q, lengths = _case(bs, 2, 2, D, 64, group, 150, [n])
    more = dict(slopes=torch.zeros(4, device="cuda")) if form == "halves" else {}
    o, lse = bs.kv4_attn_chunk(cache, q, table, lengths, out_f32=True, **more)
    want, l_ref = ref.attn_chunk(cache, q, table, [n])[:2]
    off = float((o - want).norm() / want.norm())
    assert off <= 5e-4, off
    off = float((lse - l_ref).square().mean().sqrt())
    assert off <= 1.1e-5, off


@pytest.mark.parametrize("D,group", HEADS)
@pytest.mark.parametrize("form", ["steps", "halves"])
def test_keys_with_a_common_offset(bs, D, group, form):  # noqa: F811
    """Keys near 8, queries of one sign: scores near 100 are their groups' sums.  c and the sums of q are held
    to 2^-22 each, their low halves' product is left out (2^-22), the sums of q are 32-bit ones (7 * 2^-24):
    1.2e-6 of a score; 9 steps of 32 bits: 9 * 2^-23, 1.1e-6; the argument of exp2, its maximum and the lse: 5
    roundings of 2^-24, 0.3e-6.  Of 110 at most: 2.9e-4.  (High halves alone: 2^-12 of a score and more.)"""
    cache, table, q, lengths = _case(bs, 2, 2, D, 64, group, 150, [700])
    x = (8 + 0.5 * torch.randn(cache.pages, 2, 64, D, generator=ref.gen(8), device="cuda")).bfloat16()
    code, scales = ref.quantise(x, group)
    cache.k_codes.copy_(ref.pack(code))
    cache.k_scales.copy_(scales)
    q = q.abs()
    more = dict(slopes=torch.zeros(4, device="cuda")) if form == "halves" else {}
    lse = bs.kv4_attn_chunk(cache, q, table, lengths, **more)[1]
    l_ref = ref.attn_chunk(cache, q, table, [700])[1]
    off = float((lse - l_ref).square().mean().sqrt())
    assert off <= 3e-4, (off, float(l_ref.max()))
