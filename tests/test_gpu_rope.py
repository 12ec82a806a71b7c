"""Norm + rotation and its gradient against 64-bit restatements.

Tolerances count roundings (U32 = 2^-24, UBF = 2^-8, half a step each):
forward: the row's sum of squares, root, two products and the rotation are
within 24 U32 of the sum of the two rotated terms' sizes, then one rounding to
bf16.  Backward: two row sums instead of one: 48 U32 of the terms' sizes.  The
weight gradients are sums of n rows in some order: (n + 48) U32 of the sum of
the terms' sizes."""
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


def _inputs(B, S, H, Hkv, D, wdtype, given, rot, seed=1, far=5000):
    g = ref.gen(seed)
    heads = H + 2 * Hkv
    x = (torch.randn(B, S, heads, D, generator=g, device="cuda") * 2).bfloat16()
    w = [None, None]
    if wdtype is not None:
        w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(wdtype) for _ in "qk"]
    pos = None
    if given:
        pos = torch.randint(0, far, (B, S), generator=g, device="cuda").to(torch.int32)
    return x, w, pos


def _close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.equal(got.isnan(), want.isnan()), what
    err = (got - want).abs().nan_to_num(0.0)
    assert bool((err <= tol.nan_to_num(0.0) + 1e-300).all()), (what, (err / (tol + 1e-300)).nan_to_num(0.0).max())


#       B  S    H  Hkv D    weights         rot  inter given
CASES = [
    (2, 37, 4, 2, 128, torch.bfloat16, 128, False, False),
    (1, 1, 8, 1, 128, torch.float32, 128, False, True),
    (3, 5, 1, 1, 64, torch.bfloat16, 64, True, True),
    (2, 130, 5, 5, 64, torch.float32, 32, False, True),
    (1, 259, 6, 3, 128, torch.bfloat16, 64, True, False),
    (64, 1, 32, 8, 128, torch.bfloat16, 128, False, True),
    (1, 17, 3, 1, 128, None, 16, False, True),
    (2, 9, 2, 1, 64, torch.bfloat16, 0, False, False),
    (1, 4, 2, 2, 128, None, 0, False, False),
    (1, 2000, 7, 7, 64, torch.bfloat16, 48, False, False),
]


def _case(bs, case):
    B, S, H, Hkv, D, wdtype, rot, inter, given = case
    x, w, pos = _inputs(B, S, H, Hkv, D, wdtype, given and rot > 0, rot)
    table = bs.rope_table(5000, rot) if rot else None
    turn = ref.angles(table, pos, B, S, D, inter) if rot else None
    return x, w, pos, table, turn


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(bs, case):
    B, S, H, Hkv, D, _, _, inter, _ = case
    x, w, pos, table, turn = _case(bs, case)
    q, k, v = bs.qk_norm_rope(x, H, Hkv, *w, table, pos, interleaved=inter)
    for got, lo, hi, wt in ((q, 0, H, w[0]), (k, H, H + Hkv, w[1])):
        want, size = ref.norm_rope(x[:, :, lo:hi], wt, 1e-6, turn)
        _close(got, want.transpose(1, 2), (UBF * want.abs() + 24 * U32 * size).transpose(1, 2), case)
    assert torch.equal(v, x[:, :, H + Hkv:].transpose(1, 2))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradient(bs, case):
    B, S, H, Hkv, D, _, _, inter, _ = case
    x, w, pos, table, turn = _case(bs, case)
    g = ref.gen(7)
    dq, dk, dv = (torch.randn(B, h, S, D, generator=g, device="cuda") for h in (H, Hkv, Hkv))
    dx, dwq, dwk = bs.qk_norm_rope_bwd(x, dq, dk, dv, *w, table, pos, interleaved=inter)
    assert dx.shape == x.shape and dx.is_contiguous()
    for lo, hi, d, wt, dw in ((0, H, dq, w[0], dwq), (H, H + Hkv, dk, w[1], dwk)):
        want, want_w, size, size_w = ref.norm_rope_bwd(x[:, :, lo:hi], d.transpose(1, 2), wt, 1e-6, turn)
        _close(dx[:, :, lo:hi], want, UBF * want.abs() + 48 * U32 * size, case)
        if wt is None:
            assert dw is None
        else:
            _close(dw, want_w, (B * S * (hi - lo) + 48) * U32 * size_w, case)
    assert torch.equal(dx[:, :, H + Hkv:], dv.transpose(1, 2).bfloat16())
    again = bs.qk_norm_rope_bwd(x, dq, dk, dv, *w, table, pos, interleaved=inter)
    assert all(a is b or torch.equal(a, b) for a, b in zip((dx, dwq, dwk), again))


def test_gradient_against_differences(bs):
    """The 64-bit formula that the kernel is held to, against central differences of the forward formula."""
    g = ref.gen(3)
    x = torch.randn(1, 2, 1, 64, generator=g, device="cuda", dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(64, generator=g, device="cuda", dtype=torch.float64)
    up = torch.randn(1, 2, 1, 64, generator=g, device="cuda", dtype=torch.float64)
    turn = ref.angles(bs.rope_table(9, 32), None, 1, 2, 64, True)
    dx, dw, _, _ = ref.norm_rope_bwd(x, up, w, 1e-6, turn)

    def loss(x, w):
        return float((ref.norm_rope(x, w, 1e-6, turn)[0] * up).sum())

    h = 1e-5  # error of a central difference: h^2 times third derivatives, of order 1: 1e-8
    for i in range(0, 64, 5):
        e = torch.zeros_like(x)
        e[0, 1, 0, i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - float(dx[0, 1, 0, i])) < 1e-7
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - float(dw[i])) < 1e-7


def test_strided_projection_and_given_outputs(bs):
    """x as part of a wider projection, outputs in given tensors, dx in place of x."""
    B, S, H, Hkv, D = 2, 33, 4, 2, 64
    wide = torch.randn(S, B, 12, D, generator=ref.gen(5), device="cuda").bfloat16()
    x = wide.transpose(0, 1)[:, :, 2:2 + H + 2 * Hkv]
    table = bs.rope_table(64, D)
    want = bs.qk_norm_rope(x.contiguous(), H, Hkv, table=table)
    outs = [torch.empty_like(t) for t in want]
    got = bs.qk_norm_rope(x, H, Hkv, table=table, q=outs[0], k=outs[1], v=outs[2])
    for a, b, o in zip(got, want, outs):
        assert torch.equal(a, b) and a.data_ptr() == o.data_ptr()
    grads = [torch.randn(B, h, S, D, device="cuda") for h in (H, Hkv, Hkv)]
    w = [torch.ones(D, device="cuda") for _ in "qk"]
    dx = bs.qk_norm_rope_bwd(x, *grads, *w, table)[0]
    xc = x.contiguous()
    own = bs.qk_norm_rope_bwd(xc, *grads, *w, table, dx=xc)[0]
    assert own.data_ptr() == xc.data_ptr() and torch.equal(own, dx)


def test_positions_outside_the_table_are_nan(bs):
    B, S, H, D = 1, 6, 2, 64
    x = torch.randn(B, S, 3 * H, D, generator=ref.gen(5), device="cuda").bfloat16()
    pos = torch.tensor([[0, -1, 9, 10, 2 ** 31 - 1, 3]], dtype=torch.int32, device="cuda")
    q, k, v = bs.qk_norm_rope(x, H, H, table=bs.rope_table(10, 32), positions=pos)
    bad = torch.tensor([False, True, False, True, True, False], device="cuda")
    for t in (q, k):
        assert bool(t[:, :, bad, :32].isnan().all()) and not bool(t[:, :, ~bad].isnan().any())
        assert not bool(t[:, :, :, 32:].isnan().any())
    assert not bool(v.isnan().any())


def test_table_far_positions(bs):
    """Angles of far positions keep 32-bit cos and sin: half a step each (and 64-bit rounding)."""
    n, rot = 300000, 128
    t = bs.rope_table(n, rot, theta=500000.0).double()
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    assert float((t[..., 0].cpu() - a.cos()).abs().max()) <= U32 + 1e-10
    assert float((t[..., 1].cpu() - a.sin()).abs().max()) <= U32 + 1e-10
    own = bs.rope_table(7, 32, inv_freq=torch.linspace(1, 0.01, 16))
    a = torch.arange(7, dtype=torch.float64)[:, None] * torch.linspace(1, 0.01, 16).double()
    assert float((own[..., 1].double().cpu() - a.sin()).abs().max()) <= U32 + 1e-10


def test_extreme_rows(bs):
    """A zero row stays zero (eps), a row with an infinity or NaN spoils itself only."""
    x = torch.randn(1, 4, 3, 64, generator=ref.gen(8), device="cuda").bfloat16()
    x[0, 0, 0] = 0
    x[0, 1, 0, 5] = float("inf")
    x[0, 2, 1, 7] = float("nan")
    w = [torch.ones(64, device="cuda")] * 2
    q, k, v = bs.qk_norm_rope(x, 1, 1, *w)
    assert bool((q[0, 0, 0] == 0).all())
    assert bool(k[0, 0, 2].isnan().all()) and bool(q[0, 0, 1].isnan().any())
    assert not bool(q[0, 0, 2:].isnan().any()) and not bool(k[0, 0, [0, 1, 3]].isnan().any())
    g = [torch.ones(1, 1, 4, 64, device="cuda") for _ in range(3)]
    dx = bs.qk_norm_rope_bwd(x, *g, *w)[0]
    assert not bool(dx[0, 0].isnan().any()) and not bool(dx[0, 3].isnan().any())


def test_infinities_pass_where_nothing_turns_them(bs):
    """Without norm, channels that are not rotated are copied, infinities too."""
    x = torch.randn(1, 3, 3, 64, generator=ref.gen(8), device="cuda").bfloat16()
    x[0, 1, 0, 40] = float("inf")
    for table in (None, bs.rope_table(3, 32)):
        for inter in (False, True):
            q, _, _ = bs.qk_norm_rope(x, 1, 1, table=table, interleaved=inter)
            assert float(q[0, 0, 1, 40]) == float("inf") and int(q.isfinite().sum()) == q.numel() - 1


def test_no_tokens(bs):
    table = bs.rope_table(4, 64)
    x = torch.empty(2, 0, 6, 64, dtype=torch.bfloat16, device="cuda")
    w = [torch.ones(64, device="cuda")] * 2
    q, k, v = bs.qk_norm_rope(x, 2, 2, *w, table)
    assert q.shape == k.shape == v.shape == (2, 2, 0, 64)
    g = [torch.empty(2, 2, 0, 64, device="cuda")] * 3
    dx, dwq, dwk = bs.qk_norm_rope_bwd(x, *g, *w, table)
    assert dx.shape == x.shape and not dwq.any() and not dwk.any()


def test_refusals(bs):
    x = torch.zeros(1, 4, 6, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    table = bs.rope_table(3, 64)
    with pytest.raises(ValueError, match="table has 3 positions"):
        bs.qk_norm_rope(x, 2, 2, table=table)
    with pytest.raises(ValueError, match="together"):
        bs.qk_norm_rope(x, 2, 2, w)
    with pytest.raises(ValueError, match="heads"):
        bs.qk_norm_rope(x, 3, 2)
    with pytest.raises(ValueError, match="heads"):
        bs.qk_norm_rope(x, 4, 2)
    with pytest.raises(TypeError, match="bfloat16"):
        bs.qk_norm_rope(x.float(), 2, 2)
    with pytest.raises(TypeError, match="q_weight"):
        bs.qk_norm_rope(x, 2, 2, w.half(), w.half())
    with pytest.raises(TypeError, match="k_weight"):
        bs.qk_norm_rope(x, 2, 2, w, w.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        bs.qk_norm_rope(x.transpose(1, 2).contiguous().transpose(1, 2), 2, 2)
    with pytest.raises(TypeError, match="int32"):
        bs.qk_norm_rope(x, 2, 2, table=table, positions=torch.zeros(1, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="positions need"):
        bs.qk_norm_rope(x, 2, 2, positions=torch.zeros(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="cuda"):
        bs.qk_norm_rope(x, 2, 2, w.cpu(), w.cpu())
    with pytest.raises(ValueError, match="shape"):
        bs.qk_norm_rope_bwd(x, *[torch.zeros(1, 2, 5, 64, device="cuda")] * 3)
    with pytest.raises(ValueError):
        bs.rope_table(10, 24)
    with pytest.raises(bs.BsattnError):
        bs.qk_norm_rope(x, 2, 2, w, w, eps=float("nan"))


@pytest.mark.parametrize("eps", [0.0, 1e-30, 0.01])
@pytest.mark.parametrize("H, Hkv, D", [(32, 4, 128), (16, 4, 64), (5, 5, 128), (5, 1, 64), (1, 1, 64), (3, 3, 128)], ids=str)
def test_other_eps(bs, H, Hkv, D, eps):
    """eps from zero on, with numbers of heads that leave a warp's rows empty."""
    B, S = 2, 37
    x, w, _ = _inputs(B, S, H, Hkv, D, torch.float32, False, 0)
    g = ref.gen(7)
    dq, dk, dv = (torch.randn(B, h, S, D, generator=g, device="cuda") for h in (H, Hkv, Hkv))
    q, k, _ = bs.qk_norm_rope(x, H, Hkv, *w, eps=eps)
    dx, dwq, dwk = bs.qk_norm_rope_bwd(x, dq, dk, dv, *w, eps=eps)
    for lo, hi, y, d, wt, dw in ((0, H, q, dq, w[0], dwq), (H, H + Hkv, k, dk, w[1], dwk)):
        want, size = ref.norm_rope(x[:, :, lo:hi], wt, eps, None)
        _close(y, want.transpose(1, 2), (UBF * want.abs() + 24 * U32 * size).transpose(1, 2), eps)
        want, want_w, size, size_w = ref.norm_rope_bwd(x[:, :, lo:hi], d.transpose(1, 2), wt, eps, None)
        _close(dx[:, :, lo:hi], want, UBF * want.abs() + 48 * U32 * size, eps)
        _close(dw, want_w, (B * S * (hi - lo) + 48) * U32 * size_w, eps)


def test_gradient_between_the_rows_of_its_input(bs):
    """dx beside x in one buffer, row by row: allowed where the rows lie apart, refused elsewhere."""
    B, S, H, Hkv, D = 3, 50, 4, 2, 64
    row = (H + 2 * Hkv) * D
    x, w, _ = _inputs(B, S, H, Hkv, D, torch.float32, False, 0)
    g = ref.gen(7)
    grads = [torch.randn(B, h, S, D, generator=g, device="cuda") for h in (H, Hkv, Hkv)]
    want = bs.qk_norm_rope_bwd(x, *grads, *w)
    lib, on = bs.load(), torch.cuda.current_stream().cuda_stream
    ws = torch.empty(lib.bsattn_qk_norm_rope_bwd_workspace(B, S, H, Hkv, D), dtype=torch.uint8, device="cuda")
    dw = torch.empty(2, D, device="cuda")
    both = torch.zeros(B, S, 2, row, dtype=torch.bfloat16, device="cuda")
    both[:, :, 0] = x.flatten(2)

    def call(dx):
        t = both.data_ptr()
        return lib.bsattn_qk_norm_rope_bwd(
            t, 2 * S * row, 2 * row, *(d.data_ptr() for d in grads), B, S, H, Hkv, D, *(v.data_ptr() for v in w), None,
            0, 0, None, 1e-6, bs_weight_f32, t + 2 * dx, 2 * S * row, 2 * row, dw[0].data_ptr(), dw[1].data_ptr(),
            ws.data_ptr(), ws.numel(), on)

    from block_sparse_flash_attn_gb300.rope import WEIGHT_F32 as bs_weight_f32
    assert call(row) == bs.OK
    assert torch.equal(both[:, :, 1].view_as(x), want[0]) and torch.equal(both[:, :, 0].view_as(x), x)
    assert torch.equal(dw[0], want[1]) and torch.equal(dw[1], want[2])
    for near in (8, row - 8, row + 8):
        assert call(near) == bs.ERR_INVALID_ARG
    flat = torch.empty(x.numel() + 8, dtype=torch.bfloat16, device="cuda")
    flat[:-8] = x.flatten()
    with pytest.raises(bs.BsattnError, match="invalid argument"):
        bs.qk_norm_rope_bwd(flat[:-8].view_as(x), *grads, *w, dx=flat[8:].view_as(x))
    assert torch.equal(bs.qk_norm_rope_bwd(flat[:-8].view_as(x), *grads, *w, dx=flat[:-8].view_as(x))[0], want[0])


@pytest.mark.parametrize("B, S", [(1, 3), (3, 1), (1, 1)], ids=str)
def test_given_dx_with_any_stride_along_one_entry(bs, B, S):
    """A contiguous dx; the stride of an axis of one entry means nothing."""
    x, w, _ = _inputs(B, S, 2, 2, 64, torch.float32, False, 0)
    dy = [torch.randn(B, 2, S, 64, generator=ref.gen(2), device="cuda") for _ in range(3)]
    want = bs.qk_norm_rope_bwd(x, *dy, *w)
    dx = torch.empty(B * S * 384, dtype=torch.bfloat16, device="cuda")
    dx = dx.as_strided((B, S, 6, 64), (384 * S if B > 1 else 3, 384 if S > 1 else 5, 64, 1))
    assert dx.is_contiguous()
    got = bs.qk_norm_rope_bwd(x, *dy, *w, dx=dx)
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, want))
    own = x.clone().as_strided(x.shape, dx.stride())
    assert torch.equal(bs.qk_norm_rope_bwd(own, *dy, *w, dx=own)[0], want[0])
