"""The operators used together, as a model's step would use them: training
(projection -> norm + rotation -> chosen blocks -> attention -> gradients),
serving (prompt into the cache, then tokens), captured into graphs, on other
streams and several at once."""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

import _ops_ref as ref
from _ops_ref import UBF

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


def _model(B, S, H, Hkv, D, seed=1):
    g = ref.gen(seed)
    x = torch.randn(B, S, H + 2 * Hkv, D, generator=g, device="cuda")
    x = (x + 0.7 * torch.randn(B, S // 128 + 1, 1, H + 2 * Hkv, D, generator=g, device="cuda")
         .expand(-1, -1, 128, -1, -1).reshape(B, -1, H + 2 * Hkv, D)[:, :S]).bfloat16()
    w = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in "qk"]
    return x, w


def _attention(q, k, v, mask, causal):
    """64-bit attention over a block mask (differentiable)."""
    B, H, S, D = q.shape
    k, v = (t.repeat_interleave(H // t.shape[1], 1) for t in (k, v))
    s = q @ k.transpose(-1, -2) * D ** -0.5
    allowed = mask.bool().repeat_interleave(128, -2).repeat_interleave(S // mask.shape[-1], -1)
    if causal:
        allowed = allowed & torch.ones(S, S, dtype=torch.bool, device=q.device).tril()
    return torch.softmax(s.masked_fill(~allowed, float("-inf")), -1) @ v


def test_training_step(bs):
    """Chosen blocks equal the restatement's on the same q, k; gradients of the
    projection and the weights against 64-bit differentiation of the whole chain.

    Normwise: bf16 roundings of q, k, v, o (2^-8 each), of P and dS inside the
    attention's kernels and of dx itself: a handful of 2^-8, under 8 of them in
    the root mean square."""
    B, S, H, Hkv, D = 1, 1024, 4, 2, 64
    x, w = _model(B, S, H, Hkv, D)
    table = bs.rope_table(S, D)
    q, k, v = bs.qk_norm_rope(x, H, Hkv, *w, table)
    mask = bs.select_blocks(q, k, 4, causal=True, sink=1)
    assert torch.equal(mask, ref.select_blocks(q, k, 4, causal=True, sink=1))
    plan = bs.plan(mask, causal=True)
    o, lse = bs.fwd(q, k, v, plan)
    do = torch.randn(o.shape, generator=ref.gen(9), device="cuda").bfloat16()
    dx, dwq, dwk = bs.qk_norm_rope_bwd(x, *bs.bwd(q, k, v, o, lse, do, plan), *w, table)
    bs.plan_status(plan)
    plan.close()

    xd = x.double().requires_grad_()
    wd = [t.double().requires_grad_() for t in w]
    turn = ref.angles(table, None, B, S, D, False)
    qd, kd = (ref.norm_rope(xd[:, :, lo:hi], wt, 1e-6, turn)[0].transpose(1, 2)
              for lo, hi, wt in ((0, H, wd[0]), (H, H + Hkv, wd[1])))
    od = _attention(qd, kd, xd[:, :, H + Hkv:].transpose(1, 2), mask, True)
    od.backward(do.double())
    for got, want in ((o, od.detach()), (dx, xd.grad), (dwq, wd[0].grad), (dwk, wd[1].grad)):
        err = (got.double() - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert float(err) < 8 * UBF, float(err)


def _serve(bs, cache, table, x, w, rope, H, Hkv, lengths, counts=None, selected=None, T=None):
    """One step: rows of x at their positions into the cache, and the attention over it."""
    B, T = x.shape[:2]
    pos = (lengths[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")).contiguous()
    q, k, v = bs.qk_norm_rope(x, H, Hkv, *w, rope, pos)
    bs.kv4_append(cache, k, v, table, lengths, counts)
    return q, lengths + T


@pytest.mark.parametrize("group", [32, 64])
def test_serving(bs, group):
    """A prompt, then tokens: cache attention follows the 64-bit attention on the cache's values;
    the prompt's chosen blocks run through the forward pass on keys read back from the cache."""
    B, S, H, Hkv, D, page = 2, 384, 8, 2, 64, 16
    x, w = _model(B, S + 20, H, Hkv, D, seed=4)
    rope = bs.rope_table(S + 20, D)
    cache = bs.Kv4Cache(64, Hkv, D, page_size=page, group=group)
    table = ref.table(cache, [S + 20] * B, 30, 3)
    n = _i32([0] * B)
    q, n = _serve(bs, cache, table, x[:, :S], w, rope, H, Hkv, n)
    kr, vr = bs.kv4_read(cache, table, _i32([0] * B), S)
    mask = bs.select_blocks(q, kr, 2, causal=True)
    plan = bs.plan(mask, causal=True)
    o, _ = bs.fwd(q, kr, vr, plan)
    bs.plan_status(plan)
    plan.close()
    want = _attention(q.double(), kr.double(), vr.double(), mask, True)
    assert float((o.double() - want).abs().max()) < 2e-2  # the forward pass's own tolerance
    for i in range(20):
        q, n = _serve(bs, cache, table, x[:, S + i:S + i + 1], w, rope, H, Hkv, n)
        o, lse = bs.kv4_attn(cache, q, table, n, out_f32=True)
        lengths = [S + i + 1] * B
        o_ref, l_ref, tol_o, tol_l = ref.attn(cache, q, table, lengths)
        assert bool(((o.double() - o_ref).abs() <= tol_o[..., None] + 2.0 ** -24 * o_ref.abs()).all())
        pages = bs.kv4_select(cache, q, table, n, 6)
        assert torch.equal(pages, ref.select_pages(cache, q, table, lengths, 6, 1, 1))
        o, lse = bs.kv4_attn(cache, q, table, n, pages, out_f32=True)
        o_ref, l_ref, tol_o, tol_l = ref.attn(cache, q, table, lengths, pages)
        assert bool(((o.double() - o_ref).abs() <= tol_o[..., None] + 2.0 ** -24 * o_ref.abs()).all())
    bs.kv4_status(cache)


def test_decoding_step_in_a_graph(bs):
    """One captured step replayed along the sequences: lengths, positions and tables are read on
    the device, so the graph follows them; the same as calls one by one."""
    B, H, Hkv, D, page, steps = 3, 16, 4, 128, 16, 40
    start = [0, 15, 200]
    x, w = _model(B, steps, H, Hkv, D, seed=6)
    rope = bs.rope_table(400, D)

    def fresh():
        cache = bs.Kv4Cache(40, Hkv, D, page_size=page, group=128)
        ref.fill(cache, 2)
        return cache, ref.table(cache, [s + steps for s in start], 20, 5), _i32(start)

    def step(cache, table, n, xt):
        q, k, v = bs.qk_norm_rope(xt, H, Hkv, *w, rope, n[:, None].contiguous())
        bs.kv4_append(cache, k, v, table, n)
        n += 1
        pages = bs.kv4_select(cache, q, table, n, 4, recent=2)
        return bs.kv4_attn(cache, q, table, n, pages) + bs.kv4_attn(cache, q, table, n)

    cache, table, n = fresh()
    want = [[t.clone() for t in step(cache, table, n, x[:, i:i + 1].contiguous())] for i in range(steps)]
    bs.kv4_status(cache)
    cache, table, n = fresh()
    xt = x[:, :1].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = n.clone()
        step(cache, table, n, xt)
        n.copy_(keep)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(cache, table, n, xt)
    torch.cuda.current_stream().wait_stream(side)
    n.copy_(keep)
    for i in range(steps):
        xt.copy_(x[:, i:i + 1])
        graph.replay()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b), i
    bs.kv4_status(cache)


FIRST_USE = """
import torch
import block_sparse_flash_attn_gb300 as bs
cache = bs.Kv4Cache(64, 4, 128)
table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
n = torch.tensor([100, 700], dtype=torch.int32, device="cuda")
x = torch.randn(2, 256, 24, 128, device="cuda").bfloat16()
w = torch.ones(128, device="cuda")
dy = [torch.randn(2, h, 256, 128, device="cuda") for h in (16, 4, 4)]
rope = torch.randn(256, 64, 2, device="cuda")


def step():
    q, k, v = bs.qk_norm_rope(x, 16, 4, w, w, rope)
    mask = bs.select_blocks(q, k, 2)
    grads = bs.qk_norm_rope_bwd(x, *dy, w, w, rope)
    bs.kv4_append(cache, k, v, table, n)
    one = q[:, :, -1:].contiguous()
    pages = bs.kv4_select(cache, one, table, n + 256, 4)
    return (mask, pages) + grads + bs.kv4_attn(cache, one, table, n + 256, pages) + bs.kv4_attn(cache, one, table, n)


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


def test_training_step_in_a_graph(bs):
    B, S, H, Hkv, D = 2, 256, 4, 2, 128
    x, w = _model(B, S, H, Hkv, D, seed=8)
    table = bs.rope_table(S, D)
    q, k, v = bs.qk_norm_rope(x, H, Hkv, *w, table)
    plan = bs.plan(bs.select_blocks(q, k, 1, causal=True), causal=True)
    do = torch.randn(B, H, S, D, generator=ref.gen(2), device="cuda").bfloat16()

    def step(x):
        q, k, v = bs.qk_norm_rope(x, H, Hkv, *w, table)
        mask = bs.select_blocks(q, k, 1, causal=True)
        o, lse = bs.fwd(q, k, v, plan)
        return (mask, o) + tuple(bs.qk_norm_rope_bwd(x, *bs.bwd(q, k, v, o, lse, do, plan), *w, table))

    want = [t.clone() for t in step(x)]
    xs = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(xs)
    torch.cuda.current_stream().wait_stream(side)
    xs.copy_(x)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    bs.plan_status(plan)
    plan.close()


def test_streams(bs):
    """The same calls on a given stream, and two graphs of one cache replayed at once on two
    streams (each has its own workspace), give what the default stream gives."""
    H, Hkv, D, page = 8, 2, 128, 32
    lengths = [3000, 77, 900]
    cache = bs.Kv4Cache(140, Hkv, D, page_size=page, group=64)
    ref.fill(cache, 3)
    table = ref.table(cache, lengths, 100, 1)
    n = _i32(lengths)
    q = torch.randn(3, H, 1, D, generator=ref.gen(5), device="cuda").bfloat16()
    x, w = _model(2, 300, 4, 2, 64)
    rope = bs.rope_table(300, 64)
    grads = [torch.randn(2, h, 300, 64, generator=ref.gen(7), device="cuda") for h in (4, 2, 2)]

    def calls(stream=None):
        pages = bs.kv4_select(cache, q, table, n, 5, stream=stream)
        qkv = bs.qk_norm_rope(x, 4, 2, *w, rope, stream=stream)
        return (pages, *bs.kv4_attn(cache, q, table, n, pages, stream=stream),
                *bs.kv4_attn(cache, q, table, n, stream=stream), *bs.kv4_read(cache, table, n - 20, 20, stream=stream),
                *qkv, *bs.qk_norm_rope_bwd(x, *grads, *w, rope, stream=stream))

    want = calls()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = calls(sides[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for s in sides:
        with torch.cuda.stream(s):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                outs.append(calls())
    for _ in range(20):
        for s, graph in zip(sides, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    with pytest.raises(ValueError, match="stream"):
        class Elsewhere:
            device = torch.device("cuda", 7)
        bs.kv4_attn(cache, q, table, n, stream=Elsewhere())


def test_equal_calls_give_equal_bits(bs):
    """Nothing depends on the order in which CTAs run."""
    S, H, Hkv, D = 4096, 8, 2, 128
    x, w = _model(1, S, H, Hkv, D, seed=12)
    rope = bs.rope_table(S, D)
    q, k, v = bs.qk_norm_rope(x, H, Hkv, *w, rope)
    grads = [torch.randn(1, h, S, D, generator=ref.gen(7), device="cuda") for h in (H, Hkv, Hkv)]
    cache = bs.Kv4Cache(70, Hkv, D)
    table = ref.table(cache, [S], 64, 0)
    bs.kv4_append(cache, k, v, table, _i32([0]))
    n = _i32([S])
    qt = q[:, :, -1:].contiguous()

    def calls():
        return (bs.select_blocks(q, k, 5), *bs.qk_norm_rope_bwd(x, *grads, *w, rope),
                *bs.kv4_attn(cache, qt, table, n), bs.kv4_select(cache, qt, table, n, 9))

    want = calls()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(calls(), want))
    assert np.isfinite(want[1].float().cpu().numpy()).all()
