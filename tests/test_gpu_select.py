"""Block masks chosen by block means: equal to the 64-bit restatement, entry by
entry (scores are exact by construction, ties go to the lowest index)."""
import pytest
import torch

import _ops_ref as ref

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


def _qk(B, H, Hkv, S, D, seed=1, topic=0.5):
    g = ref.gen(seed)
    out = []
    for h in (H, Hkv):
        x = torch.randn(B, h, S // 128, 128, D, generator=g, device="cuda")
        x += topic * torch.randn(B, h, S // 128, 1, D, generator=g, device="cuda")
        out.append(x.view(B, h, S, D).bfloat16())
    return out


#        B  H  Hkv S      D   kb   keep causal sink local
CASES = [
    (1, 2, 2, 128, 64, 128, 1, False, 0, 1),
    (1, 1, 1, 128, 128, 64, 1, True, 0, 0),
    (2, 4, 2, 1664, 64, 64, 5, False, 1, 1),
    (1, 3, 1, 2176, 128, 128, 4, True, 2, 2),
    (1, 2, 1, 8192, 64, 64, 13, True, 0, 0),       # 128 key blocks: 4 keys a lane and more
    (1, 1, 1, 33280, 64, 64, 40, False, 3, 1),     # 520 key blocks: keys from shared memory
    (1, 1, 1, 65664, 128, 128, 52, True, 1, 2),    # 513 query blocks
    (1, 2, 2, 1024, 128, 128, 100, True, 0, 1),    # more than there are
    (1, 2, 2, 1024, 128, 128, 1, False, 3, 2),     # fewer than are forced
    (2, 40, 8, 2176, 64, 128, 3, True, 1, 1),      # tiles of 16 rows, and of one
    (1, 80, 4, 2688, 128, 64, 6, False, 0, 1),     # of 16 and 5
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_mask(bs, case):
    B, H, Hkv, S, D, kb, keep, causal, sink, local = case
    q, k = _qk(B, H, Hkv, S, D)
    kw = dict(causal=causal, key_block=kb, sink=sink, local=local)
    got = bs.select_blocks(q, k, keep, **kw)
    assert torch.equal(got, ref.select_blocks(q, k, keep, **kw))


def test_widest_masks(bs):
    """More key blocks than 16 rows of keys fit in shared memory (4 rows a CTA)."""
    q, k = _qk(1, 1, 1, 128 * 1030, 64)
    got = bs.select_blocks(q, k, 77, causal=True, key_block=64, sink=1)
    assert torch.equal(got, ref.select_blocks(q, k, 77, causal=True, key_block=64, sink=1))


@pytest.mark.parametrize("shared", [False, True])
def test_blocks_ruled_out(bs, shared):
    B, H, S = 2, 4, 1280
    q, k = _qk(B, H, 2, S, 64)
    allow = (torch.rand(B, 1 if shared else H, 10, 10, generator=ref.gen(4), device="cuda") < 0.4)
    allow = (allow * 3).to(torch.uint8)  # any nonzero value allows
    allow[1, 0, 7] = 0                   # a row with nothing left
    for causal in (False, True):
        got = bs.select_blocks(q, k, 3, causal=causal, sink=1, allow=allow)
        assert torch.equal(got, ref.select_blocks(q, k, 3, causal=causal, sink=1, allow=allow))
        assert not bool(got[1, 0, 7].any())


def test_ties_go_to_the_lowest_index(bs):
    """Equal blocks: constant inputs, and blocks repeated."""
    S, D = 1280, 64
    one = torch.ones(1, 1, S, D, dtype=torch.bfloat16, device="cuda")
    got = bs.select_blocks(one, one, 4, local=0)
    assert bool((got[0, 0, :, :4] == 1).all()) and not bool(got[0, 0, :, 4:].any())
    zero = torch.zeros_like(one)
    assert torch.equal(bs.select_blocks(zero, zero, 4, local=0), got)
    assert torch.equal(bs.select_blocks(one, -one, 4, local=0), got)
    q, k = _qk(1, 1, 1, S, D)
    k = k[:, :, :256].repeat(1, 1, 5, 1).contiguous()
    got = bs.select_blocks(q, k, 3, local=0)
    assert torch.equal(got, ref.select_blocks(q, k, 3, local=0))
    assert torch.equal(bs.select_blocks(q, k, 3, key_block=64, local=0),
                       ref.select_blocks(q, k, 3, key_block=64, local=0))


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1.0, 1e10, 1e31])
def test_sizes_of_values(bs, scale):
    """Wide ranges of values, means on rounding borders."""
    q, k = _qk(1, 2, 1, 1024, 64, seed=3, topic=0.0)
    wide = torch.exp2(torch.randint(-12, 3, (1, 1, 1, 64), generator=ref.gen(9), device="cuda").float())
    q, k = ((x.float() * wide * scale).bfloat16() for x in (q, k))
    for kb in (64, 128):
        assert torch.equal(bs.select_blocks(q, k, 2, key_block=kb, local=0),
                           ref.select_blocks(q, k, 2, key_block=kb, local=0))
    # small whole numbers: many means fall exactly between two 7-bit values
    q, k = (torch.randint(-3, 4, x.shape, generator=ref.gen(2), device="cuda").bfloat16() for x in (q, k))
    assert torch.equal(bs.select_blocks(q, k, 2, local=0), ref.select_blocks(q, k, 2, local=0))


def test_values_that_are_not_finite_count_as_zero(bs):
    q, k = _qk(1, 1, 1, 1024, 64)
    k[0, 0, 130, 3] = float("inf")
    k[0, 0, 300, 5] = float("nan")
    q[0, 0, 0, 0] = float("-inf")
    k[0, 0, 512:640] = float("nan")
    got = bs.select_blocks(q, k, 3, local=0)
    assert torch.equal(got, ref.select_blocks(q, k, 3, local=0))


def test_given_output_and_refusals(bs):
    q, k = _qk(1, 4, 2, 256, 64)
    out = torch.full((1, 4, 2, 2), 7, dtype=torch.uint8, device="cuda")
    got = bs.select_blocks(q, k, 1, causal=True, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, ref.select_blocks(q, k, 1, causal=True))
    with pytest.raises(ValueError, match="keep"):
        bs.select_blocks(q, k, 0)
    with pytest.raises(ValueError, match="key_block"):
        bs.select_blocks(q, k, 1, key_block=32)
    with pytest.raises(ValueError, match="Hkv"):
        bs.select_blocks(q, torch.cat([k, k[:, :1]], 1), 1)
    with pytest.raises(ValueError, match="multiple of 128"):
        bs.select_blocks(q[:, :, :200].contiguous(), k[:, :, :200].contiguous(), 1)
    with pytest.raises(ValueError, match="contiguous"):
        bs.select_blocks(q.transpose(2, 3).contiguous().transpose(2, 3), k, 1)
    with pytest.raises(ValueError, match="allow"):
        bs.select_blocks(q, k, 1, allow=torch.ones(1, 2, 2, 2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="allow"):
        bs.select_blocks(q, k, 1, allow=torch.ones(1, 1, 2, 2, device="cuda"))
    with pytest.raises(TypeError):
        bs.select_blocks(q.float(), k.float(), 1)


@pytest.mark.parametrize("key_block", [128, 64])
def test_empty_batch(bs, key_block):
    """No batch entries: an empty mask, as the operators around it give empty results."""
    q, k = (torch.zeros(0, h, 256, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    mask = bs.select_blocks(q, k, 1, key_block=key_block)
    assert mask.shape == (0, 4, 2, 256 // key_block) and mask.dtype == torch.uint8
    allow = torch.zeros(0, 1, 2, 256 // key_block, dtype=torch.uint8, device="cuda")
    assert bs.select_blocks(q, k, 1, key_block=key_block, allow=allow, out=mask) is mask
    with pytest.raises(ValueError, match="keep"):
        bs.select_blocks(q, k, 0)
