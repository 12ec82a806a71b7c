"""Host-side checks of the operators around the attention (no GPU needed): every
bad argument is turned away before anything is launched."""
import ctypes

import pytest

vp = ctypes.c_void_p
FAKE = vp(0x10000)
ODD = vp(0x10008)  # not 16-byte aligned


@pytest.fixture(scope="module")
def bs():
    from block_sparse_flash_attn_gb300 import _build
    _build.build()
    import block_sparse_flash_attn_gb300 as bs
    bs.load()
    return bs


def _call(fn, good, **changes):
    args = dict(good)
    for name, value in changes.items():
        assert name in args, name
        args[name] = value
    return fn(*args.values())


ROPE = dict(x=FAKE, xb=1024, xs=512, B=1, S=2, H=4, Hkv=2, D=64, wq=FAKE, wk=FAKE, table=FAKE, n_pos=8,
            rot=64, pos=FAKE, eps=1e-6, flags=0)
ROPE_BAD = [
    (dict(x=None), 1), (dict(x=ODD), 1), (dict(B=0), 1), (dict(S=0), 1), (dict(H=3), 1), (dict(Hkv=0), 1),
    (dict(D=96), 2), (dict(xs=12), 1), (dict(xb=-8), 1), (dict(wq=None), 1), (dict(wk=ODD), 1),
    (dict(table=ODD), 1), (dict(n_pos=0), 1), (dict(rot=0), 1), (dict(rot=80), 1), (dict(rot=24), 2),
    (dict(pos=None, S=9), 1), (dict(pos=vp(0x10002)), 1), (dict(flags=4), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(B=1 << 20, S=1 << 12), 2),
    (dict(B=1 << 15, S=1 << 14), 2),
]


@pytest.mark.parametrize("change,status", ROPE_BAD, ids=lambda c: str(c))
def test_norm_rope(bs, change, status):
    lib = bs.load()
    fwd = dict(ROPE, q=FAKE, k=FAKE, v=FAKE, stream=None)
    assert _call(lib.bsattn_qk_norm_rope, fwd, **change) == status
    bwd = {}
    for name, value in ROPE.items():
        bwd[name] = value
        if name == "xs":
            bwd.update(dq=FAKE, dk=FAKE, dv=FAKE)
    bwd.update(dx=FAKE, dxb=1024, dxs=512, dwq=FAKE, dwk=FAKE, ws=FAKE, nbytes=1 << 30, stream=None)
    assert _call(lib.bsattn_qk_norm_rope_bwd, bwd, **change) == status


def test_norm_rope_outputs(bs):
    lib = bs.load()
    fwd = dict(ROPE, q=FAKE, k=FAKE, v=FAKE, stream=None)
    for name in "qkv":
        assert _call(lib.bsattn_qk_norm_rope, fwd, **{name: None}) == bs.ERR_INVALID_ARG
        assert _call(lib.bsattn_qk_norm_rope, fwd, **{name: ODD}) == bs.ERR_INVALID_ARG
    assert lib.bsattn_rope_table(None, 4, 64, FAKE, None) == bs.ERR_INVALID_ARG
    assert lib.bsattn_rope_table(FAKE, 0, 64, FAKE, None) == bs.ERR_INVALID_ARG
    assert lib.bsattn_rope_table(FAKE, 4, 24, FAKE, None) == bs.ERR_UNSUPPORTED
    assert lib.bsattn_rope_table(FAKE, 4, 144, FAKE, None) == bs.ERR_UNSUPPORTED
    args = [FAKE, 1024, 512, FAKE, FAKE, FAKE, 2, 2, 4, 2, 64, None, None, None, 0, 0, None, 1e-6, 0]
    tail = [None, None, None, 0, None]
    for dx, dxb, dxs in ((None, 1024, 512), (ODD, 1024, 512), (FAKE, 1024, 504), (FAKE, 1016, 512),
                         (FAKE, 1024, 516), (FAKE, -1024, 512)):
        assert lib.bsattn_qk_norm_rope_bwd(*args, dx, dxb, dxs, *tail) == bs.ERR_INVALID_ARG


SELECT = dict(q=FAKE, k=FAKE, B=1, H=4, Hkv=2, S=256, D=64, keep=1, sink=0, local=1, flags=0, allow=None,
              allow_heads=0, mask=FAKE, ws=FAKE, nbytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(k=ODD), 1), (dict(mask=None), 1), (dict(ws=None), 1), (dict(ws=ODD), 1),
    (dict(S=200), 1), (dict(S=0), 1), (dict(H=3), 1), (dict(Hkv=0), 1), (dict(D=32), 2), (dict(keep=0), 1),
    (dict(sink=-1), 1), (dict(local=-1), 1), (dict(flags=2), 1), (dict(allow=FAKE, allow_heads=2), 1),
    (dict(nbytes=64), 1), (dict(S=128 * 4097), 2), (dict(B=4096, S=128 * 4096), 2), (dict(B=65536), 2)],
    ids=lambda c: str(c))
def test_select_blocks(bs, change, status):
    assert _call(bs.load().bsattn_select_blocks, SELECT, **change) == status


def _cache(**changes):
    from block_sparse_flash_attn_gb300 import kv4
    f = dict(k_codes=0x10000, v_codes=0x10000, k_scales=0x10000, v_scales=0x10000, k_means=0x10000,
             status=0x10000, pages=4, kv_heads=2, page_size=16, head_dim=64, group=32)
    f.update(changes)
    return kv4._CacheStruct(**f)


APPEND = dict(cache=None, k=FAKE, kb=1024, kh=512, kt=64, v=FAKE, vb=1024, vh=512, vt=64, B=1, T=1, table=FAKE,
              stride=4, columns=4, lengths=FAKE, counts=None, stream=None)
READ = dict(cache=None, B=1, T=1, table=FAKE, stride=4, columns=4, start=FAKE, counts=None, k=FAKE, v=FAKE,
            stream=None)
PAGES = dict(cache=None, q=FAKE, B=1, H=4, T=1, table=FAKE, stride=4, columns=4, lengths=FAKE, keep=4, sink=1,
             recent=1, out=FAKE, ws=FAKE, nbytes=1 << 30, stream=None)
ATTN = dict(cache=None, q=FAKE, B=1, H=4, T=1, table=FAKE, stride=4, columns=4, lengths=FAKE, selected=None, n=0,
            scale=0.1, flags=0, out=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(k_codes=None), 1), (dict(v_scales=0x10008), 1), (dict(status=None), 1), (dict(status=0x10002), 1),
    (dict(pages=0), 1), (dict(kv_heads=0), 1), (dict(kv_heads=32768), 2), (dict(page_size=8), 2),
    (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(head_dim=96), 2), (dict(group=16), 2),
    (dict(group=128), 1)], ids=lambda c: str(c))
def test_caches(bs, change, status):
    lib = bs.load()
    c = _cache(**change)
    ref = ctypes.byref(c)
    for fn, good in ((lib.bsattn_kv4_append, APPEND), (lib.bsattn_kv4_read, READ), (lib.bsattn_kv4_select, PAGES),
                     (lib.bsattn_kv4_attn, ATTN)):
        assert _call(fn, good, cache=ref) == status
        assert _call(fn, good, cache=None) == bs.ERR_INVALID_ARG
    assert lib.bsattn_kv4_status(ref, None) == status
    assert lib.bsattn_kv4_status(None, None) == bs.ERR_INVALID_ARG


@pytest.mark.parametrize("call,good,change,status", [
    ("append", APPEND, dict(k=None), 1), ("append", APPEND, dict(v=ODD), 1), ("append", APPEND, dict(kt=4), 1),
    ("append", APPEND, dict(vh=-8), 1), ("append", APPEND, dict(T=0), 1), ("append", APPEND, dict(columns=0), 1),
    ("append", APPEND, dict(lengths=None), 1), ("append", APPEND, dict(counts=vp(0x10001)), 1),
    ("append", APPEND, dict(B=65536), 2), ("append", APPEND, dict(stride=-4), 1),
    ("read", READ, dict(k=None), 1), ("read", READ, dict(v=ODD), 1), ("read", READ, dict(start=None), 1),
    ("read", READ, dict(T=0), 1), ("read", READ, dict(B=1 << 16), 2), ("read", READ, dict(T=(1 << 30) + 1), 2),
    ("select", PAGES, dict(q=ODD), 1), ("select", PAGES, dict(H=3), 1), ("select", PAGES, dict(T=65), 2),
    ("select", PAGES, dict(keep=1), 1), ("select", PAGES, dict(recent=0), 1), ("select", PAGES, dict(sink=-1), 1),
    ("select", PAGES, dict(columns=20000, stride=20000, nbytes=8), 1), ("select", PAGES, dict(out=None), 1),
    ("attn", ATTN, dict(q=None), 1), ("attn", ATTN, dict(out=ODD), 1), ("attn", ATTN, dict(lse=None), 1),
    ("attn", ATTN, dict(T=65), 2), ("attn", ATTN, dict(scale=float("nan")), 1), ("attn", ATTN, dict(flags=1), 1),
    ("attn", ATTN, dict(selected=FAKE), 1), ("attn", ATTN, dict(n=3), 1), ("attn", ATTN, dict(H=0), 1),
    ("attn", ATTN, dict(table=None), 1), ("attn", ATTN, dict(columns=1 << 27), 2), ("attn", ATTN, dict(B=4097), 2),
    ("attn", ATTN, dict(H=5), 1)], ids=lambda c: str(c) if len(str(c)) < 40 else "")
def test_cache_calls(bs, call, good, change, status):
    c = _cache()
    assert _call(getattr(bs.load(), "bsattn_kv4_" + call), good, cache=ctypes.byref(c), **change) == status


def test_status_text(bs):
    assert "page" in bs.status_string(bs.ERR_PAGE)


def test_wrappers_check_before_the_library(bs, monkeypatch):
    """Wrong types, shapes and host tensors never reach the library."""
    import torch

    def no_load():
        raise AssertionError("the library must not be reached")

    monkeypatch.setattr(bs, "load", no_load)
    x = torch.zeros(1, 4, 6, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bfloat16"):
        bs.qk_norm_rope(x.float(), 2, 2)
    with pytest.raises(TypeError, match="CUDA"):
        bs.qk_norm_rope(x, 2, 2)
    with pytest.raises(TypeError, match="float32"):
        bs.qk_norm_rope_bwd(x, x, x, x)
    with pytest.raises(TypeError, match="CUDA"):
        bs.select_blocks(x, x, 1)
    with pytest.raises(TypeError, match="Kv4Cache"):
        bs.kv4_status(object())
    with pytest.raises(TypeError, match="CUDA device"):
        bs.Kv4Cache(1, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="multiple of 16"):
        bs.rope_table(4, 24)


BASE = 0x100000
OVERLAPS = [  # dx's distance in elements, B, S, strides of x, strides of dx (rows of 512 elements)
    (8, 1, 4, (2048, 512), (2048, 512)), (-8, 1, 4, (2048, 512), (2048, 512)), (512, 1, 4, (2048, 512), (2048, 512)),
    (2040, 1, 4, (2048, 512), (2048, 512)), (-2040, 1, 4, (2048, 512), (2048, 512)),
    (0, 1, 4, (0, 512), (0, 1024)), (0, 1, 4, (0, 0), (0, 512)), (0, 3, 4, (0, 512), (2048, 512)),  # x broadcast
    (504, 1, 4, (0, 1024), (0, 1024)), (1032, 1, 4, (0, 1024), (0, 1024)),  # between the rows, but too near
    (1024, 2, 2, (1544, 1024), (1544, 1024)), (1560, 2, 2, (1536, 512), (1536, 512)), (8, 1, 1, (0, 0), (0, 512))]


@pytest.mark.parametrize("case", OVERLAPS, ids=str)
def test_gradient_over_its_input(bs, case):
    """dx that overlaps x without being x itself: rows would be read after they were overwritten."""
    apart, B, S, (xb, xs), (dxb, dxs) = case
    dxb = max(dxb, (S - 1) * dxs + 512)
    args = [vp(BASE), xb, xs, FAKE, FAKE, FAKE, B, S, 4, 2, 64, FAKE, FAKE, None, 0, 0, None, 1e-6, 0,
            vp(BASE + 2 * apart), dxb, dxs, FAKE, FAKE, FAKE, 1 << 30, None]
    assert bs.load().bsattn_qk_norm_rope_bwd(*args) == bs.ERR_INVALID_ARG
