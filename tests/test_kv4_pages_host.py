"""Host-side checks of chunk attention and of the 4-bit cache's pages (no GPU needed): every bad
argument is turned away before anything is launched."""
import ctypes

import pytest

from test_ops_host import FAKE, ODD, _cache, _call, bs, vp  # noqa: F401

CHUNK = dict(cache=None, q=FAKE, B=1, H=4, T=40, table=FAKE, stride=4, columns=4, lengths=FAKE, counts=None,
             prefix=None, scale=0.1, cap=0.0, slopes=None, flags=0, out=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40,
             stream=None)
COPY = dict(a=None, b=None, src=FAKE, dst=FAKE, n=3, stream=None)
FORK = dict(cache=None, refs=FAKE, table=vp(0x20000), stride=4, columns=4, lengths=vp(0x30000), B=2,
            parents=vp(0x40000), n=2, new_table=vp(0x50000), new_lengths=vp(0x60000), new_refs=vp(0x70000),
            ws=vp(0x80000), nbytes=1 << 20, stream=None)
RESERVE = dict(cache=None, refs=FAKE, table=vp(0x20000), stride=4, columns=4, lengths=vp(0x30000), counts=None, T=1,
               B=2, new_table=vp(0x50000), new_stride=4, new_refs=vp(0x70000), stream=None)
COMPACT = dict(cache=None, refs=FAKE, table=vp(0x20000), stride=4, columns=4, B=2, new_table=vp(0x50000),
               new_stride=4, new_refs=vp(0x70000), map=vp(0x90000), ws=vp(0x80000), nbytes=1 << 20, stream=None)
CALLS = {"attn_chunk": CHUNK, "fork": FORK, "reserve": RESERVE, "compact": COMPACT}

BAD = [("attn_chunk", c, s) for c, s in (
    (dict(q=None), 1), (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(lse=None), 1), (dict(ws=ODD), 1),
    (dict(table=None), 1), (dict(lengths=None), 1), (dict(lengths=vp(0x10002)), 1), (dict(counts=vp(0x10001)), 1),
    (dict(prefix=vp(0x10002)), 1), (dict(slopes=vp(0x10003)), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1),
    (dict(H=5), 1), (dict(columns=0), 1), (dict(stride=-1), 1), (dict(flags=1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(cap=-1.0), 1), (dict(cap=float("inf")), 1), (dict(cap=float("nan")), 1),
    (dict(cap=1e-31), 2), (dict(cap=1e31), 2), (dict(B=65536), 2), (dict(B=40000), 2), (dict(T=1 << 24), 2),
    (dict(columns=1 << 27), 2))]
BAD += [("fork", c, s) for c, s in (
    (dict(refs=None), 1), (dict(table=None), 1), (dict(lengths=None), 1), (dict(parents=vp(0x40001)), 1),
    (dict(new_table=None), 1), (dict(new_lengths=None), 1), (dict(new_refs=vp(0x70008)), 1), (dict(B=0), 1),
    (dict(n=0), 1), (dict(columns=0), 1), (dict(stride=-1), 1), (dict(n=16385), 2), (dict(B=16385), 2),
    (dict(ws=None), 1), (dict(nbytes=8), 1), (dict(new_table=vp(0x20000)), 1), (dict(new_table=vp(0x2001C)), 1),
    (dict(new_lengths=vp(0x30004)), 1), (dict(new_lengths=vp(0x40004)), 1), (dict(new_table=vp(0x40004)), 1),
    (dict(refs=vp(0x70004)), 1))]
BAD += [("reserve", c, s) for c, s in (
    (dict(refs=None), 1), (dict(table=None), 1), (dict(lengths=None), 1), (dict(counts=vp(0x1)), 1), (dict(T=-1), 1),
    (dict(new_table=None), 1), (dict(new_refs=vp(0x70004)), 1), (dict(B=0), 1), (dict(columns=0), 1),
    (dict(stride=-4), 1), (dict(new_stride=3), 1), (dict(B=16385), 2), (dict(new_table=vp(0x20004)), 1),
    (dict(new_table=vp(0x20000), new_stride=5), 1), (dict(refs=vp(0x70004)), 1))]
BAD += [("compact", c, s) for c, s in (
    (dict(refs=None), 1), (dict(table=None), 1), (dict(new_table=None), 1), (dict(new_refs=None), 1),
    (dict(map=None), 1), (dict(B=0), 1), (dict(columns=0), 1), (dict(stride=-4), 1), (dict(new_stride=3), 1),
    (dict(ws=None), 1), (dict(nbytes=16), 1), (dict(new_table=vp(0x20004)), 1), (dict(map=FAKE), 1),
    (dict(map=vp(0x70004)), 1), (dict(refs=vp(0x70004)), 1))]


@pytest.mark.parametrize("call,change,status", BAD, ids=lambda c: str(c) if len(str(c)) < 40 else "")
def test_calls(bs, call, change, status):  # noqa: F811
    c = _cache()
    fn = getattr(bs.load(), "bsattn_kv4_" + call)
    assert _call(fn, CALLS[call], cache=ctypes.byref(c), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(src=None), 1), (dict(dst=vp(0x10002)), 1), (dict(n=0), 1), (dict(n=-1), 1)], ids=str)
def test_copy(bs, change, status):  # noqa: F811
    c = _cache()
    assert _call(bs.load().bsattn_kv4_copy, COPY, a=ctypes.byref(c), b=ctypes.byref(c), **change) == status


def test_caches(bs):  # noqa: F811
    lib = bs.load()
    good, bad = _cache(), _cache(page_size=48)
    for name, args in CALLS.items():
        fn = getattr(lib, "bsattn_kv4_" + name)
        assert _call(fn, args) == bs.ERR_INVALID_ARG
        assert _call(fn, args, cache=ctypes.byref(bad)) == bs.ERR_UNSUPPORTED
    for other in (dict(kv_heads=1), dict(page_size=32), dict(group=64), dict(head_dim=128)):
        c = _cache(**other)
        assert _call(lib.bsattn_kv4_copy, COPY, a=ctypes.byref(good), b=ctypes.byref(c)) == bs.ERR_INVALID_ARG
    assert _call(lib.bsattn_kv4_copy, COPY, a=ctypes.byref(good)) == bs.ERR_INVALID_ARG


def test_workspaces(bs):  # noqa: F811
    lib = bs.load()
    assert lib.bsattn_kv4_fork_workspace(0) == 0 and lib.bsattn_kv4_fork_workspace(5) == 40
    assert lib.bsattn_kv4_compact_workspace(-1) == 0 and lib.bsattn_kv4_compact_workspace(4) >= 36
    for sizes in ((0, 4, 2, 1, 64, 16, 4), (1, 5, 2, 1, 64, 16, 4), (1, 4, 2, 0, 64, 16, 4), (1, 4, 2, 1, 64, 16, 0)):
        assert lib.bsattn_kv4_attn_chunk_workspace(*sizes) == 0
