"""Host-side checks of pages given back (no GPU needed): bad arguments are turned away before a launch."""
import ctypes

import pytest

from test_ops_host import FAKE, _cache, _call, bs, vp  # noqa: F401

RELEASE = dict(cache=None, refs=FAKE, table=vp(0x20000), stride=4, columns=4, lengths=vp(0x30000), held=vp(0x40000),
               B=2, new_table=vp(0x50000), new_stride=4, new_refs=vp(0x70000), stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(refs=None), 1), (dict(refs=vp(0x10002)), 1), (dict(table=None), 1), (dict(lengths=None), 1),
    (dict(held=None), 1), (dict(held=vp(0x40001)), 1), (dict(new_table=vp(0x50001)), 1), (dict(new_refs=None), 1),
    (dict(new_refs=vp(0x70004)), 1), (dict(refs=vp(0x70004)), 1), (dict(B=0), 1), (dict(columns=0), 1),
    (dict(stride=-4), 1), (dict(new_stride=3), 1), (dict(new_table=vp(0x20004)), 1),
    (dict(new_table=vp(0x20000), new_stride=5), 1), (dict(B=16385), 2)], ids=str)
def test_release(bs, change, status):  # noqa: F811
    c = _cache()
    assert _call(bs.load().bsattn_kv4_release, RELEASE, cache=ctypes.byref(c), **change) == status


def test_caches(bs):  # noqa: F811
    fn = bs.load().bsattn_kv4_release
    assert _call(fn, RELEASE) == bs.ERR_INVALID_ARG
    assert _call(fn, RELEASE, cache=ctypes.byref(_cache(page_size=48))) == bs.ERR_UNSUPPORTED
