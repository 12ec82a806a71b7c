"""Pages behind a sequence that became shorter (drafts that were refused, reservations that ran out):
given back, so that refs is what the tables hold; and who reports copies of bad pages."""
import random

import pytest
import torch

import _ops_ref as ref
from test_gpu_kv4_pages import _cache, _i32, _same, _state, bs  # noqa: F401

pytestmark = pytest.mark.gpu


def _pages(n, page):
    return -(-max(n, 0) // page)


def _counted(cache, table, held):
    return ref.count_refs(cache, table.tolist(), held.tolist())


def _given_back(refs, table, lengths, held, page):
    """refs, table (lists) without the pages of columns behind `lengths` up to those of `held`."""
    refs, table = list(refs), [list(row) for row in table]
    for row, n, m in zip(table, lengths, held):
        for column in range(_pages(n, page), min(len(row), _pages(m, page))):
            if 0 <= row[column] < len(refs):
                refs[row[column]] -= 1
            row[column] = -1
    return refs, table


@pytest.mark.parametrize("place", [False, True], ids=["new", "in place"])
def test_refused_drafts(bs, place):  # noqa: F811
    """Room for 20 drafted tokens, some accepted, again and again: the pages in use stay those of the tables."""
    rng = random.Random(3)
    cache = _cache(bs, 48)
    B, columns, T = 5, 9, 20
    table, refs = torch.full((B, columns), -1, dtype=torch.int32, device="cuda"), _i32([0] * 48)
    lengths, held = _i32([0] * B), None
    for step in range(30):
        counts = _i32([rng.choice([0, 3, T]) for _ in range(B)])
        was, old_t, old_r = lengths if held is None else held, table.tolist(), refs.tolist()
        out = (table, refs) if place else None
        want_r, want_t = _given_back(old_r, old_t, lengths.tolist(), was.tolist(), 16)
        want_t, want_r = ref.reserve(want_r, want_t, lengths.tolist(), counts.tolist(), 16)
        table, refs = bs.kv4_reserve(cache, refs, table, lengths, counts, out=out, held=held)
        assert table.tolist() == want_t and refs.tolist() == want_r
        held = lengths + counts
        assert _counted(cache, table, held) == refs.tolist()
        accepted = [rng.randint(0, c) for c in counts.tolist()]
        lengths = lengths + _i32(accepted)
        lengths = torch.where(lengths > 110, 0, lengths)  # (a row that begins anew gives all of its pages back)
        if step == 15:  # (the mapping may change between)
            table, refs, _ = bs.kv4_compact(cache, refs, table)
    table, refs = bs.kv4_reserve(cache, refs, table, lengths, 0, held=held)  # nothing wanted: what is behind goes
    assert _counted(cache, table, lengths) == refs.tolist()
    bs.kv4_status(cache)


def test_a_reservation_that_ran_out_is_tried_again(bs):  # noqa: F811
    cache = _cache(bs, 6)
    table, refs = _i32([[0, -1, -1], [1, -1, -1]]), _i32([1, 1, 0, 0, 1, 0])
    n, c = _i32([16, 16]), _i32([32, 32])
    bs.kv4_reserve(cache, refs, table, n, c, out=(table, refs))
    with pytest.raises(bs.BsattnError, match="page"):  # four pages wanted, three there
        bs.kv4_status(cache)
    assert table.tolist() == [[0, 2, 3], [1, 5, -1]]
    refs[4] = 0  # another sequence's
    bs.kv4_reserve(cache, refs, table, n, c, out=(table, refs), held=n + c)
    bs.kv4_status(cache)
    assert table.tolist() == [[0, 2, 3], [1, 4, 5]] and refs.tolist() == [1] * 6
    assert _counted(cache, table, n + c) == refs.tolist()


@pytest.mark.parametrize("place", [False, True], ids=["new", "in place"])
@pytest.mark.parametrize("case", [(1, 64, 16, 64, 1, 1, 5), (2, 64, 16, 32, 7, 100, 160), (1, 64, 256, 64, 40, 700, 300),
                                  (1, 64, 16, 32, 300, 60, 40000)], ids=str)
def test_fork_with_pages_behind(bs, case, place):  # noqa: F811
    Hkv, D, page, group, rows, longest, pages = case
    rng = random.Random(5)
    cache = _cache(bs, pages, Hkv, D, page, group)
    columns = _pages(longest, page) + 3
    free = list(range(pages))
    rng.shuffle(free)
    table, lengths, held = [], [], []
    for _ in range(rows):
        n = rng.randint(0, longest)
        m = rng.choice([n, n + rng.randint(0, 2 * page), n - 3])
        row = [free.pop() for _ in range(_pages(max(n, m), page))]
        table.append(row + [rng.choice([-1, 2])] * (columns - len(row)))
        lengths.append(n)
        held.append(m)
    refs = ref.count_refs(cache, table, [max(n, m) for n, m in zip(lengths, held)])
    parents = [rng.randrange(-1, rows) for _ in range(2 * rows)]
    given, _ = _given_back(refs, table, lengths, held, page)
    want = ref.fork(given, table, lengths, parents, page)
    state = _state(cache)
    r, t = _i32(refs), _i32(table)
    got = bs.kv4_fork(cache, r, t, _i32(lengths), _i32(parents), out=(None, None, r) if place else None, held=_i32(held))
    bs.kv4_status(cache)
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
    assert ref.count_refs(cache, want[0], want[1]) == want[2]
    assert t.tolist() == table  # (the old table is read only)
    for src, dst, tokens in want[3]:
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            x = state[name].view(torch.uint8)
            x[dst, :, :tokens] = x[src, :, :tokens]
    assert _same(cache, state)


def test_bad_pages_behind(bs):  # noqa: F811
    """Entries that are not there are skipped, pages that are not there and room behind the table reported."""
    cache = _cache(bs, 8)
    table, refs = [[0, 1, -1, 3], [4, 99, 5, 6]], [1, 1, 0, 1, 1, 1, 1, 0]
    got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32([16, -3]), 0, held=_i32([64, 33]))
    with pytest.raises(bs.BsattnError, match="page"):
        bs.kv4_status(cache)
    assert got[0].tolist() == [[0, -1, -1, -1], [-1, -1, -1, 6]]
    assert got[1].tolist() == [1, 0, 0, 0, 0, 0, 1, 0]
    got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32([64, 64]), 0, held=_i32([2 ** 31 - 1, -2 ** 31]))
    with pytest.raises(bs.BsattnError, match="page"):
        bs.kv4_status(cache)
    assert got[0].tolist() == table and got[1].tolist() == refs


def test_captured(bs):  # noqa: F811
    """A step of drafts in a graph, on another stream than the current one, in place."""
    cache = _cache(bs, 30)
    table, refs = torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), _i32([0] * 30)
    lengths, held = _i32([0, 5, 40]), _i32([0, 5, 40])
    bs.kv4_reserve(cache, refs, table, _i32([0, 0, 0]), lengths, out=(table, refs))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.kv4_reserve(cache, refs, table, lengths, 20, out=(table, refs), held=held)
        held.copy_(lengths + 20)
    side = torch.cuda.Stream()
    for step in range(8):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert _counted(cache, table, held) == refs.tolist()
        lengths += _i32([step % 3, 7, 0])
    bs.kv4_status(cache)


def test_refusals(bs):  # noqa: F811
    cache = bs.Kv4Cache(4, 2, 64, page_size=16)
    refs, table, n = _i32([0] * 4), _i32([[0, 1]]), _i32([3])
    for held in (n.long(), n.cpu(), 5):
        with pytest.raises(TypeError, match="held"):
            bs.kv4_reserve(cache, refs, table, n, 1, held=held)
        with pytest.raises(TypeError, match="held"):
            bs.kv4_fork(cache, refs, table, n, n, held=held)
    with pytest.raises(ValueError, match="held"):
        bs.kv4_reserve(cache, refs, table, n, 1, held=_i32([1, 2]))
    with pytest.raises(ValueError, match="held"):
        bs.kv4_fork(cache, refs, table, n, n, held=_i32([1, 2]))
    bs.kv4_status(cache)


@pytest.mark.parametrize("src,dst", [(99, 1), (1, 99)])
def test_copies_of_bad_pages_are_reported_by_both_caches(bs, src, dst):  # noqa: F811
    cache, to = _cache(bs, 8), _cache(bs, 8, seed=2)
    state = _state(to)
    bs.kv4_copy(cache, _i32([src]), _i32([dst]), to=to)
    for c in (cache, to):
        with pytest.raises(bs.BsattnError, match="page"):
            bs.kv4_status(c)
    assert _same(to, state)
