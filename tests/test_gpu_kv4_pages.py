"""The pages of the 4-bit cache: copies, forks, reservations and compaction against plain
lists (whole numbers and codes: equal)."""
import random

import pytest
import torch

import _ops_ref as ref

pytestmark = pytest.mark.gpu
BUFFERS = ("k_codes", "v_codes", "k_scales", "v_scales", "k_means")


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


def _cache(bs, pages, Hkv=2, D=64, page=16, group=32, seed=1):
    """Every byte another one."""
    cache = bs.Kv4Cache(pages, Hkv, D, page_size=page, group=group)
    g = ref.gen(seed)
    for name in BUFFERS:
        t = getattr(cache, name)
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, device="cuda"))
    return cache


def _state(cache):
    return {n: getattr(cache, n).view(torch.uint8).clone() for n in BUFFERS}


def _same(cache, state):
    return all(torch.equal(getattr(cache, n).view(torch.uint8), state[n]) for n in BUFFERS)


def _books(rng, cache, rows, longest, columns, shared=True):
    """A table over scattered pages with rows that share full pages, lengths, refs (lists)."""
    page = cache.page_size
    free = list(range(cache.pages))
    rng.shuffle(free)
    table, lengths = [], []
    for i in range(rows):
        n = rng.randint(0, longest)
        row = []
        if shared and i and rng.random() < 0.5:  # full pages of an earlier row
            a = rng.randrange(i)
            row = table[a][:rng.randint(0, min(lengths[a], n) // page)]
        while len(row) < -(-n // page):
            row = row + [free.pop()]
        table.append(row + [rng.choice([-1, 3])] * (columns - len(row)))  # (nothing behind the length counts)
        lengths.append(n)
    return table, lengths, ref.count_refs(cache, table, lengths)


def _behind(table, lengths, page):
    return [row[:-(-n // page)] + [-1] * (len(row) - -(-n // page)) for row, n in zip(table, lengths)]


#          Hkv D    page group rows longest pages
BOOKS = [(1, 64, 16, 64, 1, 1, 3), (2, 64, 16, 32, 7, 100, 80), (3, 128, 32, 128, 20, 300, 300),
         (1, 64, 256, 64, 40, 700, 200), (2, 128, 64, 64, 33, 1000, 5000), (1, 64, 16, 32, 300, 60, 40000)]


@pytest.mark.parametrize("case", BOOKS, ids=str)
@pytest.mark.parametrize("seed", [1, 2])
def test_fork(bs, case, seed):
    Hkv, D, page, group, rows, longest, pages = case
    rng = random.Random(seed)
    cache = _cache(bs, pages, Hkv, D, page, group)
    columns = -(-longest // page) + 2
    table, lengths, refs = _books(rng, cache, rows, longest, columns)
    for n in (rows, max(1, rows // 3), 2 * rows):
        parents = [rng.randrange(-1, rows) for _ in range(n)]
        want = ref.fork(refs, table, lengths, parents, page)
        state = _state(cache)
        got = bs.kv4_fork(cache, _i32(refs), _i32(table), _i32(lengths), _i32(parents))
        if any(-1 in row[:-(-m // page)] for row, m in zip(want[0], want[1])):
            with pytest.raises(bs.BsattnError, match="page"):
                bs.kv4_status(cache)
        bs.kv4_status(cache)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
        for src, dst, tokens in want[3]:  # the tokens of the last page, and no others
            for name in BUFFERS[:4]:
                t = state[name].view(torch.uint8)
                t[dst, :, :tokens] = t[src, :, :tokens]
        assert _same(cache, state)


def test_fork_in_place(bs):
    """refs may be the argument itself; a table, lengths and refs given for the results."""
    rng = random.Random(4)
    cache = _cache(bs, 90)
    table, lengths, refs = _books(rng, cache, 12, 100, 9)
    parents = [0, 0, 0, 5, 5, -1, 11, 2]
    want = ref.fork(refs, table, lengths, parents, 16)
    r, t = _i32(refs), torch.full((8, 9), 77, dtype=torch.int32, device="cuda")
    n = torch.full((8,), 77, dtype=torch.int32, device="cuda")
    wide = torch.full((12, 30), 5, dtype=torch.int32, device="cuda")
    wide[:, 7:16] = _i32(table)
    got = bs.kv4_fork(cache, r, wide[:, 7:16], _i32(lengths), _i32(parents), out=(t, n, r))
    assert got[0] is t and got[1] is n and got[2] is r
    assert t.tolist() == want[0] and n.tolist() == want[1] and r.tolist() == want[2]
    bs.kv4_status(cache)


def test_rows_that_end_give_their_pages_back(bs):
    rng = random.Random(5)
    cache = _cache(bs, 60)
    table, lengths, refs = _books(rng, cache, 8, 90, 6)
    t, n, r = bs.kv4_fork(cache, _i32(refs), _i32(table), _i32(lengths), _i32([-1] * 8))
    assert not bool(r.any()) and bool((t == -1).all()) and not bool(n.any())
    bs.kv4_status(cache)


@pytest.mark.parametrize("case", BOOKS, ids=str)
def test_reserve(bs, case):
    Hkv, D, page, group, rows, longest, pages = case
    rng = random.Random(7)
    cache = _cache(bs, pages, Hkv, D, page, group)
    columns = -(-longest // page) + 3
    table, lengths, refs = _books(rng, cache, rows, longest, columns)
    state = _state(cache)
    for counts in ([rng.randint(-1, 2 * page) for _ in range(rows)], [1] * rows, [0] * rows):
        want = ref.reserve(refs, table, lengths, counts, page)
        short = any(-1 in row[-(-n // page):min(columns, -(-(n + max(c, 0)) // page))]
                    for row, n, c in zip(want[0], lengths, counts))
        got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32(lengths), _i32(counts))
        if short:
            with pytest.raises(bs.BsattnError, match="page"):
                bs.kv4_status(cache)
        bs.kv4_status(cache)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        t, r = _i32(table), _i32(refs)  # in place
        bs.kv4_reserve(cache, r, t, _i32(lengths), _i32(counts), out=(t, r))
        assert t.tolist() == want[0] and r.tolist() == want[1]
        if short:
            with pytest.raises(bs.BsattnError, match="page"):
                bs.kv4_status(cache)
    want = ref.reserve(refs, table, lengths, [5] * rows, page)
    got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32(lengths), 5)
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
    assert _same(cache, state)


def test_reserve_behind_the_table_and_out_of_pages(bs):
    cache = _cache(bs, 6)
    table, refs = [[0, -1, -1], [1, -1, -1]], [1, 1, 0, 0, 1, 0]
    got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32([16, 16]), _i32([100, 1]))
    with pytest.raises(bs.BsattnError, match="page"):  # three columns, and no more
        bs.kv4_status(cache)
    assert got[0].tolist() == [[0, 2, 3], [1, 5, -1]] and got[1].tolist() == [1, 1, 1, 1, 1, 1]
    got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32([16, 16]), _i32([32, 32]))
    with pytest.raises(bs.BsattnError, match="page"):  # four pages wanted, three there
        bs.kv4_status(cache)
    assert got[0].tolist() == [[0, 2, 3], [1, 5, -1]] and got[1].tolist() == [1, 1, 1, 1, 1, 1]
    got = bs.kv4_reserve(cache, _i32(refs), _i32(table), _i32([2 ** 31 - 1, -7]), _i32([2 ** 31 - 1, 17]))
    with pytest.raises(bs.BsattnError, match="page"):  # a length behind the table; one below zero is none
        bs.kv4_status(cache)
    assert got[0].tolist() == [[0, -1, -1], [2, 3, -1]]


def test_bad_entries_of_books(bs):
    """Pages that are not there, parents that are not rows, lengths behind the table."""
    cache = _cache(bs, 8)
    state = _state(cache)
    table, lengths = [[1, 99, 2], [3, -1, 4], [5, 6, 7]], [40, 48, 400]
    got = bs.kv4_fork(cache, _i32([0, 1, 1, 1, 1, 1, 1, 1]), _i32(table), _i32(lengths), _i32([0, 1, 2, 3, -9]))
    with pytest.raises(bs.BsattnError, match="page"):
        bs.kv4_status(cache)
    assert got[0].tolist() == [[1, -1, 2], [3, -1, 4], [5, 6, 7], [-1] * 3, [-1] * 3]
    assert got[2].tolist() == [0, 1, 1, 1, 1, 1, 1, 1]
    table, refs, page_map = bs.kv4_compact(cache, _i32([1] * 8), _i32([[1, 99, -3, 7]]))
    with pytest.raises(bs.BsattnError, match="page"):
        bs.kv4_status(cache)
    assert table.tolist() == [[1, 99, -3, 7]]
    bs.kv4_copy(cache, _i32([0, -1, 99, 1]), _i32([-1, 2, 3, 1 << 30]))
    with pytest.raises(bs.BsattnError, match="page"):
        bs.kv4_status(cache)
    assert _same(cache, state)


@pytest.mark.parametrize("case", BOOKS, ids=str)
@pytest.mark.parametrize("place", [False, True], ids=["new", "in place"])
def test_compact(bs, case, place):
    Hkv, D, page, group, rows, longest, pages = case
    rng = random.Random(11)
    cache = _cache(bs, pages, Hkv, D, page, group)
    table, lengths, refs = _books(rng, cache, rows, longest, -(-longest // page) + 1)
    table = _behind(table, lengths, page)
    want = ref.compact(refs, table)
    state = _state(cache)
    t, r = _i32(table), _i32(refs)
    m = torch.full((pages,), 7, dtype=torch.int32, device="cuda")
    got = bs.kv4_compact(cache, r, t, out=(t, r, m) if place else None)
    bs.kv4_status(cache)
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
    for p, q in enumerate(want[2]):
        if q >= 0 and q != p:
            for name in BUFFERS:
                state[name][q] = state[name][p]
    # (each move's source is left as it was)
    assert _same(cache, state)


@pytest.mark.parametrize("refs", [[0] * 9, [1] * 9, [0] * 8 + [2], [1] + [0] * 8, [0, 3, 0, 1, 0, 0, 2, 0, 1]], ids=str)
def test_compact_ends(bs, refs):
    cache = _cache(bs, 9)
    used = [p for p, r in enumerate(refs) if r]
    table = [used + [-1] * (9 - len(used))]
    want = ref.compact(refs, table)
    got = bs.kv4_compact(cache, _i32(refs), _i32(table))
    assert [t.tolist() for t in got] == list(want)


@pytest.mark.parametrize("case", [(1, 64, 16, 64, 1), (3, 64, 16, 32, 5), (8, 128, 256, 32, 40), (2, 128, 64, 128, 300)],
                         ids=str)
def test_copy(bs, case):
    Hkv, D, page, group, n = case
    cache, to = _cache(bs, n + 7, Hkv, D, page, group), _cache(bs, n + 2, Hkv, D, page, group, seed=2)
    src = torch.randperm(n + 7, generator=ref.gen(3, "cpu"))[:n].int().cuda()
    dst = torch.randperm(n + 2, generator=ref.gen(4, "cpu"))[:n].int().cuda()
    src[0] = -1
    state, before = _state(to), _state(cache)
    bs.kv4_copy(cache, src, dst, to=to)
    for name in BUFFERS:
        state[name][dst[1:].long()] = before[name][src[1:].long()]
    assert _same(to, state) and _same(cache, before)
    if n > 3:  # within one cache
        a, b = _i32([0, 1]), _i32([n + 1, n])
        state = _state(to)
        bs.kv4_copy(to, a, b)
        for name in BUFFERS:
            state[name][b.long()] = state[name][a.long()]
        assert _same(to, state)
    bs.kv4_copy(cache, src[:0], dst[:0], to=to)
    bs.kv4_status(cache)
    bs.kv4_status(to)


def test_a_large_cache(bs):
    """Many pages: the parts of the cluster's CTAs, and rounds of each."""
    pages, rows = 200_001, 2000
    cache = bs.Kv4Cache(pages, 1, 64, page_size=16)
    refs = (torch.rand(pages, generator=ref.gen(1), device="cuda") < 0.9).to(torch.int32)
    lengths = torch.randint(0, 100, (rows,), generator=ref.gen(2), device="cuda").to(torch.int32)
    counts = torch.randint(0, 60, (rows,), generator=ref.gen(3), device="cuda").to(torch.int32)
    table = torch.full((rows, 12), -1, dtype=torch.int32, device="cuda")
    want = ref.reserve(refs.tolist(), table.tolist(), lengths.tolist(), counts.tolist(), 16)
    got = bs.kv4_reserve(cache, refs, table, lengths, counts)
    bs.kv4_status(cache)
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
    want = ref.compact(want[1], want[0])
    cache.k_means.copy_(torch.randn(cache.k_means.shape, generator=ref.gen(4), device="cuda"))
    means = cache.k_means.clone()
    got = bs.kv4_compact(cache, got[1], got[0])
    assert [t.tolist() for t in got] == list(want)
    to = got[2].long()
    assert torch.equal(cache.k_means[to[to >= 0]], means[to >= 0])


def test_captured(bs):
    """A decoding step's reservation in place, in a graph, replayed while the lengths grow."""
    cache = _cache(bs, 50)
    table, refs = torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(50, dtype=torch.int32, device="cuda")
    n = _i32([0, 15, 16])
    bs.kv4_reserve(cache, refs, table, _i32([0, 0, 0]), n, out=(table, refs))
    want_t, want_r = ref.reserve([0] * 50, [[-1] * 8] * 3, [0] * 3, [0, 15, 16], 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.kv4_reserve(cache, refs, table, n, 1, out=(table, refs))
    for step in range(20):
        graph.replay()
        now = n.tolist()
        want_t, want_r = ref.reserve(want_r, want_t, now, [1] * 3, 16)
        n += 1
        assert table.tolist() == want_t and refs.tolist() == want_r
    fork = torch.cuda.CUDAGraph()
    parents = _i32([2, 2, 0])
    with torch.cuda.graph(fork):
        got = bs.kv4_fork(cache, refs, table, n, parents)
        moved = bs.kv4_compact(cache, got[2], got[0])
    for p in ([2, 2, 0], [1, -1, 1]):
        parents.copy_(_i32(p))
        fork.replay()
        want = ref.fork(want_r, _behind(want_t, n.tolist(), 16), n.tolist(), p, 16)
        assert got[0].tolist() == want[0] and got[2].tolist() == want[2]
        assert [t.tolist() for t in moved] == list(ref.compact(want[2], want[0]))
    bs.kv4_status(cache)


def test_refusals(bs):
    cache, other = bs.Kv4Cache(4, 2, 64, page_size=16), bs.Kv4Cache(4, 2, 64, page_size=32)
    refs, table, n = _i32([0] * 4), _i32([[0, 1]]), _i32([3])
    with pytest.raises(ValueError, match="page_size"):
        bs.kv4_copy(cache, n, n, to=other)
    with pytest.raises(ValueError, match="dst"):
        bs.kv4_copy(cache, n, _i32([1, 2]))
    with pytest.raises(TypeError, match="int32"):
        bs.kv4_copy(cache, n.long(), n)
    with pytest.raises(TypeError, match="Kv4Cache"):
        bs.kv4_copy(cache, n, n, to=3)
    with pytest.raises(ValueError, match="refs"):
        bs.kv4_fork(cache, refs[:3], table, n, n)
    with pytest.raises(ValueError, match="parents"):
        bs.kv4_fork(cache, refs, table, n, table)
    with pytest.raises(ValueError, match="rows"):
        bs.kv4_fork(cache, refs, table, n, n[:0])
    with pytest.raises(ValueError, match="out"):
        bs.kv4_fork(cache, refs, table, n, n, out=(table,))
    with pytest.raises(bs.BsattnError):  # the old table is read while the new one is written
        bs.kv4_fork(cache, refs, table, n, _i32([0]), out=(table, None, None))
    with pytest.raises(bs.BsattnError):
        bs.kv4_fork(cache, refs, table, n, _i32([0]), out=(None, n, None))
    with pytest.raises(TypeError, match="counts"):
        bs.kv4_reserve(cache, refs, table, n, 1.5)
    with pytest.raises(ValueError, match="counts"):
        bs.kv4_reserve(cache, refs, table, n, -1)
    wide = torch.zeros(5, dtype=torch.int32, device="cuda")
    with pytest.raises(bs.BsattnError):  # refs over a part of itself, and not 16-byte aligned
        bs.kv4_reserve(cache, wide[:4], table, n, 1, out=(None, wide[1:]))
    big = _i32([[0, 1, 2, 3]])
    with pytest.raises(bs.BsattnError):
        bs.kv4_reserve(cache, refs, big[:, :3], n, 1, out=(big[:, 1:], None))
    with pytest.raises(ValueError, match="block_table"):
        bs.kv4_compact(cache, refs, table[0])
    with pytest.raises(bs.BsattnError):
        bs.kv4_compact(cache, refs, table, out=(None, None, refs))
    many = torch.zeros(16385, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(bs.BsattnError, match="unsupported"):
        bs.kv4_reserve(cache, refs, many, many[:, 0].contiguous(), 1)
    bs.kv4_status(cache)
