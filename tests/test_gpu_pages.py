"""Pages of a cache on the GPU against the plain oracle: copied, forked, freed and moved together.

Everything here is whole numbers or bytes that are copied, so results are equal to the last bit."""

import random

import pytest
import torch

from oracle import pages as op
from tests.gpu_util import dev, import_library

pytestmark = pytest.mark.gpu

mxa = import_library()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=dev())


def as_table(rows, cols):
    return ints(rows).reshape(len(rows), cols)


def new_caches(layers, pages, kv_heads, page, dim, seed):
    """Caches of random bytes."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    return [mxa.KVCache(*(torch.randint(0, 256, t.shape, generator=g, device=dev(), dtype=torch.uint8)
                          for t in mxa.new_kv_cache(pages, kv_heads, page, dim, dev()))) for _ in range(layers)]


def moved(caches, copies, whole=True):
    """What the caches hold after copies (source, target, tokens) of what they held before."""
    want = [[t.clone() for t in c] for c in caches]
    for src, dst, n in copies:
        for c, w in zip(caches, want):
            for t, x in zip(c, w):
                x[dst, :, :n] = t[src, :, :n]
    return want


def assert_caches(caches, want):
    for layer, (c, w) in enumerate(zip(caches, want)):
        for name, t, x in zip(c._fields, c, w):
            assert torch.equal(t, x), (layer, name)


def sequences(r, pages, page, cols, rows, fill=0.8, outside=0):
    """Counts, table and lengths of rows that share some pages; some page numbers are held by nobody in the table."""
    order = list(range(pages))
    r.shuffle(order)
    refs, table, lens = [0] * pages, [], []
    for _ in range(outside):
        if order:
            refs[order.pop()] = r.randint(1, 3)
    left = int(len(order) * fill)
    for i in range(rows):
        n = min(cols * page, r.choice([0, 1, page - 1, page, page + 1, r.randint(0, cols * page), cols * page]))
        base = r.choice(table) if table and r.random() < 0.6 else []
        common = r.randint(0, min(len(base), op.held(n, page)))
        row = base[:common]
        while len(row) < op.held(n, page) and left > 0:
            row.append(order.pop())
            left -= 1
        n = min(n, len(row) * page)
        row = row[:op.held(n, page)]
        for q in row:
            refs[q] += 1
        table.append(row)
        lens.append(n)
    # behind a row's pages anything may stand
    return refs, [row + [r.randint(-5, pages + 5) for _ in range(cols - len(row))] for row in table], lens


def run_fork(r, pages, page, cols, rows, layers=1, kv_heads=1, dim=64, outside=0, kind=None, seed=0, in_place=False):
    refs, table, lens = sequences(r, pages, page, cols, rows, outside=outside)
    kind = kind or r.choice(["grow", "beams", "branch", "stay"])
    parents = None if kind in ("grow", "stay") else [r.randint(-1, rows) for _ in range(r.randint(1, 2 * rows + 1))]
    n = rows if parents is None else len(parents)
    new = [r.choice([0, 1, 1, 2, page, page + 1, 3 * page + 5]) for _ in range(n)]
    lead = r.choice([0, 0, 3])
    cu = [lead + sum(new[:i]) for i in range(n + 1)]
    tokens = cu[-1] + r.choice([0, 0, 2])
    wide = cols + r.choice([0, 0, 2])
    release = kind in ("grow", "beams")
    want = op.fork(refs, table, lens, page, cu, parents, release, tokens, wide)
    caches = new_caches(layers, pages, kv_heads, page, dim, seed)
    content = moved(caches, want[4])
    counts = ints(refs)
    out = (counts, torch.full((n, wide), 77, dtype=torch.int32, device=dev()), ints([55] * n),
           ints([99] * tokens, torch.int64)) if in_place else None
    got = mxa.mx_kv_fork(caches if layers > 1 else caches[0], counts, as_table(table, cols), ints(lens), ints(cu),
                         None if parents is None else ints(parents), release, tokens, None if in_place else wide, out)
    assert got.lens.tolist() == want[2]
    assert got.page_table.tolist() == want[1]
    assert got.refs.tolist() == want[0]
    assert got.slots.tolist() == want[3]
    assert_caches(caches, content)
    if not in_place:
        assert counts.tolist() == refs


@pytest.mark.parametrize("seed", range(40))
def test_fork_small(seed):
    r = random.Random(seed)
    run_fork(r, r.choice([5, 40, 130]), r.choice([16, 48]), r.choice([1, 3, 9]), r.randint(1, 9), seed=seed,
             outside=r.choice([0, 3]), in_place=seed % 3 == 0)


@pytest.mark.parametrize("dim,kv_heads,page,layers", [(64, 1, 16, 3), (96, 3, 32, 2), (128, 8, 64, 2), (192, 2, 48, 1),
                                                      (256, 2, 128, 2), (64, 1, 16, 33), (64, 1, 16, 70)])
def test_fork_shapes(dim, kv_heads, page, layers):
    r = random.Random(dim * 7 + layers)
    for seed, kind in enumerate(("beams", "branch", "grow", "stay")):
        run_fork(r, 60, page, 5, 6, layers, kv_heads, dim, kind=kind, seed=seed)


@pytest.mark.parametrize("pages,rows,cols", [(4096, 300, 40), (4097, 257, 20), (20000, 700, 33), (70000, 40, 3000)])
def test_fork_many(pages, rows, cols):
    """Several counting blocks, several blocks of children, rows of several steps."""
    r = random.Random(pages)
    for kind in ("beams", "grow", "branch"):
        run_fork(r, pages, 16, cols, rows, kind=kind, outside=pages // 20)


def test_fork_of_nothing():
    cache = mxa.new_kv_cache(4, 1, 16, 64)
    refs, table, lens = ints([0, 1, 2, 0]), ints([[1, 2], [2, 0]]), ints([20, 5])
    none = torch.empty(0, dtype=torch.int32, device=dev())
    # no children: the rows end
    got = mxa.mx_kv_fork(cache, refs, table, lens, parents=none)
    assert got.refs.tolist() == [0, 0, 0, 0] and got.page_table.shape == (0, 2)
    # no children beside them, no rows, no pages
    got = mxa.mx_kv_fork(cache, refs, table, lens, parents=none, release=False)
    assert got.refs.tolist() == [0, 1, 2, 0]
    got = mxa.mx_kv_fork(cache, refs, table[:0], lens[:0], ints([0, 1]), parents=ints([-1]))
    assert got.page_table.tolist() == [[0, -1]] and got.slots.tolist() == [0] and got.refs.tolist() == [1, 1, 2, 0]
    empty = mxa.new_kv_cache(0, 1, 16, 64)
    got = mxa.mx_kv_fork(empty, none, table * 0, lens * 0, ints([0, 1, 2]))
    assert got.lens.tolist() == [0, 0] and got.slots.tolist() == [-1, -1]
    # no new tokens: pages are shared, partly filled ones too
    got = mxa.mx_kv_fork(cache, refs, table, lens, parents=ints([0, 0, 0]))
    assert got.refs.tolist() == [0, 3, 3, 0] and got.lens.tolist() == [20, 20, 20]


def test_fork_without_children_in_an_empty_pool():
    none = torch.empty(0, dtype=torch.int32, device=dev())
    got = mxa.mx_kv_fork(mxa.new_kv_cache(0, 1, 16, 64), none, ints([[0, 0]]), ints([0]), parents=none)
    assert got.lens.shape == (0,) and got.page_table.shape == (0, 2)


@pytest.mark.parametrize("pages", [0, 50])
def test_fork_of_many_children_without_rows(pages):
    """Counts changed in place and no rows: there is nothing to begin with."""
    children, cu = 20000, [0] * 10000 + [30] * 10001
    refs, lens = ints([0] * pages), ints([1] * children)
    table, slots = ints([[5, 5]] * children), torch.full((30,), -7, device=dev())
    mxa.mx_kv_fork(mxa.new_kv_cache(pages, 1, 16, 64), refs, ints([]).view(0, 2), ints([]), ints(cu),
                   parents=ints([-1] * children), out=(refs, table, lens, slots))
    want = op.fork([0] * pages, [], [], 16, cu, [-1] * children, tokens=30, cols=2)
    assert [x.tolist() for x in (refs, table, lens, slots)] == list(want[:4])


@pytest.mark.parametrize("pages", [0, 4, 20000])
def test_fork_of_tokens_without_children(pages):
    """A padded batch that has lost its last sequence: every token is of no child."""
    none = torch.empty(0, dtype=torch.int32, device=dev())
    slots = torch.full((300,), 7, device=dev())
    out = (ints([0] * pages), none.view(0, 2), none.clone(), slots)
    got = mxa.mx_kv_fork(mxa.new_kv_cache(pages, 1, 16, 64), ints([0] * pages), none.view(0, 2), none, ints([0]),
                         parents=none, tokens=300, out=out)
    assert slots.tolist() == [-1] * 300 and not got.refs.any()


def test_fork_of_the_most_tokens():
    """2^31 - 1 new tokens of a child that no pool could hold: the count of the last step passes 31 bits."""
    most = (1 << 31) - 1
    slots = torch.full((most,), 7, device=dev())
    got = mxa.mx_kv_fork(mxa.new_kv_cache(4, 1, 16, 64), ints([0] * 4), ints([[0, 0]]), ints([0]), ints([0, most]),
                         tokens=most, out=(ints([9] * 4), ints([[9, 9]]), ints([9]), slots))
    assert got.lens.tolist() == [0] and got.refs.tolist() == [0] * 4 and got.page_table.tolist() == [[-1, -1]]
    assert int(slots.min()) == int(slots.max()) == -1


@pytest.mark.parametrize("more", [0, 20000])
def test_pages_of_a_child_too_wide_are_not_given_to_later_ones(more):
    """In one launch and, with pages in use behind the free ones, in several."""
    def fork(refs, table, lens, *args, **kw):
        cache = mxa.new_kv_cache(len(refs) + more, 1, 16, 64)
        got = mxa.mx_kv_fork(cache, ints(refs + [1] * more), ints(table), ints(lens), *args, **kw)
        assert got.refs[len(refs):].tolist() == [1] * more
        return got.refs[:len(refs)].tolist(), got.page_table.tolist(), got.lens.tolist(), got.slots.tolist()

    cu, two = ints([0, 40, 41]), [[0, 0]] * 2
    for parents in (None, ints([0, 1]), ints([-1, -1])):
        assert fork([0] * 6, two, [0, 0], cu, parents) == \
            ([0, 0, 0, 1, 0, 0], [[-1, -1], [3, -1]], [0, 1], [-1] * 40 + [48])
        assert fork([0] * 3, two, [0, 0], cu, parents) == ([0] * 3, [[-1, -1]] * 2, [0, 0], [-1] * 41)
    assert fork([1, 1] + [0] * 5, [[0, 1]], [20], cu, ints([0, 0]), release=False) == \
        ([3, 2, 0, 0, 0, 1, 0], [[0, 1], [0, 5]], [20, 21], [-1] * 40 + [84])


def test_table_of_wider_rows_and_bad_entries():
    """A table that is part of a wider one; pages outside the pool are held by nobody and not written to."""
    wide = ints([[3, 0, 1, 7], [9, 9, 2, 7], [-4, 1, 1, 7]])
    table, lens, refs = wide[:, :2], ints([20, 30, 18]), [1, 1, 0, 1, 0]
    cache = mxa.new_kv_cache(5, 1, 16, 64)
    rows = table.tolist()
    want = op.fork(refs, rows, lens.tolist(), 16, [0, 1, 2, 3], None, True, 3)
    got = mxa.mx_kv_fork(cache, ints(refs), table, lens, ints([0, 1, 2, 3]))
    assert (got.refs.tolist(), got.page_table.tolist(), got.lens.tolist(), got.slots.tolist()) == want[:4]
    assert got.slots.tolist()[1] == -1
    assert mxa.mx_kv_free(ints(refs), table, lens, 16)[0].tolist() == op.free(refs, rows, lens.tolist(), 16)[0]
    got = mxa.mx_kv_compact(cache, ints(refs), table, lens)
    want = op.compact(refs, rows, lens.tolist(), 16)
    assert (got[0].tolist(), got[1].tolist(), got[2].item()) == want[:3]


def test_lengths_outside_the_table_are_cut():
    cache = mxa.new_kv_cache(3, 1, 16, 64)
    refs, table, lens = [1, 1, 1], [[0, 1], [2, 7]], [100, -3]
    want = op.fork(refs, table, lens, 16, [0, 0, 2], None, True, 2)
    got = mxa.mx_kv_fork(cache, ints(refs), ints(table), ints(lens), ints([0, 0, 2]))
    assert (got.refs.tolist(), got.page_table.tolist(), got.lens.tolist(), got.slots.tolist()) == want[:4]
    assert [x.tolist() for x in mxa.mx_kv_free(ints(refs), ints(table), ints(lens), 16)] == list(op.free(refs, table, lens, 16))


@pytest.mark.parametrize("pages,page,cols,rows", [(1, 16, 1, 1), (50, 16, 7, 9), (5000, 64, 300, 40), (30000, 16, 33, 3000),
                                                 (70000, 16, 20000, 3), (16385, 16, 700, 800), (200000, 32, 300, 2000),
                                                 (1000000, 16, 9001, 60), (300, 16, 2, 300000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_free(pages, page, cols, rows, in_place):
    r = random.Random(pages + rows)
    refs, table, lens = sequences(r, pages, page, cols, rows)
    for keep in (None, [r.choice([-1, 0, n, n - 1, n // 2, n + 9, n - page]) for n in lens]):
        counts, length = ints(refs), ints(lens)
        got = mxa.mx_kv_free(counts, as_table(table, cols), length, page, None if keep is None else ints(keep),
                             (counts, length) if in_place else None)
        want = op.free(refs, table, lens, page, keep)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        if in_place:
            assert got[0].data_ptr() == counts.data_ptr()
        else:
            assert counts.tolist() == refs and length.tolist() == lens


@pytest.mark.parametrize("pages,rows,cols,layers,kv_heads,page,dim", [
    (1, 1, 1, 1, 1, 16, 64), (2, 1, 1, 1, 1, 16, 64), (30, 5, 3, 2, 3, 48, 96), (300, 30, 4, 33, 1, 16, 64),
    (4095, 200, 9, 1, 1, 16, 64), (4096, 200, 9, 1, 1, 16, 64), (9000, 400, 30, 1, 2, 16, 128), (40, 6, 4, 2, 8, 64, 256)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(pages, rows, cols, layers, kv_heads, page, dim, in_place):
    r = random.Random(pages + dim)
    for fill in (0.0, 0.4, 0.8, 1.0):
        refs, table, lens = sequences(r, pages, page, cols, rows, fill)
        want = op.compact(refs, table, lens, page)
        caches = new_caches(layers, pages, kv_heads, page, dim, pages)
        content = moved(caches, [(src, dst, page) for src, dst in want[3]])
        counts, rows_in = ints(refs), as_table(table, cols)
        out = (counts, rows_in, ints([-1])) if in_place else None
        got = mxa.mx_kv_compact(caches, counts, rows_in, ints(lens), out)
        assert got[2].item() == want[2]
        assert got[0].tolist() == want[0]
        assert got[1].tolist() == want[1]
        assert_caches(caches, content)


@pytest.mark.parametrize("kv_heads,page,dim,layers", [(1, 16, 64, 1), (3, 48, 96, 2), (8, 64, 128, 3), (2, 128, 256, 1),
                                                      (1, 16, 64, 40)])
@pytest.mark.parametrize("count", [0, 1, 7, 60])
def test_copy(kv_heads, page, dim, layers, count):
    r = random.Random(count)
    src, dst = new_caches(layers, 70, kv_heads, page, dim, 1), new_caches(layers, 65, kv_heads, page, dim, 2)
    a, b = r.sample(range(70), count), r.sample(range(65), count)
    if count > 5:       # pairs outside a pool are skipped
        a[2], b[4] = 70, -1
    pairs = [(x, y) for x, y in zip(a, b) if 0 <= x < 70 and 0 <= y < 65]
    want = [[t.clone() for t in c] for c in dst]
    for x, y in pairs:
        for c, w in zip(src, want):
            for t, u in zip(c, w):
                u[y] = t[x]
    mxa.mx_kv_copy(src, ints(a), dst, ints(b))
    assert_caches(dst, want)
    # within one pool, one page to several
    want = moved(src, [(3, y, page) for y in range(10, 15)])
    mxa.mx_kv_copy(src, ints([3] * 5), src, ints(list(range(10, 15))))
    assert_caches(src, want)


def test_pages_past_32_bits():
    """A pool of over 2^32 bytes of codes: the last pages are copied, forked and moved like the first."""
    pages, kv_heads, page, dim = 70000, 8, 64, 128
    cache = mxa.new_kv_cache(pages, kv_heads, page, dim)
    assert cache.k.numel() > 2 ** 32
    g = torch.Generator(device=dev()).manual_seed(5)
    for t in cache:
        t[pages - 2:] = torch.randint(0, 256, t[pages - 2:].shape, generator=g, device=dev(), dtype=torch.uint8)
    last = [t[pages - 2:].clone() for t in cache]
    mxa.mx_kv_copy(cache, ints([pages - 1, pages - 2]), cache, ints([5, pages - 3]))
    for t, x in zip(cache, last):
        assert torch.equal(t[5], x[1]) and torch.equal(t[pages - 3], x[0])
    refs = torch.ones(pages, dtype=torch.int32, device=dev())
    refs[pages - 4] = 0
    got = mxa.mx_kv_fork(cache, refs, ints([[pages - 1]]), ints([40]), ints([0, 1]), release=False)
    assert got.page_table.tolist() == [[pages - 4]] and got.slots.tolist() == [(pages - 4) * 64 + 40]
    for t, x in zip(cache, last):
        assert torch.equal(t[pages - 4, :, :48], x[1, :, :48])
    refs = torch.zeros(pages, dtype=torch.int32, device=dev())
    refs[pages - 2:] = ints([2, 3])
    got = mxa.mx_kv_compact(cache, refs, ints([[pages - 2, pages - 1]]), ints([70]))
    assert got[0][:3].tolist() == [3, 2, 0] and got[1].tolist() == [[1, 0]] and got[2].item() == 2
    for t, x in zip(cache, last):
        assert torch.equal(t[0], x[1]) and torch.equal(t[1], x[0])


def test_replayed_graph_and_other_streams():
    """A captured step (fork in place of the counts, free, compact) replayed on changing inputs, with eager calls between,
    equals the oracle each time; so does a call on a side stream."""
    page, cols, rows, pages = 16, 6, 8, 90
    r = random.Random(9)
    cache = new_caches(2, pages, 2, page, 64, 3)
    static = (ints([0] * pages), as_table([[0] * cols] * rows, cols), ints([0] * rows), ints([0] * rows),
              ints([0] * (rows + 1)))

    def step():
        refs, table, lens, parents, cu = static
        f = mxa.mx_kv_fork(cache, refs, table, lens, cu, parents, True, 40)
        c = mxa.mx_kv_compact(cache, f.refs, f.page_table, f.lens)
        return f, c, mxa.mx_kv_free(c[0], c[1], f.lens, page)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for turn in range(6):
        refs, table, lens = sequences(r, pages, page, cols, rows, 0.5)
        parents = [r.randint(0, rows - 1) for _ in range(rows)]
        new = [r.randint(0, 5) for _ in range(rows)]
        cu = [sum(new[:i]) for i in range(rows + 1)]
        for t, x in zip(static, (refs, table, lens, parents, cu)):
            t.copy_(ints(x))
        want = op.fork(refs, table, lens, page, cu, parents, True, 40)
        want_c = op.compact(want[0], want[1], want[2], page)
        content = moved([mxa.KVCache(*x) for x in moved(cache, want[4])], [(a, b, page) for a, b in want_c[3]])
        if turn % 3 == 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                f, c, z = step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
            f, c, z = outs
        assert (f.refs.tolist(), f.page_table.tolist(), f.lens.tolist(), f.slots.tolist()) == want[:4]
        assert (c[0].tolist(), c[1].tolist(), c[2].item()) == want_c[:3]
        assert z[0].tolist() == op.free(want_c[0], want_c[1], want[2], page)[0]
        assert_caches(cache, content)


def test_captured_copy():
    """The copies of more layers than one launch takes, captured, replayed on changing pages."""
    caches = new_caches(35, 30, 1, 16, 64, 4)
    src, dst = ints([0] * 6), ints([1] * 6)
    r = random.Random(2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        mxa.mx_kv_copy(caches, src * 0 - 1, caches, dst)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxa.mx_kv_copy(caches, src, caches, dst)
    for _ in range(4):
        a, b = r.sample(range(15), 6), r.sample(range(15, 30), 6)
        src.copy_(ints(a))
        dst.copy_(ints(b))
        want = moved(caches, [(x, y, 16) for x, y in zip(a, b)])
        graph.replay()
        assert_caches(caches, want)


def test_refusals():
    cache = mxa.new_kv_cache(4, 1, 16, 64)
    refs, table, lens, cu = ints([0] * 4), ints([[0, 1]]), ints([3]), ints([0, 1])
    fork = lambda **kw: mxa.mx_kv_fork(**{**dict(caches=cache, refs=refs, page_table=table, lens=lens, cu=cu), **kw})  # noqa: E731
    for kw in ({"refs": refs[:3]}, {"refs": refs.long()}, {"page_table": table.long()}, {"page_table": table[0]},
               {"lens": lens.long()}, {"lens": ints([1, 2])}, {"cu": ints([0, 1, 2])}, {"parents": ints([0, 0])},
               {"parents": ints([0], torch.int64)}, {"cols": 1}, {"tokens": -1}, {"caches": []}, {"caches": cache[:3]},
               {"caches": [cache, mxa.new_kv_cache(5, 1, 16, 64)]}, {"caches": [cache, mxa.new_kv_cache(4, 1, 32, 64)]},
               {"out": (refs, table, lens)}, {"out": (refs, table.clone(), ints([0]), ints([0]))},
               {"out": (refs, table, ints([0]), ints([0], torch.int64))}, {"refs": refs.cpu()},
               {"page_table": table.expand(2, 2), "lens": ints([3, 3]), "cu": ints([0, 1, 2])}):
        with pytest.raises(ValueError):
            fork(**kw)
    with pytest.raises(TypeError):
        fork(caches=5)
    for args in ((refs, table, ints([1, 2]), 16), (refs, table, lens, 15), (refs, table, lens, 16, ints([1, 2])),
                 (refs, table, lens, 16, None, (refs,))):
        with pytest.raises(ValueError):
            mxa.mx_kv_free(*args)
    with pytest.raises(ValueError):
        mxa.mx_kv_compact(cache, refs[:2], table, lens)
    wide = ints([[0, 1, 2], [0, 1, 2]])
    with pytest.raises(ValueError):
        mxa.mx_kv_compact(cache, refs, wide[:, :2], ints([3, 3]), (refs, wide[:, :2], ints([0])))
    other = mxa.new_kv_cache(4, 2, 16, 64)
    for args in ((cache, ints([0]), other, ints([0])), (cache, ints([0]), cache, ints([0, 1])),
                 (cache, ints([0]).long(), cache, ints([0])), ([cache], ints([0]), [cache, cache], ints([0]))):
        with pytest.raises(ValueError):
            mxa.mx_kv_copy(*args)
