"""Large pools, tables and batches of a cache's pages on the GPU: the kernels that sizes choose there.

Up to some ten thousand rows and pages against the plain oracle, beyond that against the same rules on whole tensors
(counted, sorted and indexed by torch).  Whole numbers, equal to the last one."""

import random

import pytest
import torch

from oracle import pages as op
from tests.gpu_util import dev, import_library
from tests.test_gpu_pages import as_table, assert_caches, ints, moved, new_caches, run_fork, sequences

pytestmark = pytest.mark.gpu

mxa = import_library()


@pytest.mark.parametrize("kind", ["beams", "branch", "grow", "stay"])
@pytest.mark.parametrize("pages,rows,cols", [(16384, 1025, 5), (16385, 90, 9), (20000, 700, 33)])
def test_fork_in_place(pages, rows, cols, kind):
    """Counts changed where they stand, more pages, rows or entries than one workgroup plans."""
    run_fork(random.Random(pages + rows), pages, 16, cols, rows, kind=kind, outside=pages // 20, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("release", [False, True])
@pytest.mark.parametrize("pages,rows,cols,children", [
    (9000, 4096, 3, 16384),      # the most that are counted in LDS
    (9000, 4097, 3, 6000), (9000, 700, 3, 16385), (60000, 5000, 6, 20000),
    (150000, 17000, 5, 70000)])  # more rows than a grid's workgroups take at once, more than 256 blocks of children
def test_fork_of_many_rows_and_children(pages, rows, cols, children, release, in_place):
    r = random.Random(rows + children)
    refs, table, lens = sequences(r, pages, 16, cols, rows, 0.6, outside=pages // 50)
    parents = [r.randint(-1, rows) if r.random() < 0.7 else r.randint(0, 5) for _ in range(children)]
    new = [r.choice([0, 0, 1, 1, 1, 2, 17]) for _ in range(children)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    want = op.fork(refs, table, lens, 16, cu, parents, release, cu[-1], cols)
    assert want[4], "partly filled pages must be copied"
    caches = new_caches(1, pages, 1, 16, 64, rows)
    content = caches[0].k.clone(), caches[0].v_scales.clone()
    src, dst, n = (torch.tensor(x, device=dev()) for x in zip(*want[4]))
    for t in content:
        keep = torch.arange(16, device=dev()) >= n[:, None]
        t[dst] = torch.where(keep[:, None, :, None], t[dst], t[src])
    counts = ints(refs)
    out = (counts, ints([[77] * cols]).repeat(children, 1), ints([55] * children), ints([99] * cu[-1], torch.int64))
    got = mxa.mx_kv_fork(caches, counts, as_table(table, cols), ints(lens), ints(cu), ints(parents), release, cu[-1],
                         out=out if in_place else None)
    assert got.lens.tolist() == want[2]
    assert got.page_table.tolist() == want[1]
    assert got.refs.tolist() == want[0]
    assert got.slots.tolist() == want[3]
    assert torch.equal(caches[0].k, content[0]) and torch.equal(caches[0].v_scales, content[1])
    if not in_place:
        assert counts.tolist() == refs


def holds(table, lens, keep, pages, page):
    """Lengths after a free, and how many holds each page loses: the rule on whole tensors."""
    cols = table.shape[1]
    had = lens.long().clamp(0, cols * page)
    left = torch.zeros_like(had) if keep is None else torch.minimum(had, keep.long().clamp_min(0))
    lost = torch.zeros(pages + 1, dtype=torch.int64, device=dev())
    step = max(1, 2 ** 25 // cols)
    for i in range(0, table.shape[0], step):
        j = torch.arange(cols, device=dev()) * page
        gone = (j >= -(-left[i:i + step] // page)[:, None] * page) & (j < had[i:i + step, None])
        gone &= (table[i:i + step] >= 0) & (table[i:i + step] < pages)
        lost += torch.bincount(torch.where(gone, table[i:i + step], pages).flatten().long(), minlength=pages + 1)
    return left.int(), lost[:pages]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("order", ["anywhere", "in a row", "few pages"])
@pytest.mark.parametrize("pages,rows,cols,more", [
    (16385, 1024, 512, 0),              # the fewest entries and pages that are put in order
    (100000, 1024, 700, 5),             # part of a wider table
    (2097153, 2100, 300, 3), (4194305, 3000, 250, 0), (8388608, 1 << 20, 1, 0),      # buckets of 2^14 and of 2^15 pages
    (8388609, 3000, 250, 2),            # more pages than buckets hold
    (300000, 3000, 3001, 7)])           # more than 1024 tiles
def test_free_of_many_entries(pages, rows, cols, more, order, in_place):
    page = 16
    g = torch.Generator(device=dev()).manual_seed(pages + cols)
    rand = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device=dev(), dtype=torch.int32)  # noqa: E731
    if order == "anywhere":
        table = rand(-3, pages + 3, rows, cols + more)
    elif order == "in a row":
        table = (torch.arange(rows * (cols + more), device=dev()) % pages).int().view(rows, cols + more)
    else:
        table = rand(0, 3, rows, cols + more) * (pages // 2 - 1)
    table = table[:, :cols]
    lens = rand(-20, cols * page + 20, rows)
    for keep in (None, torch.where(rand(0, 9, rows) == 0, rand(-5, cols * page, rows), lens)):
        left, lost = holds(table, lens, keep, pages, page)
        refs = (lost + rand(0, 3, pages)).int()
        want = (refs - lost).int()
        counts, length = refs.clone(), lens.clone()
        got = mxa.mx_kv_free(counts, table, length, page, keep, (counts, length) if in_place else None)
        assert torch.equal(got[0], want) and torch.equal(got[1], left)
        if not in_place:
            assert torch.equal(counts, refs) and torch.equal(length, lens)


@pytest.mark.parametrize("rows", [1 << 14, (1 << 14) + 1])
def test_free_of_the_most_entries_in_order(rows):
    """2^28 entries, and more, which are not put in order."""
    pages, cols, page = 1000000, 1 << 14, 16
    g = torch.Generator(device=dev()).manual_seed(rows)
    table = torch.randint(0, pages, (rows, cols), generator=g, device=dev(), dtype=torch.int32)
    lens = torch.randint(0, cols * page, (rows,), generator=g, device=dev(), dtype=torch.int32)
    keep = lens // 2
    left, lost = holds(table, lens, keep, pages, page)
    refs = (lost + 1).int()
    got = mxa.mx_kv_free(refs, table, lens, page, keep)
    assert bool((got[0] == 1).all()) and torch.equal(got[1], left)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pages,rows,cols,layers", [(16384, 900, 20, 1), (16385, 900, 20, 1), (70001, 3000, 30, 2),
                                                    (20480, 0, 1, 33)])
def test_compact_of_large_pools(pages, rows, cols, layers, in_place):
    r = random.Random(pages)
    for fill in (0.0, 0.4, 0.8, 1.0):
        refs, table, lens = sequences(r, pages, 16, cols, rows, fill, outside=int(pages * fill / 3))
        if fill == 1.0:         # none free
            refs = [max(n, 1) for n in refs]
        want = op.compact(refs, table, lens, 16)
        caches = new_caches(layers, pages, 1, 16, 64, pages)
        content = [[t.clone() for t in c] for c in caches]
        if want[3]:
            src, dst = torch.tensor(want[3], device=dev()).unbind(1)
            for c in content:
                for t in c:
                    t[dst] = t[src]
        counts, rows_in = ints(refs), as_table(table, cols)
        got = mxa.mx_kv_compact(caches, counts, rows_in, ints(lens), (counts, rows_in, ints([-1])) if in_place else None)
        assert got[2].item() == want[2]
        assert got[0].tolist() == want[0]
        assert got[1].tolist() == want[1]
        assert_caches(caches, content)
        if not in_place:
            assert counts.tolist() == refs and rows_in.tolist() == table


@pytest.mark.parametrize("in_place", [False, True])
def test_pool_of_more_pages_than_counting_blocks_read_at_once(in_place):
    """Over 2^24 pages a counting block goes over several runs of 4096."""
    pages, page = (1 << 24) + 5000, 16
    g = torch.Generator(device=dev()).manual_seed(3)
    cache = mxa.new_kv_cache(pages, 1, page, 64)
    # some 3000 pages in use, many of them next to the borders of runs and blocks
    at = torch.randint(0, pages // 4096, (3000,), generator=g, device=dev()) * 4096
    at = (at + torch.randint(-3, 4, (3000,), generator=g, device=dev())).clamp(0, pages - 1).unique()
    refs = torch.zeros(pages, dtype=torch.int32, device=dev())
    refs[at] = torch.randint(1, 9, at.shape, generator=g, device=dev(), dtype=torch.int32)
    used = at.numel()
    for t in cache:
        t[at] = torch.randint(0, 256, t[at].shape, generator=g, device=dev(), dtype=torch.uint8)
    before = [t[at].clone() for t in cache]
    order = torch.randperm(used, generator=g, device=dev())[:2000]
    table = at[order].int().view(40, 50)
    counts, rows = refs.clone(), table.clone()
    got = mxa.mx_kv_compact(cache, counts, rows, ints([50 * page] * 40), (counts, rows, ints([0])) if in_place else None)
    holes = (refs[:used] == 0).nonzero()[:, 0]
    goes = at.clone()
    goes[used - holes.numel():] = holes.flip(0)            # the nth free page takes the nth used one from the end
    assert bool((goes < used).all()) and got[2].item() == used
    assert torch.equal(got[1], goes[order].int().view(40, 50))
    assert torch.equal(got[0][goes], refs[at]) and not got[0][used:].any()
    for t, x in zip(cache, before):
        assert torch.equal(t[goes], x)
    # the other way round: as many free as were in use, given to three new sequences
    refs = torch.ones(pages, dtype=torch.int32, device=dev())
    refs[at] = 0
    new = [700 * page, 800 * page - 3, 5 * page]
    cu = [0, new[0], new[0] + new[1], sum(new)]
    counts = refs.clone()
    table = ints([[0] * 800] * 3)
    out = (counts, table.clone(), ints([9] * 3), ints([9] * cu[3], torch.int64)) if in_place else None
    for parents in (None, ints([-1, -1, -1])):
        counts.copy_(refs)
        got = mxa.mx_kv_fork(cache, counts, table, ints([0] * 3), ints(cu), parents, tokens=cu[3], out=out)
        assert got.lens.tolist() == new
        left = torch.full_like(got.page_table, -1)
        taken = 0
        for row, n in enumerate((700, 800, 5)):
            left[row, :n] = at[taken:taken + n].int()
            slot = (at[taken:taken + n, None] * page + torch.arange(page, device=dev())).flatten()[:new[row]]
            assert torch.equal(got.slots[cu[row]:cu[row + 1]], slot)
            taken += n
        assert torch.equal(got.page_table, left)
        want = refs.clone()
        want[at[:taken]] = 1
        assert torch.equal(got.refs, want)


def test_replayed_graph_of_large_calls():
    """A captured fork, compaction and free of the sizes that take several launches, replayed on changing inputs with eager
    calls between."""
    page, cols, rows, pages = 16, 600, 900, 30000
    r = random.Random(4)
    cache = new_caches(1, pages, 1, page, 64, 3)
    static = (ints([0] * pages), as_table([[0] * cols] * rows, cols), ints([0] * rows), ints([0] * rows), ints([0] * (rows + 1)))

    def step():
        refs, table, lens, parents, cu = static
        f = mxa.mx_kv_fork(cache, refs, table, lens, cu, parents, True, 2500)
        c = mxa.mx_kv_compact(cache, f.refs, f.page_table, f.lens)
        return f, c, mxa.mx_kv_free(c[0], c[1], f.lens, page, f.lens // 2)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for turn in range(5):
        refs, table, lens = sequences(r, pages, page, cols, rows, 0.5)
        parents = [r.randint(0, rows - 1) for _ in range(rows)]
        cu = [0]
        for _ in range(rows):
            cu.append(cu[-1] + r.randint(0, 5))
        cu = [min(n, 2500) for n in cu]
        for t, x in zip(static, (refs, table, lens, parents, cu)):
            t.copy_(ints(x))
        want = op.fork(refs, table, lens, page, cu, parents, True, 2500)
        want_c = op.compact(want[0], want[1], want[2], page)
        want_f = op.free(want_c[0], want_c[1], want[2], page, [n // 2 for n in want[2]])
        content = moved([mxa.KVCache(*x) for x in moved(cache, want[4])], [(a, b, page) for a, b in want_c[3]])
        if turn == 2:
            f, c, z = step()
        else:
            graph.replay()
            f, c, z = outs
        assert (f.refs.tolist(), f.page_table.tolist(), f.lens.tolist(), f.slots.tolist()) == want[:4]
        assert (c[0].tolist(), c[1].tolist(), c[2].item()) == want_c[:3]
        assert (z[0].tolist(), z[1].tolist()) == want_f
        assert_caches(cache, content)
