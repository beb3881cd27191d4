"""The page oracle against what it is for: every sequence reads its own tokens, and counts are holders.

A model of the cache follows it: each page holds the token that was written at each place, so that
a sequence's content can be read back through its row after any number of steps."""

import random

import pytest

from oracle import pages as op


class Model:
    """Sequences with the tokens they should hold, and pages with those they do."""

    def __init__(self, pages, page, cols, fork=op.fork):
        self.page, self.cols, self.fork = page, cols, fork
        self.refs = [0] * pages
        self.content = [[None] * page for _ in range(pages)]
        self.table, self.lens, self.want, self.stamp = [], [], [], 0

    def step(self, parents, new, release):
        cu = [sum(new[:i]) for i in range(len(new) + 1)]
        refs, table, lens, slots, copies = self.fork(self.refs, self.table, self.lens, self.page, cu, parents, release,
                                                     cu[-1], self.cols)
        for src, dst, n in copies:
            self.content[dst][:n] = self.content[src][:n]
        want = []
        for i, p in enumerate(parents):
            old = self.want[p] if 0 <= p < len(self.want) else []
            got = lens[i] - len(old)
            assert got in (0, new[i])
            assert (got == 0) == all(s < 0 for s in slots[cu[i]:cu[i + 1]])
            fresh = []
            for s in slots[cu[i]:cu[i + 1]] if got else ():
                self.stamp += 1
                self.content[s // self.page][s % self.page] = self.stamp
                fresh.append(self.stamp)
            want.append(old + fresh)
        if release:
            self.table, self.lens, self.want = table, lens, want
        else:
            self.table, self.lens, self.want = self.table + table, self.lens + lens, self.want + want
        self.refs = refs
        self.check()

    def check(self):
        count = [0] * len(self.refs)
        for row, n, want in zip(self.table, self.lens, self.want):
            used = row[:op.held(n, self.page)]
            assert [self.content[used[t // self.page]][t % self.page] for t in range(n)] == want
            for q in used:
                count[q] += 1
        assert count == self.refs


def play(seed, fork=op.fork, steps=40):
    r = random.Random(seed)
    m = Model(r.choice([12, 40, 200]), 16, r.choice([3, 8, 20]), fork)
    for _ in range(steps):
        rows = len(m.lens)
        n = r.randint(1, 6)
        parents = [r.randint(0, rows - 1) if rows and r.random() < 0.9 else -1 for _ in range(n)]
        m.step(parents, [r.choice([0, 1, 1, 1, 5, 16, 33]) for _ in range(n)], r.random() < 0.7 or rows > 12)
        if r.random() < 0.3:
            keep = [r.choice([0, n, n - 1, n - 20, n + 4]) for n in m.lens]
            m.refs, m.lens = op.free(m.refs, m.table, m.lens, m.page, keep)
            m.want = [w[:n] for w, n in zip(m.want, m.lens)]
            m.check()
        if r.random() < 0.2:
            m.refs, m.table, used, moves = op.compact(m.refs, m.table, m.lens, m.page)
            for src, dst in moves:
                m.content[dst] = list(m.content[src])
                m.content[src] = [None] * m.page
            assert used == sum(n > 0 for n in m.refs) and all(n == 0 for n in m.refs[used:])
            m.check()


@pytest.mark.parametrize("seed", range(30))
def test_sequences_read_their_own_tokens(seed):
    play(seed)


def planted_no_copy(refs, table, lens, page, cu, parents, release, tokens, cols):
    """Every writer keeps the page it shares."""
    out = op.fork(refs, table, lens, page, cu, parents, release, tokens, cols)
    return (*out[:4], []) if out[4] else out


def planted_release_twice(refs, table, lens, page, cu, parents, release, tokens, cols):
    refs, *rest = op.fork(refs, table, lens, page, cu, parents, release, tokens, cols)
    return ([max(n - 1, 0) for n in refs], *rest)


@pytest.mark.parametrize("fork", [planted_no_copy, planted_release_twice])
def test_planted_mistakes_show(fork):
    with pytest.raises(AssertionError):
        for seed in range(30):
            play(seed, fork)


def test_small_fork_by_hand():
    # a row of 20 tokens in pages 3 and 1, and its two children with one new token each: page 3 is shared, page 1 stays
    # with the first and goes to page 0, the lowest free one, for the second
    refs, table, lens, slots, copies = op.fork([0, 1, 0, 1], [[3, 1, 9]], [20], 16, [0, 1, 2], [0, 0], True, 2)
    assert (refs, table, lens) == ([1, 1, 0, 2], [[3, 1, -1], [3, 0, -1]], [21, 21])
    assert (slots, copies) == ([1 * 16 + 4, 0 * 16 + 4], [(1, 0, 16)])
    # kept beside them, the row holds its last page too: both get copies
    refs, table, _, slots, copies = op.fork([0, 1, 0, 1], [[3, 1, 9]], [20], 16, [0, 1, 2], [0, 0], False, 2)
    assert (refs, table) == ([1, 1, 1, 3], [[3, 0, -1], [3, 2, -1]])
    assert (slots, copies) == ([4, 36], [(1, 0, 16), (1, 2, 16)])
    # one free page for two children that need one each: the second keeps its length
    refs, table, lens, slots, _ = op.fork([1, 1, 0], [[0], [1]], [16, 16], 16, [0, 1, 2], None, True, 2, 2)
    assert (refs, table, lens, slots) == ([1, 1, 1], [[0, 2], [1, -1]], [17, 16], [32, -1])


def test_pages_of_a_child_too_wide_are_not_given_to_later_ones():
    # the first child would need three pages in a row of two: the second gets the fourth free one
    assert op.fork([0] * 6, [[0, 0]] * 2, [0, 0], 16, [0, 40, 41], None, True, 41) == \
        ([0, 0, 0, 1, 0, 0], [[-1, -1], [3, -1]], [0, 1], [-1] * 40 + [48], [])
    # three free pages: none is left for it
    assert op.fork([0] * 3, [[0, 0]] * 2, [0, 0], 16, [0, 40, 41], None, True, 41) == \
        ([0] * 3, [[-1, -1]] * 2, [0, 0], [-1] * 41, [])
    # a copy that the first asked for counts too: two new pages, and one for the partly filled one
    assert op.fork([1, 1] + [0] * 5, [[0, 1]], [20], 16, [0, 40, 41], [0, 0], False, 41) == \
        ([3, 2, 0, 0, 0, 1, 0], [[0, 1], [0, 5]], [20, 21], [-1] * 40 + [84], [(1, 5, 16)])


def test_small_compact_by_hand():
    refs, table, used, moves = op.compact([0, 2, 0, 0, 1, 3], [[5, 1, 4], [4, 5, 5]], [33, 10], 16)
    assert (refs, used, moves) == ([3, 2, 1, 0, 0, 0], 3, [(5, 0), (4, 2)])
    assert table == [[0, 1, 2], [2, 5, 5]]
