"""Pages of a paged cache: forked, freed, moved together (plain Python over lists).

A pool is a list of counts (0: free); a sequence a row of page numbers and a length.
Nothing here is vectorised or parallel: one sequence after the other, as the rules read.
"""


def held(n, page):
    """Pages that n tokens fill, the last one perhaps in part."""
    return -(-n // page)


def _length(n, cols, page):
    return min(max(n, 0), cols * page)


def fork(refs, table, lens, page, cu=None, parents=None, release=True, tokens=0, cols=None):
    """Returns (refs, table, lens, slots, copies), copies a list of (source page, page, tokens)."""
    pages, old_cols = len(refs), len(table[0]) if table else 0
    cols = old_cols if cols is None else cols
    refs = list(refs)
    rows = [(list(row[:held(_length(n, old_cols, page), page)]), _length(n, old_cols, page))
            for row, n in zip(table, lens)]
    parents = list(range(len(rows))) if parents is None else list(parents)
    cut = lambda x: min(max(x, 0), tokens)  # noqa: E731
    spans = [(cut(cu[i]), max(cut(cu[i]), cut(cu[i + 1]))) if cu is not None else (0, 0) for i in range(len(parents))]
    at = lambda p: rows[p] if 0 <= p < len(rows) else ([], 0)  # noqa: E731
    for p in parents:
        for q in at(p)[0]:
            if 0 <= q < pages:
                refs[q] += 1
    if release:
        for row, _ in rows:
            for q in row:
                if 0 <= q < pages:
                    refs[q] -= 1
    free = [q for q in range(pages) if refs[q] == 0]
    shared = list(refs)
    writers = {}
    for i, p in enumerate(parents):
        if spans[i][1] > spans[i][0] and at(p)[1] % page:
            writers.setdefault(p, []).append(i)
    out, new_lens, slots, copies, taken = [], [], [-1] * tokens, [], 0
    for i, p in enumerate(parents):
        row, n = list(at(p)[0]), at(p)[1]
        lo, hi = spans[i]
        after = held(n + hi - lo, page)
        if hi > lo:
            mine = writers.get(p, ())
            copy = i in mine and 0 <= row[-1] < pages and not (mine[0] == i and shared[row[-1]] == len(mine))
            need = copy + after - len(row)
            taken += need                    # also by a child that gets none of them
            if after <= cols and (need == 0 or taken <= len(free)):
                new = free[taken - need:taken]
                if copy:
                    copies.append((row[-1], new[0], -(-(n % page) // 16) * 16))
                    refs[row.pop()] -= 1
                row += new
                for q in new:
                    refs[q] = 1
                for t in range(lo, hi):
                    q, place = row[(n + t - lo) // page], (n + t - lo) % page
                    slots[t] = q * page + place if 0 <= q < pages else -1
                n += hi - lo
        out.append(row + [-1] * (cols - len(row)))
        new_lens.append(n)
    return refs, out, new_lens, slots, copies


def free(refs, table, lens, page, keep=None):
    """Returns (refs, lens)."""
    refs, cols = list(refs), len(table[0]) if table else 0
    left = []
    for i, (row, n) in enumerate(zip(table, lens)):
        n = _length(n, cols, page)
        k = min(n, 0 if keep is None else max(keep[i], 0))
        for q in row[held(k, page):held(n, page)]:
            if 0 <= q < len(refs):
                refs[q] -= 1
        left.append(k)
    return refs, left


def compact(refs, table, lens, page):
    """Returns (refs, table, pages in use, moves), moves a list of (page, its new number)."""
    refs, cols = list(refs), len(table[0]) if table else 0
    live = [q for q, n in enumerate(refs) if n != 0]
    used, goes = len(live), {}
    for q in range(used):
        if refs[q] == 0:
            goes[live.pop()] = q
    for src, dst in goes.items():
        refs[dst], refs[src] = refs[src], 0
    out = [[goes.get(q, q) if j < held(_length(n, cols, page), page) else q for j, q in enumerate(row)]
           for row, n in zip(table, lens)]
    return refs, out, used, list(goes.items())
