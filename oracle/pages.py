"""Oracle of a page pool's steps (test infrastructure): one page after another,
in lists.

A pool is ``refs`` (holders per page), and ``rows``: per request its length and
its list of pages.  ``extend`` also returns the page copies it asks for.

Written from the definitions; shares no code with the GPU package.
"""

from __future__ import annotations


def pages_of(n, block):
    return (n + block - 1) // block


def extend(refs, rows, lens, add, block, max_pages):
    """(missing, copies): rows, lens and refs are changed unless missing."""
    if any(n < 0 or a < 0 or n + a > 2 ** 31 - 1 or pages_of(n + a, block) > max_pages for n, a in zip(lens, add)):
        return -1, []
    need = []
    for row, n, a in zip(rows, lens, add):
        shared = a > 0 and n % block > 0 and 0 <= row[n // block] < len(refs) and refs[row[n // block]] > 1
        need.append((shared, pages_of(n + a, block) - pages_of(n, block) + shared))
    free = [i for i, r in enumerate(refs) if r <= 0]
    wanted = sum(w for _, w in need)
    if wanted > len(free):
        return wanted - len(free), []
    copies, at = [], 0
    for b, (shared, w) in enumerate(need):
        new = free[at:at + w]
        at += w
        if shared:
            old = rows[b][lens[b] // block]
            copies.append((old, new[0], lens[b] % block))
            rows[b][lens[b] // block] = new.pop(0)
        rows[b].extend(new)
    for page in free[:at]:
        refs[page] = 1
    for old, _, _ in copies:
        refs[old] -= 1
    for b, a in enumerate(add):
        lens[b] += a
    return 0, copies


def fork(refs, rows, lens, parents):
    """The new rows and lengths."""
    for row in rows:
        for page in row:
            if 0 <= page < len(refs):
                refs[page] -= 1
    some = [0 <= p < len(rows) for p in parents]
    new = [list(rows[p]) if s else [] for p, s in zip(parents, some)]
    for row in new:
        for page in row:
            if 0 <= page < len(refs):
                refs[page] += 1
    return new, [lens[p] if s else 0 for p, s in zip(parents, some)]


def trim(refs, rows, lens, keep, block):
    for b, k in enumerate(keep):
        if 0 <= k < lens[b]:
            for page in rows[b][pages_of(k, block):]:
                if 0 <= page < len(refs):
                    refs[page] -= 1
            rows[b] = rows[b][:pages_of(k, block)]
            lens[b] = k


def compact(refs, rows):
    """(map, moves as (src, dst), live): refs and rows are changed."""
    live = [i for i, r in enumerate(refs) if r > 0]
    n = len(live)
    moves = list(zip([i for i in live if i >= n], [i for i in range(n) if refs[i] <= 0]))
    to = {i: i for i in live if i < n}
    to.update(moves)
    for src, dst in moves:
        refs[dst], refs[src] = refs[src], 0
    for row in rows:
        row[:] = [to.get(page, page) for page in row]
    return [to.get(i, -1) for i in range(len(refs))], moves, n
