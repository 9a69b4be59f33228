"""Page tables and slot maps of a paged key/value cache, in plain Python.

Test infrastructure only (see the package docstring): written from the
definitions in include/specdec_verify.h, sharing no code with the library.
"""
from __future__ import annotations

import copy

import numpy as np

OK, INVALID, NO_PAGES = 0, -1, -7


def plan(table, held, free, n_free, start, counts, page, n=None, cu_rows=None, n_slots=None):
    """(table, held, free, n_free, map or None, status) after a plan; lists of ints in and out.

    `n` rows of a sequence in the map, or with cu_rows `n_slots` in all; neither: no map.
    """
    table, held, free = copy.deepcopy(table), list(held), list(free)
    B, max_pages, n_pages = len(table), len(table[0]) if table else 0, len(free)
    mapped = n is not None or n_slots is not None
    total = 0 if not mapped else B * n if cu_rows is None else n_slots
    slots = [-1] * total
    good = []
    if cu_rows is not None and not all(0 <= lo <= hi <= total for lo, hi in zip(cu_rows, cu_rows[1:])):
        return table, held, free, n_free, slots, INVALID
    for b in range(B):
        ok = start[b] >= 0 and counts[b] >= 0 and start[b] + counts[b] <= max_pages * page
        ok = ok and 0 <= held[b] <= max_pages
        if ok and mapped:
            if cu_rows is None:
                ok = counts[b] <= n
            else:
                ok = counts[b] <= cu_rows[b + 1] - cu_rows[b]
        good.append(ok)
    status = OK if all(good) else INVALID
    want = [-(-(start[b] + counts[b]) // page) if good[b] else held[b] for b in range(B)]
    back = [(b, x) for b in range(B) if good[b] for x in range(want[b], held[b])]
    more = [(b, x) for b in range(B) if good[b] for x in range(held[b], want[b])]
    if not 0 <= n_free <= n_pages or len(back) > n_pages - n_free:
        return table, held, free, n_free, slots if mapped else None, INVALID
    if len(more) > n_free + len(back):
        return table, held, free, n_free, slots if mapped else None, NO_PAGES
    for b, x in back:
        if not 0 <= table[b][x] < n_pages:
            status = INVALID
        free[n_free] = table[b][x]
        table[b][x] = -1
        n_free += 1
    for b, x in more:
        n_free -= 1
        table[b][x] = free[n_free]
        if not 0 <= table[b][x] < n_pages:
            status = INVALID
    held = want
    if mapped:
        for b in range(B):
            if not good[b]:
                continue
            at = b * n if cu_rows is None else cu_rows[b]
            for i in range(counts[b]):
                row = start[b] + i
                p = table[b][row // page]
                if 0 <= p < n_pages:
                    slots[at + i] = p * page + row % page
                else:
                    status = INVALID
    return table, held, free, n_free, slots if mapped else None, status


def gather(pages, table, L) -> np.ndarray:
    """Rows 0 .. L - 1 of one sequence out of pages [n_pages, page, Hkv, D]; pages that are none: zeros."""
    page = pages.shape[1]
    out = np.zeros((L, *pages.shape[2:]), dtype=np.float64)
    for j in range(L):
        p = int(table[j // page])
        if 0 <= p < pages.shape[0]:
            out[j] = pages[p, j % page]
    return out
