"""The paged cache's bookkeeping, one sequence and one page at a time.

Plain Python over numpy arrays, from the definitions: a pool is its reference
counts, a page is free when its count is 0, the lowest free page is handed out
first.  Functions change their arguments in place, as the calls do.
"""
import numpy as np


def fork(src_table, src_lengths, refs, parents):
    """(table, lengths) of the rows that continue parents[b]; refs is updated."""
    table = np.full((len(parents), src_table.shape[1]), -1, np.int32)
    lengths = np.zeros(len(parents), np.int64)
    for b, p in enumerate(parents):
        if p < 0:
            continue
        table[b], lengths[b] = src_table[p], src_lengths[p]
        for page in table[b][table[b] >= 0]:
            refs[page] += 1
    for row in src_table:                      # the old rows end
        for page in row[row >= 0]:
            refs[page] -= 1
    return table, lengths


def free(table, refs, lengths, keep, page_size):
    for b in range(len(table)):
        n = 0 if keep is None else min(int(lengths[b]), int(keep[b]))
        for j in range(-(-n // page_size), table.shape[1]):
            if table[b, j] >= 0:
                refs[table[b, j]] -= 1
                table[b, j] = -1
        lengths[b] = n


def reserve(table, refs, lengths, new, page_size):
    """The copies (old, new), or None (nothing changed) if pages do not suffice."""
    t, r, copies = table.copy(), refs.copy(), []
    idle = [int(p) for p in np.flatnonzero(refs == 0)]
    for b in range(len(t)):
        if new[b] == 0:
            continue
        first, last = int(lengths[b]) // page_size, (int(lengths[b]) + int(new[b]) - 1) // page_size
        for j in range(first, last + 1):
            old = t[b, j]
            if old >= 0 and r[old] <= 1:
                continue
            if not idle:
                return None
            got = idle.pop(0)
            r[got] = 1
            t[b, j] = got
            if old >= 0:
                r[old] -= 1
                if j == first and lengths[b] % page_size:
                    copies.append((int(old), got))
    table[:], refs[:] = t, r
    return copies


def compact(table, refs, most):
    """The moves (from, to): the highest live page into the lowest free one."""
    moves = []
    while len(moves) < most:
        live, idle = np.flatnonzero(refs > 0), np.flatnonzero(refs == 0)
        if not len(live) or not len(idle) or idle[0] > live[-1]:
            break
        src, dst = int(live[-1]), int(idle[0])
        refs[dst], refs[src] = refs[src], 0
        table[table == src] = dst
        moves.append((src, dst))
    return moves


def copy(cache, pairs):
    """cache [layers][num_pages][...]."""
    for src, dst in pairs:
        cache[:, dst] = cache[:, src]


def keep_rows(cache, lengths, keep, table, page_size):
    """cache [layers][num_pages * page_size][...]; keep: a list of positions for each sequence."""
    for b, kept in enumerate(keep):
        def row(i):
            p = int(lengths[b]) + i
            return int(table[b, p // page_size]) * page_size + p % page_size
        rows = [cache[:, row(i)].copy() for i in kept]
        for k, x in enumerate(rows):
            cache[:, row(k)] = x
