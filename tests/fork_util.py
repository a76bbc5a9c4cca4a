"""A plain statement of fa_cache_fork that covers lost tails and all-or-nothing calls."""
from paged_util import cdiv


def fork(table, lens, refs, source, room, page, whole=False):
    """(table, lens, refs, missing, tails) after a call on plain lists; tails: (from page, to page, rows).

    A sequence whose partly filled page is not in the table has lost its tail: it and its copies get no
    pages, and all that they would need from there on lack."""
    Z, M = len(table), len(table[0])
    out, new, counts = [list(r) for r in table], list(lens), list(refs)
    free = [p for p, c in enumerate(refs) if c == 0]
    missing, tails = 0, []
    for z in range(Z):
        a = z if source is None else source[z]
        n = lens[a] if a >= 0 else 0
        new[z] = n
        if a != z:
            for p in table[z]:
                if p >= 0:
                    counts[p] -= 1
            out[z] = [table[a][c] if a >= 0 and c < n // page else -1 for c in range(M)]
            for p in out[z]:
                if p >= 0:
                    counts[p] += 1
        need = cdiv(n + room, page) if a >= 0 else 0
        if a >= 0 and n % page and table[a][n // page] < 0:
            missing += need - n // page
            continue
        for c in range(n // page, need):
            if c >= M:
                missing += 1
            elif out[z][c] < 0:
                if not free:
                    missing += 1
                    continue
                p = out[z][c] = free.pop(0)
                counts[p] += 1
                if a != z and c == n // page and n % page:
                    tails.append((table[a][c], p, n % page))
    if whole and missing:
        return [list(r) for r in table], list(lens), list(refs), missing, []
    return out, new, counts, missing, tails
