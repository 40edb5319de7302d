"""Host reference of the page bookkeeping (plx_kv_update, plx_kv_compact): plain
lists, one row after the other."""


def pages_of(n, page):
    return -(-n // page)


def update(table, lens, refs, want, src, page):
    """(rows, new lens, new refs, copies): rows[b] the pages of row b afterwards,
    copies (from, to, slots)."""
    B, refs = len(lens), list(refs)
    src = list(range(B)) if src is None else src
    held = [table[b][:pages_of(lens[b], page)] for b in range(B)]
    keeps = [0 if s < 0 else max(0, min(want[b], lens[s])) for b, s in enumerate(src)]
    for b in range(B):
        for p in held[b]:
            refs[p] -= 1
    rows = [[] if s < 0 else list(held[s][:keeps[b] // page]) for b, s in enumerate(src)]
    for row in rows:
        for p in row:
            refs[p] += 1
    # Partial last pages, by page: the first row keeps it unless it is somewhere whole.
    copying = {}
    takers = {}
    for b, s in enumerate(src):
        if keeps[b] % page:
            takers.setdefault(held[s][keeps[b] // page], []).append(b)
    for p, bs in takers.items():
        if refs[p] == 0:
            rows[bs[0]].append(p)
            refs[p] = 1
            bs = bs[1:]
        for b in bs:
            copying[b] = p
    free = [p for p in range(len(refs)) if refs[p] == 0]
    new, copies, dry = [], [], False
    for b in range(B):
        need = pages_of(max(want[b], 0), page) - len(rows[b])
        dry = dry or need > len(free)
        if need > 0 and dry:
            new.append(len(rows[b]) * page if b in copying else keeps[b])
            continue
        got, free = free[:need], free[need:]
        for p in got:
            refs[p] = 1
        if b in copying:
            copies.append((copying[b], got[0], keeps[b] % page))
        rows[b] += got
        new.append(max(want[b], 0))
    return rows, new, refs, copies


def compact(table, lens, refs, page):
    """(rows, new refs, map, used)."""
    used = [p for p, n in enumerate(refs) if n > 0]
    holes = iter([p for p in range(len(used)) if refs[p] <= 0])
    to = {p: (p if p < len(used) else next(holes)) for p in used}
    new = [0] * len(refs)
    for p in used:
        new[to[p]] = refs[p]
    rows = [[to[p] for p in table[b][:pages_of(n, page)]] for b, n in enumerate(lens)]
    return rows, new, [to.get(p, -1) for p in range(len(refs))], len(used)
