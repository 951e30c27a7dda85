"""Plain host forms of shared pages: fork and compact, in Python integers."""


def blocks_of(n, page):
    return -(-n // page)


def fork(lens, parents, keep, table, page, free, count):
    """(lens, table, count, copies, free) after the fork."""
    seats, pages = len(lens), len(free)
    width = len(table[0]) if table else 0
    free = list(free)
    top = min(max(count, 0), pages)
    held = [min(max(n, 0), width * page) for n in lens]

    def is_page(p):
        return 0 <= p < pages

    take, rows = [], []
    for d in range(seats):
        p = parents[d]
        n = held[p] if 0 <= p < seats else 0
        if keep is not None:
            n = min(n, max(keep[d], 0))
        take.append(n)
        rows.append(table[p][:blocks_of(n, page)] if n else [])
    before = {e for n, row in zip(held, table) for e in row[:blocks_of(n, page)] if is_page(e)}
    after = {e for row in rows for e in row if is_page(e)}
    for e in sorted(before - after):
        if top < pages:
            free[top] = e
            top += 1
    whole = {e for n, row in zip(take, rows) for e in row[:n // page] if is_page(e)}
    ends = {}
    for d, (n, row) in enumerate(zip(take, rows)):
        if n % page and is_page(row[-1]):
            ends.setdefault(row[-1], []).append(d)
    copies = [[-1, -1] for _ in range(seats)]
    for d, (n, row) in enumerate(zip(take, rows)):
        if n % page == 0 or not is_page(row[-1]):
            continue
        tail = row[-1]
        if tail not in whole and ends[tail][0] == d:
            continue
        got = -1  # an entry of the list that is no page is none
        if top > 0:
            top -= 1
            got = free[top]
        if is_page(got):
            copies[d] = [tail, got]
            row[-1] = got
        else:
            del row[-1]
            take[d] = n - n % page
    return take, [row + [-1] * (width - len(row)) for row in rows], top, copies, free


def compact(lens, table, page, free, count):
    """(table, free, count, moves, map) after the compaction."""
    pages = len(free)
    top = min(max(count, 0), pages)
    idle = {p for p in free[:top] if 0 <= p < pages}
    used = pages - len(idle)
    number = [-1 if p in idle else p for p in range(pages)]
    holes = sorted(p for p in idle if p < used)
    movers = [p for p in range(used, pages) if p not in idle]
    assert len(holes) == len(movers)
    for a, b in zip(movers, holes):
        number[a] = b
    out = [[number[e] if b * page < n and 0 <= e < pages else e for b, e in enumerate(row)] for n, row in zip(lens, table)]
    moves = [[a, b] for a, b in zip(movers, holes)]
    moves += [[-1, -1]] * (pages // 2 - len(moves))
    return out, [pages - 1 - i for i in range(pages - used)] + [-1] * used, pages - used, moves, number
