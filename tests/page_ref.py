"""One step of page tables, request by request, from its definition."""
from __future__ import annotations


def step(table, lengths, new, free, count, q, page, block_rows):
    """Plain lists in; (positions, slots, valid, granted, table, free, lengths, count) out."""
    table, free = [list(r) for r in table], list(free)
    width = (len(table[0]) if table else 0) * page
    size, count = len(free), min(max(count, 0), len(free))
    asked = taken = 0
    positions, slots, valid, granted, after = [], [], [], [], []
    gone = []
    for r, ask in enumerate(new):
        n = min(max(lengths[r], 0), width)
        own = -(-n // page)
        add = min(max(ask, 0), q)
        if n + add > width:
            add = 0
        need = -(-(n + add) // page) - own
        asked += need
        if need and asked > count:
            add = 0
        elif need:
            for i in range(need):
                table[r][own + i] = free[count - 1 - taken]
                taken += 1
        if ask < 0:
            gone += table[r][:own]
        granted.append(add)
        after.append(0 if ask < 0 else n + add)
        for j in range(q):
            on = j < add
            pos = n + j
            at = table[r][pos // page] * block_rows + pos % page if on else -1
            positions.append(pos if on else 0)
            slots.append(at if on and table[r][pos // page] >= 0 and at < 2 ** 31 else -1)
            valid.append(pos + 1 if on else 0)
    left = count - taken
    for i, v in enumerate(gone):
        if left + i < size:
            free[left + i] = v
    return positions, slots, valid, granted, table, free, after, min(left + len(gone), size)
