"""Planning and giving back pages, from the definition in include/fa.h, one sequence at a time in whole numbers."""


def pages(n, page):
    return -(-n // page)


def plan(ring, counts, table, lens, new, page, T):
    """(table, cu, ends, positions, slots, counts, bad) after fa_cache_plan; lists in, lists out."""
    taken, given = counts
    bad = taken < 0 or given < taken or given - taken > len(ring)
    free = 0 if bad else given - taken
    table = [list(row) for row in table]
    cap = len(table[0]) * page
    cu, ends = [0], []
    positions, slots = [-1] * T, [-1] * T
    asked = 0
    for b, (had, n) in enumerate(zip(lens, new)):
        count = max(0, n) if had >= 0 else 0
        begin = cu[-1]
        cu.append(begin + count)
        if had < 0 or n < 0 or had + count > cap or begin + count > T:
            bad = True
            ends.append(had)
            continue
        first, last = pages(had, page), pages(had + count, page)
        asked += last - first
        if last > first and asked > free:
            ends.append(had)
            continue
        for at in range(first, last):
            table[b][at] = ring[(taken + asked - (last - first) + at - first) % len(ring)]
        ends.append(had + count)
        for i in range(count):
            p = table[b][(had + i) // page]
            positions[begin + i] = had + i
            if 0 <= p < len(ring):
                slots[begin + i] = p * page + (had + i) % page
            else:
                bad = True
    grew = sum(pages(e, page) - pages(h, page) for e, h in zip(ends, lens) if h >= 0)
    return table, cu, ends, positions, slots, [taken + grew, given], bad


def trim(ring, counts, table, lens, keep, page):
    """(ring, counts, bad) after fa_cache_trim."""
    taken, given = counts
    ring = list(ring)
    bad = taken < 0 or given < taken or given - taken > len(ring)
    room = 0 if bad else len(ring) - (given - taken)
    cap = len(table[0]) * page
    asked = back = 0
    for b, (had, n) in enumerate(zip(lens, keep)):
        if n < 0 or n > had or had > cap:
            bad = True
            continue
        places = range(pages(n, page), pages(had, page))
        asked += len(places)
        if len(places) and asked > room:
            bad = True
            continue
        for at in places:
            ring[(given + back) % len(ring)] = table[b][at]
            bad |= not 0 <= table[b][at] < len(ring)
            back += 1
    return ring, [taken, given + back], bad
