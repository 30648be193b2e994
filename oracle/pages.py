"""Oracle: pages of a free list to requests and back (test infrastructure
only).  Plain loops over requests, pages and tokens.

The serving systems that the explainers name keep the KV cache in fixed-size
pages behind a block table; the free list is a stack whose top is
free_pages[free_count - 1].
"""


def page_map(kv_len, new_len, table, count, free, free_count, page, num_pages, T=None):
    """Returns (error, table, count, free_count, slots, starts) with new
    lists; error is None, "pages" or "invalid" (then nothing changed)."""
    B = len(kv_len)
    max_pages = len(table[0])
    bad = not 0 <= free_count <= num_pages
    for b in range(B):
        bad |= kv_len[b] < 0 or new_len[b] < 0 or not 0 <= count[b] <= max_pages
        bad |= kv_len[b] + new_len[b] > max_pages * page
    if bad or (T is not None and sum(new_len) > T):
        return "invalid", table, count, free_count, None, None
    need = [max(count[b], -(-(kv_len[b] + new_len[b]) // page)) for b in range(B)]
    if sum(need) - sum(count) > free_count:
        return "pages", table, count, free_count, None, None
    table = [list(r) for r in table]
    for b in range(B):
        for p in range(count[b], need[b]):
            free_count -= 1
            table[b][p] = free[free_count]
    slots, starts = [], [0]
    for b in range(B):
        for pos in range(kv_len[b], kv_len[b] + new_len[b]):
            slots.append(table[b][pos // page] * page + pos % page)
        starts.append(len(slots))
    if T is not None:
        slots += [-1] * (T - len(slots))
    return None, table, need, free_count, slots, starts


def page_release(keep_len, table, count, free, free_count, page):
    """Returns (table, count, free, free_count) with new lists."""
    table, count, free = [list(r) for r in table], list(count), list(free)
    given = []
    for b in range(len(keep_len)):
        if keep_len[b] < 0:
            continue
        keep = min(count[b], -(-keep_len[b] // page))
        for p in range(keep, count[b]):
            given.append(table[b][p])
            table[b][p] = -1
        count[b] = keep
    for page_id in reversed(given):  # the first one taken comes to lie on top
        free[free_count] = page_id
        free_count += 1
    return table, count, free, free_count
