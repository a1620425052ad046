"""gemv_block_tables by its definition: one request after the other, one token after the other."""
MAX32 = 2 ** 31 - 1


def block_tables(lens, new, table, page, width, num_pages, free, free_next, room):
    """Returns the call's outputs as lists; ``table`` (a list of lists) is changed in place."""
    slots, positions = [-1] * room, [0] * room
    token_start, page_start, new_lens, status = [], [], [], []
    avail = max(0, len(free) - free_next) if free_next >= 0 else 0
    tok = asked = used = 0
    for r, (n, add) in enumerate(zip(lens, new)):
        count = max(0, add)
        first, end = tok, tok + count
        tok = end
        token_start.append(min(first, MAX32))
        if n < 0 or add < 0:
            state = 4
        elif n + add > width * page:
            state = 2
        elif count and end > room:
            state = 3
        else:
            state = 0
        have = -(-n // page) if state == 0 else 0
        need = -(-(n + count) // page) - have if state == 0 else 0
        asked += need
        if need and asked > avail:
            state = 1
        if state:
            page_start.append(-1)
            new_lens.append(n)
            status.append(state)
            continue
        begin = free_next + asked - need
        page_start.append(begin)
        new_lens.append(n + count)
        status.append(0)
        used += need
        for i in range(need):
            table[r][have + i] = free[begin + i]
        for i in range(count):
            pos = n + i
            positions[first + i] = pos
            g = table[r][pos // page]
            if 0 <= g < num_pages:
                slots[first + i] = g * page + pos % page
    token_start.append(min(tok, MAX32))
    return dict(slots=slots, positions=positions, token_start=token_start, page_start=page_start, new_lens=new_lens,
                status=status, free_next=free_next + used, table=table)
