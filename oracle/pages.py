"""Oracle of a serving step's bookkeeping: one request and one token after the other, in Python integers."""


def build_page_tables(query_lens, context_lens, block_table, free_pages, free_head, page_size, max_tokens):
    """Lists in, a dict of lists out: cu_seqlens, seq_lens, positions, slot_map, free_head, shortage and the
    updated block_table."""
    top = 2 ** 31 - 1
    table = [list(row) for row in block_table]
    cols = len(table[0])
    head = min(max(free_head, 0), len(free_pages))
    wanted = short = 0
    cu, lens = [0], []
    pos, slot = [0] * max_tokens, [-1] * max_tokens
    for n, (q, c) in enumerate(zip(query_lens, context_lens)):
        q, c = max(q, 0), max(c, 0)
        new = min(q, max_tokens - cu[-1])
        held = min(-(-c // page_size), cols)
        full = -(-(c + new) // page_size)
        for j in range(held, min(full, cols)):
            at = head + wanted
            wanted += 1
            table[n][j] = free_pages[at] if at < len(free_pages) else -1
        short += full - min(full, cols)
        for i in range(new):
            p = c + i
            t = cu[-1] + i
            pos[t] = min(p, top)
            j = p // page_size
            if j < cols and table[n][j] >= 0:
                s = table[n][j] * page_size + p % page_size
                slot[t] = s if s <= top else -1
        cu.append(cu[-1] + new)
        lens.append(min(c + new, top))
    return dict(cu_seqlens=cu, seq_lens=lens, positions=pos, slot_map=slot, block_table=table,
                free_head=min(head + wanted, len(free_pages)),
                shortage=max(head + wanted - len(free_pages), 0) + short)
