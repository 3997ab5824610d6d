"""A serving step's bookkeeping from its request lengths (oracle, plain loops).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Request b has seq_lens[b] tokens, the last query_lens[b] of them new.  Walking the
requests in order and each request's new tokens in order gives the step's rows.  A new
token at the first place of a page enters that page: the next entry of the free list
goes into the block table (-1 past the list's end).  Negative lengths count as 0.
"""

import numpy as np

PAGE = 64


def step_map(seq_lens, query_lens, block_table, num_rows, free_pages=None, free_start=0,
             gathered=False):
    """dict of the outputs, and the block table after the step."""
    table = np.array(block_table, dtype=np.int32)
    out = {"slot_mapping": np.full(num_rows, -1, np.int64), "positions": np.zeros(num_rows, np.int64),
           "row_seq": np.full(num_rows, -1, np.int32), "ks": np.zeros(num_rows, np.int32),
           "ke": np.zeros(num_rows, np.int32)}
    offsets, row, taken = [0], 0, int(free_start) if free_pages is not None else 0
    for b in range(len(seq_lens)):
        length, new = max(int(seq_lens[b]), 0), max(int(query_lens[b]), 0)
        held = -(-max(length - new, 0) // PAGE)
        for pos in range(length - new, length):
            if row < num_rows:
                page_no = pos // PAGE
                if 0 <= pos and page_no < table.shape[1]:
                    if free_pages is not None and page_no >= held:
                        at = taken + page_no - held
                        page = int(free_pages[at]) if 0 <= at < len(free_pages) else -1
                        if pos % PAGE == 0:
                            table[b, page_no] = page
                    else:
                        page = int(table[b, page_no])
                    if page >= 0:
                        out["slot_mapping"][row] = page * PAGE + pos % PAGE
                base = offsets[-1] if gathered else 0
                out["positions"][row] = pos
                out["row_seq"][row] = b
                out["ks"][row] = base
                out["ke"][row] = base + pos + 1
            row += 1
        taken += -(-length // PAGE) - held
        offsets.append(offsets[-1] + length)
    out["cu_seq_offsets"] = np.array(offsets, np.int64)
    out["free_next"] = np.array([taken], np.int64)
    return out, table
