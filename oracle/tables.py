"""Oracle: block tables, slots and the free list of a step.

TEST INFRASTRUCTURE ONLY (see the package docstring).

What it computes, one sequence after the other.  "Speculative Decoding"
(atlas), "Committed tokens versus cached states": a step writes states for new
tokens and the rejected suffix is removed; pages holding no kept position may
be released.  The readings here:
  * a free list is a stack: pages are taken from its end and put back there;
  * sequences are served in order; one whose pages do not fit is refused
    whole, and so is every later one that needs pages (the running sum counts
    the refused ones);
  * a token falls on slot page * page_size + offset, -1 where there is none.
"""
import numpy as np

BAD_LEN, NO_PAGES, BAD_PAGE = 16, 32, 64
MOST = 2 ** 31 - 1


def extend(ctx_len, add_len, block_table, free_list, free_count, page_size, max_tokens):
    """The values spec_extend_tables leaves, and the updated table."""
    P, table = int(page_size), np.array(block_table, dtype=np.int64, copy=True)
    B, width = table.shape
    pool = len(free_list)
    count = min(max(int(free_count), 0), pool)
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.full(max_tokens, -1, dtype=np.int64)
    cu, new_len, status = [0], [], []
    upto = taken = 0
    for b in range(B):
        c, a = int(ctx_len[b]), int(add_len[b])
        first = cu[-1]
        cu.append(first + max(a, 0))
        have, want = -(-c // P), -(-(c + a) // P)
        if c < 0 or a < 0 or want > width or cu[-1] > max_tokens:
            status.append(BAD_LEN)
            new_len.append(c)
            continue
        need = want - have
        upto += need
        if need and upto > count:
            status.append(NO_PAGES)
            new_len.append(c)
            continue
        for j in range(need):
            table[b, have + j] = free_list[count - 1 - (upto - need + j)]
        taken = upto if need else taken
        bad = False
        for t in range(a):
            page = int(table[b, (c + t) // P])
            if 0 <= page < pool:
                slots[first + t] = page * P + (c + t) % P
                positions[first + t] = c + t
            else:
                bad = True
        # a page taken past the last token does not happen: every new page holds one
        status.append(BAD_PAGE if bad else 0)
        new_len.append(c if bad else c + a)
    return dict(block_table=table, slot_map=slots, positions=positions,
                cu_len=np.minimum(cu, MOST), new_len=np.array(new_len, dtype=np.int64),
                free_count=count - taken, status=np.array(status, dtype=np.int64))


def release(block_table, length, keep_pages, free_list, free_count, page_size):
    """(free list, count, status) after the pages behind the kept ones went back."""
    P, lst = int(page_size), np.array(free_list, dtype=np.int64, copy=True)
    width, pool = np.asarray(block_table).shape[1], len(lst)
    count = min(max(int(free_count), 0), pool)
    upto, end, status = count, count, []
    for b in range(len(length)):
        n, k = int(length[b]), int(keep_pages[b])
        held = -(-n // P)
        if n < 0 or k < 0 or k > held or held > width:
            status.append(BAD_LEN)
            continue
        give = held - k
        upto += give
        if give and upto > pool:
            status.append(NO_PAGES)
            continue
        bad = False
        for j in range(give):
            page = int(block_table[b][k + j])
            ok = 0 <= page < pool
            lst[upto - give + j] = page if ok else -1
            bad = bad or not ok
        end = upto if give else end
        status.append(BAD_PAGE if bad else 0)
    return lst, end, np.array(status, dtype=np.int64)
