"""Oracle of the decoder's attention operators: block tables and slot maps,
the append to a paged cache, paged and cross attention.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain NumPy and Python
loops: one request, one head and one query row at a time, in float64 (whole
numbers for the tables).
"""

import numpy as np


def kv_tables(cached, added, free_blocks, block_table, page, tokens):
    """(block_table, lens, starts, slots, taken) of a step.

    Request b holds cached[b] tokens in the first ceil(cached / page) entries
    of its row and gets added[b] more. It takes the next free blocks for the
    entries its longer length needs, as far as its row is wide; a new token's
    slot is its block times page plus its offset, -1 where there is no block.
    """
    table = np.array(block_table, dtype=np.int64, copy=True)
    width = table.shape[1]
    lens, starts, slots, taken = [], [0], [], 0
    for b in range(len(cached)):
        old, new = max(0, int(cached[b])), max(0, int(added[b]))
        length = min(old + new, width * page)
        for i in range(-(-old // page), -(-length // page)):
            table[b, i] = free_blocks[taken] if taken < len(free_blocks) else -1
            taken += 1
        for p in range(old, old + new):
            block = table[b, p // page] if p // page < width else -1
            slots.append(block * page + p % page if block >= 0 else -1)
        lens.append(length)
        starts.append(starts[-1] + new)
    slots = (slots + [-1] * tokens)[:tokens]
    return (table, np.array(lens, dtype=np.int64), np.minimum(np.array(starts, dtype=np.int64), tokens),
            np.array(slots, dtype=np.int64), taken)


def attend(q, k, v, scale):
    """softmax(scale * q . k) v of one query row q [D] over k, v [n, D]:
    zeros where the weights sum to zero (no key, every score -infinity)."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    if len(k) == 0:
        return np.zeros(v.shape[1])
    with np.errstate(invalid="ignore", over="ignore"):
        score = (k * q).sum(axis=1) * scale
        top = score.max()
        weight = np.exp(score - (0.0 if top == -np.inf else top))
        if weight.sum() == 0:
            return np.zeros(v.shape[1])
        return (weight[:, None] * v).sum(axis=0) / weight.sum()


def paged_rows(cache, table_row, length, page):
    """Positions below `length` of one request whose block exists, as rows
    [n, heads, D] of a cache [blocks, heads, page, D]."""
    rows = []
    for t in range(max(0, min(length, len(table_row) * page))):
        block = int(table_row[t // page])
        if 0 <= block < cache.shape[0]:
            rows.append(cache[block, :, t % page])
    return np.array(rows).reshape(len(rows), cache.shape[1], cache.shape[3])


def paged_attention(q, k_cache, v_cache, block_table, lens, max_len, scale):
    """q [B, Hq, D] over caches [blocks, Hkv, page, D] -> float64 [B, Hq, D]."""
    out = np.zeros(q.shape)
    group = q.shape[1] // k_cache.shape[1]
    for b in range(q.shape[0]):
        n = min(int(lens[b]), max_len)
        k = paged_rows(k_cache, block_table[b], n, k_cache.shape[2])
        v = paged_rows(v_cache, block_table[b], n, k_cache.shape[2])
        for h in range(q.shape[1]):
            out[b, h] = attend(q[b, h], k[:, h // group], v[:, h // group], scale)
    return out


def cross_attention(q, k, v, lens, scale):
    """q [B, Tq, Hq, D] over k, v [B, Tk, Hkv, D] -> float64 [B, Tq, Hq, D];
    rows at lens[b] and beyond are left out (lens None: none are)."""
    out = np.zeros(q.shape)
    group = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        n = k.shape[1] if lens is None else max(0, min(int(lens[b]), k.shape[1]))
        for t in range(q.shape[1]):
            for h in range(q.shape[2]):
                out[b, t, h] = attend(q[b, t, h], k[b, :n, h // group], v[b, :n, h // group], scale)
    return out
