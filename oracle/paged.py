"""Oracle of the paged key-value cache: page upkeep on plain integers, and
attention over the pages in fp64.

TEST INFRASTRUCTURE: see the package header for who may import this.

A pool is a numpy array [planes, num_pages, n_kv_heads, page_size, head_dim]; refs,
table and lengths are integer arrays.  The functions change what they are given, one
slot and one page at a time, in the order the contract states.

Parity pins (tests/test_paged_cpu.py): growing, forking and freeing keeps every
page's count equal to its holders; compaction leaves what the sequences hold
unchanged; attention over pages equals attention over the same rows laid out
contiguously.
"""
import numpy as np

from .attention import attend


def held(length, page):
    return -(-int(length) // page)


def fork(parent, refs, table, lengths, page):
    """Slots become forks of other slots (parent[s] = s keeps, -1 frees), at once."""
    before, lens = table.copy(), lengths.copy()
    for s, p in enumerate(parent):
        if p == s:
            continue
        for j in range(held(lens[s], page)):
            refs[before[s, j]] -= 1
            table[s, j] = -1
        lengths[s] = lens[p] if p >= 0 else 0
        for j in range(held(lengths[s], page)):
            table[s, j] = before[p, j]
            refs[before[p, j]] += 1


def grow(add, data, refs, table, lengths):
    """Room for add[s] more tokens; returns granted (list of 0 / 1)."""
    page = data.shape[3]
    free = [i for i in range(len(refs)) if refs[i] == 0]
    shared = refs > 1                       # as the call found them
    at, granted = 0, []
    for s in range(len(lengths)):
        a = max(0, int(add[s]))
        old, new = int(lengths[s]), int(lengths[s]) + a
        if held(new, page) > table.shape[1]:
            granted.append(0)
            continue
        tail = old // page
        copy = a > 0 and old % page != 0 and shared[table[s, tail]]
        want = held(new, page) - held(old, page) + bool(copy)
        mine = free[at:at + want]
        at += want
        if want and at > len(free):
            granted.append(0)
            continue
        if copy:
            src, dst = table[s, tail], mine[0]
            data[:, dst, :, :old % page] = data[:, src, :, :old % page]
            refs[src] -= 1
            refs[dst] += 1
            table[s, tail] = dst
            mine = mine[1:]
        for i, p in enumerate(mine):
            table[s, held(old, page) + i] = p
            refs[p] += 1
        lengths[s] = new
        granted.append(1)
    return granted


def compact(data, refs, table, lengths):
    """Live pages numbered n_live and up move into the free pages below; returns remap."""
    page = data.shape[3]
    n = int((refs > 0).sum())
    holes = [i for i in range(n) if refs[i] == 0]
    remap = np.where(refs > 0, np.arange(len(refs)), -1)
    for hole, p in zip(holes, [i for i in range(n, len(refs)) if refs[i] > 0]):
        data[:, hole] = data[:, p]
        refs[hole], refs[p] = refs[p], 0
        remap[p] = hole
    for s in range(len(lengths)):
        for j in range(held(lengths[s], page)):
            table[s, j] = remap[table[s, j]]
    return remap


def rows(pages, table_row, length):
    """The first `length` rows of a sequence: [length, n_kv_heads, head_dim]."""
    page = pages.shape[2]
    out = np.zeros((length, pages.shape[1], pages.shape[3]), dtype=pages.dtype)
    for i in range(length):
        out[i] = pages[table_row[i // page], :, i % page]
    return out


def append(k, v, k_pages, v_pages, table, lengths, q_start):
    """Rows q_start[s] .. q_start[s+1] - 1 are the last tokens of sequence s."""
    page = k_pages.shape[2]
    for s in range(len(lengths)):
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            pos = lengths[s] - n + i
            if pos >= 0:
                k_pages[table[s, pos // page], :, pos % page] = k[q_start[s] + i]
                v_pages[table[s, pos // page], :, pos % page] = v[q_start[s] + i]


def attention(q, k_pages, v_pages, table, lengths, q_start):
    """q [tokens, heads, D] -> dict(o, lse, spread): spread[t, h, d] = sum_j p_j |v_j[d]|,
    the scale that rounding the terms of o is measured against.  Tokens that see no
    position get o = 0, lse = -inf; rows that no sequence counts get NaN."""
    T, H, D = q.shape
    G = k_pages.shape[1]
    o, lse, spread = np.full((T, H, D), np.nan), np.full((T, H), np.nan), np.full((T, H, D), np.nan)
    for s in range(len(lengths)):
        a, b = q_start[s], q_start[s + 1]
        L, n = int(lengths[s]), b - a
        k, v = (np.repeat(rows(x, table[s], L), H // G, axis=1) for x in (k_pages, v_pages))
        for t in range(a, b):
            seen = L - n + (t - a) + 1
            if seen <= 0:
                o[t], lse[t], spread[t] = 0, -np.inf, 0
                continue
            x = np.einsum("hd,jhd->hj", q[t], k[:seen]) / np.sqrt(D)
            top = x.max(axis=1, keepdims=True)
            e = np.exp(x - top)
            z = e.sum(axis=1, keepdims=True)
            o[t] = np.einsum("hj,jhd->hd", e / z, v[:seen])
            spread[t] = np.einsum("hj,jhd->hd", e / z, np.abs(v[:seen]))
            lse[t] = (np.log(z) + top)[:, 0]
    return dict(o=o, lse=lse, spread=spread)


def contiguous(q, k, v):
    """attend() of q [n, H, D] as the last tokens of k, v [L, G, D], for the pins."""
    return attend(q[None], k[None], v[None], q_pos0=k.shape[0] - q.shape[0])[0]
