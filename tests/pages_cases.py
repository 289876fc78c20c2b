"""Plain implementations (Python and NumPy, one entry after the other) of the operators for shared
pages, and the states of their tests. Written from the operators' definitions; nothing here uses
the library."""
from __future__ import annotations

import numpy as np

from tests.step_cases import blocks_of


def fork(src, dst, lens_wanted, seq_lens, table, page, shares, free_pages, free_count):
    table, lens, shares = table.copy(), seq_lens.copy(), shares.copy()
    old_table, S, NB = table.copy(), len(seq_lens), len(shares)
    count = min(max(int(free_count), 0), len(free_pages))
    n = len(src)
    shared, cs, cd = (np.full(n, -1, np.int32) for _ in range(3))
    named, no_pages, refused = set(), False, 0
    for i in range(n):
        s, d, m = int(src[i]), int(dst[i]), int(lens_wanted[i])
        if s == -1:
            continue
        ok = 0 <= s < S and 0 <= d < S and 0 <= m
        ok = ok and m <= seq_lens[s] and m <= table.shape[1] * page and seq_lens[d] == 0 and d not in named
        named.add(d)
        if ok and m % page:
            no_pages = no_pages or count == 0
            ok = not no_pages
        if not ok:
            refused += 1
            continue
        full = m // page
        for b in range(full):
            p = int(old_table[s, b])
            table[d, b] = p
            if 0 <= p < NB:
                shares[p] += 1
        if m % page:
            count -= 1
            p, q = int(old_table[s, full]), int(free_pages[count])
            table[d, full] = q
            if 0 <= p < NB and 0 <= q < NB:
                cs[i], cd[i] = p, q
        shared[i], lens[d] = full, m
    return dict(table=table, seq_lens=lens, shares=shares, free_count=count, shared_blocks=shared,
                copy_src=cs, copy_dst=cd, refused=refused)


def release(keep_lens, seq_lens, table, page, shares, free_pages, free_count):
    lens, left, stack = seq_lens.copy(), shares.astype(np.int64), free_pages.copy()
    NB, cap, W = len(shares), len(free_pages), table.shape[1]
    count = min(max(int(free_count), 0), cap)
    dropped_entries, refused = [], 0
    for s in range(len(seq_lens)):
        keep, length = int(keep_lens[s]), int(seq_lens[s])
        if not 0 <= keep < length:
            continue
        if keep % page and keep // page < W:
            p = int(table[s, keep // page])
            if 0 <= p < NB and shares[p] > 0:
                refused += 1
                continue
        lens[s] = keep
        for b in range(blocks_of(keep, page), min(blocks_of(length, page), W)):
            p = int(table[s, b])
            if 0 <= p < NB:
                dropped_entries.append(p)
                left[p] -= 1
    back, seen = [], set()
    for p in dropped_entries:
        if left[p] < 0 and p not in seen:
            seen.add(p)
            back.append(p)
    left[list(seen)] = 0
    pushed = back[::-1][:cap - count]
    stack[count:count + len(pushed)] = pushed
    return dict(seq_lens=lens, shares=left.astype(np.int32), free_pages=stack,
                free_count=count + len(pushed), dropped=len(back) - len(pushed), refused=refused)


def compact(seq_lens, table, page, shares, free_pages, free_count, max_moves):
    NB, W = len(shares), table.shape[1]
    table, shares, stack = table.copy(), shares.copy(), free_pages.copy()
    count = min(max(int(free_count), 0), len(free_pages))
    held = [(s, b) for s in range(len(seq_lens)) for b in range(min(blocks_of(max(int(seq_lens[s]), 0), page), W))
            if 0 <= table[s, b] < NB]
    used = {int(table[e]) for e in held}
    idle = {int(p) for p in free_pages[:count] if 0 <= p < NB} - used
    moves = {}
    cs, cd = np.full(max_moves, -1, np.int32), np.full(max_moves, -1, np.int32)
    for i, (u, f) in enumerate(zip(sorted(used, reverse=True), sorted(idle))):
        if i >= max_moves or f > u:
            break
        moves[u], cs[i], cd[i] = f, u, f
    for e in held:
        table[e] = moves.get(int(table[e]), table[e])
    for u, f in moves.items():
        shares[f], shares[u] = shares[u], 0
    idle = (idle - set(moves.values())) | set(moves)
    used = (used - set(moves)) | set(moves.values())
    stack[:len(idle)] = sorted(idle, reverse=True)
    return dict(table=table, shares=shares, free_pages=stack, free_count=len(idle), copy_src=cs,
                copy_dst=cd, pages_end=max(used) + 1 if used else 0)


def family(rng, seqs, page, longest, spare, width=None, empty=0.3):
    """Sequences of random lengths over a random pool; `empty` of them have none and some of the others
    share the whole pages of an earlier one's beginning. Returns lens, table, shares, stack, count."""
    lens = rng.integers(1, longest + 1, seqs)
    lens[rng.random(seqs) < empty] = 0
    width = width or max(blocks_of(longest, page), 1)
    total = sum(blocks_of(int(n), page) for n in lens) + spare
    perm = list(rng.permutation(total))
    table = np.full((seqs, width), -1, np.int32)
    shares = np.zeros(total, np.int32)
    for s in range(seqs):
        n = blocks_of(int(lens[s]), page)
        whole = 0
        if s and rng.random() < 0.6:
            o = int(rng.integers(0, s))
            whole = int(rng.integers(0, min(int(lens[s]), int(lens[o])) // page + 1))
            table[s, :whole] = table[o, :whole]
            np.add.at(shares, table[s, :whole], 1)
        for b in range(whole, n):
            table[s, b] = perm.pop()
    stack = np.full(total + 5, -9, np.int32)
    stack[:len(perm)] = perm
    return lens.astype(np.int32), table, shares, stack, len(perm)


def check_state(lens, table, page, shares, free_pages, free_count):
    """Every page is free once or held, and its shares are its holders beyond the first."""
    holders = np.zeros(len(shares), np.int64)
    for s in range(len(lens)):
        for p in table[s, :blocks_of(int(lens[s]), page)]:
            holders[p] += 1
    free = free_pages[:free_count]
    assert len(set(free.tolist())) == len(free)
    assert np.array_equal(np.sort(free), np.nonzero(holders == 0)[0])
    assert np.array_equal(shares, np.maximum(holders - 1, 0))
