"""Plain implementations (Python and NumPy, 64 bits) of the step-planning, index-cache and
selection operators, and the inputs of their tests. Written from the operators' definitions;
nothing here uses the library."""
from __future__ import annotations

import numpy as np

from workloads.gen import bf16_from_f32, f32_from_bf16

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
DIM, GROUP, ROW = 128, 16, 72


def blocks_of(n, page):
    return -(-n // page)


# ------------------------------------------------------------------------------ planning
def plan_step(new_lens, seq_lens, table, page, free_pages, free_count, max_tokens):
    """One sequence after the other: its pages from the top of the stack, its tokens behind the
    last one's. Returns a dict of everything the step writes."""
    table, lens = table.copy(), seq_lens.copy()
    count = min(max(int(free_count), 0), len(free_pages))
    no_pages = no_rows = False
    ids, pos, slots, cu, refused = [], [], [], [0], 0
    for s in range(len(new_lens)):
        n, length = int(new_lens[s]), int(seq_lens[s])
        ok = n >= 0 and length >= 0 and length + n <= table.shape[1] * page
        if ok:
            first = blocks_of(length, page)
            need = blocks_of(length + n, page) - first
            if need > 0 and (no_pages or need > count):
                no_pages, ok = True, False
            elif n > 0 and (no_rows or len(ids) + n > max_tokens):
                no_rows, ok = True, False
                # a request without rows keeps its claim on pages before later ones
                no_pages = no_pages or need > 0
        if ok:
            for i in range(need):
                table[s, first + i] = free_pages[count - 1 - i]
            count -= need
            for p in range(length, length + n):
                ids.append(s)
                pos.append(p)
                pg = int(table[s, p // page])
                slots.append(pg * page + p % page if pg >= 0 else -1)
            lens[s] = length + n
        elif n != 0:
            refused += 1
        cu.append(len(ids))
    fill = max_tokens - len(ids)
    return dict(seq_ids=np.array(ids + [-1] * fill, np.int32),
                positions=np.array(pos + [-1] * fill, np.int32),
                slots=np.array(slots + [-1] * fill, np.int64), cu_tokens=np.array(cu, np.int32),
                seq_lens=lens, table=table, free_count=count, refused=refused)


def truncate(keep_lens, seq_lens, table, page, free_pages, free_count):
    lens, stack, cap = seq_lens.copy(), free_pages.copy(), len(free_pages)
    count = min(max(int(free_count), 0), cap)
    back = []
    for s in range(len(seq_lens)):
        keep, length = int(keep_lens[s]), int(seq_lens[s])
        if 0 <= keep < length:
            for b in range(blocks_of(keep, page), min(blocks_of(length, page), table.shape[1])):
                if table[s, b] >= 0:
                    back.append(int(table[s, b]))
            lens[s] = keep
    pushed = back[::-1][:cap - count]
    stack[count:count + len(pushed)] = pushed
    return dict(seq_lens=lens, free_pages=stack, free_count=count + len(pushed),
                dropped=len(back) - len(pushed))


# --------------------------------------------------------------------------- index cache
def _e4m3_values():
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append((1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6)
    return np.array(v)


E4M3 = _e4m3_values()


def quantize(x):
    """bf16 bit patterns [..., 128] -> codes [..., 128], scale bytes [..., 8] (nearest, ties even)."""
    v = f32_from_bf16(x).astype(np.float64).reshape(*x.shape[:-1], DIM // GROUP, GROUP)
    want = np.abs(v).max(-1) / 6
    up = np.clip(np.searchsorted(E4M3, want), 1, 126)
    lo, hi = E4M3[up - 1], E4M3[up]
    scale = np.where((want - lo < hi - want) | ((want - lo == hi - want) & (up % 2 == 1)), up - 1, up)
    s = E4M3[scale][..., None]
    # saturation: far beyond 6 s the distances would round to equal doubles
    off = np.abs(np.minimum(np.abs(v), 6 * s)[..., None] - GRID * s[..., None])
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first: they win ties
    code = order[np.argmin(off[..., order], -1)] + 8 * np.signbit(v)
    code = np.where(s > 0, code, 0)
    return code.reshape(*x.shape).astype(np.uint8), scale.astype(np.uint8)


def values(codes, scales):
    g = np.concatenate([GRID, -GRID])[codes].reshape(*codes.shape[:-1], DIM // GROUP, GROUP)
    return (g * E4M3[scales][..., None]).reshape(*codes.shape)


def row_at(pool, stride, page, blk, row):
    """Views of a row's 64 code bytes and 8 scale bytes."""
    base = blk * stride
    c = base + row * 64
    s = base + page * 64 + row * 8
    return pool[c:c + 64], pool[s:s + 8]


def resolve(seq, pos, table, page, num_blocks):
    if seq < 0 or seq >= table.shape[0] or pos < 0 or pos // page >= table.shape[1]:
        return None
    blk = int(table[seq, pos // page])
    return (blk, pos % page) if 0 <= blk < num_blocks else None


def index_append(keys, seq_ids, positions, table, page, pool, num_blocks, stride):
    codes, scales = quantize(keys)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    bad = 0
    for t in range(len(seq_ids)):
        at = resolve(int(seq_ids[t]), int(positions[t]), table, page, num_blocks)
        if at is None:
            bad += int(seq_ids[t]) != -1
            continue
        c, s = row_at(pool, stride, page, *at)
        c[:] = packed[t]
        s[:] = scales[t]
    return bad


def read_row(pool, stride, page, blk, row):
    c, s = row_at(pool, stride, page, blk, row)
    codes = np.empty(DIM, np.uint8)
    codes[0::2], codes[1::2] = c & 15, c >> 4
    return values(codes, s)


def random_tables(rng, lens, page, spare=3, width=None):
    pages = [blocks_of(int(n), page) for n in lens]
    perm = rng.permutation(sum(pages) + spare).astype(np.int32)
    table = np.full((len(lens), width or max(max(pages), 1)), -1, np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, perm[at:].copy(), len(perm)


def random_pool(rng, num_blocks, page, stride):
    """A pool whose rows are all index rows of N(0,1) keys; what lies between them is noise."""
    pool = rng.integers(0, 256, num_blocks * stride, dtype=np.uint8)
    keys = bf16_from_f32(rng.standard_normal((num_blocks * page, DIM)))
    codes, scales = quantize(keys)
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(num_blocks, page * 64)
    v = pool.reshape(num_blocks, stride)
    v[:, :page * 64] = packed
    v[:, page * 64:page * ROW] = scales.reshape(num_blocks, page * 8)
    return pool


# ----------------------------------------------------------------------------- selection
def select(q_index, weights, q_seq, q_pos, table, page, pool, num_blocks, stride, num, block=1,
           sink=0, recent=0):
    """Every score in 64 bits, then a stable sort."""
    num_q, H, _ = q_index.shape
    q = values(*quantize(q_index))
    out = np.full((num_q, num * block), -1, np.int32)
    cached = {}
    for t in range(num_q):
        s, p = int(q_seq[t]), int(q_pos[t])
        if s < 0 or s >= table.shape[0] or p < 0:
            continue
        seen = min(p + 1, table.shape[1] * page)
        if s not in cached:
            k = np.full((table.shape[1] * page, DIM), np.nan)
            for b in range(table.shape[1]):
                if 0 <= table[s, b] < num_blocks:
                    for r in range(page):
                        k[b * page + r] = read_row(pool, stride, page, int(table[s, b]), r)
            cached[s] = k
        dots = cached[s][:seen] @ q[t].T
        score = np.where(dots < 0, 0.0, dots) @ weights[t].astype(np.float64)
        score = np.where(np.isnan(score), -np.inf, score)
        nb = blocks_of(seen, block)
        best = np.full(nb * block, -np.inf)
        best[:seen] = score
        best = best.reshape(nb, block).max(1)
        idx = np.arange(nb)
        forced = (idx < sink) | (idx >= nb - recent)
        order = np.lexsort((idx, -best, ~forced))[:num]
        pos = (np.sort(order)[:, None] * block + np.arange(block)).reshape(-1)
        pos = pos[pos < seen]
        out[t, :len(pos)] = pos
    return out
