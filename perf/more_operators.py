"""Dense attention of a step's new tokens, and the page operators: cases, inputs and plain forms.

Measured here are the causal attention of prompt chunks, drafts and single tokens over the paged
latent cache, and what manages pages that several sequences share: forking sequences (with the copy
of the pages that cannot be shared), releasing them, and compacting a pool. `run` computes them in
elementary torch operations, or, where `own` is true, through nvfp4_compressed_mla_gb300.
"""
import math

import torch

own = False

DEV = "cuda:0"
LATENT, ROPE, GROUP = 512, 64, 16
CODE_BYTES, SCALE_BYTES = LATENT // 2, LATENT // GROUP
NVFP4_ROW, FP8_ROW, INDEX_ROW = CODE_BYTES + SCALE_BYTES + ROPE, LATENT + ROPE, 72   # 352, 576, 72 bytes
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes
SM_SCALE = 1.0 / 24.0                            # 1 / sqrt(576)
FLOPS = 2.0 * (LATENT + ROPE + LATENT)           # a head, a token and a key that it sees
SCORES = 1 << 27                                 # scores that the plain form holds at a time


# ---------------------------------------------------------------------------------- cases
def _chunk(name, **kw):
    # new: "one" (a decode step), "draft" (1..`most` tokens each), "chunk" (`most` tokens each), "mixed" (decode
    # steps, one sequence in eight a prompt of up to `most`); pad: rows behind the last token
    return {"name": name, "op": "chunk", "page": 64, "fp8": False, "ragged": 0.0, "pad": 0, **kw}


def _fork(name, **kw):
    # prompts of up to `longest` tokens (shortest: `longest` * (1 - ragged)), each forked `samples` times at its end
    return {"name": name, "op": "fork", "page": 64, **kw}


def _release(name, **kw):
    # families of `samples` sequences that share their prompt; `cut` of all sequences end or drop their answers
    return {"name": name, "op": "release", "page": 64, **kw}


def _compact(name, **kw):
    # a pool of which `used` is in use, at random places; up to `moves` pages move
    return {"name": name, "op": "compact", "page": 64, **kw}


def listed():
    return [
        # the smallest call: seven tokens behind a short context, 16 heads; latency counts
        _chunk("chunk_tiny", seqs=1, longest=307, new="chunk", most=7, heads=16),
        # a decode step of 66 sessions that attends to everything (a layer without a selection)
        _chunk("chunk_decode", seqs=66, longest=32768, ragged=0.5, new="one", most=1, heads=128),
        # drafts of a verification step: 1..15 tokens on each of 32 long sequences
        _chunk("chunk_drafts", seqs=32, longest=65536, ragged=0.1, new="draft", most=15, heads=128, pad=37),
        # a step of continuous batching: decode steps and a few prompts, half of the heads
        _chunk("chunk_mixed", seqs=61, longest=12001, ragged=0.9, new="mixed", most=2048, heads=64, pad=19),
        # a prompt chunk of 4096 tokens behind 12288
        _chunk("chunk_prompt", seqs=1, longest=16384, new="chunk", most=4096, heads=128),
        # whole prompts of FP8 rows, 32 heads, ragged
        _chunk("chunk_fp8", seqs=5, longest=5003, ragged=0.6, new="chunk", most=2011, heads=32, fp8=True),
        # four samples of each of eight prompts
        _fork("fork_samples", seqs=8, longest=4000, ragged=0.7, samples=4),
        # eight beams of each of 120 sequences, many pages to copy
        _fork("fork_beams", seqs=120, longest=8000, ragged=0.5, samples=8),
        # the beams that a step drops
        _release("release_beams", seqs=16, longest=6000, ragged=0.5, samples=8, answer=300, cut=0.4, whole=True),
        # many requests over common prompts end, or take back part of their answers
        _release("release_many", seqs=100, longest=30000, ragged=0.8, samples=10, answer=3000, cut=0.3, whole=False),
        # a few stray pages of a small pool
        _compact("compact_few", seqs=16, longest=4000, ragged=0.6, used=0.8, moves=64),
        # a pool of 23000 pages gives up its upper third
        _compact("compact_pool", seqs=100, longest=16000, ragged=0.8, used=0.65, moves=16384),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "fork", "release", "compact"])
    page = rng.choice([16, 32, 48, 64, 64, 64, 128])
    ragged = round(rng.choice([0.0, rng.random()]), 3)
    if op == "chunk":
        heads = rng.choice([1, 8, 16, 16, 24, 32, 33, 64, 64, 128, 128])
        new = rng.choice(["one", "draft", "chunk", "chunk", "mixed"])
        seqs = _log_int(rng, 1, 200)
        most = {"one": 1, "draft": rng.randint(2, 16), "chunk": _log_int(rng, 16, max(16, 8192 // seqs)),
                "mixed": _log_int(rng, 16, 2048)}[new]
        case = {"op": op, "page": page, "fp8": rng.random() < 0.3, "ragged": ragged, "pad": rng.choice([0, rng.randint(1, 300)]),
                "seqs": seqs, "longest": most + 1, "new": new, "most": most, "heads": heads}
        # at most the work of the prompt chunk, and a pool of at most 3 million rows
        tokens = sum(_new_tokens(case))
        case["longest"] = _log_int(rng, most + 1, max(most + 1, min(200_000, 3_000_000 // seqs, 7_300_000_000 // (tokens * heads))))
        while work(case)["flops"] > 1.6e13:
            case["longest"] = max(most + 1, case["longest"] // 2)
            case["seqs"] = (case["seqs"] + 1) // 2
        return case
    if op == "fork":
        samples = rng.randint(1, 12)
        seqs = _log_int(rng, 1, 1000 // samples)
        return {"op": op, "page": page, "seqs": seqs, "longest": _log_int(rng, 20, min(100000, 900_000 // seqs)),
                "ragged": ragged, "samples": samples}
    if op == "release":
        samples = rng.randint(1, 12)
        seqs = _log_int(rng, 1, 1000 // samples)
        return {"op": op, "page": page, "seqs": seqs, "longest": _log_int(rng, 20, min(100000, 4_000_000 // seqs)),
                "ragged": ragged, "samples": samples, "answer": _log_int(rng, 2, min(20000, 4_000_000 // (seqs * samples))),
                "cut": round(rng.uniform(0.05, 1.0), 3), "whole": rng.random() < 0.5}
    seqs = _log_int(rng, 1, 600)
    longest = _log_int(rng, 20, min(100000, 600_000 // seqs))
    return {"op": op, "page": page, "seqs": seqs, "longest": longest, "ragged": ragged, "used": round(rng.uniform(0.4, 0.95), 3),
            "moves": _log_int(rng, 1, 16384)}


# --------------------------------------------------------------------------------- inputs
def _spread(count, low, high):
    """Whole numbers spread evenly over low .. high: a case has the same ones for every seed, in another order."""
    return [int(low + (high - low) * (j + 0.5) / count) for j in range(count)]


def _shuffled(values, g):
    v = torch.tensor(values, device=DEV)
    return v[torch.randperm(v.numel(), generator=g, device=DEV)]


def _contexts(case):
    return _spread(case["seqs"], max(1, case["longest"] * (1 - case["ragged"])), case["longest"])


def _new_tokens(case):
    S, most = case["seqs"], case["most"]
    if case["new"] == "draft":
        return _spread(S, 1, most + 1)
    if case["new"] == "mixed":
        prompts = max(1, S // 8)
        return _spread(prompts, 1, most + 1) + [1] * (S - prompts)
    return [most] * S


def _tables(pages, width, pool, g):
    """Block table [S, width] over random pages of a pool, and the pages left over."""
    total = int(pages.sum())
    perm = torch.randperm(pool, generator=g, device=DEV)
    at = (pages.cumsum(0) - pages)[:, None] + torch.arange(width, device=DEV)
    used = torch.arange(width, device=DEV) < pages[:, None]
    table = torch.where(used, perm[at.clamp(max=max(total - 1, 0))], -1)
    return table.int().contiguous(), perm[total:].int().contiguous(), pool


def _quantize(x):
    """E2M1 codes (two a byte) and E4M3 scales of each 16 values of x [n, 512]."""
    a = x.unflatten(-1, (SCALE_BYTES, GROUP))
    s = (a.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    q = torch.where(s.float() > 0, a / s.float(), 0.0)
    codes = (torch.bucketize(q.abs(), edges).int() + 8 * (q < 0).int()).flatten(-2).to(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), s.squeeze(-1).view(torch.uint8)


def _fill_rows(rows, fp8, g):
    """Cache rows [n, row bytes] of N(0, 1) latents (one in a hundred times 8) and ropes."""
    for r in rows.split(1 << 17):
        x = torch.randn(r.shape[0], LATENT, generator=g, device=DEV)
        x *= torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.01, 8.0, 1.0)
        rope = torch.randn(r.shape[0], ROPE, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
        if fp8:
            r[:, :LATENT] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            r[:, :CODE_BYTES], r[:, CODE_BYTES:CODE_BYTES + SCALE_BYTES] = _quantize(x)
        r[:, -ROPE:] = rope


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    P, S = case["page"], case["seqs"]
    st = {"case": dict(case)}
    i32 = torch.int32
    if case["op"] == "chunk":
        H, row = case["heads"], FP8_ROW if case["fp8"] else NVFP4_ROW
        lens, new = _shuffled(_contexts(case), g), _shuffled(_new_tokens(case), g)
        lens = torch.maximum(lens, new)
        width = (max(case["longest"], case["most"]) + P - 1) // P
        pages = (lens + P - 1) // P
        table, _, blocks = _tables(pages, width, int(pages.sum()) + 3, g)
        pool = torch.empty(blocks * P, row, device=DEV, dtype=torch.uint8)
        _fill_rows(pool, case["fp8"], g)
        cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
        n = int(cu[-1]) + case["pad"]
        q = torch.randn(n, H, LATENT + ROPE, generator=g, device=DEV) * 2
        st.update(q_latent=q[..., :LATENT].bfloat16().contiguous(), q_rope=q[..., LATENT:].bfloat16().contiguous(),
                  cu=cu, lens=lens.int(), table=table, pool=pool.view(-1), blocks=blocks,
                  out=torch.zeros(n, H, LATENT, device=DEV, dtype=torch.bfloat16), lse=torch.zeros(n, H, device=DEV),
                  workspace={})
        return st
    if case["op"] == "fork":
        k = case["samples"]
        total = S * (1 + k)
        lens = torch.zeros(total, device=DEV, dtype=torch.long)
        lens[:S] = _shuffled(_contexts(case), g)
        width = (case["longest"] + P - 1) // P
        pages = (lens + P - 1) // P
        table, free, blocks = _tables(pages, width, int(pages.sum()) + S * k + 7, g)
        src = torch.arange(S, device=DEV).repeat_interleave(k)
        dst = S + torch.randperm(S * k, generator=g, device=DEV)
        shares = torch.zeros(blocks, device=DEV, dtype=i32)
        st.update(src=src.int(), dst=dst.int(), fork_lens=lens[src].int(), pools=[])
        for row in (NVFP4_ROW, INDEX_ROW):  # the latent pool and the index keys' pool of a layer
            st["pools"].append((torch.randint(0, 256, (blocks * P * row,), generator=g, device=DEV, dtype=torch.uint8), P * row))
        for name in ("shared", "copy_src", "copy_dst"):
            st[name] = torch.empty(S * k, device=DEV, dtype=i32)
    elif case["op"] == "release":
        # prompt s and its samples s * k .. s * k + k - 1, all of them sequences with answers of their own
        k = case["samples"]
        prompt = _shuffled(_contexts(case), g)
        answer = _shuffled(_spread(S * k, 1, case["answer"]), g)
        lens = prompt.repeat_interleave(k) + answer
        width = (case["longest"] + case["answer"] + P - 1) // P
        common = prompt.repeat_interleave(k) // P                        # whole pages that a family shares
        own_pages = (lens + P - 1) // P - common
        pages = torch.cat([prompt // P, own_pages])
        most = int((prompt // P).sum() + ((answer + P - 1) // P).sum()) + S * k + 11
        flat, free, blocks = _tables(pages, int(pages.max().clamp(min=1)), most, g)
        col = torch.arange(width, device=DEV)
        family = torch.arange(S, device=DEV).repeat_interleave(k)
        w = flat.shape[1] - 1
        shared = flat[family[:, None], col.clamp(max=w)]
        mine = flat[S + torch.arange(S * k, device=DEV)[:, None], (col - common[:, None]).clamp(0, w)]
        used = col < ((lens + P - 1) // P)[:, None]
        table = torch.where(used, torch.where(col < common[:, None], shared, mine), -1).int().contiguous()
        shares = torch.zeros(blocks, device=DEV, dtype=i32)
        held = flat[:S][torch.arange(flat.shape[1], device=DEV) < (prompt // P)[:, None]].long()
        shares[held] = k - 1
        cut = torch.rand(S * k, generator=g, device=DEV) < case["cut"]
        less = torch.rand(S * k, generator=g, device=DEV) * answer
        keep = torch.zeros_like(lens) if case["whole"] else torch.where(
            torch.rand(S * k, generator=g, device=DEV) < 0.5, 0, lens - less.long())
        st.update(keep=torch.where(cut, keep, lens).int())
    else:
        lens = _shuffled(_contexts(case), g)
        width = (case["longest"] + P - 1) // P
        pages = (lens + P - 1) // P
        table, free, blocks = _tables(pages, width, int(int(pages.sum()) / case["used"]) + 5, g)
        shares = torch.zeros(blocks, device=DEV, dtype=i32)
        for s in range(0, S - 1, 5):  # some of the sequences share the first half of another's pages
            n = int(min(lens[s], lens[s + 1])) // P // 2
            shares[table[s, :n].long()] += 1
            gone = table[s + 1, :n].clone()
            table[s + 1, :n] = table[s, :n]
            free = torch.cat([free, gone])
        st.update(pools=[(torch.randint(0, 256, (blocks * P * NVFP4_ROW,), generator=g, device=DEV, dtype=torch.uint8),
                          P * NVFP4_ROW)],
                  table_out=torch.empty_like(table), free_out=torch.full((blocks,), -1, device=DEV, dtype=i32),
                  copy_src=torch.empty(case["moves"], device=DEV, dtype=i32),
                  copy_dst=torch.empty(case["moves"], device=DEV, dtype=i32), end=torch.zeros(1, device=DEV, dtype=i32),
                  workspace={})
    stack = torch.full((blocks,), -1, device=DEV, dtype=i32)
    stack[:free.numel()] = free
    st["count"] = torch.tensor([free.numel()], device=DEV, dtype=i32)
    st.update(lens=lens.int(), table=table, free=stack, shares=shares, blocks=blocks, lens_out=torch.empty_like(lens, dtype=i32),
              shares_out=torch.empty_like(shares), count_out=torch.empty_like(st["count"]))
    return st


# ---------------------------------------------------------------------------- plain forms
def _decode_rows(rows, fp8, dtype):
    """The 512 latent and 64 rope values that cache rows [n, row bytes] stand for."""
    rope = rows[:, -ROPE:].contiguous().view(torch.float8_e4m3fn).to(dtype)
    if fp8:
        return rows[:, :LATENT].contiguous().view(torch.float8_e4m3fn).to(dtype), rope
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=DEV, dtype=dtype)
    codes = rows[:, :CODE_BYTES]
    v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(1).int()]
    s = rows[:, CODE_BYTES:CODE_BYTES + SCALE_BYTES].contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (v.unflatten(1, (SCALE_BYTES, GROUP)) * s[..., None]).flatten(1), rope


def _plain_chunk(st):
    case = st["case"]
    P, H, fp8 = case["page"], case["heads"], case["fp8"]
    row = FP8_ROW if fp8 else NVFP4_ROW
    pages = st["pool"].view(st["blocks"], P * row)
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    out, lse = torch.zeros_like(st["out"]), torch.zeros_like(st["lse"])
    for s, length in enumerate(lens):
        n = cu[s + 1] - cu[s]
        if n == 0:
            continue
        rows = pages[st["table"][s, :(length + P - 1) // P].long()].view(-1, row)[:length]
        lat, rope = _decode_rows(rows, fp8, torch.float32)
        keys = torch.cat([lat, rope], 1).t()
        step = max(1, SCORES // (H * length))
        for t in range(0, n, step):
            m = min(step, n - t)
            at = slice(cu[s] + t, cu[s] + t + m)
            seen = length - n + t + m  # the last of these tokens sees so many
            q = torch.cat([st["q_latent"][at], st["q_rope"][at]], -1).float().view(m * H, -1)
            z = torch.matmul(q, keys[:, :seen]).mul_(SM_SCALE).view(m, H, seen)
            pos = length - n + t + torch.arange(m, device=DEV)
            z.masked_fill_(torch.arange(seen, device=DEV) > pos[:, None, None], -math.inf)
            top = z.amax(-1, keepdim=True)
            e = z.sub_(top).exp_()
            total = e.sum(-1, keepdim=True)
            o = torch.matmul(e.view(m * H, seen), lat[:seen]).view(m, H, LATENT) / total
            out[at] = o.bfloat16()
            lse[at] = (top + total.log()).squeeze(-1)
    return {"out": out, "lse": lse}


def _copy_plain(pool, size, src, dst):
    pages = pool.view(-1, size)
    live = (src >= 0) & (dst >= 0)
    pages[dst[live].long()] = pages[src[live].long()]


def _plain_fork(st):
    P = st["case"]["page"]
    table, free, shares = st["table"], st["free"], st["shares"]
    S, W = table.shape
    NB = shares.numel()
    src, dst, n = st["src"].long(), st["dst"].long(), st["fork_lens"].long()
    lens = st["lens"].long()
    i = torch.arange(src.numel(), device=DEV)
    count = st["count"].long().clamp(0, free.numel())
    inside = (src >= 0) & (src < S) & (dst >= 0) & (dst < S)
    sc, dc = src.clamp(0, S - 1), dst.clamp(0, S - 1)
    first = torch.full((S,), i.numel(), device=DEV).scatter_reduce(
        0, dc, torch.where((src != -1) & (dst >= 0) & (dst < S), i, i.numel()), "amin")
    ok = inside & (n >= 0) & (n <= lens[sc]) & (n <= W * P) & (lens[dc] == 0) & (first[dc] == i)
    need = (ok & (n % P != 0)).long()
    rank = need.cumsum(0)
    ok = ok & ((need == 0) | (rank <= count))
    need = torch.where(ok, need, 0)
    full = torch.where(ok, n // P, 0)
    fresh = free[(count - rank).clamp(0, free.numel() - 1)].long()
    last = table[sc, full.clamp(max=W - 1)].long()
    col = torch.arange(W, device=DEV)
    taken = col < full[:, None]
    rows = torch.where(taken, table[sc], torch.where((col == full[:, None]) & (need > 0)[:, None], fresh[:, None].int(), table[dc]))
    held = table[sc][taken].long()
    held = held[(held >= 0) & (held < NB)]
    new_shares = shares + torch.bincount(held, minlength=NB).int()
    new_table, new_lens = table.clone(), lens.int()
    new_table[dc[ok]] = rows[ok]
    new_lens[dc[ok]] = n[ok].int()
    pair = (need > 0) & (last >= 0) & (last < NB) & (fresh >= 0) & (fresh < NB)
    copy_src, copy_dst = torch.where(pair, last, -1).int(), torch.where(pair, fresh, -1).int()
    for pool, size in st["pools"]:
        _copy_plain(pool, size, copy_src, copy_dst)
    return {"block_table": new_table, "seq_lens": new_lens, "page_shares": new_shares,
            "free_count": (count - need.sum()).int(), "shared_blocks": torch.where(ok, full, -1).int(),
            "copy_src": copy_src, "copy_dst": copy_dst, "latent": st["pools"][0][0], "index": st["pools"][1][0]}


def _plain_release(st):
    P = st["case"]["page"]
    table, free, shares = st["table"], st["free"], st["shares"]
    S, W = table.shape
    NB, cap = shares.numel(), free.numel()
    lens, keep = st["lens"].long(), st["keep"].long()
    cut = (keep >= 0) & (keep < lens)
    inner = table.gather(1, (keep // P).clamp(0, W - 1)[:, None]).squeeze(1).long()
    in_pool = (inner >= 0) & (inner < NB)
    stuck = cut & (keep % P != 0) & (keep // P < W) & in_pool & (shares[torch.where(in_pool, inner, 0)] > 0)
    cut = cut & ~stuck
    col = torch.arange(W, device=DEV)
    drop = (cut[:, None] & (col >= ((keep + P - 1) // P)[:, None]) & (col < ((lens + P - 1) // P)[:, None])
            & (table >= 0) & (table < NB))
    page = table[drop].long()
    seq = torch.arange(S, device=DEV)[:, None].expand(S, W)[drop]
    drops = torch.bincount(page, minlength=NB)
    first = torch.full((NB,), S, device=DEV).scatter_reduce(0, page, seq, "amin")
    gone = drops > shares
    back = page[gone[page] & (first[page] == seq)]  # by sequence, then block
    count = st["count"].long().clamp(0, cap)
    at = count + back.numel() - 1 - torch.arange(back.numel(), device=DEV)
    stack = free.clone()
    stack[at[at < cap]] = back[at < cap].int()
    return {"seq_lens": torch.where(cut, keep, lens).int(), "page_shares": torch.where(gone, 0, shares - drops).int(),
            "free_pages": stack, "free_count": (count + back.numel()).clamp(max=cap).int()}


def _plain_compact(st):
    case = st["case"]
    P = case["page"]
    table, free, shares = st["table"], st["free"], st["shares"]
    NB, W = shares.numel(), table.shape[1]
    lens = st["lens"].long()
    count = st["count"].long().clamp(0, free.numel())
    held = torch.arange(W, device=DEV) < ((lens + P - 1) // P)[:, None]
    ids = table[held].long()
    used = torch.zeros(NB, device=DEV, dtype=torch.bool)
    used[ids[(ids >= 0) & (ids < NB)]] = True
    spare = free[torch.arange(free.numel(), device=DEV) < count].long()
    idle = torch.zeros_like(used)
    idle[spare[(spare >= 0) & (spare < NB)]] = True
    idle &= ~used
    low, high = idle.nonzero().squeeze(1), used.nonzero().squeeze(1).flip(0)
    n = min(low.numel(), high.numel(), case["moves"])
    m = int((low[:n] < high[:n]).sum())
    src, dst = high[:m], low[:m]
    to = torch.arange(NB, device=DEV)
    to[src] = dst
    valid = held & (table >= 0) & (table < NB)
    new_table = torch.where(valid, to[torch.where(valid, table, 0).long()].int(), table)
    new_shares = shares.clone()
    new_shares[dst] = shares[src]
    new_shares[src] = 0
    used[src], used[dst], idle[src], idle[dst] = False, True, True, False
    left = idle.nonzero().squeeze(1).flip(0).int()
    stack = torch.full_like(free, -1)
    stack[:left.numel()] = left
    copy_src, copy_dst = (torch.full((case["moves"],), -1, device=DEV, dtype=torch.int32) for _ in range(2))
    copy_src[:m], copy_dst[:m] = src.int(), dst.int()
    pool, size = st["pools"][0]
    _copy_plain(pool, size, copy_src, copy_dst)
    top = torch.where(used, torch.arange(1, NB + 1, device=DEV), 0).amax()
    return {"block_table": new_table, "page_shares": new_shares, "free_pages": stack,
            "free_count": torch.tensor([left.numel()], device=DEV, dtype=torch.int32), "copy_src": copy_src,
            "copy_dst": copy_dst, "pages_end": top.int().view(1), "latent": pool}


# ----------------------------------------------------------------------------- one pass
def _own(st):
    import nvfp4_compressed_mla_gb300 as nm
    case = st["case"]
    P, blocks = case["page"], st["blocks"]
    if case["op"] == "chunk":
        n, H = st["out"].shape[:2]
        if not st["workspace"]:  # kept by the program from its first step on
            size = nm.dense_mla_chunk_workspace_size(n, H, case["seqs"])
            st["workspace"]["buffer"] = torch.empty(size, device=DEV, dtype=torch.uint8)
        fmt = nm.ROW_FP8_576 if case["fp8"] else nm.ROW_NVFP4_352
        nm.dense_mla_chunk(st["q_latent"], st["q_rope"], st["cu"], st["table"], st["lens"], P, st["pool"], blocks,
                           P * nm.ROW_BYTES[fmt], fmt, SM_SCALE, out=st["out"], lse=st["lse"],
                           workspace=st["workspace"]["buffer"])
        return {"out": st["out"], "lse": st["lse"]}
    outs = {"page_shares_out": st["shares_out"], "free_count_out": st["count_out"]}
    if case["op"] == "fork":
        nm.nvfp4_mla_fork(st["src"], st["dst"], st["fork_lens"], st["lens"], st["table"], P, st["shares"], st["free"],
                          st["count"], seq_lens_out=st["lens_out"], shared_blocks=st["shared"], copy_src=st["copy_src"],
                          copy_dst=st["copy_dst"], **outs)
        for pool, size in st["pools"]:
            nm.nvfp4_mla_copy_pages(st["copy_src"], st["copy_dst"], pool, blocks, size, size)
        return {"block_table": st["table"], "seq_lens": st["lens_out"], "page_shares": st["shares_out"],
                "free_count": st["count_out"], "shared_blocks": st["shared"], "copy_src": st["copy_src"],
                "copy_dst": st["copy_dst"], "latent": st["pools"][0][0], "index": st["pools"][1][0]}
    if case["op"] == "release":
        nm.nvfp4_mla_release(st["keep"], st["lens"], st["table"], P, st["shares"], st["free"], st["count"],
                             seq_lens_out=st["lens_out"], **outs)
        return {"seq_lens": st["lens_out"], "page_shares": st["shares_out"], "free_pages": st["free"],
                "free_count": st["count_out"]}
    if not st["workspace"]:
        st["workspace"]["buffer"] = torch.empty(nm.nvfp4_mla_compact_workspace_size(blocks), device=DEV, dtype=torch.uint8)
    nm.nvfp4_mla_compact(st["lens"], st["table"], P, st["shares"], st["free"], st["count"], case["moves"],
                         block_table_out=st["table_out"], free_pages_out=st["free_out"], copy_src=st["copy_src"],
                         copy_dst=st["copy_dst"], pages_end=st["end"], workspace=st["workspace"]["buffer"], **outs)
    pool, size = st["pools"][0]
    nm.nvfp4_mla_copy_pages(st["copy_src"], st["copy_dst"], pool, blocks, size, size)
    return {"block_table": st["table_out"], "page_shares": st["shares_out"], "free_pages": st["free_out"],
            "free_count": st["count_out"], "copy_src": st["copy_src"], "copy_dst": st["copy_dst"],
            "pages_end": st["end"], "latent": pool}


def run(state):
    if own:
        return _own(state)
    return {"chunk": _plain_chunk, "fork": _plain_fork, "release": _plain_release,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- the work
def work(case):
    P, S = case["page"], case["seqs"]
    mean = sum(_contexts(case)) / S
    if case["op"] == "chunk":
        H, row, new = case["heads"], FP8_ROW if case["fp8"] else NVFP4_ROW, _new_tokens(case)
        total = sum(new)
        mean = max(mean, total / S)
        # a sequence's n new tokens see its keys but, between them, n (n - 1) / 2
        seen = total * mean - sum(n * (n - 1) / 2 for n in new)
        return {"bytes": S * mean * row + total * H * (2.0 * (LATENT + ROPE) + 2 * LATENT + 4) + 4 * S * mean / P,
                "flops": max(seen, total) * H * FLOPS}
    if case["op"] == "fork":  # table entries read and written, their counts; the pages copied of both pools
        forks = S * case["samples"]
        return {"bytes": forks * (mean // P) * 8 + S * (mean // P) * 8
                + forks * (1 - 1 / P) * 2 * P * (NVFP4_ROW + INDEX_ROW) + 32.0 * forks, "flops": 0.0}
    if case["op"] == "release":  # entries of the sequences that are cut, their counts and the stack
        k = case["samples"]
        share = 1.0 if case["whole"] else 0.5
        entries = S * k * case["cut"] * (share * (mean + case["answer"] / 2) + (1 - share) * case["answer"] / 4) / P
        return {"bytes": entries * 12 + S * k * 12.0, "flops": 0.0}
    # the tables once in and out, the counts, the stack, and the pages that move
    entries = S * mean / P
    pool = entries / case["used"]
    moved = min(case["moves"], entries * (1 - case["used"]))
    return {"bytes": entries * 8 + pool * 8 + (pool - entries) * 8 + moved * (2.0 * P * NVFP4_ROW + 8), "flops": 0.0}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The attention token by token in 64 bits, from the row format's bits; the page operators give whole numbers only."""
    if case["op"] != "chunk" or work(case)["flops"] > 1e13:
        return None
    st = prepare(case, seed)
    P, H, fp8 = case["page"], case["heads"], case["fp8"]
    row = FP8_ROW if fp8 else NVFP4_ROW
    f64 = torch.float64
    byte = torch.arange(256, device=DEV)
    exp, man = (byte >> 3) & 15, (byte & 7).to(f64)
    e4m3 = torch.where(exp > 0, (1 + man / 8) * torch.pow(2.0, (exp - 7).to(f64)), man / 8 * 2.0 ** -6)
    e4m3 = torch.where(byte >= 128, -e4m3, e4m3)
    code = torch.arange(16, device=DEV)
    e2, m2 = (code >> 1) & 3, (code & 1).to(f64)
    e2m1 = torch.where(e2 > 0, (1 + m2 / 2) * torch.pow(2.0, (e2 - 1).to(f64)), m2 / 2) * torch.where(code >= 8, -1.0, 1.0).to(f64)
    rows_all = st["pool"].view(st["blocks"] * P, row)
    out = torch.zeros(st["out"].shape, device=DEV, dtype=f64)
    lse = torch.zeros(st["lse"].shape, device=DEV, dtype=f64)
    for s in range(case["seqs"]):
        a, b, length = int(st["cu"][s]), int(st["cu"][s + 1]), int(st["lens"][s])
        pos = torch.arange(length, device=DEV)
        rows = rows_all[st["table"][s].long()[pos // P] * P + pos % P]
        if fp8:
            lat = e4m3[rows[:, :LATENT].int()]
        else:
            lat = torch.empty(length, LATENT, device=DEV, dtype=f64)
            lat[:, 0::2], lat[:, 1::2] = e2m1[(rows[:, :CODE_BYTES] & 15).int()], e2m1[(rows[:, :CODE_BYTES] >> 4).int()]
            lat *= e4m3[rows[:, CODE_BYTES:CODE_BYTES + SCALE_BYTES].int()].repeat_interleave(GROUP, 1)
        rope = e4m3[rows[:, row - ROPE:].int()]
        span = max(1, (1 << 26) // (H * length))
        for t in range(a, b, span):
            u = min(t + span, b)
            last = length - (b - t) + 1 + torch.arange(u - t, device=DEV)  # keys that each token sees
            z = SM_SCALE * (torch.einsum("thd,jd->thj", st["q_latent"][t:u].to(f64), lat)
                            + torch.einsum("thd,jd->thj", st["q_rope"][t:u].to(f64), rope))
            z = torch.where(pos < last[:, None, None], z, -math.inf)
            lse[t:u] = torch.logsumexp(z, -1)
            out[t:u] = torch.einsum("thj,jd->thd", torch.exp(z - lse[t:u, :, None]), lat)
    return {"out": out, "lse": lse}
