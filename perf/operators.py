"""The step-planning, index-cache and selection operators: their cases, inputs and plain forms.

Around a sparse MLA decode step stand the operators measured here: building the step's block tables
and slot maps from request lengths (and giving pages back when requests shrink or end), writing and
reading the NVFP4 index-key cache, and choosing the blocks of the context that a query token attends
to. `run` computes them in elementary torch operations, or, where `own` is true, through
nvfp4_compressed_mla_gb300.
"""
import math

import torch

own = False

DEV = "cuda:0"
DIM = 128            # index key width
GROUP = 16           # values per E4M3 scale
CODE_BYTES = DIM // 2
SCALE_BYTES = DIM // GROUP
ROW_BYTES = CODE_BYTES + SCALE_BYTES   # 72 bytes of an index row
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes
MAX_TOPK = 65536


# ---------------------------------------------------------------------------------- cases
def _plan(name, **kw):
    # new: "one" (a decode step), "draft" (1..`most` tokens each), "mixed" (decode steps and prompts up to `most`)
    return {"name": name, "op": "plan", "page": 64, "spare": 1.25, **kw}


def _truncate(name, **kw):
    # cut: share of sequences that shrink; whole: they end (all pages return) instead of dropping up to `most` tokens
    return {"name": name, "op": "truncate", "page": 64, **kw}


def _index(name, **kw):
    return {"name": name, "op": "index", "page": 64, "pad": 0, **kw}


def _select(name, **kw):
    return {"name": name, "op": "select", "page": 64, "sink": 0, "recent": 0, "ragged": 0.0, "slack": 0, **kw}


def listed():
    return [
        # one decode step of the 66 agent sessions: one new token each, every 64th opens a page
        _plan("plan_agent", seqs=66, longest=150000, tokens=66, new="one", most=1),
        # a step of continuous batching: 1021 requests, prompts among them, within a 131072-token budget
        _plan("plan_mixed", seqs=1021, longest=65536, tokens=131072, new="mixed", most=16384),
        # draft tokens that a verification step rejected: a few tokens off each of 66 sessions
        _truncate("truncate_drafts", seqs=66, longest=150000, cut=0.9, whole=False, most=15),
        # a quarter of 1021 requests ends and returns its pages
        _truncate("truncate_release", seqs=1021, longest=65536, cut=0.25, whole=True, most=0),
        # index keys of one decode step: 66 tokens, read back
        _index("index_step", seqs=66, longest=150000, tokens=66, run_len=1),
        # index keys of a prompt chunk: 8 sequences x 4096 tokens, read back, the batch padded
        _index("index_chunk", seqs=8, longest=16384, tokens=32768, run_len=4096, pad=37),
        # the smallest selection: one sequence of 4096 tokens, 16 heads, the top 256 tokens
        _select("select_tiny", seqs=1, longest=4096, per_seq=1, heads=16, block=1, num=256),
        # a decode step of the 66 agent sessions: the top 2048 tokens of up to 150000
        _select("select_agent", seqs=66, longest=150000, ragged=0.053, per_seq=1, heads=64, block=1, num=2048),
        # the same sessions by whole pages: 32 blocks of 64, the first and the two newest always among them
        _select("select_agent_blocks", seqs=66, longest=150000, ragged=0.053, per_seq=1, heads=64, block=64, num=32,
                sink=1, recent=2),
        # 15 draft tokens on each of 32 sequences of 65536 tokens
        _select("select_multi_token", seqs=32, longest=65536, per_seq=15, heads=64, block=1, num=2048),
        # a prompt chunk: 512 query tokens on each of 4 sequences of 16384, blocks of 16
        _select("select_prefill", seqs=4, longest=16384, per_seq=512, heads=32, block=16, num=128, sink=1, recent=4),
        # one request with a million tokens: the long axis alone has to fill the device
        _select("select_long", seqs=1, longest=1000003, per_seq=1, heads=64, block=1, num=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "truncate", "index", "select", "select", "select"])
    page = rng.choice([16, 32, 48, 64, 64, 64, 128])
    if op in ("plan", "truncate"):
        seqs = _log_int(rng, 1, 1500)
        longest = _log_int(rng, 50, min(150000, 60_000_000 // seqs))
        if op == "truncate":
            return {"op": op, "page": page, "seqs": seqs, "longest": longest, "cut": round(rng.uniform(0.05, 1.0), 3),
                    "whole": rng.random() < 0.5, "most": rng.randint(1, 40)}
        new = rng.choice(["one", "draft", "mixed"])
        most = {"one": 1, "draft": rng.randint(2, 16), "mixed": _log_int(rng, 64, 16384)}[new]
        tokens = _log_int(rng, 1, 131072) if new == "mixed" else max(1, int(seqs * most * rng.uniform(0.5, 1.2)))
        return {"op": op, "page": page, "spare": round(rng.uniform(0.3, 1.5), 3), "seqs": seqs, "longest": longest,
                "tokens": tokens, "new": new, "most": most}
    if op == "index":
        seqs = _log_int(rng, 1, 300)
        run_len = _log_int(rng, 1, max(1, 32768 // seqs))
        return {"op": op, "page": page, "pad": rng.choice([0, rng.randint(1, 64)]), "seqs": seqs,
                "longest": run_len + _log_int(rng, 1, 20000), "tokens": seqs * run_len, "run_len": run_len}
    heads = rng.choice([1, 4, 8, 16, 24, 32, 33, 48, 64, 64, 96, 128])
    per_seq = rng.choice([1, 1, 1, rng.randint(2, 16), _log_int(rng, 16, 512)])
    seqs = _log_int(rng, 1, max(1, 512 // per_seq))
    # keys seen x heads at most those of the agent decode step
    most = min(300000, int(66 * 150000 * 64 / (seqs * per_seq * heads)), 24_000_000 // (seqs * per_seq))
    block = rng.choice([1, 1, 2, 4, 8, 16, 32, 64, 128])
    longest = _log_int(rng, min(16 * block, most), most)
    sink = rng.choice([0, 0, 1, 2])
    recent = rng.choice([0, 0, 1, 3])
    # some blocks are left to choose from, beside the forced ones
    num = sink + recent + _log_int(rng, 1, max(1, min(4096, 16384 // block, longest * 3 // (4 * block)) - sink - recent))
    return {"op": op, "page": page, "seqs": seqs, "longest": longest, "ragged": round(rng.choice([0.0, rng.random()]), 3),
            "slack": rng.choice([0, rng.randint(1, 2000)]), "per_seq": per_seq, "heads": heads, "block": block, "num": num,
            "sink": sink, "recent": recent}


# --------------------------------------------------------------------------------- inputs
def _lens(case, g, least=1):
    """Sequence lengths: U[longest * (1 - ragged), longest] for a selection, log-uniform otherwise."""
    u = torch.rand(case["seqs"], generator=g, device=DEV, dtype=torch.float64)
    top = case["longest"]
    if "ragged" in case:
        n = top * (1 - case["ragged"] * u)
    else:
        n = torch.exp(u * math.log(max(top, 2)))
    return n.floor().long().clamp(least, max(top, least))


def _tables(lens, page, width, extra, g):
    """Block table [S, width] over a random permutation of the pool's pages (-1 = unused), and the pages left over."""
    pages = (lens + page - 1) // page
    total = int(pages.sum())
    perm = torch.randperm(total + extra, generator=g, device=DEV)
    at = (pages.cumsum(0) - pages)[:, None] + torch.arange(width, device=DEV)
    used = torch.arange(width, device=DEV) < pages[:, None]
    table = torch.where(used, perm[at.clamp(max=max(total - 1, 0))], -1)
    return table.int().contiguous(), perm[total:].int().contiguous(), total


def _quantize(x):
    """E2M1 codes (0..15) and E4M3 scales of each 16 values of x [..., 128]."""
    a = x.float().unflatten(-1, (SCALE_BYTES, GROUP))
    amax = a.abs().amax(-1, keepdim=True)
    scale = (amax.double() / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    m = a.abs()
    mag = ((m > 0.25 * s).int() + (m >= 0.75 * s).int() + (m > 1.25 * s).int() + (m >= 1.75 * s).int()
           + (m > 2.5 * s).int() + (m >= 3.5 * s).int() + (m > 5.0 * s).int())
    codes = torch.where(s > 0, mag + 8 * torch.signbit(a).int(), 0)
    return codes.flatten(-2).to(torch.uint8), scale.squeeze(-1).view(torch.uint8)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pool_views(pool, case):
    """Codes [pages, P, 64] and scales [pages, P, 8] of a pool [pages, P * 72]."""
    P = case["page"]
    n = pool.shape[0]
    return (pool[:, :P * CODE_BYTES].view(n, P, CODE_BYTES),
            pool[:, P * CODE_BYTES:P * ROW_BYTES].view(n, P, SCALE_BYTES))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    P, S = case["page"], case["seqs"]
    st = {"case": dict(case)}
    if case["op"] == "plan":
        lens = _lens(case, g)
        if case["new"] == "one":
            new = torch.ones(S, device=DEV, dtype=torch.long)
        else:
            new = torch.randint(1, case["most"] + 1, (S,), generator=g, device=DEV)
            if case["new"] == "mixed":  # one request in eight is a prompt, the others decode
                prompt = torch.rand(S, generator=g, device=DEV) < 0.125
                new = torch.where(prompt, new, 1)
        need = int(((lens + new + P - 1) // P - (lens + P - 1) // P).sum())
        width = (case["longest"] + case["most"] + P - 1) // P
        table, free, _ = _tables(lens, P, width, max(16, int(need * case["spare"])), g)
        st.update(new_lens=new.int(), seq_lens=lens.int(), table=table, free=free,
                  count=torch.tensor([free.numel()], device=DEV, dtype=torch.int32))
    elif case["op"] == "truncate":
        lens = _lens(case, g)
        width = (case["longest"] + P - 1) // P
        table, free, _ = _tables(lens, P, width, 1000, g)
        cut = torch.rand(S, generator=g, device=DEV) < case["cut"]
        less = lens if case["whole"] else torch.randint(1, case["most"] + 1, (S,), generator=g, device=DEV)
        keep = torch.where(cut, (lens - less).clamp(min=0), lens)
        stack = torch.full((free.numel() + S * width,), -1, device=DEV, dtype=torch.int32)
        stack[:free.numel()] = free
        st.update(keep_lens=keep.int(), seq_lens=lens.int(), table=table, free=stack,
                  count=torch.tensor([free.numel()], device=DEV, dtype=torch.int32))
    elif case["op"] == "index":
        n = case["run_len"]
        lens = _lens(case, g, least=n)
        width = (max(case["longest"], n) + P - 1) // P
        table, _, total = _tables(lens, P, width, 0, g)
        seq = torch.arange(S, device=DEV).repeat_interleave(n)
        pos = (lens - n).repeat_interleave(n) + torch.arange(n, device=DEV).repeat(S)
        pad = torch.full((case["pad"],), -1, device=DEV)
        keys = torch.randn(S * n + case["pad"], DIM, generator=g, device=DEV)
        # one page more than the operator is told of: the plain form puts padding there
        st.update(keys=keys.bfloat16(), seq_ids=torch.cat([seq, pad]).int(), positions=torch.cat([pos, pad]).int(),
                  table=table, blocks=total, pool=torch.zeros(total + 1, P * ROW_BYTES, device=DEV, dtype=torch.uint8))
    else:
        lens = _lens(case, g, least=1)
        q = case["per_seq"]
        width = (case["longest"] + case["slack"] + P - 1) // P  # the table may be wider than the longest sequence
        table, _, total = _tables(lens, P, width, 0, g)
        pool = torch.empty(total, P * ROW_BYTES, device=DEV, dtype=torch.uint8)
        codes, scales = _quantize(torch.randn(total * P, DIM, generator=g, device=DEV).bfloat16())
        c, s = _pool_views(pool, case)
        c.copy_(_pack(codes).view_as(c))
        s.copy_(scales.view_as(s))
        del codes, scales
        seq = torch.arange(S, device=DEV).repeat_interleave(q)
        pos = (lens - q).repeat_interleave(q) + torch.arange(q, device=DEV).repeat(S)  # < 0: a token before the start
        H = case["heads"]
        qi = torch.randn(S * q, H, DIM, generator=g, device=DEV).bfloat16()
        w = torch.randn(S * q, H, generator=g, device=DEV) / math.sqrt(H * DIM)
        st.update(q_index=qi, weights=w, q_seq=seq.int(), q_pos=pos.int(), table=table, pool=pool, blocks=total)
    if case["op"] == "plan":  # the step's buffers, as a serving loop keeps them
        n = case["tokens"]
        st.update(lens_out=torch.empty_like(st["seq_lens"]), count_out=torch.empty_like(st["count"]),
                  ids=torch.empty(n, device=DEV, dtype=torch.int32), pos=torch.empty(n, device=DEV, dtype=torch.int32),
                  slots=torch.empty(n, device=DEV, dtype=torch.int64),
                  cu=torch.empty(S + 1, device=DEV, dtype=torch.int32))
    elif case["op"] == "truncate":
        st.update(lens_out=torch.empty_like(st["seq_lens"]), count_out=torch.empty_like(st["count"]))
    elif case["op"] == "index":
        st.update(out=torch.empty_like(st["keys"]))
    else:
        st.update(idx=torch.empty(S * case["per_seq"], case["num"] * case["block"], device=DEV, dtype=torch.int32),
                  workspace={})
    return st


# ---------------------------------------------------------------------------- plain forms
def _plain_plan(st):
    c = st["case"]
    P, n = c["page"], c["tokens"]
    table, free = st["table"], st["free"]
    S, width = table.shape
    lens, new = st["seq_lens"].long(), st["new_lens"].long()
    count = st["count"].long().clamp(0, free.numel())
    blocks = (lens + P - 1) // P
    fits = (new >= 0) & (lens >= 0) & (lens + new <= width * P)
    need = torch.where(fits, (lens + new + P - 1) // P - blocks, 0)
    paged = fits & ((need == 0) | (need.cumsum(0) <= count))
    want = torch.where(paged, new, 0)
    served = paged & ((new == 0) | (want.cumsum(0) <= n))
    add = torch.where(served, new, 0)
    take = torch.where(served, need, 0)
    end, first = add.cumsum(0), take.cumsum(0) - take
    t = torch.arange(n, device=DEV)
    live = t < end[-1]
    s = torch.searchsorted(end, t, right=True).clamp(max=S - 1)
    pos = lens[s] + t - (end[s] - add[s])
    fresh = pos // P - blocks[s]
    taken = free[(count - 1 - first[s] - fresh).clamp(0, free.numel() - 1)].long()
    page = torch.where(fresh >= 0, taken, table[s, (pos // P).clamp(0, width - 1)].long())
    slot = torch.where(live & (page >= 0), page * P + pos % P, -1)
    k = torch.arange(width, device=DEV) - blocks[:, None]
    opened = (k >= 0) & (k < take[:, None])
    new_table = torch.where(opened, free[(count - 1 - first[:, None] - k).clamp(0, free.numel() - 1)], table)
    return {"seq_ids": torch.where(live, s, -1).int(), "positions": torch.where(live, pos, -1).int(), "slots": slot,
            "cu_tokens": torch.cat([end.new_zeros(1), end]).int(), "seq_lens": (lens + add).int(),
            "block_table": new_table, "free_count": (count - take.sum()).int()}


def _plain_truncate(st):
    P = st["case"]["page"]
    table, free = st["table"], st["free"]
    cap = free.numel()
    lens, keep = st["seq_lens"].long(), st["keep_lens"].long()
    cut = (keep >= 0) & (keep < lens)
    col = torch.arange(table.shape[1], device=DEV)
    back = (cut[:, None] & (col >= ((keep + P - 1) // P)[:, None]) & (col < ((lens + P - 1) // P)[:, None])
            & (table >= 0)).flatten()
    count = st["count"].long().clamp(0, cap)
    n = back.sum()
    at = count + n - back.cumsum(0)  # the first page returned ends on top
    at = torch.where(back & (at < cap), at, cap)
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at, table.flatten())[:cap]
    return {"seq_lens": torch.where(cut, keep, lens).int(), "free_pages": stack,
            "free_count": (count + n).clamp(max=cap).int()}


def _rows(st, seq, pos):
    """Page and row in the page of each token, and whether it resolves."""
    P, table = st["case"]["page"], st["table"]
    ok = (seq >= 0) & (seq < table.shape[0]) & (pos >= 0) & (pos < table.shape[1] * P)
    page = table[seq.clamp(0, table.shape[0] - 1), (pos // P).clamp(0, table.shape[1] - 1)].long()
    ok = ok & (page >= 0) & (page < st["blocks"])
    return torch.where(ok, page, 0), pos.clamp(min=0) % P, ok


def _values(codes, scales, dtype):
    """The values that packed codes [..., 64] with scales [..., 8] stand for: [..., 128]."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=DEV, dtype=dtype)
    nib = torch.stack([codes & 15, codes >> 4], -1)
    v = grid.index_select(0, nib.flatten().int()).view(*codes.shape[:-1], SCALE_BYTES, GROUP)
    return (v * scales.view(torch.float8_e4m3fn).to(dtype)[..., None]).flatten(-2)


def _plain_index(st):
    c, s = _pool_views(st["pool"], st["case"])
    seq, pos = st["seq_ids"].long(), st["positions"].long()
    page, row, ok = _rows(st, seq, pos)
    codes, scales = _quantize(st["keys"])
    to = torch.where(ok, page, st["blocks"])
    c[to, row] = _pack(codes)
    s[to, row] = scales
    got = _values(c[page, row], s[page, row], torch.float32)
    return {"values": torch.where(ok[:, None], got, 0).bfloat16()}


def _plain_select(st):
    # 64 bits: scores next to the border of the selection decide which tokens are chosen
    case = st["case"]
    P, B, K, H = case["page"], case["block"], case["num"], case["heads"]
    table = st["table"].long()
    S, width = table.shape
    L = width * P
    c, s = _pool_views(st["pool"], case)
    keys = _values(c, s, torch.float64)[table.clamp(min=0)].view(S, L, DIM)
    q_seq, q_pos = st["q_seq"].long(), st["q_pos"].long()
    codes, scales = _quantize(st["q_index"])
    q = _values(_pack(codes), scales, torch.float64)
    dots = torch.matmul(q, keys[q_seq].transpose(1, 2)).clamp_(min=0)           # [Q, H, L]
    score = torch.matmul(st["weights"].double()[:, None], dots).squeeze(1)     # [Q, L]
    del dots, keys
    at = torch.arange(L, device=DEV)
    seen = (at <= q_pos[:, None])
    stored = ((table >= 0) & (table < st["blocks"])).repeat_interleave(P, 1)[q_seq]
    low = -math.inf
    score = torch.where(seen & stored & ~score.isnan(), score, low)
    nb = (L + B - 1) // B
    score = torch.nn.functional.pad(score, (0, nb * B - L), value=low).view(-1, nb, B).amax(-1)
    blocks = torch.where(q_pos < 0, 0, q_pos // B + 1)[:, None]                  # visible blocks of each query
    b = torch.arange(nb, device=DEV)
    always = (b < case["sink"]) | (b >= blocks - case["recent"])
    # by rank: forced blocks, visible blocks by score, the rest; equal scores by the lower index
    rank = torch.where(b < blocks, torch.where(always, 1.0, 0.0), -1.0)
    order = torch.sort(torch.where(rank == 0, score, torch.where(rank > 0, math.inf, low)), dim=1, descending=True,
                       stable=True).indices
    order = order.gather(1, torch.sort(rank.gather(1, order), dim=1, descending=True, stable=True).indices)[:, :K]
    order = torch.nn.functional.pad(order, (0, K - order.shape[1]), value=nb)
    order = torch.where(order < blocks, order, nb).sort(1).values
    pos = (order[:, :, None] * B + torch.arange(B, device=DEV)).flatten(1)
    return {"topk_idx": torch.where((pos <= q_pos[:, None]) & (order < nb).repeat_interleave(B, 1), pos, -1).int()}


# ----------------------------------------------------------------------------- one pass
def _own(st):
    import nvfp4_compressed_mla_gb300 as nm
    case = st["case"]
    P = case["page"]
    if case["op"] == "plan":
        nm.nvfp4_mla_plan_step(st["new_lens"], st["seq_lens"], st["table"], P, st["free"], st["count"], case["tokens"],
                               seq_lens_out=st["lens_out"], free_count_out=st["count_out"], seq_ids=st["ids"],
                               positions=st["pos"], slots=st["slots"], cu_tokens=st["cu"])
        return {"seq_ids": st["ids"], "positions": st["pos"], "slots": st["slots"], "cu_tokens": st["cu"],
                "seq_lens": st["lens_out"], "block_table": st["table"], "free_count": st["count_out"]}
    if case["op"] == "truncate":
        nm.nvfp4_mla_truncate(st["keep_lens"], st["seq_lens"], st["table"], P, st["free"], st["count"],
                              seq_lens_out=st["lens_out"], free_count_out=st["count_out"])
        return {"seq_lens": st["lens_out"], "free_pages": st["free"], "free_count": st["count_out"]}
    if case["op"] == "index":
        nm.nvfp4_mla_index_append(st["keys"], st["seq_ids"], st["positions"], st["table"], P, st["pool"], st["blocks"],
                                  P * ROW_BYTES)
        out = nm.nvfp4_mla_index_read(st["seq_ids"], st["positions"], st["table"], P, st["pool"], st["blocks"],
                                      P * ROW_BYTES, keys=st["out"])
        return {"values": out}
    if not st["workspace"]:  # kept by the program from its first step on
        n = nm.sparse_mla_select_workspace_size(st["q_seq"].numel(), case["heads"], st["table"].shape[1], P, case["block"])
        st["workspace"]["buffer"] = torch.empty(n, device=DEV, dtype=torch.uint8)
    idx = nm.sparse_mla_select(st["q_index"], st["weights"], st["q_seq"], st["q_pos"], st["table"], P, st["pool"],
                               st["blocks"], P * ROW_BYTES, case["num"], select_block=case["block"],
                               sink_blocks=case["sink"], recent_blocks=case["recent"], topk_idx=st["idx"],
                               workspace=st["workspace"]["buffer"])
    return {"topk_idx": idx}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "truncate": _plain_truncate, "index": _plain_index,
            "select": _plain_select}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- the work
def work(case):
    P, S = case["page"], case["seqs"]
    if case["op"] == "plan":  # lengths in and out, offsets; 16 bytes a token; a new page's id read and written
        return {"bytes": 16.0 * S + 16.0 * case["tokens"] + 8.0 * case["tokens"] / P, "flops": 0.0}
    if case["op"] == "truncate":  # lengths; a returned page's id read and written
        mean = case["longest"] / math.log(max(case["longest"], 2)) if case["whole"] else case["most"] / 2
        return {"bytes": 12.0 * S + 8.0 * S * case["cut"] * max(1.0, mean / P), "flops": 0.0}
    if case["op"] == "index":  # a bf16 key in, its row out; the row in, the bf16 values out; ids
        return {"bytes": (case["tokens"] + case["pad"]) * (2.0 * (2 * DIM + ROW_BYTES) + 16), "flops": 0.0}
    q, H = S * case["per_seq"], case["heads"]
    mean = case["longest"] * (1 - case["ragged"] / 2)
    keys = S * mean
    seen = q * max(1.0, mean - (case["per_seq"] - 1) / 2)
    return {"bytes": keys * ROW_BYTES + q * (H * (2.0 * DIM + 4) + 8 + 4 * case["num"] * case["block"]) + 4 * keys / P,
            "flops": seen * H * (2.0 * DIM + 3)}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The stored values from the format's definition: the nearest scale of all E4M3 values, the nearest code of all
    E2M1 values. The other operators give whole numbers only."""
    if case["op"] != "index":
        return None
    st = prepare(case, seed)
    x = st["keys"].double().view(-1, SCALE_BYTES, GROUP)
    scales = torch.arange(127, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    want = x.abs().amax(-1) / 6
    up = torch.searchsorted(scales, want).clamp(1, 126)
    lo, hi = scales[up - 1], scales[up]
    down = (want - lo < hi - want) | ((want - lo == hi - want) & ((up - 1) % 2 == 0))
    s = torch.where(down, lo, hi)[..., None]
    grid = torch.tensor(GRID, device=DEV, dtype=torch.float64)
    off = (x.abs()[..., None] - grid * s[..., None]).abs()
    # a tie goes to the even code: looked for among the even codes first
    first = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=DEV)
    code = first[off[..., first].argmin(-1)]
    v = torch.where(s > 0, grid[code] * s * torch.sign(x), 0).flatten(-2)
    return {"values": torch.where((st["seq_ids"] >= 0)[:, None], v, 0)}
