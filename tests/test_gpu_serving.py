"""GPU: the dense attention of a step and the operators for shared pages together, over one cache, as a
server calls them: plan a step, write its rows, attend, fork, take tokens back, end requests, compact.
The host side keeps its own pool through the oracle and the plain forms."""
import numpy as np
import pytest
import torch

import oracle
from tests import pages_cases as pc, step_cases as sc
from tests.chunk_cases import FP8, NVFP4, ROW, Case
from tests.gpu_cases import dev_tensor as dev
from workloads.gen import bf16_from_f32

pytestmark = pytest.mark.gpu

SEQS, FORKS, MOVES, ROWS = 7, 3, 4, 80


class Server(Case):
    """State on both sides (the host's under the names that Case.check reads), and static buffers for a
    step of at most ROWS tokens."""

    def __init__(self, seed, heads, fmt, page, width, blocks):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.fmt, self.page, self.S, self.width, self.blocks = heads, fmt, page, SEQS, width, blocks
        self.latent_scale, self.rope_scale, self.sm_scale = (0.5, 0.25, 0.04) if fmt == FP8 else (1.0, 1.0, 0.04)
        self.stride = page * ROW[fmt]
        self.num_q = ROWS
        self.lens, self.table = np.zeros(SEQS, np.int32), np.full((SEQS, width), -1, np.int32)
        self.stack, self.count = rng.permutation(blocks).astype(np.int32), blocks
        self.shares = np.zeros(blocks, np.int32)
        # what no token was written to is NaN
        self.pool = np.full((blocks, self.stride), 0xFF, np.uint8)
        zeros = lambda *shape, t=torch.int32: torch.zeros(shape, dtype=t, device="cuda:0")
        bf = torch.bfloat16
        self.d = dict(lens=dev(self.lens), table=dev(self.table), stack=dev(self.stack), shares=dev(self.shares),
                      count=dev(np.array([blocks], np.int32)), pool=dev(self.pool).view(-1), new=zeros(SEQS),
                      src=zeros(FORKS), dst=zeros(FORKS), want=zeros(FORKS), keep=zeros(SEQS),
                      rows=zeros(ROWS, 512, t=bf), rope=zeros(ROWS, 64, t=bf), ql=zeros(ROWS, heads, 512, t=bf),
                      qr=zeros(ROWS, heads, 64, t=bf), end=zeros(1))

    def device_step(self):
        import nvfp4_compressed_mla_gb300 as nm
        d, page, blocks, size = self.d, self.page, self.blocks, self.stride
        ids, pos, _, cu = nm.nvfp4_mla_plan_step(d["new"], d["lens"], d["table"], page, d["stack"], d["count"], ROWS)
        nm.nvfp4_mla_append(d["rows"], d["rope"], ids, pos, d["table"], page, d["pool"], blocks, size, self.fmt,
                            self.latent_scale, self.rope_scale)
        got = nm.dense_mla_chunk(d["ql"], d["qr"], cu, d["table"], d["lens"], page, d["pool"], blocks, size, self.fmt,
                                 self.sm_scale, self.latent_scale, self.rope_scale, out_fp32=True)
        _, a, b = nm.nvfp4_mla_fork(d["src"], d["dst"], d["want"], d["lens"], d["table"], page, d["shares"],
                                    d["stack"], d["count"])
        nm.nvfp4_mla_copy_pages(a, b, d["pool"], blocks, size, size)
        nm.nvfp4_mla_release(d["keep"], d["lens"], d["table"], page, d["shares"], d["stack"], d["count"])
        a, b = nm.nvfp4_mla_compact(d["lens"], d["table"], page, d["shares"], d["stack"], d["count"], MOVES,
                                    pages_end=d["end"])
        nm.nvfp4_mla_copy_pages(a, b, d["pool"], blocks, size, size)
        return got

    def inputs(self):
        """A step's inputs, and what the plain forms make of them."""
        rng, page = self.rng, self.page
        new = np.where(rng.random(SEQS) < 0.5, rng.choice([1, 1, 4, 30], SEQS), 0).astype(np.int32)
        ended = (self.lens == 0) & (rng.random(SEQS) < 0.5)
        new[ended] = 0
        if not self.lens.any():
            new[0] = 60
        h = dict(new=new)
        for name in ("rows", "rope", "ql", "qr"):
            h[name] = bf16_from_f32(rng.standard_normal(tuple(self.d[name].shape)).astype(np.float32))
        plan = sc.plan_step(new, self.lens, self.table, page, self.stack, self.count, ROWS)
        now = plan["seq_lens"]
        h["src"] = rng.integers(-1, SEQS, FORKS).astype(np.int32)
        h["dst"] = rng.integers(0, SEQS, FORKS).astype(np.int32)
        h["want"] = np.array([rng.integers(0, now[s] + 1) if s >= 0 else 0 for s in h["src"]], np.int32)
        fork = pc.fork(h["src"], h["dst"], h["want"], now, plan["table"], page, self.shares, self.stack,
                       plan["free_count"])
        now = fork["seq_lens"]
        h["keep"] = np.where(rng.random(SEQS) < 0.3, (now * rng.choice([0, 0.8], SEQS)).astype(np.int32), now)
        rel = pc.release(h["keep"], now, fork["table"], page, fork["shares"], self.stack, fork["free_count"])
        com = pc.compact(rel["seq_lens"], fork["table"], page, rel["shares"], rel["free_pages"], rel["free_count"],
                         MOVES)
        for name, v in h.items():
            self.d[name].copy_(dev(v, torch.bfloat16) if v.dtype == np.uint16 else dev(v.astype(np.int32)))
        return h, plan, fork, rel, com

    def copy(self, src, dst):
        old = self.pool.copy()
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                self.pool[b] = old[a]

    def check_step(self, refs, got):
        h, plan, fork, rel, com = refs
        ids, pos, cu = (np.asarray(plan[k]) for k in ("seq_ids", "positions", "cu_tokens"))
        n = int((ids >= 0).sum())
        flat = self.pool.reshape(-1)
        assert oracle.append(h["rows"][:n], h["rope"][:n], ids[:n], pos[:n], plan["table"], self.page, flat,
                             self.blocks, self.stride, self.fmt, self.latent_scale, self.rope_scale) == 0
        self.lens, self.table, self.cu, self.n = plan["seq_lens"], plan["table"], cu.astype(np.int32), n
        self.new = np.diff(cu).astype(np.int32)
        self.ql, self.qr = h["ql"], h["qr"]
        torch.cuda.synchronize()
        self.check(*got, out_fp32=True)
        self.copy(fork["copy_src"], fork["copy_dst"])
        self.copy(com["copy_src"], com["copy_dst"])
        self.lens, self.table, self.shares = rel["seq_lens"], com["table"], com["shares"]
        self.stack, self.count = com["free_pages"], com["free_count"]
        d, host = self.d, lambda t: t.cpu().numpy()
        for name in ("lens", "table", "shares"):
            assert np.array_equal(host(d[name]), getattr(self, name)), name
        assert int(d["count"]) == self.count
        assert np.array_equal(host(d["stack"])[:self.count], self.stack[:self.count])
        assert np.array_equal(host(d["pool"]).reshape(self.pool.shape), self.pool)
        return n


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("heads,fmt,page", [(16, NVFP4, 64), (128, NVFP4, 16), (16, FP8, 64), (5, FP8, 24)])
def test_steps_of_a_server_with_shared_pages(heads, fmt, page, captured):
    s = Server(heads + page, heads, fmt, page, width=-(-320 // page), blocks=6 * 320 // page)
    graph, tokens, forked, longest = None, 0, 0, 0
    for _ in range(14):
        refs = s.inputs()
        if captured and graph is None:
            saved = {k: v.clone() for k, v in s.d.items()}
            s.device_step()  # the library is loaded outside the capture
            torch.cuda.synchronize()
            for k, v in saved.items():
                s.d[k].copy_(v)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = s.device_step()
        if captured:
            graph.replay()
        else:
            got = s.device_step()
        tokens += s.check_step(refs, got)
        forked += int((refs[2]["shared_blocks"] > 0).sum())
        longest = max(longest, int(s.lens.max()))
    assert tokens > 100 and forked > 0 and longest > 64, (tokens, forked, longest)


def test_beams_read_what_they_share():
    """Forked sequences attend to their prompt's pages as the prompt does, each within the bound of its
    roundings. The bits may differ: the step's work is divided among the clusters without regard to
    sequences, and the parts of a cut row have FP16 weights relative to references of their own."""
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(61, [500, 0, 0, 0], [1, 0, 0, 0], 16)
    args = c.device()
    out, lse = nm.dense_mla_chunk(*args)
    d32 = lambda *v: dev(np.array(v, np.int32))
    shares = torch.zeros(c.blocks, dtype=torch.int32, device="cuda:0")
    free = sorted(set(range(c.blocks)) - set(c.table[c.table >= 0].tolist()))
    _, a, b = nm.nvfp4_mla_fork(d32(0, 0, 0), d32(1, 2, 3), d32(500, 500, 500), args[4], args[3], c.page, shares,
                                d32(*free), d32(len(free)))
    nm.nvfp4_mla_copy_pages(a, b, args[6], c.blocks, c.stride, c.stride)
    four = [args[0].expand(4, 16, 512).contiguous(), args[1].expand(4, 16, 64).contiguous(), d32(0, 1, 2, 3, 4)]
    out4, lse4 = nm.dense_mla_chunk(*four, *args[3:])
    torch.cuda.synchronize()
    assert int(shares.max()) == 3
    c.check(out, lse)
    for i in range(4):
        c.check(out4[i:i + 1], lse4[i:i + 1])
