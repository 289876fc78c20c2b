"""GPU: the operators of a serving step together, as a server calls them: plan the step, write the
latent and the index rows, select, attend, and give back what a truncation frees. The host side
keeps its own pools and tables through the oracle and the plain forms."""
import numpy as np
import pytest
import torch

import oracle
from tests import step_cases as sc
from tests.gpu_cases import assert_parity, dev_tensor as dev
from workloads.gen import bf16_from_f32

pytestmark = pytest.mark.gpu

PAGE, SEQS, WIDTH, BLOCKS, ROWS = 64, 5, 8, 30, 96
LATENT, INDEX = PAGE * 352, PAGE * sc.ROW
HEADS, INDEX_HEADS, SCALE = 16, 8, 0.05


class Server:
    """State on both sides, and static buffers for a step of at most ROWS tokens."""

    def __init__(self, seed, num, block):
        self.rng = np.random.default_rng(seed)
        self.num, self.block = num, block
        self.lens = np.zeros(SEQS, np.int32)
        self.table = np.full((SEQS, WIDTH), -1, np.int32)
        self.stack = self.rng.permutation(BLOCKS).astype(np.int32)
        self.count = BLOCKS
        self.latent = np.zeros(BLOCKS * LATENT, np.uint8)
        self.index = np.zeros(BLOCKS * INDEX, np.uint8)
        i32 = torch.int32
        self.d = dict(lens=dev(self.lens), table=dev(self.table), stack=dev(self.stack),
                      count=dev(np.array([BLOCKS], np.int32)), latent=dev(self.latent),
                      index=dev(self.index), new=torch.zeros(SEQS, dtype=i32, device="cuda:0"),
                      bad=torch.zeros(1, dtype=i32, device="cuda:0"),
                      index_bad=torch.zeros(1, dtype=i32, device="cuda:0"),
                      refused=torch.zeros(1, dtype=i32, device="cuda:0"))
        for name, shape in (("rows", (ROWS, 512)), ("rope", (ROWS, 64)), ("keys", (ROWS, 128)),
                            ("ql", (ROWS, HEADS, 512)), ("qr", (ROWS, HEADS, 64)),
                            ("qi", (ROWS, INDEX_HEADS, 128))):
            self.d[name] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda:0")
        self.d["w"] = torch.zeros((ROWS, INDEX_HEADS), device="cuda:0")

    def device_step(self):
        import nvfp4_compressed_mla_gb300 as nm
        d = self.d
        ids, pos, _, _ = nm.nvfp4_mla_plan_step(d["new"], d["lens"], d["table"], PAGE, d["stack"],
                                                d["count"], ROWS, refused_count=d["refused"])
        nm.nvfp4_mla_append(d["rows"], d["rope"], ids, pos, d["table"], PAGE, d["latent"], BLOCKS,
                            LATENT, invalid_count=d["bad"])
        nm.nvfp4_mla_index_append(d["keys"], ids, pos, d["table"], PAGE, d["index"], BLOCKS, INDEX,
                                  invalid_count=d["index_bad"])
        top = nm.sparse_mla_select(d["qi"], d["w"], ids, pos, d["table"], PAGE, d["index"], BLOCKS,
                                   INDEX, self.num, self.block)
        out, lse = nm.sparse_mla_decode(d["ql"], d["qr"], ids, top, d["table"], d["lens"], PAGE,
                                        d["latent"], BLOCKS, LATENT, nm.ROW_NVFP4_352, SCALE,
                                        out_fp32=True)
        return ids, pos, top, out, lse

    def inputs(self, new):
        h = dict(new=np.asarray(new, np.int32))
        for name in ("rows", "rope", "keys", "ql", "qr", "qi"):
            h[name] = bf16_from_f32(self.rng.standard_normal(tuple(self.d[name].shape)))
            self.d[name].copy_(dev(h[name], torch.bfloat16))
        h["w"] = self.rng.standard_normal((ROWS, INDEX_HEADS)).astype(np.float32)
        self.d["w"].copy_(dev(h["w"]))
        self.d["new"].copy_(dev(h["new"]))
        return h

    def check(self, h, got):
        ref = sc.plan_step(h["new"], self.lens, self.table, PAGE, self.stack, self.count, ROWS)
        self.table, self.lens, self.count = ref["table"], ref["seq_lens"], ref["free_count"]
        ids, pos = np.asarray(ref["seq_ids"]), np.asarray(ref["positions"])
        n = int((ids >= 0).sum())
        assert oracle.append(h["rows"][:n], h["rope"][:n], ids[:n], pos[:n], self.table, PAGE,
                             self.latent, BLOCKS, LATENT, 0, 1.0, 1.0) == 0
        assert sc.index_append(h["keys"], ids, pos, self.table, PAGE, self.index, BLOCKS,
                               INDEX) == 0
        top = sc.select(h["qi"], h["w"], ids, pos, self.table, PAGE, self.index, BLOCKS, INDEX,
                        self.num, self.block)
        out, lse, _ = oracle.sparse_mla_decode(h["ql"], h["qr"], ids, top, self.table, self.lens,
                                               PAGE, self.latent, BLOCKS, LATENT, 0, SCALE)
        torch.cuda.synchronize()
        assert np.array_equal(got[0].cpu().numpy(), ids) and np.array_equal(got[1].cpu().numpy(), pos)
        d = self.d
        assert np.array_equal(d["lens"].cpu().numpy(), self.lens)
        assert np.array_equal(d["table"].cpu().numpy(), self.table)
        assert int(d["count"]) == self.count
        assert np.array_equal(d["latent"].cpu().numpy(), self.latent)
        assert np.array_equal(d["index"].cpu().numpy(), self.index)
        assert np.array_equal(got[2].cpu().numpy(), top)
        assert (top[n:] == -1).all()
        assert_parity(got[3].double().cpu().numpy(), got[4].double().cpu().numpy(), out, lse)

    def truncate(self, keep):
        import nvfp4_compressed_mla_gb300 as nm
        d, keep = self.d, np.asarray(keep, np.int32)
        nm.nvfp4_mla_truncate(dev(keep), d["lens"], d["table"], PAGE, d["stack"], d["count"])
        ref = sc.truncate(keep, self.lens, self.table, PAGE, self.stack, self.count)
        self.lens, self.stack, self.count = ref["seq_lens"], ref["free_pages"], ref["free_count"]
        torch.cuda.synchronize()
        assert np.array_equal(d["lens"].cpu().numpy(), self.lens)
        assert int(d["count"]) == self.count
        assert np.array_equal(d["stack"].cpu().numpy()[:self.count], self.stack[:self.count])


# prompts in chunks, single tokens, drafts of which some are taken back, a request that ends and
# whose pages another one takes, one that does not fit any more
STEPS = [([60, 30, 1, 0, 5], None), ([60, 0, 0, 36, 0], None), ([1, 1, 1, 1, 1], None),
         ([4, 4, 0, 4, 4], [122, 33, 2, 38, 7]), ([1, 1, 1, 1, 1], [0, 34, 3, 39, 8]),
         ([70, 1, 1, 1, 1], None), ([0, 0, 0, 0, 0], None), ([2, 90, 1, 1, 4], None)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("num,block", [(64, 1), (5, 16)])
def test_steps_of_a_server(captured, num, block):
    s = Server(num, num, block)
    graph, padding = None, 0
    for new, keep in STEPS:
        h = s.inputs(new)
        if captured and graph is None:
            s.d["new"].zero_()
            s.device_step()  # nothing to do; the library is loaded outside the capture
            torch.cuda.synchronize()
            s.d["bad"].zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = s.device_step()
            s.d["new"].copy_(dev(h["new"]))
        if captured:
            graph.replay()
        else:
            got = s.device_step()
        s.check(h, got)
        padding += int((got[0] < 0).sum())
        if keep is not None:
            s.truncate(keep)
    # nvfp4_mla_append counts every token that does not resolve, padding among them
    assert int(s.d["bad"]) == padding and int(s.d["index_bad"]) == 0
    assert int(s.d["refused"]) == 1


def test_the_stream_that_a_call_takes():
    import nvfp4_compressed_mla_gb300 as nm
    assert nm._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert nm._stream(None) == side.cuda_stream
        with torch.cuda.stream(torch.cuda.default_stream()):
            assert nm._stream(None) == torch.cuda.default_stream().cuda_stream
    assert nm._stream(side) == side.cuda_stream == nm._stream(side.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert nm._stream(None) == torch.cuda.current_stream().cuda_stream
        torch.zeros(1, device="cuda:0")
