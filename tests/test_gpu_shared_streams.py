"""GPU: the dense attention and the operators for shared pages on other streams than the current one, from
a host thread without a context, and in captured graphs that share a workspace."""
import numpy as np
import pytest
import torch

from tests import pages_cases as pc
from tests.chunk_cases import FP8, Case
from tests.gpu_cases import dev_tensor as dev
from tests.test_gpu_streams import allocated
from tests.test_gpu_thread_first_call import in_new_thread

pytestmark = pytest.mark.gpu

I32 = torch.int32


def one(v):
    return dev(np.array([v], np.int32))


def pages(seed):
    """A fork's arguments (in place), and its reference."""
    rng = np.random.default_rng(seed)
    lens, table, shares, stack, count = pc.family(rng, 300, 16, 400, 200)
    src, dst = np.nonzero(lens > 0)[0].astype(np.int32), np.nonzero(lens == 0)[0].astype(np.int32)
    n = min(len(src), len(dst))
    src, dst = src[:n], dst[:n]
    ref = pc.fork(src, dst, lens[src], lens, table, 16, shares, stack, count)
    return n, [dev(x) for x in (src, dst, lens[src], lens, table)] + [16, dev(shares), dev(stack), one(count)], ref, stack


def test_buffers_that_calls_allocate():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(80, [900, 700], [30, 1], 128)
    args = c.device()
    want = nm.dense_mla_chunk(*args)
    got, shared = allocated(lambda s: nm.dense_mla_chunk(*args, stream=s), ((31, 128, 512), torch.bfloat16),
                            ((31, 128), torch.float32))
    assert not shared and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    n, d, ref, stack = pages(81)
    got, shared = allocated(lambda s: nm.nvfp4_mla_fork(*d, stream=s), *[((n,), I32)] * 3)
    assert not shared
    for t, name in zip(got, ("shared_blocks", "copy_src", "copy_dst")):
        assert np.array_equal(t.cpu().numpy(), ref[name])
    want = pc.compact(ref["seq_lens"], ref["table"], 16, ref["shares"], stack, ref["free_count"], 90)
    got, shared = allocated(lambda s: nm.nvfp4_mla_compact(d[3], d[4], 16, *d[6:], 90, stream=s), *[((90,), I32)] * 2)
    assert not shared
    for t, name in zip(got, ("copy_src", "copy_dst")):
        assert np.array_equal(t.cpu().numpy(), want[name])


def test_workspace_is_the_launch_streams():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(82, [900], [3], 16)
    args = c.device()
    need = nm.dense_mla_chunk_workspace_size(3, 16, 1)
    out = torch.empty((3, 16, 512), dtype=torch.bfloat16, device="cuda:0")
    lse = torch.empty((3, 16), device="cuda:0")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    nm.dense_mla_chunk(*args, out=out, lse=lse, stream=side)
    mine = [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]
    torch.cuda.synchronize()
    assert sum(s["total_size"] for s in mine) >= need
    c.check(out, lse)


def test_first_calls_of_a_host_thread():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(83, [900], [3], 16, FP8)
    args, ref = c.device(), c.reference()
    out = torch.empty((3, 16, 512), dtype=torch.bfloat16, device="cuda:0")
    lse = torch.empty((3, 16), device="cuda:0")
    ws = torch.empty(nm.dense_mla_chunk_workspace_size(3, 16, 1), dtype=torch.uint8, device="cuda:0")
    in_new_thread(lambda: nm.dense_mla_chunk(*args, out=out, lse=lse, workspace=ws, stream=0))
    c.check(out, lse, ref=ref)
    n, d, ref, stack = pages(84)
    outs = [torch.empty(n, dtype=I32, device="cuda:0") for _ in range(3)]
    in_new_thread(lambda: nm.nvfp4_mla_fork(*d, shared_blocks=outs[0], copy_src=outs[1], copy_dst=outs[2], stream=0))
    for t, name in zip(outs, ("shared_blocks", "copy_src", "copy_dst")):
        assert np.array_equal(t.cpu().numpy(), ref[name])
    keep = (ref["seq_lens"] // 2).astype(np.int32)
    want = pc.release(keep, ref["seq_lens"], ref["table"], 16, ref["shares"], stack, ref["free_count"])
    keep = dev(keep)
    in_new_thread(lambda: nm.nvfp4_mla_release(keep, d[3], d[4], 16, *d[6:], stream=0))
    assert np.array_equal(d[6].cpu().numpy(), want["shares"]) and int(d[8]) == want["free_count"]
    ws = torch.empty(nm.nvfp4_mla_compact_workspace_size(d[6].numel()), dtype=torch.uint8, device="cuda:0")
    moves = [torch.empty(90, dtype=I32, device="cuda:0") for _ in range(2)]
    in_new_thread(lambda: nm.nvfp4_mla_compact(d[3], d[4], 16, *d[6:], 90, copy_src=moves[0], copy_dst=moves[1],
                                               workspace=ws, stream=0))
    com = pc.compact(want["seq_lens"], ref["table"], 16, want["shares"], want["free_pages"], want["free_count"], 90)
    assert np.array_equal(moves[0].cpu().numpy(), com["copy_src"])
    pool = torch.arange(d[6].numel(), dtype=I32, device="cuda:0").view(-1, 1).expand(-1, 4).contiguous()
    before = pool.cpu().numpy()
    in_new_thread(lambda: nm.nvfp4_mla_copy_pages(*moves, pool.view(-1), len(pool), 16, 16, stream=0))
    for a, b in zip(com["copy_src"], com["copy_dst"]):
        if a >= 0:
            before[b] = before[a]
    assert np.array_equal(pool.cpu().numpy(), before)


def test_two_captured_graphs_share_a_workspace():
    import nvfp4_compressed_mla_gb300 as nm
    cases = [Case(85, [5000], [1], 128), Case(86, [300, 60], [80, 9], 32)]
    size = max(nm.dense_mla_chunk_workspace_size(c.num_q, c.H, c.S) for c in cases)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda:0")
    graphs, outs, refs = [], [], [c.reference() for c in cases]
    for c in cases:
        args = c.device()
        nm.dense_mla_chunk(*args, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((args, nm.dense_mla_chunk(*args, workspace=ws)))
        graphs.append(graph)
    for order in ((0, 1, 1, 0), (1, 0, 1, 0)):
        for _, got in outs:
            got[0].fill_(3), got[1].fill_(3)
        ws.fill_(0xFF)  # nothing is kept there from one call for the next
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for c, (_, got), ref in zip(cases, outs, refs):
            c.check(*got, ref=ref)


def test_results_dropped_inside_a_capture():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(87, [700, 90], [5, 2], 16)
    args, ref = c.device(), c.reference()
    side = torch.cuda.Stream()
    nm.dense_mla_chunk(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        first = nm.dense_mla_chunk(*args, stream=side)
        nm.dense_mla_chunk(*args, stream=side)
        second = nm.dense_mla_chunk(*args, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        first[0].fill_(-9), second[0].fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        c.check(*first, ref=ref)
        c.check(*second, ref=ref)
