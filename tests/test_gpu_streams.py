"""GPU: buffers that a call allocates for work on another stream than the current one. Memory that
the current stream has given up may still be read by its pending work, so it is not the call's."""
import numpy as np
import pytest
import torch

from tests import step_cases as sc
from tests.test_gpu_select import Case, dev
from tests.test_gpu_thread_first_call import LATENT, decode_args

pytestmark = pytest.mark.gpu

I32 = torch.int32


def allocated(call, *shapes):
    """Whether call(stream) returns memory that the current stream gave up just before: blocks of
    the results' own sizes, all work done."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    given_up = [torch.empty(s, dtype=t, device="cuda:0") for s, t in shapes]
    spans = [(x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()) for x in given_up]
    del given_up
    got = call(side)
    torch.cuda.synchronize()
    got = got if isinstance(got, tuple) else (got,)
    return got, any(a <= t.data_ptr() < b for t in got for a, b in spans)


def test_select():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(70, [700, 1300], 400, 16)
    args = c.device()
    (out,), shared = allocated(lambda s: nm.sparse_mla_select(*args, 64, stream=s),
                               ((800, 64), I32))
    assert not shared
    assert np.array_equal(out.cpu().numpy(), c.ref(64))


def test_plan_step():
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(71)
    lens = rng.integers(0, 300, 70).astype(np.int32)
    new = np.full(70, 900, np.int32)
    table, free, _ = sc.random_tables(rng, lens, 16, 5000, 90)
    ref = sc.plan_step(new, lens, table, 16, free, len(free), 70000)
    d = [dev(x) for x in (new, lens, table, free, np.array([len(free)], np.int32))]
    got, shared = allocated(
        lambda s: nm.nvfp4_mla_plan_step(d[0], d[1], d[2], 16, d[3], d[4], 70000, stream=s),
        (70000, I32), (70000, I32), (70000, torch.int64), (71, I32))
    assert not shared
    for t, name in zip(got, ("seq_ids", "positions", "slots", "cu_tokens")):
        assert np.array_equal(t.cpu().numpy(), ref[name])


def test_index_read():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(72, [700, 1300], 400, 1)
    a = c.device()
    (keys,), shared = allocated(
        lambda s: nm.nvfp4_mla_index_read(a[2], a[3], a[4], 64, a[6], c.blocks, c.stride, stream=s),
        ((800, 128), torch.bfloat16))
    assert not shared
    assert bool((keys != 0).any(1).all())


@pytest.mark.parametrize("splits", [1, 2])
def test_decode(splits):
    # with splits, the workspace too is the launch stream's: it is given up before the work ends
    import nvfp4_compressed_mla_gb300 as nm
    args = decode_args(128)
    want = nm.sparse_mla_decode(*args, nm.ROW_NVFP4_352, 0.05, num_splits=splits)
    spare = ((1, 128, 512), torch.bfloat16), ((1, 128), torch.float32)
    got, shared = allocated(
        lambda s: nm.sparse_mla_decode(*args, nm.ROW_NVFP4_352, 0.05, num_splits=splits, stream=s),
        *spare)
    assert not shared
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_workspace():
    import nvfp4_compressed_mla_gb300 as nm
    args = decode_args(128)
    need = nm.sparse_mla_decode_workspace_size(1, 128, 256, 2)
    out = torch.empty((1, 128, 512), dtype=torch.bfloat16, device="cuda:0")
    lse = torch.empty((1, 128), device="cuda:0")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    nm.sparse_mla_decode(*args, nm.ROW_NVFP4_352, 0.05, out=out, lse=lse, num_splits=2, stream=side)
    # all segments that the call brought belong to the stream it ran on
    mine = [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]
    torch.cuda.synchronize()
    assert sum(s["total_size"] for s in mine) >= need


def test_merge_and_stage():
    import nvfp4_compressed_mla_gb300 as nm
    args = decode_args()
    parts = torch.randn((2, 64, 16, 512), device="cuda:0"), torch.randn((2, 64, 16), device="cuda:0")
    want = nm.sparse_mla_merge_states(*parts)
    got, shared = allocated(lambda s: nm.sparse_mla_merge_states(*parts, stream=s),
                            ((64, 16, 512), torch.bfloat16), ((64, 16), torch.float32))
    assert not shared
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _, _, seq, top, table, lens = args[:6]
    want = nm.nvfp4_mla_stage_fp8(seq, top, table, lens, 64, args[7], 4, LATENT)
    got, shared = allocated(
        lambda s: nm.nvfp4_mla_stage_fp8(seq, top, table, lens, 64, args[7], 4, LATENT, stream=s),
        (256 * 576, torch.uint8), ((1, 256), I32))
    assert not shared
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_result_that_the_current_stream_still_reads_is_not_handed_out_again():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(74, [700, 1300], 400, 16)
    args, ref = c.device(), c.ref(64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = nm.sparse_mla_select(*args, 64, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(400_000_000)  # about 0.2 s, behind which the result is read
    kept = out.clone()
    at = out.data_ptr()
    del out
    again = nm.sparse_mla_select(*args, 64, stream=side)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(again.cpu().numpy(), ref)


@pytest.mark.parametrize("handle", [False, True])
def test_the_default_stream_given_while_another_is_current(handle):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(75, [700, 1300], 400, 16)
    args, ref = c.device(), c.ref(64)
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = nm.sparse_mla_select(*args, 64, stream=0 if handle else default)
    torch.cuda.synchronize()
    at = out.data_ptr()
    mine = [s for s in torch.cuda.memory_snapshot()
            if s["address"] <= at < s["address"] + s["total_size"]]
    assert [s["stream"] for s in mine] == [0]
    assert np.array_equal(out.cpu().numpy(), ref)


def test_buffers_of_another_stream_in_a_captured_graph():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(76, [700, 1300], 2, 16)
    args, ref = c.device(), c.ref(64)
    side = torch.cuda.Stream()
    nm.sparse_mla_select(*args, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        first = nm.sparse_mla_select(*args, 64, stream=side)
        nm.sparse_mla_select(*args, 64, stream=side)  # dropped inside the capture
        second = nm.sparse_mla_select(*args, 64, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        first.fill_(-9), second.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(first.cpu().numpy(), ref) and np.array_equal(second.cpu().numpy(), ref)
