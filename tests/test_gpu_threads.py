"""GPU: two host threads that call the same operator with other sizes at the same time. A kernel's
limit of shared memory belongs to the process: one thread's call may not lower the other's."""
import sys
import threading

import numpy as np
import pytest
import torch

from tests import step_cases as sc
from tests.test_gpu_select import Case, dev

pytestmark = pytest.mark.gpu

CALLS = 8000


def together(*calls):
    """Each of `calls`, which returns a status, CALLS times in a thread of its own."""
    bad, start = [], threading.Barrier(len(calls))

    def loop(call):
        start.wait()
        for i in range(CALLS):
            status = call()
            if status != 0:
                bad.append(status)
            if i % 100 == 99:
                torch.cuda.synchronize()

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    torch.cuda.synchronize()
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not bad, (len(bad), set(bad))


def lib():
    from nvfp4_compressed_mla_gb300 import _native
    return _native.load()


def ptr(*tensors):
    return [t.data_ptr() for t in tensors]


def test_select_from_two_threads():
    # other sizes of both kernels: runs of one and of four query tokens, and rows that need
    # nearly all and next to none of the shared memory that the choice can have
    import nvfp4_compressed_mla_gb300 as nm
    f, calls, made = lib().sparse_mla_select, [], []
    for c, width in ((Case(60, [700], 1, 64), 400), (Case(61, [500], 8, 64), 8)):
        ref = c.ref(64)
        wide = np.full((1, width), -1, np.int32)
        wide[:, :c.table.shape[1]] = c.table
        n = len(c.seq)
        q, w, seq, pos, _, _, pool = c.device()[:7]
        table, stream = dev(wide), torch.cuda.Stream()
        out = torch.empty((n, 64), dtype=torch.int32, device="cuda:0")
        size = nm.sparse_mla_select_workspace_size(n, 64, width, 64)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda:0")
        args = [*ptr(q, w, seq, pos), n, 64, *ptr(table), 1, width, 64, *ptr(pool), c.blocks,
                c.stride, 1, 64, 0, 0, *ptr(out, ws), size, stream.cuda_stream]
        calls.append(lambda args=args: f(*args))
        made.append((out, ref, (q, w, seq, pos, table, pool, ws, stream)))
    together(*calls)
    for out, ref, _ in made:
        assert np.array_equal(out.cpu().numpy(), ref)


def test_plan_step_from_two_threads():
    f, calls, made = lib().nvfp4_mla_plan_step, [], []
    for seqs in (16384, 4200):
        lens, new = np.full(seqs, 3, np.int32), np.zeros(seqs, np.int32)
        new[seqs - 1] = 5
        table, free = np.full((seqs, 1), 9, np.int32), np.array([4], np.int32)
        ref = sc.plan_step(new, lens, table, 16, free, 1, 8)
        d = [dev(x) for x in (new, lens, table, free, np.array([1], np.int32))]
        o = [torch.empty_like(d[1]), torch.empty_like(d[4])]
        r = [torch.empty(8, dtype=t, device="cuda:0")
             for t in (torch.int32, torch.int32, torch.int64)]
        stream = torch.cuda.Stream()
        args = [*ptr(d[0], d[1]), seqs, *ptr(d[2]), 1, 16, *ptr(d[3]), 1, *ptr(d[4]), 8, *ptr(*o),
                *ptr(*r), None, None, stream.cuda_stream]
        calls.append(lambda args=args: f(*args))
        made.append((ref, d, o, r, stream))
    together(*calls)
    for ref, _, o, r, _ in made:
        assert np.array_equal(o[0].cpu().numpy(), ref["seq_lens"])
        assert np.array_equal(r[2].cpu().numpy(), ref["slots"])


def test_truncate_from_two_threads():
    f, calls, made = lib().nvfp4_mla_truncate, [], []
    for seqs in (16384, 13000):
        lens = np.full(seqs, 30, np.int32)
        keep = lens.copy()
        keep[7], keep[seqs - 1] = 16, 0
        table, stack = np.arange(2 * seqs, dtype=np.int32).reshape(seqs, 2), np.zeros(9, np.int32)
        ref = sc.truncate(keep, lens, table, 16, stack, 2)
        d = [dev(x) for x in (keep, lens, table, stack, np.array([2], np.int32))]
        o = [torch.empty_like(d[1]), torch.empty_like(d[4])]
        stream = torch.cuda.Stream()
        args = [*ptr(d[0], d[1]), seqs, *ptr(d[2]), 2, 16, *ptr(d[3]), 9, *ptr(d[4]), *ptr(*o),
                None, stream.cuda_stream]
        calls.append(lambda args=args: f(*args))
        made.append((ref, d, o, stream))
    together(*calls)
    for ref, d, o, _ in made:
        assert np.array_equal(o[0].cpu().numpy(), ref["seq_lens"])
        assert int(o[1]) == ref["free_count"]
        assert np.array_equal(d[3].cpu().numpy(), ref["free_pages"])
