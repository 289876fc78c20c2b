"""GPU: numbers of sequences at which a kernel's shared memory reaches the 48 KB that it has without asking,
its static part included, and the largest allowed."""
import numpy as np
import pytest
import torch

from tests import pages_cases as pc, step_cases as sc
from tests.gpu_cases import dev_tensor as dev

pytestmark = pytest.mark.gpu

PAGE, WIDTH, BLOCKS = 16, 4, 900


def state(seqs):
    rng = np.random.default_rng(seqs)
    lens = np.where(rng.random(seqs) < 200 / seqs, rng.integers(1, PAGE * WIDTH, seqs), 0).astype(np.int32)
    table, free, _ = sc.random_tables(rng, lens, PAGE, BLOCKS)
    new = np.where(rng.random(seqs) < 100 / seqs, 1, 0).astype(np.int32)
    return rng, lens, table, free, new


def on_device(*arrays):
    return [dev(np.asarray(a, np.int32)) for a in arrays]


# 12 bytes a sequence of the plan, 4 of a truncation and of a fork, 12 and 16 KB of a release
@pytest.mark.parametrize("seqs", [2710, 2730, 4070, 4080, 4096, 12225, 12288, 16384])
def test_operators(seqs):
    import nvfp4_compressed_mla_gb300 as nm
    rng, lens, table, free, new = state(seqs)
    keep = np.where(rng.random(seqs) < 0.5, lens // 2, lens).astype(np.int32)

    for rows in (200, 9000):  # one CTA, and a cluster
        d = on_device(new, lens, table, free, [len(free)])
        got = nm.nvfp4_mla_plan_step(d[0], d[1], d[2], PAGE, d[3], d[4], rows)
        ref = sc.plan_step(new, lens, table, PAGE, free, len(free), rows)
        for t, name in zip(got, ("seq_ids", "positions", "slots", "cu_tokens")):
            assert np.array_equal(t.cpu().numpy(), ref[name]), name
        assert np.array_equal(d[1].cpu().numpy(), ref["seq_lens"])

    d = on_device(keep, lens, table, np.concatenate([free, np.zeros(seqs, np.int32)]), [len(free)])
    nm.nvfp4_mla_truncate(d[0], d[1], d[2], PAGE, d[3], d[4])
    ref = sc.truncate(keep, lens, table, PAGE, np.concatenate([free, np.zeros(seqs, np.int32)]), len(free))
    assert np.array_equal(d[1].cpu().numpy(), ref["seq_lens"]) and int(d[4]) == ref["free_count"]

    blocks = int(max(table.max(), free.max())) + 1
    shares = np.zeros(blocks, np.int32)
    live, idle = np.nonzero(lens)[0], np.nonzero(lens == 0)[0]
    src, dst = rng.choice(live, 40), rng.choice(idle, 40, replace=False)
    d = on_device(src, dst, lens[src], lens, table, shares, free, [len(free)])
    got = nm.nvfp4_mla_fork(d[0], d[1], d[2], d[3], d[4], PAGE, d[5], d[6], d[7])
    ref = pc.fork(src, dst, lens[src], lens, table, PAGE, shares, free, len(free))
    for t, name in zip(got, ("shared_blocks", "copy_src", "copy_dst")):
        assert np.array_equal(t.cpu().numpy(), ref[name]), name
    assert np.array_equal(d[4].cpu().numpy(), ref["table"]) and np.array_equal(d[5].cpu().numpy(), ref["shares"])

    keep = np.where(rng.random(seqs) < 0.5, 0, ref["seq_lens"]).astype(np.int32)
    stack = np.concatenate([free, np.zeros(seqs, np.int32)])
    d = on_device(keep, ref["seq_lens"], ref["table"], ref["shares"], stack, [ref["free_count"]])
    nm.nvfp4_mla_release(d[0], d[1], d[2], PAGE, d[3], d[4], d[5])
    ref = pc.release(keep, ref["seq_lens"], ref["table"], PAGE, ref["shares"], stack, ref["free_count"])
    assert np.array_equal(d[3].cpu().numpy(), ref["shares"]) and int(d[5]) == ref["free_count"]
    assert np.array_equal(d[4].cpu().numpy()[:ref["free_count"]], ref["free_pages"][:ref["free_count"]])
    torch.cuda.synchronize()
