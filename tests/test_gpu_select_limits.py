"""GPU: the selection where sizes, tables and weights reach their limits, against 64-bit scores and
a stable sort. The chosen positions have to be equal."""
import numpy as np
import pytest

from tests import step_cases as sc
from tests.test_gpu_select import Case, reference_on_device
from workloads.gen import bf16_from_f32

pytestmark = pytest.mark.gpu


# Tables of more than 32768 blocks: a cluster of CTAs a query token, whose row may be short.
@pytest.mark.parametrize("lens,per_seq,num,block,sink,recent", [
    ([900], 1, 40, 1, 0, 0), ([900, 5, 2000], 3, 64, 1, 0, 0), ([900, 1300], 2, 10, 1, 3, 7),
    ([2600, 40], 1, 9, 16, 1, 2), ([2600, 3000], 19, 9, 16, 0, 0), ([900, 17000], 1, 100, 1, 0, 0),
])
def test_short_rows_of_a_wide_table(lens, per_seq, num, block, sink, recent):
    c = Case(sum(lens) + num, lens, per_seq, 16)
    ref = c.ref(num, block, sink, recent)
    wide = np.full((len(lens), 16384), -1, np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    got = c.run(num, block, sink, recent)
    bad = np.nonzero((got != ref).any(1))[0]
    assert bad.size == 0, (bad[:5], got[bad[0]][:20], ref[bad[0]][:20])


# Few different keys, so that thousands of blocks tie at the border, in rows that shared memory does
# not hold: each step reads the scores, and the marks of what is decided, from memory.
@pytest.mark.parametrize("length,keys,heads,num,block,per_seq", [
    (20000, 8, 16, 3000, 1, 1), (20000, 8, 16, 6000, 1, 2), (20011, 3, 1, 2048, 1, 1),
    (70000, 16, 64, 2048, 1, 1), (40000, 5, 8, 5001, 2, 1), (70000, 4, 16, 4000, 4, 3),
])
@pytest.mark.parametrize("sink,recent", [(0, 0), (2, 3)])
def test_ties_in_rows_that_shared_memory_does_not_hold(length, keys, heads, num, block, per_seq,
                                                       sink, recent):
    c = Case(length + keys, [length], per_seq, heads)
    rng = np.random.default_rng(keys)
    pages = c.pool.reshape(c.blocks, c.stride)
    codes, scales = pages[0, :64 * 64].reshape(64, 64), pages[0, 64 * 64:64 * 72].reshape(64, 8)
    for p in range(1, c.blocks):
        pick = rng.integers(0, keys, 64)
        pages[p, :64 * 64] = codes[pick].reshape(-1)
        pages[p, 64 * 64:64 * 72] = scales[pick].reshape(-1)
    c.check(num, block, sink, recent)


# Sums over the heads that pass the largest fp32 number, downwards, upwards or both ways: fp32
# settles nothing, and fp64 decides. At most as many blocks as the list of candidates holds; more;
# rows that are sampled first.
@pytest.mark.parametrize("size", [1e35, 2e37, 3e38])
@pytest.mark.parametrize("signs", ["negative", "positive", "both"])
@pytest.mark.parametrize("lens,per_seq,heads,num,block", [
    ([700, 900], 1, 64, 100, 1), ([700, 300], 2, 3, 100, 1), ([2600, 1300], 1, 16, 9, 16),
    ([2600, 700], 1, 33, 5, 64), ([5000], 1, 16, 300, 1), ([5000], 1, 8, 700, 4),
    ([20000], 1, 4, 512, 1),
])
def test_weights_whose_sums_pass_fp32(size, signs, lens, per_seq, heads, num, block):
    c = Case(len(signs) + heads, lens, per_seq, heads)
    rng = np.random.default_rng(heads)
    w = size * rng.uniform(0.5, 1.0, c.w.shape)
    c.w = {"negative": -w, "positive": w,
           "both": w * rng.choice([-1.0, 1.0], w.shape)}[signs].astype(np.float32)
    assert np.isfinite(c.w).all()
    c.check(num, block)


def test_equal_large_weights_choose_by_score():
    c = Case(50, [700], 1, 64)
    c.w[:] = np.float32(-2e37)
    assert not np.array_equal(c.ref(100)[0], np.arange(100))
    c.check(100)


def test_pages_that_do_not_resolve_rank_last_beside_large_weights():
    c = Case(51, [900, 900], 1, 16)
    c.w = (np.sign(c.w) * 2e37).astype(np.float32)
    c.table[0, 3], c.table[1, 2:9] = -1, 10 ** 6
    c.check(64)
    c.check(860)  # some of them have to be taken
    c.check(5, 64)


def long_case(length, per_seq, heads, keys=None):
    """One sequence of random codes, or of few different keys under weights that are powers of two:
    their scores are exact in any order of summation, and thousands of them are equal."""
    rng = np.random.default_rng(length + per_seq)
    c = Case.__new__(Case)
    c.page, c.stride, c.lens = 64, 64 * sc.ROW, np.array([length])
    c.table, _, c.blocks = sc.random_tables(rng, c.lens, 64, 2)
    rows = np.empty((c.blocks, c.stride), np.uint8)
    n = c.blocks * 64 if keys is None else keys
    codes = rng.integers(0, 256, (n, 64), dtype=np.uint8)
    scales = rng.integers(0x28, 0x48, (n, 8), dtype=np.uint8)
    pick = np.arange(n) if keys is None else rng.integers(0, keys, c.blocks * 64)
    rows[:, :64 * 64] = codes[pick].reshape(c.blocks, -1)
    rows[:, 64 * 64:] = scales[pick].reshape(c.blocks, -1)
    c.pool = rows.reshape(-1)
    c.seq = np.zeros(per_seq, np.int32)
    c.pos = np.arange(length - per_seq, length).astype(np.int32)
    c.q = bf16_from_f32(rng.standard_normal((per_seq, heads, 128)))
    c.w = (rng.standard_normal((per_seq, heads)) / np.sqrt(heads)).astype(np.float32)
    if keys is not None:
        c.w = (2.0 ** rng.integers(-2, 2, c.w.shape) * np.sign(c.w)).astype(np.float32)
    return c


# More chosen than a list has room for; rows of more blocks than the list's place has bits; several
# stored scores a block in a row that shared memory does not hold; the smaller CTAs of many tokens.
@pytest.mark.parametrize("length,per_seq,heads,num,block,keys", [
    (131072, 2, 16, 16384, 1, None), (131072, 1, 16, 65536, 1, None), (70000, 1, 4, 7000, 1, None),
    (70000, 1, 4, 7000, 1, 9), (131072, 1, 16, 16384, 4, 30),
    (1048576, 1, 4, 2048, 1, None), (1048577, 1, 4, 2048, 1, None), (1200003, 2, 4, 2048, 1, None),
    (1100003, 1, 4, 30, 64, None), (1100003, 1, 2, 400, 64, 3000), (2200001, 1, 2, 100, 128, 9000),
    (17000, 320, 8, 300, 1, 12), (17000, 320, 8, 9000, 1, None),
])
def test_long_rows_of_every_form(length, per_seq, heads, num, block, keys):
    c = long_case(length, per_seq, heads, keys)
    got, ref = c.run(num, block), reference_on_device(c, num, block)
    bad = np.nonzero((got != ref).any(1))[0]
    assert bad.size == 0, (bad.size, bad[:5], got[bad[0]][:20], ref[bad[0]][:20])
