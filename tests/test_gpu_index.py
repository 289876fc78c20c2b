"""GPU: rows of the index-key cache. Codes and scales are decided exactly: bytes have to be equal,
and so have the values read back (a code times a scale has at most 6 significant bits)."""
import numpy as np
import pytest
import torch

from tests import step_cases as sc
from workloads.gen import bf16_from_f32, f32_from_bf16

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.view(dtype) if dtype is not None else t).to("cuda:0")


def check(keys, seq, pos, table, page, num_blocks, stride):
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(9)
    pool = rng.integers(0, 256, num_blocks * stride, dtype=np.uint8)
    got = dev(pool)
    bad = torch.zeros(2, dtype=torch.int32, device="cuda:0")
    args = (dev(seq), dev(pos), dev(table), page)
    nm.nvfp4_mla_index_append(dev(keys, torch.bfloat16), *args, got, num_blocks, stride,
                              invalid_count=bad[:1])
    back = nm.nvfp4_mla_index_read(*args, got, num_blocks, stride, invalid_count=bad[1:])
    torch.cuda.synchronize()
    want_bad = sc.index_append(keys, seq, pos, table, page, pool, num_blocks, stride)
    assert np.array_equal(got.cpu().numpy(), pool)
    assert bad.tolist() == [want_bad, want_bad]
    back = back.double().cpu().numpy()
    for t in range(len(seq)):
        at = sc.resolve(int(seq[t]), int(pos[t]), table, page, num_blocks)
        ref = np.zeros(128) if at is None else sc.read_row(pool, stride, page, *at)
        assert np.array_equal(back[t], ref), t
    return want_bad


@pytest.mark.parametrize("n,page,pad", [(1, 64, 0), (31, 64, 16), (33, 48, 0), (66, 2, 48),
                                        (700, 128, 4096), (129, 1024, 16)])
def test_rows_of_a_scattered_pool(n, page, pad):
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 400, 9)
    table, _, num_blocks = sc.random_tables(rng, lens, page, 2)
    every = [(s, p) for s in range(9) for p in range(lens[s])]
    pick = rng.permutation(len(every))[:n]
    seq = np.array([every[i][0] for i in pick], np.int32)
    pos = np.array([every[i][1] for i in pick], np.int32)
    keys = bf16_from_f32(rng.standard_normal((len(pick), 128)) * 10 ** rng.uniform(-3, 3, (len(pick), 1)))
    assert check(keys, seq, pos, table, page, num_blocks, page * sc.ROW + pad) == 0


def test_every_bf16_magnitude_and_edge_of_the_grid():
    rng = np.random.default_rng(0)
    bits = np.arange(0x7F80, dtype=np.uint16)  # every finite non-negative bf16
    rows = [np.resize(bits | (0x8000 if i % 2 else 0), (255, 128)) for i in range(2)]
    # midpoints of the code grid times exact scales, and their neighbours
    scale = 2.0 ** rng.integers(-9, 9, (64, 8, 1)) * (1 + rng.integers(0, 8, (64, 8, 1)) / 8)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = (np.tile(mids, 2) * scale).reshape(64, 128)
    near = [bf16_from_f32(x), bf16_from_f32(x) + 1, bf16_from_f32(x) - 1]
    keys = np.concatenate(rows + near + [np.zeros((3, 128), np.uint16), np.full((2, 128), 0x8000, np.uint16)])
    n = len(keys)
    assert np.isfinite(f32_from_bf16(keys)).all()
    table = np.arange(-(-n // 64), dtype=np.int32)[None]
    check(keys.astype(np.uint16), np.zeros(n, np.int32), np.arange(n, dtype=np.int32), table, 64,
          table.shape[1], 64 * sc.ROW)


def test_tokens_that_do_not_resolve_are_skipped_and_counted():
    rng = np.random.default_rng(4)
    table = np.array([[2, -1, 5], [7, 0, 99]], np.int32)
    seq = np.array([0, 0, 0, 0, 1, 1, -1, 2, -5, 1, -1], np.int32)
    pos = np.array([0, 16, 47, 48, -1, 40, -1, 0, 3, 17, 5], np.int32)
    keys = bf16_from_f32(rng.standard_normal((len(seq), 128)))
    # bad: no page, past the table, negative, page out of the pool, sequences 2 and -5
    assert check(keys, seq, pos, table, 16, 8, 16 * sc.ROW) == 6


def test_a_pool_past_4_gib():
    import nvfp4_compressed_mla_gb300 as nm
    page, stride, num_blocks = 64, 1 << 20, 4500
    pool = torch.zeros(num_blocks * stride, dtype=torch.uint8, device="cuda:0")
    keys = torch.randn(64, 128, device="cuda:0").bfloat16()
    table = torch.tensor([[num_blocks - 1, 0]], dtype=torch.int32, device="cuda:0")
    seq = torch.zeros(64, dtype=torch.int32, device="cuda:0")
    pos = torch.arange(64, dtype=torch.int32, device="cuda:0")
    nm.nvfp4_mla_index_append(keys, seq, pos, table, page, pool, num_blocks, stride)
    last = pool[(num_blocks - 1) * stride:][:page * sc.ROW].cpu().numpy()
    ref = np.zeros(page * sc.ROW, np.uint8)
    sc.index_append(keys.cpu().view(torch.int16).numpy().view(np.uint16), np.zeros(64, np.int32),
                    np.arange(64, dtype=np.int32), np.array([[0]], np.int32), page, ref, 1,
                    page * sc.ROW)
    assert np.array_equal(last, ref)
    assert int(pool[:(num_blocks - 1) * stride].count_nonzero()) == 0
