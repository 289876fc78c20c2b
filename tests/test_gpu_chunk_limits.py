"""GPU: the dense attention of a step where keys are missing."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import FP8, NVFP4, Case

pytestmark = pytest.mark.gpu

I32 = torch.int32


def zero():
    return torch.zeros(1, dtype=I32, device="cuda:0")


def unresolved(case):
    """Positions of the sequences with new tokens whose page does not resolve."""
    n = 0
    for s in np.nonzero(case.new)[0]:
        pages = case.table[s, np.arange(case.lens[s]) // case.page]
        n += int(((pages < 0) | (pages >= case.blocks)).sum())
    return n


@pytest.mark.parametrize("page", [1, 3, 16, 32, 48, 64, 100, 128, 192])
@pytest.mark.parametrize("heads,fmt", [(16, NVFP4), (16, FP8), (128, NVFP4), (128, FP8)])
def test_missing_pages_of_every_size(page, heads, fmt):
    """Holes of a key, of parts of a piece of 64 keys and of whole pieces, in both halves of key tiles, one
    tile after the other."""
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(40 + page, [700, 333, 3 * 64, 1500], [30, 5, 1, 0], heads, fmt, page=page)
    rng = np.random.default_rng(page)
    live = c.table >= 0
    holes = live & (rng.random(c.table.shape) < 0.3)
    holes[0, 0], holes[1, live[1].sum() - 1] = True, True
    c.table[holes] = rng.choice(np.array([-1, c.blocks, -2 ** 31, 2 ** 31 - 1], np.int32), holes.sum())
    bad = zero()
    tokens = set(range(0, 30, 7)) | {29, 30, 32, 34, 35}
    out, lse = nm.dense_mla_chunk(*c.device(), invalid_count=bad)
    c.check(out, lse, tokens=tokens)
    assert int(bad) == unresolved(c)


@pytest.mark.parametrize("page", [1, 48, 64])
@pytest.mark.parametrize("fmt", [NVFP4, FP8])
def test_missing_pages_of_a_context_that_many_clusters_share(page, fmt):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(50 + page, [7000], [3], 128, fmt, page=page)
    rng = np.random.default_rng(page)
    holes = rng.random(c.table.shape) < 0.5
    holes[0, :4000 // page] |= rng.random(4000 // page) < 0.9
    c.table[holes] = -1
    for _ in range(3):  # the words of an earlier call must not matter
        out, lse = nm.dense_mla_chunk(*c.device(), out_fp32=True)
        c.check(out, lse, True)
