"""GPU: the operators for shared pages at the largest sizes that their arguments can have. Expected
values are written out: a plain form would walk billions of entries."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1  # of an int32


@pytest.fixture(autouse=True)
def memory_goes_back():
    yield
    torch.cuda.empty_cache()  # tens of gigabytes


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda:0")


@pytest.mark.parametrize("blocks", [60, 5000])  # one CTA ranks the pages, and a cluster
def test_lists_of_as_many_moves_as_an_int_holds(blocks):
    """"All pages" as the largest number there is: two lists of 8.6 GB, -1 behind the last move."""
    import nvfp4_compressed_mla_gb300 as nm
    top = blocks - 1
    table = ints(top, top - 1, 3, -1).view(1, 4)
    lens, shares, count = ints(20), torch.zeros(blocks, dtype=torch.int32, device="cuda:0"), ints(4)
    shares[top] = 5
    stack = ints(0, 1, 4, top - 2, -7, -7)
    src, dst, end = (torch.full((n,), -7, dtype=torch.int32, device="cuda:0") for n in (MOST, MOST, 1))
    nm.nvfp4_mla_compact(lens, table, 7, shares, stack, count, MOST, copy_src=src, copy_dst=dst, pages_end=end)
    assert src[:3].tolist() == [top, top - 1, -1] and dst[:3].tolist() == [0, 1, -1]
    for t in (src, dst):
        assert all(bool((part == -1).all()) for part in t[2:].split(1 << 28))
    assert table.tolist() == [[0, 1, 3, -1]] and int(end) == 4
    assert int(count) == 4 and stack.tolist() == [top, top - 1, top - 2, 4, -7, -7]
    assert int(shares[0]) == 5 and int(shares.sum()) == 5
