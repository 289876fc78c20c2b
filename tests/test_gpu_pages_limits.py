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


def test_rows_of_as_many_pages_as_an_int_holds():
    """Pages of one token, so that a row of the table is 8.6 GB. Sequence 0 fills it, without pages but for
    a few at its ends and in the middle."""
    import nvfp4_compressed_mla_gb300 as nm
    table = torch.full((2, MOST), -1, dtype=torch.int32, device="cuda:0")
    at = torch.tensor([0, 1, 1023, 1024, 2 ** 30, MOST - 1024, MOST - 1023, MOST - 2, MOST - 1], device="cuda:0")
    held = ints(40, 41, 42, 43, 44, 45, 46, 47, 48)
    table[0, at] = held
    lens, shares = ints(MOST, 0), torch.zeros(60, dtype=torch.int32, device="cuda:0")
    stack, count = torch.arange(39, -1, -1, dtype=torch.int32, device="cuda:0"), ints(40)

    def entries(row):
        return int((table[row] != -1).sum())

    shared, src, dst = nm.nvfp4_mla_fork(ints(0), ints(1), ints(MOST), lens, table, 1, shares, stack, count)
    assert [int(shared), int(src), int(dst), int(count)] == [MOST, -1, -1, 40]
    assert lens.tolist() == [MOST, MOST] and entries(1) == 9
    assert torch.equal(table[1, at], held)
    assert shares[40:49].tolist() == [1] * 9 and int(shares.sum()) == 9

    end = ints(-7)
    src, dst = nm.nvfp4_mla_compact(lens, table, 1, shares, stack, count, 4, pages_end=end)
    assert src.tolist() == [48, 47, 46, 45] and dst.tolist() == [0, 1, 2, 3]
    held = ints(40, 41, 42, 43, 44, 3, 2, 1, 0)
    assert torch.equal(table[0, at], held) and torch.equal(table[1, at], held)
    assert entries(0) == entries(1) == 9 and int(end) == 45 and int(count) == 40
    assert stack.tolist() == list(range(48, 44, -1)) + list(range(39, 3, -1))
    assert shares[:4].tolist() + shares[40:45].tolist() == [1] * 9 and int(shares.sum()) == 9

    stack = torch.cat([stack, stack.new_zeros(20)])
    nm.nvfp4_mla_release(ints(MOST, 0), lens, table, 1, shares, stack, count)
    assert lens.tolist() == [MOST, 0] and int(count) == 40 and not shares.any()
    nm.nvfp4_mla_release(ints(1, 0), lens, table, 1, shares, stack, count)
    assert lens.tolist() == [1, 0] and int(count) == 48
    assert stack[40:48].tolist() == [0, 1, 2, 3, 44, 43, 42, 41]
