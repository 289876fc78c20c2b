"""Host-side checks of the operators for shared pages, and of their plain forms (no GPU)."""
import numpy as np
import pytest

from tests import pages_cases as pc

FAKE = 0x10000  # 16-byte aligned non-null address; never dereferenced on these paths
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    from nvfp4_compressed_mla_gb300 import _native
    return _native.load()


def _fork(lib, **kw):
    a = dict(src=FAKE, dst=FAKE, want=FAKE, n=3, seq_lens=FAKE, num_seqs=4, block_table=FAKE, max_blocks=10,
             page_size=64, shares=FAKE, num_blocks=50, free_pages=FAKE, free_capacity=10, free_count=FAKE,
             seq_lens_out=FAKE, shares_out=FAKE, free_count_out=FAKE, shared=FAKE, copy_src=FAKE,
             copy_dst=FAKE, refused=None, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_fork(*a.values())


def _release(lib, **kw):
    a = dict(keep=FAKE, seq_lens=FAKE, num_seqs=4, block_table=FAKE, max_blocks=10, page_size=64,
             shares=FAKE, num_blocks=50, free_pages=FAKE, free_capacity=10, free_count=FAKE,
             seq_lens_out=FAKE, shares_out=FAKE, free_count_out=FAKE, dropped=None, refused=None,
             stream=None)
    a.update(kw)
    return lib.nvfp4_mla_release(*a.values())


def _compact(lib, **kw):
    a = dict(seq_lens=FAKE, num_seqs=4, block_table=FAKE, max_blocks=10, page_size=64, shares=FAKE,
             num_blocks=50, free_pages=FAKE, free_capacity=10, free_count=FAKE, max_moves=5,
             table_out=FAKE, shares_out=FAKE, free_pages_out=FAKE, free_count_out=FAKE, copy_src=FAKE,
             copy_dst=FAKE, end=None, ws=FAKE, ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_compact(*a.values())


def _copy(lib, **kw):
    a = dict(copy_src=FAKE, copy_dst=FAKE, n=3, cache=FAKE, num_blocks=50, stride=4096, page_bytes=4096,
             invalid=None, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_copy_pages(*a.values())


COMMON = [
    (dict(num_seqs=0), SHAPE), (dict(num_seqs=16385), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=(1 << 20) + 1), SHAPE),
    (dict(max_blocks=1 << 25, page_size=64), SHAPE), (dict(free_capacity=-1), SHAPE),
    (dict(num_blocks=0), SHAPE), (dict(seq_lens=None), NULL), (dict(block_table=None), NULL),
    (dict(free_pages=None), NULL), (dict(free_count=None), NULL), (dict(shares=None), NULL),
    (dict(shares_out=None), NULL), (dict(free_count_out=None), NULL)]


@pytest.mark.parametrize("call", [_fork, _release, _compact])
@pytest.mark.parametrize("kw,status", COMMON)
def test_common_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("call,kw,status", [
    (_fork, dict(n=-1), SHAPE), (_fork, dict(n=16385), SHAPE), (_fork, dict(src=None), NULL),
    (_fork, dict(dst=None), NULL), (_fork, dict(want=None), NULL), (_fork, dict(shared=None), NULL),
    (_fork, dict(copy_src=None), NULL), (_fork, dict(copy_dst=None), NULL),
    (_fork, dict(seq_lens_out=None), NULL), (_release, dict(keep=None), NULL),
    (_release, dict(seq_lens_out=None), NULL), (_compact, dict(max_moves=-1), SHAPE),
    (_compact, dict(table_out=None), NULL), (_compact, dict(free_pages_out=None), NULL),
    (_compact, dict(copy_src=None), NULL), (_compact, dict(copy_dst=None), NULL),
    (_compact, dict(ws=None), WORKSPACE), (_compact, dict(ws_bytes=100), WORKSPACE),
    (_compact, dict(ws=FAKE + 8), ALIGN), (_copy, dict(n=-1), SHAPE), (_copy, dict(copy_src=None), NULL),
    (_copy, dict(copy_dst=None), NULL), (_copy, dict(cache=None), NULL), (_copy, dict(num_blocks=0), SHAPE),
    (_copy, dict(num_blocks=1 << 31), SHAPE), (_copy, dict(page_bytes=0), SHAPE),
    (_copy, dict(page_bytes=4112), SHAPE), (_copy, dict(page_bytes=4088), ALIGN),
    (_copy, dict(stride=4100), ALIGN), (_copy, dict(cache=FAKE + 8), ALIGN),
    (_copy, dict(stride=1 << 62), SHAPE)])
def test_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_sizes_and_nothing_to_copy(lib):
    assert _copy(lib, n=0, copy_src=None) == 0
    size = lib.nvfp4_mla_compact_workspace_size
    assert size(0) == size(-1) == (1 << 64) - 1
    assert 36 <= size(1) <= 128 and 2 * 128 + 4000 <= size(1000) <= 8000
    assert size(2 ** 31 - 1) > 2 ** 33


def test_valid_arguments_without_gpu_report_device(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_fork, _release, _compact, _copy):
        assert call(lib) in (4, 9)


def test_plain_forms_keep_a_pool_whole():
    """Forks, releases and compactions in turn: every page is free or held, as its shares say."""
    rng = np.random.default_rng(3)
    lens, table, shares, stack, count = pc.family(rng, 40, 8, 150, 120)
    pc.check_state(lens, table, 8, shares, stack, count)
    for _ in range(6):
        live, idle = np.nonzero(lens > 0)[0], np.nonzero(lens == 0)[0]
        src, dst = rng.choice(live, 9).astype(np.int32), rng.choice(idle, 9).astype(np.int32)
        want = (lens[src] * rng.random(9)).astype(np.int32)
        f = pc.fork(src, dst, want, lens, table, 8, shares, stack, count)
        assert f["refused"] > 0 or len(set(dst)) == 9
        pc.check_state(f["seq_lens"], f["table"], 8, f["shares"], stack, f["free_count"])
        keep = np.where(rng.random(40) < 0.4, (f["seq_lens"] * rng.random(40)).astype(np.int32), f["seq_lens"])
        r = pc.release(keep, f["seq_lens"], f["table"], 8, f["shares"], stack, f["free_count"])
        pc.check_state(r["seq_lens"], f["table"], 8, r["shares"], r["free_pages"], r["free_count"])
        c = pc.compact(r["seq_lens"], f["table"], 8, r["shares"], r["free_pages"], r["free_count"], 7)
        pc.check_state(r["seq_lens"], c["table"], 8, c["shares"], c["free_pages"], c["free_count"])
        lens, table, shares, stack, count = (r["seq_lens"], c["table"], c["shares"], c["free_pages"],
                                             c["free_count"])
