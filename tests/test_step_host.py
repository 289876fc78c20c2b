"""Host-side checks of the step-planning, index-cache and selection entry points (no GPU)."""
import pytest

FAKE = 0x10000  # 16-byte aligned non-null address; never dereferenced on these paths
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    from nvfp4_compressed_mla_gb300 import _native
    return _native.load()


def _plan(lib, **kw):
    a = dict(new_lens=FAKE, seq_lens=FAKE, num_seqs=4, block_table=FAKE, max_blocks=10,
             page_size=64, free_pages=FAKE, free_capacity=10, free_count=FAKE, max_tokens=8,
             seq_lens_out=FAKE, free_count_out=FAKE, seq_ids=FAKE, positions=FAKE, slots=None,
             cu=None, refused=None, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_plan_step(*a.values())


def _truncate(lib, **kw):
    a = dict(keep=FAKE, seq_lens=FAKE, num_seqs=4, block_table=FAKE, max_blocks=10, page_size=64,
             free_pages=FAKE, free_capacity=10, free_count=FAKE, seq_lens_out=FAKE,
             free_count_out=FAKE, dropped=None, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_truncate(*a.values())


COMMON = [
    (dict(num_seqs=0), SHAPE), (dict(num_seqs=16385), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=(1 << 20) + 1), SHAPE),
    (dict(max_blocks=1 << 25, page_size=64), SHAPE), (dict(free_capacity=-1), SHAPE),
    (dict(seq_lens=None), NULL), (dict(block_table=None), NULL), (dict(free_pages=None), NULL),
    (dict(free_count=None), NULL), (dict(seq_lens_out=None), NULL), (dict(free_count_out=None), NULL),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(max_tokens=-1), SHAPE), (dict(new_lens=None), NULL), (dict(seq_ids=None), NULL),
    (dict(positions=None), NULL)])
def test_plan_rejects_bad_arguments(lib, kw, status):
    assert _plan(lib, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(keep=None), NULL)])
def test_truncate_rejects_bad_arguments(lib, kw, status):
    assert _truncate(lib, **kw) == status


def _append(lib, **kw):
    a = dict(keys=FAKE, seq=FAKE, pos=FAKE, n=4, bt=FAKE, num_seqs=2, max_blocks=3, page_size=64,
             cache=FAKE, num_blocks=5, stride=64 * 72, invalid=None, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_index_append(*a.values())


def _read(lib, **kw):
    a = dict(seq=FAKE, pos=FAKE, n=4, bt=FAKE, num_seqs=2, max_blocks=3, page_size=64, cache=FAKE,
             num_blocks=5, stride=64 * 72, keys=FAKE, invalid=None, stream=None)
    a.update(kw)
    return lib.nvfp4_mla_index_read(*a.values())


@pytest.mark.parametrize("call", [_append, _read])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(keys=None), NULL), (dict(seq=None), NULL), (dict(pos=None), NULL),
    (dict(bt=None), NULL), (dict(cache=None), NULL), (dict(num_seqs=0), SHAPE),
    (dict(max_blocks=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=63), SHAPE),
    (dict(num_blocks=0), SHAPE), (dict(stride=64 * 72 - 16), SHAPE), (dict(stride=64 * 72 + 8), ALIGN),
    (dict(keys=FAKE + 8), ALIGN), (dict(cache=FAKE + 4), ALIGN)])
def test_index_rejects_bad_arguments(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_index_zero_tokens_is_a_noop(lib):
    assert _append(lib, n=0, keys=None) == 0
    assert _read(lib, n=0, keys=None) == 0


def _select(lib, **kw):
    a = dict(q=FAKE, w=FAKE, seq=FAKE, pos=FAKE, num_q=2, heads=16, bt=FAKE, num_seqs=2,
             max_blocks=30, page_size=64, cache=FAKE, num_blocks=50, stride=64 * 72, block=1,
             num=100, sink=0, recent=0, out=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.sparse_mla_select(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(num_q=-1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=129), SHAPE),
    (dict(block=0), SHAPE), (dict(block=3), SHAPE), (dict(block=256), SHAPE), (dict(block=-2), SHAPE),
    (dict(num=0), SHAPE), (dict(num=65537), SHAPE), (dict(num=1025, block=64), SHAPE),
    (dict(num=2 ** 31 - 1, block=128), SHAPE), (dict(sink=-1), SHAPE), (dict(recent=-1), SHAPE),
    (dict(sink=60, recent=41), SHAPE), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), SHAPE),
    (dict(max_blocks=0), SHAPE), (dict(max_blocks=1 << 25), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=33), SHAPE), (dict(num_seqs=0), SHAPE), (dict(num_blocks=0), SHAPE),
    (dict(stride=64 * 72 - 16), SHAPE), (dict(stride=64 * 72 + 4), ALIGN), (dict(q=None), NULL),
    (dict(w=None), NULL), (dict(seq=None), NULL), (dict(pos=None), NULL), (dict(bt=None), NULL),
    (dict(cache=None), NULL), (dict(out=None), NULL), (dict(q=FAKE + 2), ALIGN),
    (dict(cache=FAKE + 8), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(ws=FAKE + 8), ALIGN)])
def test_select_rejects_bad_arguments(lib, kw, status):
    assert _select(lib, **kw) == status


def test_select_workspace(lib):
    size = lib.sparse_mla_select_workspace_size
    big = (1 << 64) - 1
    assert size(-1, 16, 10, 64, 1) == big and size(1, 0, 10, 64, 1) == big
    assert size(1, 16, 0, 64, 1) == big and size(1, 16, 10, 64, 3) == big
    assert size(0, 16, 10, 64, 1) == 0
    assert _select(lib, num_q=0, q=None) == 0
    one, many = size(1, 16, 1000, 64, 1), size(10 ** 6, 16, 1000, 64, 1)
    assert 64000 * 4 <= one < many <= 1 << 30     # a large batch shares a bounded workspace
    assert size(1, 16, 1000, 64, 64) < one        # one score for 32 positions
    assert size(1, 128, (1 << 31) // 64 - 8, 64, 1) < 1 << 34


def test_valid_arguments_without_gpu_report_device(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_plan, _truncate, _append, _read, _select):
        assert call(lib) in (4, 9)


def test_plain_forms_agree_with_each_other():
    """The tests' own planning and truncation undo each other, and prefix rules hold."""
    import numpy as np

    from tests import step_cases as sc
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 200, 30).astype(np.int32)
    new = rng.integers(0, 50, 30).astype(np.int32)
    table, free, _ = sc.random_tables(rng, lens, 16, 200, 20)
    step = sc.plan_step(new, lens, table, 16, free, len(free), 2000)
    assert step["refused"] == 0 and step["cu_tokens"][-1] == new.sum()
    live = step["slots"][:new.sum()]
    assert len(set(live.tolist())) == live.size
    back = sc.truncate(lens, step["seq_lens"], step["table"], 16, free, step["free_count"])
    assert np.array_equal(back["free_pages"], free) and back["free_count"] == len(free)
