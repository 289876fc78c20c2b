"""Host-side checks of the dense chunk attention's entry point and of its tests' plain form (no GPU)."""
import numpy as np
import pytest

FAKE = 0x10000  # 16-byte aligned non-null address; never dereferenced on these paths
NULL, SHAPE, ALIGN, WORKSPACE, FORMAT, VALUE = 1, 2, 3, 5, 7, 8


@pytest.fixture(scope="module")
def lib():
    from nvfp4_compressed_mla_gb300 import _native
    return _native.load()


def _chunk(lib, **kw):
    a = dict(ql=FAKE, qr=FAKE, cu=FAKE, num_q=7, heads=16, bt=FAKE, num_seqs=3, max_blocks=10, lens=FAKE,
             page_size=64, cache=FAKE, num_blocks=50, stride=64 * 352, fmt=0, sm=0.04, lat=1.0, rope=1.0,
             out=FAKE, f32=0, lse=None, ws=FAKE, ws_bytes=1 << 30, invalid=None, stream=None)
    a.update(kw)
    return lib.dense_mla_chunk(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(num_q=-1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=129), SHAPE), (dict(num_seqs=0), SHAPE),
    (dict(num_seqs=16385), SHAPE), (dict(num_q=1 << 25, heads=128), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=(1 << 20) + 1), SHAPE), (dict(max_blocks=1 << 25), SHAPE),
    (dict(num_blocks=0), SHAPE), (dict(stride=64 * 352 - 16), SHAPE), (dict(fmt=1), SHAPE),
    (dict(stride=1 << 62), SHAPE), (dict(stride=64 * 352 + 8), ALIGN), (dict(ql=FAKE + 2), ALIGN),
    (dict(qr=FAKE + 8), ALIGN), (dict(cache=FAKE + 4), ALIGN), (dict(out=FAKE + 8), ALIGN),
    (dict(ws=FAKE + 8), ALIGN), (dict(ql=None), NULL), (dict(qr=None), NULL), (dict(cu=None), NULL),
    (dict(bt=None), NULL), (dict(lens=None), NULL), (dict(cache=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE), (dict(fmt=2), FORMAT),
    (dict(sm=float("nan")), VALUE), (dict(sm=float("inf")), VALUE), (dict(lat=0.0), VALUE),
    (dict(rope=-1.0), VALUE), (dict(rope=float("inf")), VALUE)])
def test_refusals(lib, kw, status):
    assert _chunk(lib, **kw) == status


def test_workspace_and_nothing_to_do(lib):
    size = lib.dense_mla_chunk_workspace_size
    big = (1 << 64) - 1
    assert size(-1, 16, 3) == size(1, 0, 3) == size(1, 129, 3) == size(1, 16, 0) == size(1 << 25, 128, 1) == big
    assert size(0, 16, 3) == 0 and _chunk(lib, num_q=0, ql=None) == 0
    assert 0 < size(1, 1, 1) <= size(131072, 128, 1000) < 1 << 26


def test_valid_arguments_without_gpu_report_device(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _chunk(lib) in (4, 9)


@pytest.mark.parametrize("fmt", [0, 1])
def test_plain_form_agrees_with_the_oracle(fmt):
    """A step's tokens are decoded by the oracle over the positions that they see."""
    import oracle
    from tests.chunk_cases import Case
    c = Case(3, [70, 1, 130], [5, 1, 3], 4, fmt, latent_scale=0.5, rope_scale=2.0)
    out, lse, _, _ = c.reference()
    seq = np.repeat(np.arange(3), c.new).astype(np.int32)
    idx = np.full((c.n, 130), -1, np.int32)
    for t in range(c.n):
        s = seq[t]
        idx[t, :c.lens[s] - c.new[s] + t - c.cu[s] + 1] = np.arange(c.lens[s] - c.new[s] + t - c.cu[s] + 1)
    ref, ref_lse, bad = oracle.sparse_mla_decode(c.ql, c.qr, seq, idx, c.table, c.lens, 64, c.pool.reshape(-1),
                                                 c.blocks, c.stride, fmt, np.float32(c.sm_scale), 0.5, 2.0)
    assert np.abs(out - ref).max() < 1e-6 and np.abs(lse - ref_lse).max() < 1e-6
