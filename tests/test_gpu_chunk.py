"""GPU: the dense attention of a step's new tokens against the definition in 64 bits, at the sizes
and masks where it can go wrong."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import FP8, NVFP4, Case

pytestmark = pytest.mark.gpu

I32 = torch.int32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def run(case, **kw):
    import nvfp4_compressed_mla_gb300 as nm
    out, lse = nm.dense_mla_chunk(*case.device(), **kw)
    torch.cuda.synchronize()
    return out, lse


# lengths and new tokens of a step's sequences
STEPS = {
    "one token": ([1], [1]),
    "first tokens of a prompt": ([5], [5]),
    "single tokens": ([1, 63, 64, 65, 127, 128, 129, 700], [1] * 8),
    "drafts": ([300, 17, 64, 200], [3, 17, 2, 15]),
    "a chunk behind a context": ([777], [130]),
    "mixed, with idle sequences": ([0, 400, 90, 257, 1, 0, 300], [0, 1, 90, 0, 1, 0, 70]),
}


@pytest.mark.parametrize("step", STEPS)
@pytest.mark.parametrize("heads", [1, 3, 16, 33, 128])
@pytest.mark.parametrize("fmt", [NVFP4, FP8])
def test_steps(step, heads, fmt):
    lens, new = STEPS[step]
    c = Case(len(step) + heads, lens, new, heads, fmt)
    out, lse = run(c)
    c.check(out, lse)


@pytest.mark.parametrize("page,lens,new", [(1, [70, 9], [3, 9]), (3, [200], [40]), (16, [130, 64], [1, 1]),
                                           (48, [500, 47, 48], [60, 47, 1]), (100, [333], [200]), (1000, [900], [2]),
                                           (128, [129, 256], [129, 3])])
@pytest.mark.parametrize("fmt,pad", [(NVFP4, 0), (NVFP4, 48), (FP8, 16)])
def test_page_sizes_and_strides(page, lens, new, fmt, pad):
    c = Case(page, lens, new, 16, fmt, page=page, stride_pad=pad, width=1100 if page < 16 else 40)
    out, lse = run(c)
    c.check(out, lse)


@pytest.mark.parametrize("heads,lens,new", [
    (128, [6000], [1]),               # a few rows: the keys are dealt out to many clusters
    (16, [9001], [3]),
    (128, [5000, 40, 3000], [1, 1, 1]),
    (128, [3500], [30]),              # pairs, every row tile cut several times
    (64, [2500, 2500, 1], [100, 1, 1]),
    (127, [1500] * 5, [11] * 5),
])
@pytest.mark.parametrize("fmt", [NVFP4, FP8])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_long_contexts_are_split_and_merged(heads, lens, new, fmt, out_fp32):
    c = Case(heads + len(lens), lens, new, heads, fmt, q_scale=2.0)
    tokens = sorted(set(np.linspace(0, c.n - 1, 12).astype(int).tolist()))
    out, lse = run(c, out_fp32=out_fp32)
    c.check(out, lse, out_fp32, tokens=tokens)


def test_many_row_tiles():
    # more row tiles than one round of the planning's threads, and than clusters
    rng = np.random.default_rng(3)
    new = rng.integers(0, 40, 700)
    lens = new + rng.integers(0, 60, 700)
    c = Case(4, lens, new, 16)
    tokens = set(rng.integers(0, c.n, 200).tolist())
    out, lse = run(c)
    c.check(out, lse, tokens=tokens)
    c = Case(5, [2000], [2000], 128)
    tokens = set(rng.integers(0, c.n, 20).tolist()) | {0, 1, c.n - 1}
    out, lse = run(c)
    c.check(out, lse, tokens=tokens)


@pytest.mark.parametrize("latent_scale,rope_scale", [(1.0, 0.5), (0.25, 2.0), (0.37, 1.7)])
@pytest.mark.parametrize("fmt", [NVFP4, FP8])
def test_scales(latent_scale, rope_scale, fmt):
    c = Case(11, [300, 90], [20, 1], 16, fmt, latent_scale=latent_scale, rope_scale=rope_scale)
    out, lse = run(c)
    c.check(out, lse)


@pytest.mark.parametrize("sm_scale", [0.0, -0.05, 1e-6, 0.4])
@pytest.mark.parametrize("new", [1, 40])
def test_softmax_scales(sm_scale, new):
    # 0.4: scores of hundreds, the reference of most rows moves again and again
    c = Case(12, [900], [new], 16, sm_scale=sm_scale, q_scale=3.0)
    out, lse = run(c)
    c.check(out, lse)


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("fmt", [NVFP4, FP8])
def test_scores_that_grow_along_the_context(new, fmt):
    """Every tile's scores exceed those before: each moves the references and rescales O."""
    c = Case(13, [1300], [new], 128 if new == 1 else 8, fmt, q_scale=1.0)
    rows = c.pool[:, :c.page * c.stride // c.page].reshape(c.blocks, c.page, -1)
    for b in range(c.width):
        rows[c.table[0, b], :, -64:] = 0x38 if b % 2 else 0x30   # rope values 1 and 0.5
        rows[c.table[0, b], :, -64:] += np.uint8(min(b, 16))     # growing by an eighth
    c.qr[:] = 0x4080  # 4.0
    out, lse = run(c)
    c.check(out, lse)


@pytest.mark.parametrize("new", [1, 30])
def test_pages_that_do_not_resolve(new):
    c = Case(14, [700, 64 * 3, 130], [new, 5, 2], 16 if new == 1 else 64)
    c.table[0, [1, 4]], c.table[0, 7] = [-1, c.blocks], -2 ** 31
    c.table[1] = -5  # a sequence without any page
    bad = torch.zeros(1, dtype=I32, device="cuda:0")
    out, lse = run(c, invalid_count=bad)
    c.check(out, lse)
    assert int(bad) == 3 * 64 + 3 * 64
    assert bool((out[c.cu[1]:c.cu[2]] == 0).all()) and bool(torch.isneginf(lse[c.cu[1]:c.cu[2]]).all())


def test_first_pages_missing_leaves_rows_that_see_nothing_of_a_part():
    c = Case(15, [9000], [20], 16)
    c.table[0, :70] = -1
    out, lse = run(c)
    c.check(out, lse, tokens=[0, 7, 19])


@pytest.mark.parametrize("fmt", [NVFP4, FP8])
@pytest.mark.parametrize("heads", [16, 128])
def test_nan_rows_reach_only_the_tokens_that_see_them(fmt, heads):
    """The last 4 of 9 new tokens were appended as NaN; what lies behind the sequence is NaN too."""
    c = Case(16, [200], [9], heads, fmt)
    flat = c.pool.reshape(c.blocks, c.page, -1)
    clean = c.pool.copy()
    for pos in range(196, 256):
        row = flat[c.table[0, pos // 64], pos % 64]
        if fmt == NVFP4:
            row[256:288] = 0x7F
        else:
            row[:512] = 0xFF
        row[-64:] = 0x7F
    out, lse = run(c)
    assert bool(torch.isnan(out[5:9].float()).all()) and bool(torch.isnan(lse[5:9]).all())
    c.pool = clean
    c.check(out, lse, tokens=range(5))


def test_rows_behind_the_last_token_are_left_alone():
    import nvfp4_compressed_mla_gb300 as nm
    for heads, new in ((16, [1, 1]), (128, [30, 7])):
        c = Case(17, [100, 300], new, heads, pad=13)
        out = torch.full((c.num_q, heads, 512), 7.5, dtype=torch.bfloat16, device="cuda:0")
        lse = torch.full((c.num_q, heads), -3.25, device="cuda:0")
        run(c, out=out, lse=lse)
        c.check(out, lse)
        assert bool((out[c.n:] == 7.5).all()) and bool((lse[c.n:] == -3.25).all())
    empty = Case(18, [100, 300], [0, 0], 16, pad=5)
    out = torch.full((5, 16, 512), 7.5, dtype=torch.bfloat16, device="cuda:0")
    run(empty, out=out)
    assert bool((out == 7.5).all())
    none = Case(19, [100], [0], 16)
    assert run(none)[0].shape == (0, 16, 512)


def test_malformed_sequences_are_skipped_and_counted():
    c = Case(20, [100, 300, 50, 80, 64], [10, 5, 7, 20, 3], 16)
    args, ref = c.device(), c.reference()
    out = torch.full((c.num_q, 16, 512), 7.5, dtype=torch.bfloat16, device="cuda:0")
    bad = torch.zeros(1, dtype=I32, device="cuda:0")
    import nvfp4_compressed_mla_gb300 as nm
    lens = c.lens.copy()
    lens[1], lens[3] = 4, c.width * c.page + 1  # fewer than its new tokens; beyond its table
    args[4] = dev(lens)
    _, lse = nm.dense_mla_chunk(*args, out=out, invalid_count=bad)
    assert int(bad) == 2
    keep = [t for s in (0, 2, 4) for t in range(c.cu[s], c.cu[s + 1])]
    c.check(out, lse, ref=ref, tokens=keep)
    for s in (1, 3):
        assert bool((out[c.cu[s]:c.cu[s + 1]] == 7.5).all())
    # offsets that leave the rows, descend or overlap: no fault, and the others are right
    for cu in ([0, 10, 10 ** 6, 22, 42, 45], [-5, 10, 15, 22, 42, 45], [0, 10, 15, 12, 42, 45],
               [0, 45, 0, 45, 0, 45]):
        args[2] = dev(np.array(cu, np.int32))
        nm.dense_mla_chunk(*args, out=out)
    args[2], args[4] = dev(c.cu), dev(c.lens)
    out, lse = nm.dense_mla_chunk(*args)
    c.check(out, lse, ref=ref)


def test_offsets_past_32_bits():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(21, [500, 200], [3, 40], 16)
    far = torch.zeros(200000 * c.stride, dtype=torch.uint8, device="cuda:0").view(200000, c.stride)  # 4.5 GB
    table = c.table.copy()
    for s in range(c.S):
        for b in range(c.width):
            if table[s, b] >= 0:
                table[s, b] = 199999 - c.table[s, b]
                far[int(table[s, b])] = dev(c.pool[c.table[s, b]])
    args = c.device()
    args[3], args[6], args[7] = dev(table), far.view(-1), 200000
    out, lse = nm.dense_mla_chunk(*args)
    c.check(out, lse)


@pytest.mark.parametrize("heads,new", [(16, 1), (128, 20)])
def test_captured_and_replayed_with_other_contents(heads, new):
    import nvfp4_compressed_mla_gb300 as nm
    cases = [Case(seed, lens, [new] * 3, heads, width=10) for seed, lens in ((22, [600, 300, 20]), (23, [80, 20, 640]))]
    blocks = max(c.blocks for c in cases)
    for c in cases:
        c.pool = np.concatenate([c.pool, np.zeros((blocks - c.blocks, c.stride), np.uint8)])
        c.blocks = blocks
    held = cases[0].device()
    out = torch.zeros((cases[0].num_q, heads, 512), dtype=torch.bfloat16, device="cuda:0")
    lse = torch.zeros((cases[0].num_q, heads), device="cuda:0")
    nm.dense_mla_chunk(*held, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nm.dense_mla_chunk(*held, out=out, lse=lse)
    for c in (cases[1], cases[0]):
        for a, b in zip(held, c.device()):
            if torch.is_tensor(a):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_two_streams_at_once_and_results_that_repeat():
    import nvfp4_compressed_mla_gb300 as nm
    a, b = Case(24, [3000], [40], 128), Case(25, [5000, 700], [1, 1], 64)
    da, db = a.device(), b.device()
    one, two = run(a), run(b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append((nm.dense_mla_chunk(*da, stream=s), nm.dense_mla_chunk(*db, stream=t)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], one[0]) and torch.equal(x[1], one[1])
        assert torch.equal(y[0], two[0]) and torch.equal(y[1], two[1])
    a.check(*one, tokens=[0, 20, 39])


@pytest.mark.parametrize("heads,new,fmt", [(16, 1, NVFP4), (128, 20, NVFP4), (128, 20, FP8), (128, 600, NVFP4)])
def test_waits_that_run_out_make_every_row_nan(heads, new, fmt):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(26, [900, 700], [new, new], heads, fmt, pad=3)
    args = c.device()
    out = torch.full((c.num_q, heads, 512), 7.5, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.zeros((c.num_q, heads), device="cuda:0")
    nm.nvfp4_mla_set_wait_limit(300)
    try:
        nm.dense_mla_chunk(*args, out=out, lse=lse)
        torch.cuda.synchronize()
    finally:
        nm.nvfp4_mla_set_wait_limit(0)
    assert bool(torch.isnan(out[:c.n].float()).all()) and bool(torch.isnan(lse[:c.n]).all())
    assert bool((out[c.n:] == 7.5).all())
    nm.dense_mla_chunk(*args, out=out, lse=lse)
    c.check(out, lse, tokens=[0, new // 2, c.n - 1])


def test_against_the_sparse_decode_over_the_same_rows():
    """A step of single tokens attends to what the decode attends to when it is given every position."""
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(27, [900, 64, 333], [1, 1, 1], 128)
    out, lse = run(c, out_fp32=True)
    a = c.device()
    idx = np.full((3, 900), -1, np.int32)
    for s in range(3):
        idx[s, :c.lens[s]] = np.arange(c.lens[s])
    ref, ref_lse = nm.sparse_mla_decode(a[0], a[1], dev(np.arange(3, dtype=np.int32)), dev(idx), a[3], a[4], 64,
                                        a[6], c.blocks, c.stride, NVFP4, c.sm_scale, out_fp32=True)
    assert float((out - ref).norm() / ref.norm()) < 1e-3
    assert float((lse - ref_lse).abs().max()) < 1e-3


def test_thousands_of_sequences():
    """More sequences and row tiles than the plan takes at a time, among them idle ones."""
    rng = np.random.default_rng(29)
    lens = rng.integers(0, 60, 2600)
    new = np.minimum(lens, rng.choice([0, 1, 1, 1, 3], 2600))
    c = Case(29, lens, new, 16, page=16)
    c.check(*run(c))


@pytest.mark.parametrize("heads,fmt", [(16, NVFP4), (128, FP8)])
def test_queries_that_are_no_numbers_stay_in_their_rows(heads, fmt):
    c = Case(30, [300, 90], [20, 3], heads, fmt)
    ref = c.reference()
    c.ql[3, 2, 17], c.qr[21, 1, 5] = 0x7FC0, 0x7FC0  # NaN
    c.ql[7, 4, 0], c.qr[9, 0, 63] = 0x7F80, 0xFF80   # infinities
    out, lse = run(c)
    for t, h in ((3, 2), (21, 1)):
        assert bool(torch.isnan(out[t, h].float()).all()) and bool(torch.isnan(lse[t, h]))
    for t, h in ((3, 2), (21, 1), (7, 4), (9, 0)):
        out[t, h] = dev(ref[0][t, h]).to(out.dtype)
        lse[t, h] = float(ref[1][t, h])
    c.check(out, lse, ref=ref)


def test_bindings_refuse_what_they_can_see():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(28, [100], [2], 16)
    good = c.device()

    def bad(error, i, value, **kw):
        args = list(good)
        args[i] = value
        with pytest.raises(error):
            nm.dense_mla_chunk(*args, **kw)

    bad(ValueError, 0, good[0].float())
    bad(ValueError, 0, good[0][..., :256].contiguous())
    bad(ValueError, 0, good[0].transpose(0, 1))
    bad(ValueError, 1, good[1][:1])
    bad(ValueError, 2, good[2][:1])
    bad(ValueError, 3, good[3].long())
    bad(ValueError, 4, good[4].cpu())
    bad(ValueError, 6, good[6][:-16])
    bad(nm.NativeError, 5, 0)
    bad(nm.NativeError, 9, 5)
    bad(nm.NativeError, 10, float("nan"))
    bad(nm.NativeError, 11, 0.0)
    bad(ValueError, 0, good[0], out=torch.zeros(1, device="cuda:0"))
    bad(ValueError, 0, good[0], lse=torch.zeros(1, device="cuda:0"))
    bad(nm.NativeError, 0, good[0], workspace=torch.zeros(16, dtype=torch.uint8, device="cuda:0"))
