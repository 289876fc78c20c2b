"""GPU: the dense attention of a step where keys are missing, where its planning's shared memory, the count of
missing positions and the time that a result takes reach their limits, and where operands leave FP16's normal range."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import FP8, NVFP4, ROW, Case
from tests.gpu_cases import dev_tensor as dev
from workloads.gen import f32_from_bf16

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


@pytest.mark.parametrize("fmt", [NVFP4, FP8])
def test_results_that_take_longer_than_a_wait_may(fmt):
    """72 tokens behind a million: 36 row tiles of 8192 key tiles, about 10 ms each, under a limit of 2 million
    cycles (1 ms; a wait for one key tile is a microsecond). All of the context is one page."""
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(55, [64], [1], 128, fmt, spare=0)
    rng = np.random.default_rng(55)
    n, length = 72, 1 << 20
    q = torch.from_numpy(rng.standard_normal((n, 128, 576)).astype(np.float32)).to("cuda:0").bfloat16()
    args = c.device()
    args[0], args[1] = q[..., :512].contiguous(), q[..., 512:].contiguous()
    args[2] = torch.tensor([0, n], dtype=I32, device="cuda:0")
    args[3] = torch.zeros((1, length // 64), dtype=I32, device="cuda:0")
    args[4] = torch.tensor([length], dtype=I32, device="cuda:0")
    nm.nvfp4_mla_set_wait_limit(2_000_000)
    try:
        out, lse = nm.dense_mla_chunk(*args, out_fp32=True)
        torch.cuda.synchronize()
    finally:
        nm.nvfp4_mla_set_wait_limit(0)
    lat, rope, _ = c.keys(0)
    keys = np.concatenate([lat, rope], 1)
    for t in (0, 35, 71):
        seen = length - n + t + 1
        often = seen // 64 + (np.arange(64) < seen % 64)  # so many of the keys that the token sees are this row
        x = q[t].double().cpu().numpy()
        z = x @ keys.T * c.sm_scale
        top = z.max(1, keepdims=True)
        w = often * np.exp(z - top)
        total = w.sum(1, keepdims=True)
        w /= total
        # scores over 37 steps in fp32; the sum of weights over a third of the pieces of 64 keys, and a few more;
        # the output over 65536 steps of 16 keys, each off by 2^-23 of the magnitudes' sum, and FP16 weights
        dz = (np.abs(x) @ np.abs(keys).T).max(1) * c.sm_scale * 37 * 2.0 ** -23
        dsum = (seen / 64 / 3 + 40) * 2.0 ** -24 + 2.0 ** -20
        bound = (w @ np.abs(lat)) * (2.0 ** -11 + seen / 16 * 2.0 ** -23 + dsum + 2 * dz)[:, None]
        assert (np.abs(out[t].double().cpu().numpy() - w @ lat) <= bound).all()
        error = np.abs(lse[t].double().cpu().numpy() - (top + np.log(total))[:, 0])
        assert (error <= dz + dsum + 2.0 ** -20 * np.abs(top[:, 0] + np.log(total[:, 0]))).all()


def test_count_of_missing_positions_that_passes_32_bits():
    """Two sequences of pages that do not exist, 2146435072 positions each (about two seconds)."""
    import nvfp4_compressed_mla_gb300 as nm
    page, width = 1 << 20, 2047
    c = Case(60, [5, 5], [1, 1], 1, page=64)
    args = c.device()
    args[3] = torch.full((2, width), -1, dtype=I32, device="cuda:0")
    args[4] = torch.full((2,), page * width, dtype=I32, device="cuda:0")
    args[6] = torch.zeros(page * ROW[NVFP4], dtype=torch.uint8, device="cuda:0")
    args[5], args[7], args[8] = page, 1, page * ROW[NVFP4]
    bad = zero()
    out, lse = nm.dense_mla_chunk(*args, invalid_count=bad)
    assert not out.any() and bool(torch.isneginf(lse).all())
    assert int(bad) == 2 ** 31 - 1


@pytest.mark.parametrize("before,after", [(0, 200), (-50, 150), (2 ** 31 - 201, 2 ** 31 - 1), (2 ** 31 - 200, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_count_of_missing_positions_is_added(before, after):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(61, [300, 120, 40], [2, 1, 1], 16, page=16)
    c.table[0, :5], c.table[1, :] = -1, c.blocks  # 80 positions and 120
    bad = torch.tensor([before], dtype=I32, device="cuda:0")
    nm.dense_mla_chunk(*c.device(), invalid_count=bad)
    assert int(bad) == after


def small_operands(c, tokens):
    """The case's reference, its bounds widened for operands below FP16's normal range.

    The kernel's operands are q_latent and q_rope * rope_scale (/ latent_scale for FP8 rows) in FP16. Below 2^-14
    the step is 2^-24, so that an operand is off by 2^-25 at most, and a score by |sm_scale| (times latent_scale
    for FP8 rows) 2^-25 sum |k_d|, k being a row's values before the scales and d the dimensions of such
    operands. A score that is off by dz moves its weight by a factor of exp(dz) and the sum of weights by one of
    exp(max dz) at most, lse by max dz."""
    out, lse, tol, ltol = c.reference(tokens)
    lat_scale = c.latent_scale if c.fmt == FP8 else 1.0
    tiny = lambda q: (np.abs(q) < 2.0 ** -14) & (q != 0)
    for s in range(c.S):
        lat, rope, ok = c.keys(s)
        base = int(c.lens[s]) - int(c.new[s])
        for i in range(int(c.new[s])):
            t = int(c.cu[s]) + i
            if t not in tokens:
                continue
            k, r = lat[:base + i + 1], rope[:base + i + 1]
            ql, qr = f32_from_bf16(c.ql[t]).astype(np.float64), f32_from_bf16(c.qr[t]).astype(np.float64)
            z = c.sm_scale * (ql @ k.T + qr @ r.T)
            dz = abs(c.sm_scale) * lat_scale * 2.0 ** -25 * (
                tiny(ql) @ np.abs(k / lat_scale).T + tiny(qr * c.rope_scale / lat_scale) @ np.abs(r / c.rope_scale).T)
            w = np.exp(z - lse[t][:, None])
            tol[t] += (w * np.expm1(dz + dz.max(1, keepdims=True))) @ np.abs(k)
            ltol[t] += dz.max(1)
    return out, lse, tol, ltol


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("fmt,latent_scale,rope_scale,sm_scale,part", [
    (FP8, 1.0, 2.0 ** -14, 64.0, "rope"),       # the ratio of the scales makes q_rope's operand subnormal
    (FP8, 2.0 ** 10, 2.0 ** -4, 1.0, "rope"),
    (FP8, 2.0 ** 10, 2.0 ** -10, 8.0, "rope"),
    (NVFP4, 1.0, 2.0 ** -14, 64.0, "rope"),
    (NVFP4, 1.0, 1.0, 2048.0, "latent"),        # small q_latent
    (FP8, 2.0 ** -3, 1.0, 4096.0, "latent"),
    (FP8, 1.0, 2.0 ** -14, 1 / 24, "both"),
])
def test_operands_below_the_normal_range_of_fp16(heads, fmt, latent_scale, rope_scale, sm_scale, part):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(70, [150, 80], [6, 1], heads, fmt, latent_scale=latent_scale, rope_scale=rope_scale, sm_scale=sm_scale)
    if part == "rope":
        c.ql[:] = 0
    if part == "latent":
        c.ql -= np.where(c.ql & 0x7F80, 17 << 7, 0).astype(np.uint16)  # times 2^-17
        c.qr[:] = 0
    tokens = range(c.n)
    ref = small_operands(c, tokens)
    out, lse = nm.dense_mla_chunk(*c.device(), out_fp32=True)
    c.check(out, lse, True, ref=ref)


@pytest.mark.parametrize("seqs", [10240, 10241, 12225, 12288, 16384])
def test_sequences_around_the_plan_s_shared_memory(seqs):
    """4 bytes a sequence; most of them are idle."""
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(seqs)
    new = np.where(rng.random(seqs) < 150 / seqs, rng.integers(1, 6, seqs), 0)
    new[[0, seqs - 1]] = 1
    lens = np.where(rng.random(seqs) < 0.1, rng.integers(0, 60, seqs), 0)
    lens = np.maximum(lens, new)
    c = Case(seqs, lens, new, 16, page=16)
    c.table[seqs - 1, 0] = -1
    args, lens = c.device(), c.lens.copy()
    lens[np.nonzero(c.new == 0)[0][::7]] = -1  # of a sequence without new tokens nothing is read
    args[4] = dev(lens)
    bad = zero()
    out, lse = nm.dense_mla_chunk(*args, invalid_count=bad)
    c.check(out, lse)
    assert int(bad) == unresolved(c) > 0


@pytest.mark.parametrize("heads,new", [(16, 1), (128, 1), (64, 20)])
def test_a_few_row_tiles_over_any_number_of_key_tiles(heads, new):
    """Wherever the clusters' shares cut them: 1 to 20 key tiles, and a border beside a multiple of 128 keys."""
    import nvfp4_compressed_mla_gb300 as nm
    for k in range(1, 21):
        for length in (128 * k - 1, 128 * k, 128 * k + 1 + (k % 5) * 20):
            c = Case(80 + k, [length], [new], heads)
            out, lse = nm.dense_mla_chunk(*c.device(), out_fp32=True)
            c.check(out, lse, True, tokens=sorted({0, new // 2, new - 1}))
