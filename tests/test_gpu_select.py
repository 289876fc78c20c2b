"""GPU: the selection against 64-bit scores and a stable sort. The chosen positions have to be
equal: the operator decides as 64-bit arithmetic does, ties by the lower index."""
import numpy as np
import pytest
import torch

from tests import step_cases as sc
from workloads.gen import bf16_from_f32

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.view(dtype) if dtype is not None else t).to("cuda:0")


class Case:
    def __init__(self, seed, lens, per_seq, heads, page=64, pad=0, width=None, order=None):
        rng = np.random.default_rng(seed)
        self.page, self.stride = page, page * sc.ROW + pad
        self.lens = np.asarray(lens)
        self.table, _, self.blocks = sc.random_tables(rng, self.lens, page, 2, width)
        self.pool = sc.random_pool(rng, self.blocks, page, self.stride)
        seq = np.repeat(np.arange(len(lens)), per_seq)
        pos = np.concatenate([np.arange(n - per_seq, n) for n in self.lens])
        if order is not None:
            seq, pos = seq[order], pos[order]
        self.seq, self.pos = seq.astype(np.int32), pos.astype(np.int32)
        self.q = bf16_from_f32(rng.standard_normal((len(seq), heads, 128)))
        self.w = (rng.standard_normal((len(seq), heads)) / np.sqrt(heads)).astype(np.float32)

    def ref(self, num, block=1, sink=0, recent=0):
        return sc.select(self.q, self.w, self.seq, self.pos, self.table, self.page, self.pool,
                         self.blocks, self.stride, num, block, sink, recent)

    def device(self):
        return (dev(self.q, torch.bfloat16), dev(self.w), dev(self.seq), dev(self.pos),
                dev(self.table), self.page, dev(self.pool), self.blocks, self.stride)

    def run(self, num, block=1, sink=0, recent=0, **kw):
        import nvfp4_compressed_mla_gb300 as nm
        out = nm.sparse_mla_select(*self.device(), num, select_block=block, sink_blocks=sink,
                                   recent_blocks=recent, **kw)
        torch.cuda.synchronize()
        return out.cpu().numpy()

    def check(self, num, block=1, sink=0, recent=0, **kw):
        got, ref = self.run(num, block, sink, recent, **kw), self.ref(num, block, sink, recent)
        bad = np.nonzero((got != ref).any(1))[0]
        assert bad.size == 0, (bad[:5], got[bad[0]][:20], ref[bad[0]][:20])


@pytest.mark.parametrize("heads", [1, 2, 16, 31, 32, 33, 64, 65, 100, 128])
def test_head_counts(heads):
    Case(heads, [700, 1, 129, 2000], 1, heads).check(100)


@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("sink,recent", [(0, 0), (1, 2), (0, 5)])
def test_block_sizes(block, sink, recent):
    Case(block, [block * 40 + 3, block * 9, 5 * block + 1, 1], 2, 8).check(6, block, sink, recent)


@pytest.mark.parametrize("page,pad", [(2, 0), (16, 16), (48, 0), (64, 64 * 352), (128, 0), (1000, 0)])
def test_page_sizes_and_strides(page, pad):
    Case(page, [1500, 333], 1, 24, page=page, pad=pad).check(64)


@pytest.mark.parametrize("per_seq", [1, 2, 3, 5, 15, 64])
def test_several_query_tokens_of_a_sequence(per_seq):
    Case(per_seq, [900, 40, 2100], per_seq, 32).check(128)


def test_query_tokens_in_any_order():
    rng = np.random.default_rng(3)
    Case(3, [900, 1200, 500, 70], 9, 16, order=rng.permutation(36)).check(50)


@pytest.mark.parametrize("num", [1, 2, 255, 256, 1000, 2047, 2999, 3000, 5000])
def test_numbers_selected(num):
    Case(num, [3000, 2999, 10], 1, 16).check(num)


def test_lengths_around_a_tile():
    Case(8, [1, 2, 127, 128, 129, 255, 256, 257, 383, 385], 1, 16).check(100)


def test_long_context():
    Case(11, [60011], 2, 64).check(2048)


def test_a_table_wider_than_the_sequences():
    Case(12, [300, 7], 1, 16, width=500).check(40)


def test_query_tokens_that_see_nothing_or_past_the_table():
    c = Case(13, [300, 500], 3, 16)
    c.seq[0], c.pos[1], c.seq[2] = -1, -1, 2
    c.pos[3] = 10 ** 6  # sees the whole table
    c.pos[4] = 2 ** 31 - 1
    c.check(40)
    got = c.run(40)
    assert (got[:3] == -1).all()


def test_pages_that_do_not_resolve_rank_last():
    c = Case(14, [900, 900], 1, 16)
    c.table[0, 3], c.table[0, 5], c.table[1, 0] = -1, 10 ** 6, -1
    c.table[1, 2:9] = -1
    c.check(64)
    c.check(700)  # some of them have to be taken: the lowest ones
    c.check(5, 64)


def test_equal_scores_go_to_the_lower_index():
    c = Case(15, [1000, 1000, 1000], 1, 16)
    c.w[0] = 0.0                      # every score 0
    c.q[1] = 0
    row = c.pool.reshape(c.blocks, c.stride)
    one = row[:, :64].copy()[0], row[:, 64 * 64:64 * 64 + 8].copy()[0]
    for b in c.table[2][:9]:          # sequence 2: the same key 576 times, then others
        row[b, :64 * 64] = np.tile(one[0], 64)
        row[b, 64 * 64:64 * sc.ROW] = np.tile(one[1], 64)
    c.check(100)
    c.check(700)
    c.check(9, 64)


def test_more_candidates_than_the_list_holds():
    # one head: half of the scores are exactly 0, and the border lies among them
    c = Case(16, [9000, 5000], 1, 1)
    c.w[:] = 1.0
    c.check(6000)
    c = Case(17, [9000], 2, 2)
    c.w[:] = -1.0
    c.check(3000)
    c.check(100, 32)


def test_scores_next_to_each_other():
    # keys that differ in one code of a small group: scores a few parts in 2^24 apart
    rng = np.random.default_rng(18)
    c = Case(18, [2000], 1, 64)
    row = c.pool.reshape(c.blocks, c.stride)
    base = rng.integers(0, 256, 64, dtype=np.uint8)
    for b in c.table[0]:
        codes = row[b, :64 * 64].reshape(64, 64)
        codes[:] = base
        codes[np.arange(64), 0] = rng.integers(0, 256, 64)
        row[b, 64 * 64:64 * sc.ROW] = np.tile(np.array([1] + [126] * 7, np.uint8), 64)
    c.check(500)
    c.check(10, 16)


def test_weights_and_keys_over_a_wide_range():
    rng = np.random.default_rng(19)
    c = Case(19, [3000, 3000], 1, 64)
    c.w *= (10.0 ** rng.uniform(-6, 6, c.w.shape)).astype(np.float32)
    c.q = bf16_from_f32(rng.standard_normal(c.q.shape) * 10.0 ** rng.uniform(-4, 2, c.q.shape))
    c.check(300)
    c.w *= np.float32(1e-38)  # subnormal weights among them
    c.check(300)


def test_workspace_of_the_stated_size_is_enough_and_its_contents_do_not_matter():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(20, [700, 1300], 5, 16)
    n = nm.sparse_mla_select_workspace_size(10, 16, c.table.shape[1], 64, 4)
    buf = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda:0")
    got = c.run(20, 4, workspace=buf[:n])
    assert bool((buf[n:] == 255).all())
    assert np.array_equal(got, c.ref(20, 4))
    with pytest.raises(nm.NativeError):
        c.run(20, 4, workspace=buf[:n - 16])


def test_replayed_graphs_that_share_a_workspace_in_order():
    import nvfp4_compressed_mla_gb300 as nm
    a, b = Case(21, [700, 1300], 1, 16), Case(22, [500, 90, 2000], 1, 64)
    n = max(nm.sparse_mla_select_workspace_size(len(c.seq), c.q.shape[1], c.table.shape[1], 64)
            for c in (a, b))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda:0")
    made = []
    for c in (a, b):
        args = c.device()
        out = torch.empty((len(c.seq), 64), dtype=torch.int32, device="cuda:0")
        nm.sparse_mla_select(*args, 64, topk_idx=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nm.sparse_mla_select(*args, 64, topk_idx=out, workspace=ws)
        made.append((g, out, args, c.ref(64)))
    for g, out, _, _ in made:
        out.fill_(-9)
    for g, _, _, _ in made * 3:
        g.replay()
    torch.cuda.synchronize()
    for _, out, _, ref in made:
        assert np.array_equal(out.cpu().numpy(), ref)


def test_another_stream():
    c = Case(23, [700, 1300], 2, 16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(64, stream=s)
    assert np.array_equal(got, c.ref(64))


def test_results_repeat():
    c = Case(24, [5000, 3000], 4, 64)
    first = c.run(512)
    for _ in range(5):
        assert np.array_equal(c.run(512), first)


def reference_on_device(c, num, block=1, sink=0, recent=0):
    """The same definition in torch, fp64, for sizes past the Python loops."""
    nib = torch.tensor(np.concatenate([sc.GRID, -sc.GRID]), device="cuda:0")
    pool = dev(c.pool).view(c.blocks, c.stride)
    codes = pool[:, :c.page * 64].reshape(c.blocks, c.page, 64)
    scale = pool[:, c.page * 64:c.page * sc.ROW].reshape(c.blocks, c.page, 8)
    v = nib[torch.stack([codes & 15, codes >> 4], -1).long()].view(c.blocks, c.page, 8, 16)
    keys = (v * scale.view(torch.float8_e4m3fn).double()[..., None]).view(c.blocks, c.page, 128)
    out = np.full((len(c.seq), num * block), -1, np.int32)
    q = torch.from_numpy(sc.values(*sc.quantize(c.q))).to("cuda:0")
    w = dev(c.w).double()
    for t in range(len(c.seq)):
        seen = int(c.pos[t]) + 1
        k = keys[torch.from_numpy(c.table[c.seq[t]][:sc.blocks_of(seen, c.page)]).long().to("cuda:0")]
        score = torch.relu(k.reshape(-1, 128)[:seen] @ q[t].T) @ w[t]
        nb = sc.blocks_of(seen, block)
        best = torch.nn.functional.pad(score, (0, nb * block - seen), value=-np.inf)
        best = best.view(nb, block).amax(1)
        idx = torch.arange(nb, device="cuda:0")
        best[(idx < sink) | (idx >= nb - recent)] = np.inf
        chosen = torch.sort(best, descending=True, stable=True).indices[:num].sort().values
        pos = (chosen[:, None] * block + torch.arange(block, device="cuda:0")).reshape(-1)
        pos = pos[pos < seen].cpu().numpy()
        out[t, :len(pos)] = pos
    return out


# every CTA of the score kernel goes many times round its stages and slots
@pytest.mark.parametrize("seqs,length,per_seq,heads,num,block,page", [
    (40, 40000, 1, 64, 2048, 1, 64), (40, 30000, 1, 32, 512, 4, 64), (20, 40000, 1, 128, 1000, 1, 16),
    (20, 40000, 1, 96, 32, 64, 256), (6, 30000, 15, 64, 2048, 1, 64), (4, 20000, 64, 64, 64, 16, 64),
    (30, 40000, 1, 64, 700, 1, 48), (4, 20000, 32, 128, 300, 1, 96), (3, 20000, 200, 24, 128, 16, 64),
    (1, 600000, 1, 16, 2048, 1, 64), (330, 3000, 1, 64, 16, 64, 64), (400, 20000, 1, 16, 256, 1, 64),
])
def test_sizes_that_fill_the_device(seqs, length, per_seq, heads, num, block, page):
    rng = np.random.default_rng(seqs + length)
    lens = rng.integers(length * 9 // 10, length + 1, seqs)
    c = Case.__new__(Case)
    c.page, c.stride, c.lens = page, page * sc.ROW, lens
    c.table, _, c.blocks = sc.random_tables(rng, lens, page, 2)
    c.pool = rng.integers(0, 256, c.blocks * c.stride, dtype=np.uint8)
    rows = c.pool.reshape(c.blocks, c.stride)
    scales = rng.integers(0x28, 0x48, (c.blocks, page * 8), dtype=np.uint8)
    rows[:, page * 64:] = scales
    seq = np.repeat(np.arange(seqs), per_seq)
    pos = np.concatenate([np.arange(n - per_seq, n) for n in lens])
    c.seq, c.pos = seq.astype(np.int32), pos.astype(np.int32)
    c.q = bf16_from_f32(rng.standard_normal((len(seq), heads, 128)))
    c.w = (rng.standard_normal((len(seq), heads)) / np.sqrt(heads)).astype(np.float32)
    got, ref = c.run(num, block), reference_on_device(c, num, block)
    bad = np.nonzero((got != ref).any(1))[0]
    assert bad.size == 0, (bad.size, bad[:5], got[bad[0]][:20], ref[bad[0]][:20])


def test_more_query_tokens_than_the_workspace_takes_at_a_time():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(23, [700, 333], 80, 16, width=8192)
    per_q = nm.sparse_mla_select_workspace_size(1, 16, 8192, 64)
    n = nm.sparse_mla_select_workspace_size(160, 16, 8192, 64)
    assert n < 140 * per_q  # parts of fewer than 160
    c.check(40)


def test_on_a_stream_of_its_own():
    c = Case(24, [700, 2000], 3, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    import nvfp4_compressed_mla_gb300 as nm
    args = c.device()
    torch.cuda.synchronize()
    a = nm.sparse_mla_select(*args, 64, stream=side)
    with torch.cuda.stream(side):
        b = nm.sparse_mla_select(*args, 64)
    e = nm.sparse_mla_select(*args, 64, stream=side.cuda_stream)
    side.synchronize()
    for got in (a, b, e):
        assert np.array_equal(got.cpu().numpy(), c.ref(64))


def test_two_calls_at_once():
    cases = [Case(25, [9000, 2000], 1, 64), Case(26, [3000, 100, 7000], 2, 32)]
    import nvfp4_compressed_mla_gb300 as nm
    args, refs = [c.device() for c in cases], [c.ref(256) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(nm.sparse_mla_select(*args[i], 256))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert np.array_equal(g.cpu().numpy(), refs[i])


def test_python_arguments_that_are_refused():
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(27, [300, 40], 1, 16)
    args = c.device()

    def bad(i, t):
        a = list(args)
        a[i] = t
        with pytest.raises(ValueError):
            nm.sparse_mla_select(*a, 16)

    q, w, seq, pos, table, _, pool = args[:7]
    bad(0, q.float())                       # type
    bad(0, q[:, :, :64])                    # width
    bad(0, q.cpu())                         # device
    bad(0, q.transpose(0, 1))               # strides
    bad(1, w[:, :8])
    bad(1, w.double())
    bad(2, seq[:1])                         # too few
    bad(3, pos.long())
    bad(4, table.view(-1))
    bad(4, table.cpu())
    bad(6, pool[:-1])                       # a page short
    with pytest.raises(ValueError):
        nm.sparse_mla_select(*args, 16, topk_idx=torch.empty((2, 15), dtype=torch.int32, device="cuda"))
    for kw in (dict(select_block=3), dict(select_block=256), dict(sink_blocks=-1),
               dict(sink_blocks=9, recent_blocks=8)):
        with pytest.raises(nm.NativeError):
            nm.sparse_mla_select(*args, 16, **kw)
    with pytest.raises(nm.NativeError):
        nm.sparse_mla_select(*args, 0)
    assert np.array_equal(c.run(16), c.ref(16))


# page 64: tensor copies; page 48: copies row by row
@pytest.mark.parametrize("page", [64, 48])
@pytest.mark.parametrize("heads,per_seq", [(16, 1), (64, 4), (128, 2)])
def test_waits_that_run_out_give_minus_two_and_the_next_launch_is_correct(page, heads, per_seq):
    import nvfp4_compressed_mla_gb300 as nm
    # ten steps or more an SM, so that stages are taken a second time: a long
    # sequence that has the same pages again and again
    c = Case(28, [4000, 333], per_seq, heads, page=page)
    c.table = np.tile(c.table[:, :4000 // page], (1, 100))
    c.pos[:per_seq] += c.table.shape[1] * page - 4000
    args = c.device()
    want = nm.sparse_mla_select(*args, 64).clone()
    nm.nvfp4_mla_set_wait_limit(200)
    try:
        for _ in range(3):
            got = nm.sparse_mla_select(*args, 64)
            torch.cuda.synchronize()
            assert bool((got == -2).all()), "no wait ran out under a 200-cycle bound"
    finally:
        nm.nvfp4_mla_set_wait_limit(0)
    assert torch.equal(nm.sparse_mla_select(*args, 64), want)


@pytest.mark.parametrize("heads,block,num,lens", [
    (1, 1, 50, [9000, 2592, 40]), (1, 1, 6000, [9000, 2592]), (1, 128, 4, [5240, 2000, 5239]),
    (4, 16, 14, [2592, 2591, 700]), (3, 4, 100, [9000, 333]), (1, 64, 30, [9000]),
    (2, 1, 2048, [70000]), (1, 2, 3000, [40000]),
])
def test_weights_of_one_sign(heads, block, num, lens):
    # without a positive weight the highest scores are zeros, and ties go to the lower index
    c = Case(heads * block + num, lens, 2, heads)
    c.w = -np.abs(c.w) - np.float32(1e-3)
    c.check(num, block)
    c.check(num, block, min(2, num // 2), min(1, num // 2))
    c.w = -c.w  # the lowest scores are zeros
    c.check(num, block)


@pytest.mark.parametrize("block,num", [(1, 700), (1, 5000), (8, 60), (128, 5)])
def test_scores_that_cancel(block, num):
    # two equal heads with opposite weights: every score is 0, by a sum that fp32 bounds but
    # does not settle, or by dot products that are all 0
    c = Case(29, [9000, 1300], 2, 2)
    c.q[:, 1] = c.q[:, 0]
    c.w[:, 0], c.w[:, 1] = 0.7, -0.7
    c.check(num, block)
    # and a third head that tells some of them apart
    d = Case(30, [9000, 1300], 2, 3)
    d.q[:, 1] = d.q[:, 0]
    d.w[:, 0], d.w[:, 1], d.w[:, 2] = 0.7, -0.7, 1e-9
    d.check(num, block)


@pytest.mark.parametrize("page", [64, 48])
def test_a_layer_of_a_pool_that_holds_several(page):
    # page p of layer l at (p * layers + l) pages: the last layer's last page ends the pool
    import nvfp4_compressed_mla_gb300 as nm
    layers, bytes_ = 3, page * sc.ROW
    cases = [Case(31, [900, 1300], 2, 16, page=page) for _ in range(layers)]
    pool = torch.empty(cases[0].blocks * layers * bytes_, dtype=torch.uint8, device="cuda:0")
    whole = pool.view(cases[0].blocks, layers, bytes_)
    for i, c in enumerate(cases):
        c.pool = sc.random_pool(np.random.default_rng(40 + i), c.blocks, page, bytes_)
        whole[:, i] = dev(c.pool).view(c.blocks, bytes_)
    for i, c in enumerate(cases):
        a = c.device()
        view = pool[i * bytes_:]
        got = nm.sparse_mla_select(*a[:6], view, c.blocks, layers * bytes_, 40)
        assert np.array_equal(got.cpu().numpy(), c.ref(40))
        keys = torch.randn((1, 128), device="cuda:0").bfloat16()
        at = [dev(np.array([x], np.int32)) for x in (1, 1299)]
        nm.nvfp4_mla_index_append(keys, *at, a[4], page, view, c.blocks, layers * bytes_)
        k = nm.nvfp4_mla_index_read(*at, a[4], page, view, c.blocks, layers * bytes_)
        codes, scales = sc.quantize(keys.view(torch.int16).cpu().numpy().view(np.uint16))
        assert np.array_equal(k.float().cpu().numpy(), sc.values(codes, scales))
        with pytest.raises(ValueError):  # a byte short of the last page's end
            nm.sparse_mla_select(*a[:6], pool[i * bytes_:pool.numel() - (layers - 1 - i) * bytes_ - 1],
                                 c.blocks, layers * bytes_, 40)


@pytest.mark.parametrize("page", [64, 48])
def test_pages_past_4_gib(page):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(32, [1500, 700], 3, 32, page=page)
    stride = (160 << 20) + 16
    pool = torch.empty(c.blocks * stride, dtype=torch.uint8, device="cuda:0")
    assert pool.numel() > 5 << 30
    pool.view(c.blocks, stride)[:, :page * sc.ROW] = dev(c.pool).view(c.blocks, -1)
    a = c.device()
    for block, num in ((1, 50), (16, 6)):
        got = nm.sparse_mla_select(*a[:6], pool, c.blocks, stride, num, block)
        assert np.array_equal(got.cpu().numpy(), c.ref(num, block))
