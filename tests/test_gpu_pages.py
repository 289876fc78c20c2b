"""GPU: forking, releasing, compacting and copying pages, against plain Python. Everything is whole
numbers: results have to be equal."""
import numpy as np
import pytest
import torch

from tests import pages_cases as pc
from tests import step_cases as sc

pytestmark = pytest.mark.gpu

I32 = torch.int32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def one(v):
    return dev(np.array([v], np.int32))


def host(t):
    return t.cpu().numpy()


def assert_same(got, ref):
    assert got.keys() == ref.keys()
    for k in ref:
        assert np.array_equal(got[k], ref[k]), k


def run_fork(src, dst, want, lens, table, page, shares, stack, count, in_place):
    import nvfp4_compressed_mla_gb300 as nm
    d = dict(src=dev(src), dst=dev(dst), want=dev(want), lens=dev(lens), table=dev(table),
             shares=dev(shares), stack=dev(stack), count=one(count))
    outs = {} if in_place else dict(seq_lens_out=torch.full_like(d["lens"], -7),
                                    page_shares_out=torch.full_like(d["shares"], -7),
                                    free_count_out=one(-7))
    refused = one(0)
    shared, cs, cd = nm.nvfp4_mla_fork(d["src"], d["dst"], d["want"], d["lens"], d["table"], page,
                                       d["shares"], d["stack"], d["count"], refused_count=refused, **outs)
    torch.cuda.synchronize()
    assert np.array_equal(host(d["stack"]), stack)
    if not in_place:
        assert np.array_equal(host(d["lens"]), lens) and np.array_equal(host(d["shares"]), shares)
        assert int(d["count"]) == count
    return dict(table=host(d["table"]), seq_lens=host(outs.get("seq_lens_out", d["lens"])),
                shares=host(outs.get("page_shares_out", d["shares"])),
                free_count=int(outs.get("free_count_out", d["count"])), shared_blocks=host(shared),
                copy_src=host(cs), copy_dst=host(cd), refused=int(refused))


def run_release(keep, lens, table, page, shares, stack, count, in_place):
    import nvfp4_compressed_mla_gb300 as nm
    d = dict(lens=dev(lens), table=dev(table), shares=dev(shares), stack=dev(stack), count=one(count))
    outs = {} if in_place else dict(seq_lens_out=torch.full_like(d["lens"], -7),
                                    page_shares_out=torch.full_like(d["shares"], -7),
                                    free_count_out=one(-7))
    dropped, refused = one(0), one(0)
    nm.nvfp4_mla_release(dev(keep), d["lens"], d["table"], page, d["shares"], d["stack"], d["count"],
                         dropped_count=dropped, refused_count=refused, **outs)
    torch.cuda.synchronize()
    assert np.array_equal(host(d["table"]), table)
    if not in_place:
        assert np.array_equal(host(d["lens"]), lens) and np.array_equal(host(d["shares"]), shares)
        assert int(d["count"]) == count
    return dict(seq_lens=host(outs.get("seq_lens_out", d["lens"])),
                shares=host(outs.get("page_shares_out", d["shares"])), free_pages=host(d["stack"]),
                free_count=int(outs.get("free_count_out", d["count"])), dropped=int(dropped),
                refused=int(refused))


def run_compact(lens, table, page, shares, stack, count, moves, in_place):
    import nvfp4_compressed_mla_gb300 as nm
    d = dict(lens=dev(lens), table=dev(table), shares=dev(shares), stack=dev(stack), count=one(count))
    outs = {} if in_place else dict(block_table_out=torch.full_like(d["table"], -7),
                                    page_shares_out=torch.full_like(d["shares"], -7),
                                    free_pages_out=dev(stack), free_count_out=one(-7))
    end = one(-7)
    cs, cd = nm.nvfp4_mla_compact(d["lens"], d["table"], page, d["shares"], d["stack"], d["count"], moves,
                                  pages_end=end, **outs)
    torch.cuda.synchronize()
    assert np.array_equal(host(d["lens"]), lens)
    if not in_place:
        assert np.array_equal(host(d["table"]), table) and np.array_equal(host(d["shares"]), shares)
        assert np.array_equal(host(d["stack"]), stack) and int(d["count"]) == count
    return dict(table=host(outs.get("block_table_out", d["table"])),
                shares=host(outs.get("page_shares_out", d["shares"])),
                free_pages=host(outs.get("free_pages_out", d["stack"])),
                free_count=int(outs.get("free_count_out", d["count"])), copy_src=host(cs),
                copy_dst=host(cd), pages_end=int(end))


@pytest.mark.parametrize("seqs,page,longest,forks,spare", [
    (2, 64, 64, 1, 0),           # whole pages only: no page is needed
    (2, 64, 1, 1, 1),            # a part of a page only
    (5, 7, 40, 9, 3),
    (66, 64, 5000, 40, 60),
    (300, 16, 700, 250, 60),     # pages run out on the way
    (40, 1, 3000, 20, 5),        # a page per token, rows of more than one chunk
    (2500, 48, 300, 2100, 900),  # more than one round of the prefix sum
])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(seqs, page, longest, forks, spare, in_place):
    rng = np.random.default_rng(seqs + page)
    lens, table, shares, stack, count = pc.family(rng, seqs, page, longest, spare, empty=0.5)
    lens[0] = longest if seqs == 2 else lens[0]
    if seqs == 2:
        lens[1] = 0
        table, stack, total = sc.random_tables(rng, lens, page, spare)
        shares, count = np.zeros(total, np.int32), len(stack)
    live, idle = np.nonzero(lens > 0)[0], np.nonzero(lens == 0)[0]
    src = rng.choice(live, forks).astype(np.int32)
    dst = rng.choice(idle, forks).astype(np.int32)
    dst[:min(forks, idle.size)] = rng.permutation(idle)[:min(forks, idle.size)]
    want = np.array([rng.choice([lens[s], lens[s] // page * page, rng.integers(0, lens[s] + 1)]) for s in src],
                    np.int32)
    if forks > 8:  # what is refused, and padding
        src[3], src[5], dst[2], dst[6] = -1, seqs, -1, seqs
        want[4], want[7], dst[1] = lens[src[4]] + 1, -2, live[0]
    ref = pc.fork(src, dst, want, lens, table, page, shares, stack, count)
    if seqs > 2:
        assert ref["refused"] > 0
    assert_same(run_fork(src, dst, want, lens, table, page, shares, stack, count, in_place), ref)


def test_fork_of_nothing_and_of_bad_pages():
    rng = np.random.default_rng(5)
    lens, table, shares, stack, count = pc.family(rng, 20, 16, 200, 20)
    none = np.zeros(0, np.int32)
    assert_same(run_fork(none, none, none, lens, table, 16, shares, stack, count, False),
                pc.fork(none, none, none, lens, table, 16, shares, stack, count))
    lens[:4], lens[4:8] = [64, 70, 70, 70], 0
    table[0, :4], table[1, :5], table[2, 4], table[3, 4] = [-1, 2, 10 ** 6, -5], [1, -1, 3, 4, -1], 10 ** 6, 7
    stack[count - 1] = 2 ** 31 - 1  # a page id outside of the pool is handed out as it is, but not copied into
    src, dst, want = (np.array(x, np.int32) for x in ([0, 3, 1, 2], [4, 5, 6, 7], [64, 70, 70, 70]))
    ref = pc.fork(src, dst, want, lens, table, 16, shares, stack, count)
    assert (ref["copy_src"] == -1).all() and ref["refused"] == 0
    assert_same(run_fork(src, dst, want, lens, table, 16, shares, stack, count, True), ref)
    for c in (-3, 0, 2, 10 ** 6):  # counts outside the stack are clamped
        ref = pc.fork(src, dst, want, lens, table, 16, shares, stack[:30], c)
        assert_same(run_fork(src, dst, want, lens, table, 16, shares, stack[:30], c, True), ref)


@pytest.mark.parametrize("seqs,page,longest,cut,whole", [
    (1, 64, 64, 1.0, True), (3, 64, 200, 1.0, False), (8, 1, 500, 0.9, False), (66, 64, 5000, 0.5, True),
    (300, 16, 700, 0.6, False), (2500, 48, 300, 0.4, False), (4, 2, 20000, 0.8, True),
    (3, 1, 400000, 1.0, False)])  # more than 4096 units of 256 entries
@pytest.mark.parametrize("in_place", [False, True])
def test_release(seqs, page, longest, cut, whole, in_place):
    rng = np.random.default_rng(seqs + page + longest)
    lens, table, shares, stack, count = pc.family(rng, seqs, page, longest, 10, empty=0.1)
    if seqs < 4:
        lens[:] = np.maximum(lens, 0)
    stack = np.concatenate([stack, np.full(len(shares), -8, np.int32)])
    keep = lens.copy()
    gone = rng.random(seqs) < cut
    keep[gone] = 0 if whole else (lens * rng.random(seqs)).astype(np.int32)[gone]
    keep[rng.random(seqs) < 0.05] = -1
    ref = pc.release(keep, lens, table, page, shares, stack, count)
    got = run_release(keep, lens, table, page, shares, stack, count, in_place)
    assert_same(got, ref)
    if page > 1 and not whole and seqs > 60:
        assert ref["refused"] > 0
    pc.check_state(got["seq_lens"], table, page, got["shares"], got["free_pages"], got["free_count"])


def test_release_without_room_on_the_stack_and_of_bad_pages():
    rng = np.random.default_rng(8)
    lens, table, shares, stack, count = pc.family(rng, 60, 16, 400, 10, empty=0.1)
    keep = np.where(rng.random(60) < 0.5, 0, lens).astype(np.int32)
    for room in (0, 5, 40):
        short = stack[:count + room].copy()
        ref = pc.release(keep, lens, table, 16, shares, short, count)
        assert ref["dropped"] > 0
        assert_same(run_release(keep, lens, table, 16, shares, short, count, True), ref)
    bad = table.copy()
    bad[:, 0], lens[7], keep[7] = -4, 10 ** 6, 3
    bad[::3, 1] = len(shares)
    stack = np.concatenate([stack, np.full(len(shares), -8, np.int32)])
    ref = pc.release(keep, lens, bad, 16, shares, stack, count)
    assert_same(run_release(keep, lens, bad, 16, shares, stack, count, False), ref)


@pytest.mark.parametrize("seqs,page,longest,spare,moves", [
    (1, 64, 64, 1, 3), (3, 64, 200, 40, 1), (8, 1, 500, 300, 10 ** 5), (66, 64, 5000, 5000, 700),
    (300, 16, 700, 2000, 10 ** 6), (2500, 48, 300, 100, 5000), (20, 1, 2500, 0, 100), (5, 16, 300, 200, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(seqs, page, longest, spare, moves, in_place):
    rng = np.random.default_rng(seqs + page + longest)
    lens, table, shares, stack, count = pc.family(rng, seqs, page, longest, spare)
    ref = pc.compact(lens, table, page, shares, stack, count, moves)
    got = run_compact(lens, table, page, shares, stack, count, moves, in_place)
    assert_same(got, ref)
    pc.check_state(lens, got["table"], page, got["shares"], got["free_pages"], got["free_count"])
    n = int((ref["copy_src"] >= 0).sum())
    if n < moves:  # nothing is left to move: the pages in use are the lowest
        assert ref["pages_end"] == len(shares) - ref["free_count"]


def test_compact_leaves_pages_alone_that_nobody_names():
    rng = np.random.default_rng(9)
    lens, table, shares, stack, count = pc.family(rng, 60, 16, 400, 300)
    stack[3:40] = np.array([stack[2], -1, 10 ** 7, int(table[table >= 0][0])] * 10, np.int32)[:37]
    for c in (count, -1, 5, 10 ** 6):
        ref = pc.compact(lens, table, 16, shares, stack, c, 200)
        assert_same(run_compact(lens, table, 16, shares, stack, c, 200, True), ref)
    bad = table.copy()
    bad[::5, 0], bad[1::5, 0] = -3, len(shares)
    lens[11], lens[12] = -5, 10 ** 6
    ref = pc.compact(lens, bad, 16, shares, stack, count, 200)
    assert_same(run_compact(lens, bad, 16, shares, stack, count, 200, False), ref)


@pytest.mark.parametrize("n,page_bytes,pad", [(1, 16, 0), (3, 64 * 352, 0), (500, 64 * 72, 48),
                                              (700, 16 * 576, 0), (20, 1 << 20, 16), (4000, 352 * 16, 0)])
def test_copy_pages(n, page_bytes, pad):
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(n)
    stride, blocks = page_bytes + pad, 2 * n + 5
    pool = rng.integers(0, 256, (blocks, stride), dtype=np.uint8)
    ids = rng.permutation(blocks).astype(np.int32)
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    bad = 0
    if n > 10:
        src[::5], dst[1::7] = -1, -1
        src[3], dst[4], src[8], dst[8], dst[9] = blocks, 2 ** 31 - 1, -2, 0, src[9]
        bad = sum(1 for a, b in zip(src, dst) if a != -1 and b != -1 and not (0 <= a < blocks and 0 <= b < blocks))
    d, count = dev(pool), one(0)
    nm.nvfp4_mla_copy_pages(dev(src), dev(dst), d.view(-1), blocks, stride, page_bytes, invalid_count=count)
    ref = pool.copy()
    for a, b in zip(src, dst):
        if 0 <= a < blocks and 0 <= b < blocks:
            ref[b, :page_bytes] = pool[a, :page_bytes]
    assert np.array_equal(host(d), ref)
    assert int(count) == bad and (n <= 10 or bad >= 3)


def test_copy_pages_past_four_gigabytes():
    import nvfp4_compressed_mla_gb300 as nm
    stride, blocks = 64 * 352, 200000  # 4.5 GB
    pool = torch.zeros(blocks, stride, dtype=torch.uint8, device="cuda:0")
    pool[blocks - 2] = 7
    pool[3] = 9
    nm.nvfp4_mla_copy_pages(dev(np.array([blocks - 2, 3], np.int32)), dev(np.array([5, blocks - 1], np.int32)),
                            pool.view(-1), blocks, stride, stride)
    assert bool((pool[5] == 7).all()) and bool((pool[blocks - 1] == 9).all()) and int(pool[6].max()) == 0


@pytest.mark.parametrize("captured", [False, True])
def test_a_life_of_forks_releases_and_compactions(captured):
    """Prompts grow, fork, end and are compacted, in place; the pool's rows follow."""
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(12)
    S, page, W, blocks, rows = 24, 16, 12, 150, 128
    stride = page * 32
    lens, table = np.zeros(S, np.int32), np.full((S, W), -1, np.int32)
    stack, count, shares = rng.permutation(blocks).astype(np.int32), blocks, np.zeros(blocks, np.int32)
    pool = np.zeros((blocks, page, 32), np.uint8)
    d = dict(lens=dev(lens), table=dev(table), stack=dev(stack), count=one(count), shares=dev(shares),
             pool=dev(pool), new=dev(lens), keep=dev(lens), src=dev(np.full(8, -1, np.int32)),
             dst=dev(np.zeros(8, np.int32)), want=dev(np.zeros(8, np.int32)), data=dev(np.zeros((rows, 32), np.uint8)))

    def step():
        _, _, slots, _ = nm.nvfp4_mla_plan_step(d["new"], d["lens"], d["table"], page, d["stack"], d["count"], rows)
        at = torch.where(slots >= 0, slots, blocks * page)
        big = torch.cat([d["pool"].view(-1, 32), d["data"][:1]])
        big.index_copy_(0, at, d["data"])
        d["pool"].view(-1, 32).copy_(big[:-1])
        _, a, b = nm.nvfp4_mla_fork(d["src"], d["dst"], d["want"], d["lens"], d["table"], page, d["shares"],
                                    d["stack"], d["count"])
        nm.nvfp4_mla_copy_pages(a, b, d["pool"].view(-1), blocks, stride, stride)
        nm.nvfp4_mla_release(d["keep"], d["lens"], d["table"], page, d["shares"], d["stack"], d["count"])
        a, b = nm.nvfp4_mla_compact(d["lens"], d["table"], page, d["shares"], d["stack"], d["count"], 5)
        nm.nvfp4_mla_copy_pages(a, b, d["pool"].view(-1), blocks, stride, stride)

    text = [[] for _ in range(S)]  # what each sequence holds
    graph = None
    for turn in range(25):
        new = np.where(rng.random(S) < 0.4, rng.integers(0, 12, S), 0).astype(np.int32)
        new[(lens == 0) & (rng.random(S) < 0.7)] = 0
        step1 = sc.plan_step(new, lens, table, page, stack, count, rows)
        data = rng.integers(0, 256, (rows, 32), dtype=np.uint8)
        src, dst = rng.integers(-1, S, 8).astype(np.int32), rng.integers(0, S, 8).astype(np.int32)
        now = step1["seq_lens"]
        want = np.array([rng.integers(0, now[s] + 1) if s >= 0 else 0 for s in src], np.int32)
        step2 = pc.fork(src, dst, want, now, step1["table"], page, shares, stack, step1["free_count"])
        now = step2["seq_lens"]
        keep = np.where(rng.random(S) < 0.25, (now * rng.choice([0, 0.7], S)).astype(np.int32), now).astype(np.int32)
        step3 = pc.release(keep, now, step2["table"], page, step2["shares"], stack, step2["free_count"])
        step4 = pc.compact(step3["seq_lens"], step2["table"], page, step3["shares"], step3["free_pages"],
                           step3["free_count"], 5)
        for name, v in (("new", new), ("data", data), ("src", src), ("dst", dst), ("want", want), ("keep", keep)):
            d[name].copy_(dev(v))
        if captured and graph is None:
            saved = {k: v.clone() for k, v in d.items()}
            step()  # the library is loaded outside the capture
            torch.cuda.synchronize()
            for k, v in saved.items():
                d[k].copy_(v)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if captured:
            graph.replay()
        else:
            step()
        for i in range(int((step1["seq_ids"] >= 0).sum())):
            text[step1["seq_ids"][i]].append(data[i])
        old = [list(t) for t in text]
        for i in range(8):
            if step2["shared_blocks"][i] >= 0:
                text[dst[i]] = old[src[i]][:want[i]]
        lens, table, shares = step3["seq_lens"], step4["table"], step4["shares"]
        stack, count = step4["free_pages"], step4["free_count"]
        text = [t[:n] for t, n in zip(text, lens)]
        torch.cuda.synchronize()
        for name, v in (("lens", lens), ("table", table), ("shares", shares)):
            assert np.array_equal(host(d[name]), v), (turn, name)
        assert int(d["count"]) == count and np.array_equal(host(d["stack"])[:count], stack[:count])
        pc.check_state(lens, table, page, shares, stack, count)
        pool = host(d["pool"]).reshape(blocks, page, 32)
        for s in range(S):
            for i, row in enumerate(text[s]):
                assert np.array_equal(pool[table[s, i // page], i % page], row), (turn, s, i)
    assert max(len(t) for t in text) > page


def test_results_on_another_stream():
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(13)
    lens, table, shares, stack, count = pc.family(rng, 40, 16, 400, 50)
    src, dst = np.nonzero(lens > 0)[0][:5].astype(np.int32), np.nonzero(lens == 0)[0][:5].astype(np.int32)
    n = min(len(src), len(dst))
    src, dst = src[:n], dst[:n]
    ref = pc.fork(src, dst, lens[src], lens, table, 16, shares, stack, count)
    d = [dev(x) for x in (src, dst, lens[src], lens, table, shares, stack)] + [one(count)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = nm.nvfp4_mla_fork(d[0], d[1], d[2], d[3], d[4], 16, d[5], d[6], d[7], stream=side)
    cs, cd = nm.nvfp4_mla_compact(d[3], d[4], 16, d[5], d[6], d[7], 30, stream=side)
    side.synchronize()
    for t, k in zip(got, ("shared_blocks", "copy_src", "copy_dst")):
        assert np.array_equal(host(t), ref[k])
    ref = pc.compact(ref["seq_lens"], ref["table"], 16, ref["shares"], stack, ref["free_count"], 30)
    assert np.array_equal(host(cs), ref["copy_src"]) and np.array_equal(host(cd), ref["copy_dst"])


def test_bindings_refuse_what_they_can_see():
    import nvfp4_compressed_mla_gb300 as nm
    i = torch.zeros(4, dtype=I32, device="cuda:0")
    t = torch.zeros((4, 3), dtype=I32, device="cuda:0")
    c, w = i[:1], torch.zeros(8, dtype=torch.int64, device="cuda:0")
    with pytest.raises(ValueError):
        nm.nvfp4_mla_fork(i, i[:3], i, i, t, 64, i, i, c)
    with pytest.raises(ValueError):
        nm.nvfp4_mla_fork(i, i, i, i, t, 64, w, i, c)
    with pytest.raises(ValueError):
        nm.nvfp4_mla_release(i[:3], i, t, 64, i, i, c)
    with pytest.raises(ValueError):
        nm.nvfp4_mla_release(i, i, t.view(-1), 64, i, i, c)
    with pytest.raises(ValueError):
        nm.nvfp4_mla_compact(i, t, 64, i.cpu(), i, c, 3)
    with pytest.raises(nm.NativeError):
        nm.nvfp4_mla_compact(i, t, 64, i, i, c, -1)
    with pytest.raises(nm.NativeError):
        nm.nvfp4_mla_compact(i, t, 64, i, i, c, 3, workspace=w[:1])
    with pytest.raises(ValueError):
        nm.nvfp4_mla_copy_pages(i, i, torch.zeros(100, dtype=torch.uint8, device="cuda:0"), 3, 64, 64)
