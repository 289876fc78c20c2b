"""GPU: block tables and slot maps of a step, and the pages that come back, against plain Python.
Everything is whole numbers: results have to be equal."""
import numpy as np
import pytest
import torch

from tests import step_cases as sc

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def run_plan(new, lens, table, page, free, count, max_tokens, in_place=False):
    import nvfp4_compressed_mla_gb300 as nm
    d = dict(new=dev(new), lens=dev(lens), table=dev(table), free=dev(free),
             count=dev(np.array([count], np.int32)))
    refused = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    lens_out = None if in_place else torch.full_like(d["lens"], -7)
    count_out = None if in_place else torch.full_like(d["count"], -7)
    ids, pos, slots, cu = nm.nvfp4_mla_plan_step(
        d["new"], d["lens"], d["table"], page, d["free"], d["count"], max_tokens,
        seq_lens_out=lens_out, free_count_out=count_out, refused_count=refused)
    torch.cuda.synchronize()
    assert np.array_equal(d["free"].cpu().numpy(), free)
    if not in_place:
        assert np.array_equal(d["lens"].cpu().numpy(), lens)
        assert int(d["count"]) == count
    return dict(seq_ids=ids.cpu().numpy(), positions=pos.cpu().numpy(), slots=slots.cpu().numpy(),
                cu_tokens=cu.cpu().numpy(),
                seq_lens=(d["lens"] if in_place else lens_out).cpu().numpy(),
                table=d["table"].cpu().numpy(),
                free_count=int(d["count"] if in_place else count_out), refused=int(refused))


def assert_same(got, ref):
    for k in ref:
        assert np.array_equal(got[k], ref[k]), k


@pytest.mark.parametrize("seqs,page,most_len,most_new,tokens,spare", [
    (1, 64, 0, 1, 1, 2),              # the first token of the first request
    (1, 64, 64, 1, 1, 0),             # a full page and no page left
    (3, 48, 200, 1, 3, 4),
    (66, 64, 5000, 1, 66, 70),
    (66, 1, 40, 5, 400, 400),         # a page per token
    (257, 16, 300, 40, 4096, 10),     # pages run out on the way
    (257, 16, 300, 40, 1000, 3000),   # rows run out on the way
    (1021, 64, 3000, 90, 40000, 2000),
    (1500, 32, 900, 120, 65536, 100000),
    (5000, 64, 100, 3, 9000, 8000),
    (16384, 16, 30, 2, 20000, 20000),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_step(seqs, page, most_len, most_new, tokens, spare, in_place):
    rng = np.random.default_rng(seqs + page + tokens)
    lens = rng.integers(0, most_len + 1, seqs).astype(np.int32)
    new = rng.integers(0, most_new + 1, seqs).astype(np.int32)
    if seqs == 1:
        lens[0], new[0] = most_len, most_new
    width = max(sc.blocks_of(most_len + most_new, page), 1)
    table, free, _ = sc.random_tables(rng, lens, page, spare, width)
    if seqs > 50:  # requests that are refused for what they are
        new[7], lens[11], new[13] = -3, -1, 2 ** 31 - 1
        new[17] = width * page - lens[17] + 1
    ref = sc.plan_step(new, lens, table, page, free, len(free), tokens)
    assert_same(run_plan(new, lens, table, page, free, len(free), tokens, in_place), ref)


def test_plan_long_prompt_and_idle_sequences():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 500, 700).astype(np.int32)
    new = np.zeros(700, np.int32)
    new[3], new[350], new[699] = 100000, 1, 20011
    table, free, _ = sc.random_tables(rng, lens, 64, 2000, 1700)
    ref = sc.plan_step(new, lens, table, 64, free, len(free), 131072)
    assert ref["refused"] == 0
    assert_same(run_plan(new, lens, table, 64, free, len(free), 131072), ref)


@pytest.mark.parametrize("page", [1, 3, 7, 48, 1000, 2 ** 20 - 1, 2 ** 20])
@pytest.mark.parametrize("tokens", [3000, 12000])  # one CTA, a cluster
def test_plan_page_sizes_and_lengths_up_to_the_last_token(page, tokens):
    rng = np.random.default_rng(page)
    width = min((2 ** 31 - 1) // page, 2047)
    room = width * page
    lens = np.minimum([0, page, page * 5 + 1, 2 * page - 1, room - 700, room - 900], room)
    lens = np.maximum(lens, 0).astype(np.int32)
    new = np.minimum([300, 1, 700, 2, 700, 901], room - lens).astype(np.int32)
    new[5] = room - lens[5] + 1  # one too many
    if tokens > 3000:
        new[2] = min(9000, room - int(lens[2]))
    table, free, _ = sc.random_tables(rng, lens, page, 4000, width)
    ref = sc.plan_step(new, lens, table, page, free, len(free), tokens)
    assert ref["refused"] >= 1
    assert_same(run_plan(new, lens, table, page, free, len(free), tokens), ref)
    after = ref["seq_lens"]
    stack = np.concatenate([free[:ref["free_count"]], np.full(9000, -7, np.int32)])
    back = sc.truncate(lens, after, ref["table"], page, stack, ref["free_count"])
    got = run_truncate(lens, after, ref["table"], page, stack, ref["free_count"])
    assert_same(got, back)
    assert np.array_equal(back["free_pages"][:len(free)], free)


def test_plan_nothing_to_do_and_no_rows():
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 500, 40).astype(np.int32)
    table, free, _ = sc.random_tables(rng, lens, 64, 5, 9)
    zero = np.zeros(40, np.int32)
    for new, tokens in ((zero, 0), (zero, 10), (zero + 1, 0)):
        ref = sc.plan_step(new, lens, table, 64, free, len(free), tokens)
        assert_same(run_plan(new, lens, table, 64, free, len(free), tokens), ref)


@pytest.mark.parametrize("count", [-5, 0, 3, 1000])
def test_plan_page_counts_outside_the_stack_are_clamped(count):
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 200, 20).astype(np.int32)
    table, free, _ = sc.random_tables(rng, lens, 16, 9, 20)
    new = np.full(20, 17, np.int32)
    ref = sc.plan_step(new, lens, table, 16, free, count, 400)
    assert_same(run_plan(new, lens, table, 16, free, count, 400), ref)


def test_plan_table_entry_without_a_page_gives_no_slot():
    lens, new = np.array([5], np.int32), np.array([3], np.int32)
    table, free = np.array([[-1, -1]], np.int32), np.array([4], np.int32)
    ref = sc.plan_step(new, lens, table, 8, free, 1, 4)
    assert list(ref["slots"]) == [-1, -1, -1, -1]
    assert_same(run_plan(new, lens, table, 8, free, 1, 4), ref)


def run_truncate(keep, lens, table, page, stack, count, in_place=False):
    import nvfp4_compressed_mla_gb300 as nm
    d = [dev(x) for x in (keep, lens, table, stack, np.array([count], np.int32))]
    dropped = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    lens_out = None if in_place else torch.full_like(d[1], -7)
    count_out = None if in_place else torch.full_like(d[4], -7)
    nm.nvfp4_mla_truncate(d[0], d[1], d[2], page, d[3], d[4], seq_lens_out=lens_out,
                          free_count_out=count_out, dropped_count=dropped)
    torch.cuda.synchronize()
    assert np.array_equal(d[2].cpu().numpy(), table)
    return dict(seq_lens=(d[1] if in_place else lens_out).cpu().numpy(),
                free_pages=d[3].cpu().numpy(),
                free_count=int(d[4] if in_place else count_out), dropped=int(dropped))


@pytest.mark.parametrize("seqs,page,most_len,room", [
    (1, 64, 1, 10), (1, 64, 20000, 400), (5, 48, 700, 200), (33, 16, 900, 4000),
    (66, 64, 20000, 30000), (1021, 64, 3000, 50000), (1021, 64, 3000, 40), (4000, 16, 60, 30000),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_truncate(seqs, page, most_len, room, in_place):
    rng = np.random.default_rng(seqs + page + room)
    lens = rng.integers(0, most_len + 1, seqs).astype(np.int32)
    lens[0] = most_len
    table, free, _ = sc.random_tables(rng, lens, page, 7)
    keep = np.where(rng.random(seqs) < 0.3, 0,
                    lens - rng.integers(-3, 40, seqs)).astype(np.int32)  # negative: unchanged
    if seqs > 1:  # a page that was never assigned and a length past the table are skipped
        table[1, : table.shape[1] // 2] = -1
        lens[2], keep[2] = table.shape[1] * page + 100, 0
    stack = np.full(room + len(free), -9, np.int32)
    stack[:len(free)] = free
    ref = sc.truncate(keep, lens, table, page, stack, len(free))
    got = run_truncate(keep, lens, table, page, stack, len(free), in_place)
    assert_same(got, ref)


def test_truncating_a_step_restores_the_stack():
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 3000, 300).astype(np.int32)
    new = rng.integers(0, 200, 300).astype(np.int32)
    table, free, _ = sc.random_tables(rng, lens, 64, 2000, 60)
    dl, dt, df = dev(lens), dev(table), dev(free)
    before = dl.clone()
    count = dev(np.array([len(free)], np.int32))
    nm.nvfp4_mla_plan_step(dev(new), dl, dt, 64, df, count, int(new.sum()))
    assert int(count) < len(free) and np.array_equal(dl.cpu().numpy(), lens + new)
    nm.nvfp4_mla_truncate(before, dl, dt, 64, df, count)
    assert int(count) == len(free)
    assert np.array_equal(df.cpu().numpy(), free) and np.array_equal(dl.cpu().numpy(), lens)


def test_steps_replayed_from_a_graph_advance_the_state():
    import nvfp4_compressed_mla_gb300 as nm
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 300, 70).astype(np.int32)
    new = rng.integers(0, 9, 70).astype(np.int32)
    table, free, _ = sc.random_tables(rng, lens, 16, 400, 40)
    dn, dl, dt, df = dev(new), dev(lens), dev(table), dev(free)
    count = dev(np.array([len(free)], np.int32))
    out = dict(seq_ids=torch.empty(600, dtype=torch.int32, device="cuda:0"),
               positions=torch.empty(600, dtype=torch.int32, device="cuda:0"),
               slots=torch.empty(600, dtype=torch.int64, device="cuda:0"),
               cu_tokens=torch.empty(71, dtype=torch.int32, device="cuda:0"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nm.nvfp4_mla_plan_step(dn, dl, dt, 16, df, count, 600, **out)
    have = len(free)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        ref = sc.plan_step(new, lens, table, 16, free, have, 600)
        for k in out:
            assert np.array_equal(out[k].cpu().numpy(), ref[k]), k
        lens, table, have = ref["seq_lens"], ref["table"], ref["free_count"]
        assert np.array_equal(dl.cpu().numpy(), lens) and int(count) == have
        assert np.array_equal(dt.cpu().numpy(), table)
