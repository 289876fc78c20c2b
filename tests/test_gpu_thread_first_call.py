"""GPU: a host thread whose first CUDA work is a call of this library. No context is bound to it yet."""
import threading

import numpy as np
import pytest
import torch

from tests.test_gpu_select import Case

pytestmark = pytest.mark.gpu

I32 = torch.int32
LATENT = 64 * 352


def decode_args(heads=16, topk=256):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(73)
    bf = dict(dtype=torch.bfloat16, device="cuda:0", generator=g)
    cache = torch.zeros(4 * LATENT, dtype=torch.uint8, device="cuda:0")
    table = torch.arange(4, dtype=I32, device="cuda:0").view(1, 4)
    seq = torch.zeros(256, dtype=I32, device="cuda:0")
    pos = torch.arange(256, dtype=I32, device="cuda:0")
    import nvfp4_compressed_mla_gb300 as nm
    nm.nvfp4_mla_append(torch.randn((256, 512), **bf), torch.randn((256, 64), **bf), seq, pos,
                        table, 64, cache, 4, LATENT)
    top = pos.view(1, -1)[:, :topk].contiguous()
    return (torch.randn((1, heads, 512), **bf), torch.randn((1, heads, 64), **bf), seq[:1], top,
            table, torch.full((1,), 256, dtype=I32, device="cuda:0"), 64, cache, 4, LATENT)


def in_new_thread(call):
    got, errors = [], []

    def work():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            errors.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    return got[0]


@pytest.mark.parametrize("page", [64, 48])  # codes by tensor copies, row by row
def test_select(page):
    import nvfp4_compressed_mla_gb300 as nm
    c = Case(80, [700, 1300], 2, 16, page=page)
    args = c.device()
    out = torch.empty((4, 64), dtype=torch.int32, device="cuda:0")
    ws = torch.empty(nm.sparse_mla_select_workspace_size(4, 16, c.table.shape[1], page),
                     dtype=torch.uint8, device="cuda:0")
    in_new_thread(lambda: nm.sparse_mla_select(*args, 64, topk_idx=out, workspace=ws, stream=0))
    assert np.array_equal(out.cpu().numpy(), c.ref(64))


def test_decode():
    import nvfp4_compressed_mla_gb300 as nm
    args = decode_args(128)
    want = nm.sparse_mla_decode(*args, nm.ROW_NVFP4_352, 0.05, num_splits=1)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(max(nm.sparse_mla_decode_workspace_size(1, 128, 256, 1), 16),
                     dtype=torch.uint8, device="cuda:0")
    in_new_thread(lambda: nm.sparse_mla_decode(*args, nm.ROW_NVFP4_352, 0.05, num_splits=1, out=out,
                                               lse=lse, workspace=ws, stream=0))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
