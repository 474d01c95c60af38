"""What contexts hold on the device: room for the parts of the tree attention from its first call on."""
import pytest
import torch

from parity import tsl
from test_gpu_tree import BF, DEV, Case

pytestmark = pytest.mark.gpu


def _free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


def test_contexts_without_drafts_hold_no_room_for_them():
    """Sixteen contexts of bf16 pools take what those of fp32 pools take, to the granularity of the allocations (2 MB each)."""
    T = tsl()
    used = []
    for kind in (T.TS_KV_F32, T.TS_KV_BF16):
        before = _free()
        held = [T.Context(32, 8, 128, kind, 1, 4, 8) for _ in range(16)]
        used.append(before - _free())
        for c in held:
            c.close()
    assert used[1] <= used[0] + 16 * 2 * 2 ** 20


def test_the_first_call_makes_the_room():
    """Also one without rows, and one that is captured; the calls behind it make no more."""
    T = tsl()
    c = Case(8, 4, 128, lens=[9000, 50], trees=[40, 7], seed=26)
    c.run()
    want, wl = c.out.clone(), c.lse.clone()
    now = _free()
    c.run()
    assert _free() == now
    args = (c.k_pool, c.v_pool, c.dev(c.table), c.dev(c.lens))
    # without rows
    c.ctx = T.Context(32, 8, 128, T.TS_KV_BF16, 2, c.table.shape[1], c.pages)
    none = torch.zeros(0, 32, 128, dtype=BF, device=DEV)
    c.ctx.tree_attend(none, *args, c.dev([0, 0, 0]), None, none)
    now = _free()
    c.out.fill_(0)
    c.run()
    assert _free() == now and torch.equal(c.out, want)
    # captured
    c.ctx = T.Context(32, 8, 128, T.TS_KV_BF16, 2, c.table.shape[1], c.pages)
    more = (c.dev(c.cu), c.mask_tensor(), c.out, c.lse)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        c.ctx.tree_attend(c.q, *args, *more)
    for _ in range(2):
        c.out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(c.lse, wl)
    assert c.ctx.status() == 0
