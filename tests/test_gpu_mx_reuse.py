"""A grouping that is reused: whatever the workspace holds, the MXFP4 product stays inside its
buffers, and the next call is right again."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_linear_amd as nv
from test_gpu_mx import act_operand, acts, dev, rng_of, routes, say, up, weight  # noqa: F401

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


# (tokens, experts, top_k): by slots with and without list tiles, tiles of 64 and of 128
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(16, 64, 17), (100, 64, 4), (700, 512, 8), (300, 40, 4), (1100, 16, 4)])
def test_any_workspace_stays_in_bounds(dev, T, E, k, kind):
    N, K = 64, 96
    rng = rng_of(30, T, E, k)
    ids, tw = routes(rng, T, E, k)
    (xd, xs), _ = act_operand(acts(rng, T, K), kind, dev)
    wd, idd, twd = [up(a, dev) for a in weight(rng, E, N, K)], up(ids, dev), up(tw, dev)
    # the workspace and the output lie between guards
    size = nv.mxfp4_grouped_workspace_size(T, k, N, K, E, nv.OUT_COMBINE)
    arena = torch.full((GUARD + size + GUARD,), 0xA5, dtype=torch.uint8, device=dev)
    ws = arena[GUARD:GUARD + size]
    board = torch.full((T + 8192, N), 7.0, device=dev)
    out = board[4096:4096 + T]

    def combine(**kw):
        return nv.mxfp4_grouped_linear(xd, *wd, idd, topk_w=twd, x_scales=xs, out_mode=nv.OUT_COMBINE, out=out, workspace=ws, **kw)

    def other_grouping(t, e, top_k):
        i = up(routes(rng, t, e, top_k)[0], dev)
        (x, s), _ = act_operand(acts(rng, t, K), kind, dev)
        own = torch.zeros((nv.mxfp4_grouped_workspace_size(t, top_k, N, K, e, nv.OUT_ROUTES),), dtype=torch.uint8, device=dev)
        nv.mxfp4_grouped_linear(x, wd[0][:1].expand(e, -1, -1).contiguous(), wd[1][:1].expand(e, -1, -1).contiguous(), i, x_scales=s, workspace=own)
        n = min(size, own.numel())
        ws[:n] = own[:n]

    want = combine().clone()
    ints = lambda low, high: torch.from_numpy(rng.integers(low, high, size // 4, dtype=np.int64).astype(np.int32)).to(dev).view(torch.uint8)  # noqa: E731
    fills = {
        "another batch's routes": lambda: other_grouping(T, E, k), "more tokens": lambda: other_grouping(3 * T, E, k),
        "more experts": lambda: other_grouping(T, 2 * E, k), "zeros": lambda: ws.zero_(), "ones": lambda: ws.fill_(0xFF),
        "large": lambda: ws.fill_(0x7F), "least": lambda: ws.copy_(torch.full((size // 4,), -2 ** 31, dtype=torch.int32, device=dev).view(torch.uint8)),
        "any": lambda: ws.copy_(ints(-2 ** 31, 2 ** 31)), "near": lambda: ws.copy_(ints(-3, T * k + 3)), "experts": lambda: ws.copy_(ints(0, E)),
    }
    for name, fill in fills.items():
        say("reused workspace", kind, T, E, k, name)
        fill()
        combine(reuse_grouping=True)
        torch.cuda.synchronize()
        assert (arena[:GUARD] == 0xA5).all() and (arena[GUARD + size:] == 0xA5).all(), name
        assert (board[:4096] == 7).all() and (board[4096 + T:] == 7).all(), name
        assert torch.equal(combine(), want), name
