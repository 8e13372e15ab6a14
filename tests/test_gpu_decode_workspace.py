"""The layer for a few tokens refuses a workspace that its kernels cannot write:
host memory, and a view whose elements do not lie one after the other."""

import pytest
import torch

import mixture_experts_routed_route_amd as moe

pytestmark = pytest.mark.gpu


def test_workspaces_that_are_refused():
    T, D, F, E, k = 2, 128, 128, 4, 2
    g = torch.Generator().manual_seed(0)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    x, w = mk(T, D), (mk(E, F, D), mk(E, F, D), mk(E, D, F))
    lg = torch.randn(T, E, generator=g).cuda()
    y, _ = moe.moe_decode(x, *w, k, logits=lg)
    n = moe.moe_decode_workspace_bytes(T, E, k, D, F, moe.MOE_BF16, moe.MOE_BF16)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
                torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            moe.moe_decode(x, *w, k, logits=lg, workspace=bad)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.moe_decode(x, *w, k, logits=lg, workspace=ws)[0], y)
