"""
Sizes just below 2^31, where a sum in 32 bits (N + 127, N + 15) would pass it.
"""

import pytest
import torch

import f8_ref as R
import mixture_experts_routed_route_amd as moe

pytestmark = pytest.mark.gpu

VALUES = torch.tensor([1.0, -0.3, 0.01, 0.0, 7.0, -2.5, 0.6, 3.0])


@pytest.fixture(autouse=True)
def _give_memory_back():
    yield
    torch.cuda.empty_cache()


def _same(got, want):
    """Every eight codes of got are want's, read as one whole number."""
    return bool((got.view(torch.int64) == want.view(torch.int64).cuda()).all())


def test_quant_one_row():
    K = 2 ** 31 - 8
    q, s = moe.moe_quant_f8(VALUES.to(torch.bfloat16).cuda().repeat(K // 8)[None])
    rq, rs = R.quant_rows(VALUES.to(torch.bfloat16)[None])
    assert q.shape == (1, K) and s.shape == (1, 2 ** 24)
    assert bool((s == rs[0, 0].cuda()).all()) and _same(q.flatten(), rq.flatten())


def test_quant_weights_of_many_rows():
    N = 2 ** 31 - 1
    w = VALUES.to(torch.bfloat16).cuda().expand(N, 8).contiguous()
    q, s = moe.moe_quant_f8_weights(w)
    del w
    rq, rs = R.quant_rows(VALUES.to(torch.bfloat16)[None])
    assert q.shape == (N, 8) and s.shape == (2 ** 24, 1)
    assert bool((s == rs[0, 0].cuda()).all()) and _same(q.flatten(), rq.flatten())


@pytest.mark.parametrize("M", [1, 17])
def test_product_of_many_weight_rows(M):
    """Rows of ones, every 2^20th and the last of twos: sums of 16 and 32."""
    N = 2 ** 31 - 1 if M == 1 else 2 ** 31 - 17
    one = torch.tensor(1.0).to(R.F8)
    q = torch.empty(N, 16, dtype=R.F8, device="cuda")
    q.view(torch.uint8).fill_(int(one.view(torch.uint8)))
    twos = torch.tensor(2.0).to(R.F8).cuda()
    q[::2 ** 20] = twos
    q[-1] = twos
    s = torch.ones(2 ** 24, 1, device="cuda")
    x = (torch.ones(M, 16).to(R.F8).cuda(), torch.ones(M, 1, device="cuda"))
    out = moe.moe_gemm_f8(x, (q, s), out_dtype=torch.bfloat16)
    del q, s
    assert out.shape == (M, N)
    for r in range(M):
        assert bool((out[r, ::2 ** 20] == 32).all()) and float(out[r, -1]) == 32
        out[r, ::2 ** 20] = 16
        out[r, -1] = 16
        assert bool((out[r] == 16).all())
