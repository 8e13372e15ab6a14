"""
The sums of the layer on 8-bit weights: products that cancel, whose rest the
8-bit matrix unit would drop, on every route.
"""

import pytest
import torch

import f8_ref as R
import mixture_experts_routed_route_amd as moe
from test_gpu_f8 import DT

pytestmark = pytest.mark.gpu

ONE = 448.0   # a block whose largest magnitude this is has scale 1


def _blocks_of_one(n, N, K):
    """Weights of zeros whose first block of every 128 rows has scale 1: its
    largest value stands in column 100, where x is zero."""
    w = torch.zeros(n, N, K)
    w[:, ::128, 100] = ONE
    return w


def _call(x, logits, ws, y_dtype):
    p = moe.moe_plan_create(logits.cuda(), 2)
    y = moe.moe_forward(p, x.cuda(), *(moe.moe_quant_f8_weights(w.cuda()) for w in ws),
                        options=moe.make_options(swiglu_limit=0.0), y_dtype=y_dtype)
    v = moe.moe_plan_get_views(p)
    return y.cpu().double(), v["topk_id"].cpu().long(), v["topk_w"].cpu().double()


@pytest.mark.parametrize("T", [1, 8, 40, 300])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gate_up_products_that_cancel(dt, T):
    """Every row of x is 448, 448, then six values a; W_up is 448, -448, then
    six values c: u = 6 a c, where the first two products are 2^13 times the
    others and more. All sums are whole numbers below 2^24: exact in f32."""
    n, D, F = 2, 256, 128
    a = torch.tensor([2.0, 4.0, 8.0])[torch.arange(T) % 3]
    c = torch.tensor([1.0, 2.0])[torch.arange(F) % 2]
    x = torch.zeros(T, D)
    x[:, :2] = ONE
    x[:, 2:8] = a[:, None]
    wg, wu = _blocks_of_one(n, F, D), _blocks_of_one(n, F, D)
    wg[:, :, 2:8] = 0.125
    wu[:, :, 0], wu[:, :, 1], wu[:, :, 2:8] = ONE, -ONE, c[None, :, None]
    wd = torch.rand(n, D, F, generator=torch.Generator().manual_seed(1)) + 0.5
    logits = torch.randn(T, n, generator=torch.Generator().manual_seed(T))
    y, ids, w = _call(x.to(DT[dt]), logits, (wg, wu, wd), DT[dt])
    g = 0.75 * a.double()
    h = (g * torch.sigmoid(g) * 6.0 * a.double())[:, None] * c.double()   # codes 224 and 448
    m = R.weights_f64(*R.quant_weights(wd))
    ref = sum(w[:, j, None] * torch.einsum("tf,tdf->td", h, m[ids[:, j]]) for j in range(2))
    # every term positive: silu 16 u, the block's scale and codes 2, the sums 131
    # and two products, the weights 1e-6, the sum of the pairs 4; for a 16-bit
    # output the down product may drop 7 2^-13 of eight products' largest, and
    # y is rounded once
    tol = 1e-6 + 160 * R.U + 7 * 2.0 ** -13 + R.half_step(DT[dt])
    assert bool(((y - ref).abs() <= tol * ref).all()), float(((y - ref).abs() / ref).max())
