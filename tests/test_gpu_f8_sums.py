"""
The sums of the layer on 8-bit weights: products that cancel, whose rest the
8-bit matrix unit would drop, and the layer's error in the norm, on rows of
every route.
"""

import pytest
import torch

import f8_ref as R
import mixture_experts_routed_route_amd as moe
from test_gpu_f8 import DT, _check, _layer, _product, _run

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


@pytest.mark.parametrize("T", [1, 8, 40, 300])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_down_products_that_cancel(dt, T):
    """h's codes are 448, -448 and six of 2, W_down's rows 448, 448 and six
    values c: a pair's output is 12 c times h's scale. y is f32."""
    n, D, F = 2, 256, 128
    x = torch.zeros(T, D)
    x[:, 0] = ONE
    wg, wu, wd = _blocks_of_one(n, F, D), _blocks_of_one(n, F, D), torch.zeros(n, D, F)
    wg[:, :, 0] = 2.0 ** -6           # gate 7
    wu[:, 0, 0], wu[:, 1, 0], wu[:, 2:8, 0] = ONE, -ONE, 2.0
    c = torch.tensor([[1.0, 2.0], [3.0, 0.5]]).repeat(1, D // 2)
    wd[:, :, :2] = ONE
    wd[:, :, 2:8] = c[:, :, None]
    logits = torch.randn(T, n, generator=torch.Generator().manual_seed(T))
    y, ids, w = _call(x.to(DT[dt]), logits, (wg, wu, wd), torch.float32)
    g = torch.tensor(7.0, dtype=torch.float64)
    ref = 12.0 * float(g * torch.sigmoid(g)) * ONE * (w[:, :, None] * c.double()[ids]).sum(1)
    # silu 16 u, the scale 1, two products and sums, the weights 1e-6, the sum
    # of the pairs 4
    tol = 1e-6 + 32 * R.U
    assert bool(((y - ref).abs() <= tol * ref).all()), float(((y - ref).abs() / ref).max())


def _likely(a, w):
    """What f32 sums of a . w^T are off by: n roundings, each uniform up to u
    of a partial sum, which for terms of random sign is about sqrt(sum of
    their squares / 2). Their sum's deviation is u sqrt(n / 6 sum (a w)^2);
    five times that (one of 10^6 such sums is further off)."""
    n = a.shape[1] + 3 * -(-a.shape[1] // 128)
    return 5 * R.U * ((n / 6) * (a.square() @ w.square().t())).sqrt()


def _norm_bound(x, w_gate, w_up, w_down, ids, w, keep, E, n_shared, limit):
    """The f64 layer and, for each token, a bound of its error's norm. Codes of
    h within h's error of a border may move; each counts once, with the norm of
    its column of W_down (all against each value of y would be 20 times as
    much)."""
    T, k = ids.shape
    xq = R.rows_f64(*R.quant_rows(x))
    y, e = torch.zeros(T, x.shape[1], dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    for ex in range(E + n_shared):
        if ex < E:
            t, j = torch.nonzero((ids == ex) & keep, as_tuple=True)
            pw = w[t, j].double()
        else:
            t, pw = torch.arange(T), torch.ones(T, dtype=torch.float64)
        if not t.numel():
            continue
        wg, wu, wd = (R.weights_f64(q[ex], s[ex]) for q, s in (w_gate, w_up, w_down))
        g, u = xq[t] @ wg.t(), xq[t] @ wu.t()
        eg, eu = _likely(xq[t], wg), _likely(xq[t], wu)
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
        h = g * torch.sigmoid(g) * u
        # as in R.expert: |silu'| <= 1.1, the exponential's and products' steps
        eh = 1.1 * u.abs() * eg + (g * torch.sigmoid(g)).abs() * eu + 16 * R.U * h.abs()
        b, eb = (v.view(len(t), -1, 128) for v in (h, eh))
        a = torch.clamp_min(b.abs().amax(-1, keepdim=True), R.TINY)
        val = (b * (448.0 / a)).clamp(-448, 448).to(R.F8).double() * a / 448.0
        lo, hi = R._codes_between(b, eb, a, eb.amax(-1, keepdim=True))
        off = torch.maximum(hi - val, val - lo).clamp_min(0).view_as(h)
        o = val.view_as(h) @ wd.t()
        b = off @ wd.norm(dim=0) + _likely(val.view_as(h), wd).norm(dim=1)
        y.index_add_(0, t, pw[:, None] * o)
        e.index_add_(0, t, pw * (b + (1e-6 + (k + 3) * R.U) * (o.norm(dim=1) + b)))
    return y, e + R.U * y.norm(dim=1)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,D,F,E,k,shared", [
    (1, 512, 256, 8, 2, 1), (8, 512, 256, 8, 2, 0), (40, 512, 256, 16, 2, 0), (300, 512, 256, 4, 2, 1),
    (600, 256, 384, 6, 1, 0)])
def test_error_in_the_norm(dt, T, D, F, E, k, shared):
    """f32 sums throughout: what is left are codes of h beside a border."""
    wl, ws = _layer(T, D, F, E, k, dt, shared, seed=T + D)
    p, y = _run(wl, ws, torch.float32)
    v = moe.moe_plan_get_views(p)
    ref, bound = _norm_bound(wl["x"], ws["w_gate"], ws["w_up"], ws["w_down"], v["topk_id"].cpu().long(),
                             v["topk_w"].cpu(), v["tok2pair"].cpu() >= 0, E, shared, wl["swiglu_limit"])
    err = (y.cpu().double() - ref).norm(dim=1)
    print(f"error {float(err.norm() / ref.norm()):.2e}, bound {float(bound.norm() / ref.norm()):.2e} of y's norm")
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(300, 512, 8208), (130, 257, 16528), (70, 300, 8192)])
def test_product_of_long_rows(M, N, K, out):
    """More than 64 and 128 blocks of K on the tile: its weights' scales are
    loaded again, 64 blocks at a time."""
    got, ref, bound = _product(M, N, K, out, seed=K)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,F", [(8320, 128), (128, 8320)])
def test_layer_of_long_rows(dt, D, F):
    wl, ws = _layer(150, D, F, 2, 2, dt, seed=D)
    _check(wl, ws, torch.float32)
