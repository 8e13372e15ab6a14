"""
NaN and infinities in the routed layer: a weight that is one makes every token
of its expert NaN and leaves the others as they are, a row of x that holds one
makes its token NaN, on every route and in every weight format.
"""

import pytest
import torch

import mixture_experts_routed_route_amd as moe
import workloads as W

pytestmark = pytest.mark.gpu

# Four experts of which each token takes two: one-token launches, decode-shaped
# calls, groups of up to 16 rows or split K, the full tiles.
TOKENS = [1, 8, 40, 300]
E, K, D, F = 4, 2, 256, 256


def _layer(T, dtype, w_dtype=None):
    wl = W.make_layer(T, D, F, E, K, dtype, w_dtype=w_dtype, w_std=0.05, seed=T)
    return wl, {n: wl[n] for n in ("w_gate", "w_up", "w_down")}


def _forward(wl, ws, x=None):
    p = moe.moe_plan_create(wl["logits"].cuda(), K)
    y = moe.moe_forward(p, (wl["x"] if x is None else x).cuda(), *(ws[n] for n in ("w_gate", "w_up", "w_down")))
    ids = moe.moe_plan_get_views(p)["topk_id"].cpu()
    return y.cpu(), ids


def _expect(y, clean, bad):
    """Rows `bad` are NaN throughout, the others the clean run's."""
    assert bool(bad.any())
    assert bool(torch.isnan(y[bad]).all())
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("which", ["w_gate", "w_up", "w_down"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T", TOKENS)
def test_8bit_weight(T, dt, which, value):
    wl, ws = _layer(T, dt)
    quant = lambda w: moe.moe_quant_f8_weights(w.float().cuda())  # noqa: E731
    good = {n: quant(w) for n, w in ws.items()}
    clean, ids = _forward(wl, good)
    assert bool(torch.isfinite(clean).all())
    e = int(ids[0, 0])
    w = ws[which].float().clone()
    w[e, 130, 140] = float(value)
    y, _ = _forward(wl, dict(good, **{which: quant(w)}))
    bad = (ids == e).any(1)
    if which != "w_down":
        _expect(y, clean, bad)
    else:   # the block's own columns
        _expect(y[:, 128:], clean[:, 128:], bad)
        assert torch.equal(y[:, :128], clean[:, :128])


@pytest.mark.parametrize("dt,wdt", [("bf16", "f8"), ("f16", "f8"), ("f32", None), ("bf16", None), ("f16", None),
                                    ("f16", "q4b32"), ("f16", "q4a32"), ("f16", "q4a64")])
@pytest.mark.parametrize("T", TOKENS)
def test_row_of_x(T, dt, wdt):
    wl, ws = _layer(T, dt, None if wdt == "f8" else wdt)
    if wdt == "f8":
        ws = {n: moe.moe_quant_f8_weights(w.float().cuda()) for n, w in ws.items()}
    else:
        ws = {n: tuple(t.cuda() for t in w) if isinstance(w, tuple) else w.cuda() for n, w in ws.items()}
    clean, _ = _forward(wl, ws)
    x = wl["x"].clone()
    bad = torch.zeros(T, dtype=torch.bool)
    for t, v in ((0, "nan"), (T - 1, "nan")):
        x[t, 77] = float(v)
        bad[t] = True
    y, _ = _forward(wl, ws, x)
    _expect(y, clean, bad)


@pytest.mark.parametrize("which", ["w_gate", "w_up"])
@pytest.mark.parametrize("dt,wdt", [("f32", None), ("bf16", None), ("f16", None), ("f16", "q4b32")])
@pytest.mark.parametrize("T", TOKENS)
def test_weight(T, dt, wdt, which):
    wl, ws = _layer(T, dt, wdt)
    dev = lambda w: tuple(t.cuda() for t in w) if isinstance(w, tuple) else w.cuda()  # noqa: E731
    good = {n: dev(w) for n, w in ws.items()}
    clean, ids = _forward(wl, good)
    e = int(ids[0, 0])
    if wdt:
        w = (ws[which][0], ws[which][1].clone())
        w[1][e, 130, 3] = float("nan")
    else:
        w = ws[which].clone()
        w[e, 130, 140] = float("nan")
    y, _ = _forward(wl, dict(good, **{which: dev(w)}))
    _expect(y, clean, (ids == e).any(1))
