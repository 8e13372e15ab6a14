"""
The norms around a block on the GPU against f64, forward and backward, at
every row shape of the kernels, and one layer step of all the operators that
meet there.
"""

import pytest
import torch

import f8_ref as R
import mixture_experts_routed_route_amd as moe

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _inputs(T, D, res, blk, par, post, gate, unit, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shift = 0.0 if unit else 1.0
    v = dict(r=(rn(T, D) * torch.exp(rn(T, 1))).to(DT[res]), u=rn(T, D).to(DT[blk]),
             w=(shift + 0.2 * rn(D)).to(DT[par]), p=None, g=None)
    if post:
        v["p"] = (shift + 0.2 * rn(D)).to(DT[par])
    if gate == "channel":
        v["g"] = rn(D).to(DT[par])
    elif gate == "token":
        v["g"] = rn(T, 1).to(DT[par])
    v["dx"] = rn(T, D)
    v["dr"] = rn(T, D).to(DT[res])
    return v


def _f64(v, *names):
    return [None if v[n] is None else v[n].double() for n in names]


def _dev(t):
    return None if t is None else t.cuda()


SHAPES = [(1, 8), (5, 72), (3, 512), (130, 520), (9, 1024), (700, 1032), (33, 2048), (7, 2056),
          (65, 4096), (3, 4104), (11, 8192), (2, 8200), (4, 16384)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("res,blk,x,par,post,gate,unit", [
    ("f32", "f32", "f32", "f32", True, "channel", False),
    ("f32", "bf16", "bf16", "bf16", True, "token", True),
    ("bf16", "bf16", "bf16", "f32", False, "channel", False),
    ("f16", "f32", "f16", "f16", True, "none", True)])
def test_forward_against_f64(T, D, res, blk, x, par, post, gate, unit):
    v = _inputs(T, D, res, blk, par, post, gate, unit, seed=T + D)
    got_r, got_x = moe.moe_norm(*(_dev(v[n]) for n in ("r", "u", "w", "p", "g")), alpha=0.7,
                                eps=1e-5, unit_offset=unit, x_dtype=DT[x])
    r, xx, er, ex = R.norm(*_f64(v, "r", "u", "w", "p", "g"), 0.7, 1e-5, unit)
    assert got_r.dtype == DT[res] and got_x.dtype == DT[x]
    for got, ref, e in ((got_r, r, er), (got_x, xx, ex)):
        b = e + R.half_step(got.dtype) * (ref.abs() + e) + R.smallest(got.dtype)
        err = (got.cpu().double() - ref).abs()
        assert bool((err <= b).all()), float((err / b).max())


@pytest.mark.parametrize("T,D", [(1, 8), (4, 136), (3, 1000), (50, 2048), (9, 4224), (2, 16384)])
def test_forward_quantised(T, D):
    v = _inputs(T, D, "f32", "bf16", "bf16", True, "channel", False, seed=D)
    args = [_dev(v[n]) for n in ("r", "u", "w", "p", "g")]
    out, (q, s) = moe.moe_norm(*args, alpha=0.7, x_dtype=R.F8)
    out2, x = moe.moe_norm(*args, alpha=0.7, x_dtype=torch.float32)
    assert torch.equal(out, out2)
    # the codes and scales of the f32 row the same kernel writes
    rq, rs = R.quant_rows(x.cpu())
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu().float(), rq.float())


def test_forward_parts_and_in_place():
    v = _inputs(37, 640, "f32", "bf16", "bf16", True, "none", False, seed=2)
    r, u, w, p = (_dev(v[n]) for n in ("r", "u", "w", "p"))
    out, x = moe.moe_norm(r, weight=w)                       # before the first block
    assert out is r
    _, ref, _, e = R.norm(*_f64(v, "r"), None, *_f64(v, "w"), None, None, 1.0, 1e-6, False)
    b = e + R.half_step(x.dtype) * (ref.abs() + e)
    assert bool(((x.cpu().double() - ref).abs() <= b).all())
    out, x = moe.moe_norm(r, u, post_weight=p)               # after the last one
    assert x is None
    ref, _, e, _ = R.norm(*_f64(v, "r", "u"), None, *_f64(v, "p"), None, 1.0, 1e-6, False)
    b = e + R.half_step(torch.float32) * (ref.abs() + e)
    assert bool(((out.cpu().double() - ref).abs() <= b).all())
    # the C entry in place: residual_out over residual
    import ctypes
    d = moe.NormDesc(37, 640, moe.MOE_F32, moe.MOE_BF16, moe.MOE_BF16, moe.MOE_BF16, moe.MOE_F32,
                     0, 0, 1.0, 1e-6)
    x1 = torch.empty(37, 640, dtype=torch.bfloat16, device="cuda")
    full, x2 = moe.moe_norm(r, u, w, p)
    st = moe.library().moe_norm_forward(
        ctypes.byref(d), r.data_ptr(), u.data_ptr(), p.data_ptr(), None, w.data_ptr(),
        r.data_ptr(), x1.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert st == moe.MOE_OK and torch.equal(r, full) and torch.equal(x1, x2)


def test_forward_of_a_view():
    """A residual that is a view at an odd offset, without a block: it comes
    back as it is."""
    base = torch.randn(6, 72, device="cuda")
    r = base[::2, 3:67]
    w = torch.ones(64, device="cuda")
    out, x = moe.moe_norm(r, weight=w, x_dtype=torch.float32)
    assert out is r
    assert torch.equal(x, moe.moe_norm(r.clone(), weight=w, x_dtype=torch.float32)[1])


def test_forward_many_rows():
    """More workgroups than a launch holds along one axis (2^32 threads)."""
    T = (1 << 26) + 5
    r = torch.full((T, 8), 2.0, dtype=torch.bfloat16, device="cuda")
    r[-1] = -4.0
    out, x = moe.moe_norm(r, r, weight=torch.full((8,), 3.0, dtype=torch.bfloat16, device="cuda"), eps=0.0)
    assert bool((out[:-1] == 4.0).all()) and bool((out[-1] == -8.0).all())
    assert bool((x[:-1] == 3.0).all()) and bool((x[-1] == -3.0).all())


def test_forward_special_rows():
    """A row of zeros norms to zeros; NaN and infinities stay in their rows."""
    v = _inputs(6, 256, "f32", "f32", "f32", True, "none", False, seed=5)
    ref, xref = moe.moe_norm(*(_dev(v[n]) for n in ("r", "u", "w", "p")))
    v["r"][1] = 0.0
    v["u"][1] = 0.0
    v["u"][2, 7] = float("nan")
    v["r"][4, 9] = float("inf")
    out, x = moe.moe_norm(*(_dev(v[n]) for n in ("r", "u", "w", "p")))
    assert bool((out[1] == 0).all()) and bool((x[1] == 0).all())
    assert torch.isnan(x[2]).all() and torch.isnan(x[4, 9])
    for i in (0, 3, 5):
        assert torch.equal(out[i], ref[i]) and torch.equal(x[i], xref[i])
    empty = torch.empty(0, 64, device="cuda")
    out, x = moe.moe_norm(empty, empty, torch.ones(64, device="cuda"))
    assert out.shape == (0, 64) and x.shape == (0, 64)


def _grads(v, unit, dxt, dr=True):
    return moe.moe_norm_backward(_dev(v["r"]), _dev(v["u"]), _dev(v["dx"].to(dxt)),
                                 _dev(v["dr"]) if dr else None, _dev(v["w"]), _dev(v["p"]),
                                 _dev(v["g"]), alpha=0.7, eps=1e-5, unit_offset=unit)


def _grad_bounds(v, ref, unit, T, D):
    """Bounds for each gradient: the terms of its formula in absolute value
    times the roundings that may meet. Rows: under 64 roundings a value of
    each term (two sums over the row, the inverse norms, the products).
    Columns: each of T rows' terms has that relative error and is added at
    most T + 64 times in any order the partial sums take."""
    one = 1.0 if unit else 0.0
    r, u, w, p, g, dr, dx = _f64(v, "r", "u", "w", "p", "g", "dr", "dx")
    C = 160 * R.U
    inv = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-5)
    n = r * inv
    t = (dx * (w + one)).abs()
    ad = dr.abs() + inv * (t + n.abs() * (t * n.abs()).mean(1, keepdim=True))
    got = {"dresidual": C * ad}
    col = lambda terms: (C + (T + 64) * R.U) * terms.sum(0)  # noqa: E731
    got["dweight"] = col((dx * n).abs())
    vu, ap, inv_u = u.abs(), torch.ones(D, dtype=torch.float64), 1.0
    if p is not None:
        inv_u = 1 / torch.sqrt(u.square().mean(1, keepdim=True) + 1e-5)
        vu, ap = (u * inv_u).abs(), (p + one).abs()
    ag = g.abs() if g is not None else 1.0
    adz = 0.7 * ag * ad
    got["dblock"] = C * adz
    if p is not None:
        tp = adz * ap
        got["dblock"] = C * inv_u * (tp + vu * (tp * vu).mean(1, keepdim=True))
        got["dpost_weight"] = col(adz * vu)
    if g is not None:
        terms = 0.7 * ad * vu * ap
        got["dgate"] = col(terms) if g.dim() == 1 else C * terms.sum(1, keepdim=True)
    return got


@pytest.mark.parametrize("T,D", SHAPES + [(1500, 256), (1100, 1536)])
@pytest.mark.parametrize("res,blk,dxt,par,post,gate,unit", [
    ("f32", "f32", "f32", "f32", True, "channel", False),
    ("f32", "bf16", "bf16", "bf16", True, "token", True),
    ("bf16", "bf16", "f32", "f32", False, "channel", False),
    ("f16", "f16", "f16", "f32", True, "none", True)])
def test_backward_against_f64(T, D, res, blk, dxt, par, post, gate, unit):
    v = _inputs(T, D, res, blk, par, post, gate, unit, seed=T + D + 1)
    v["dx"] = v["dx"].to(DT[dxt]).float()
    got = _grads(v, unit, DT[dxt])
    ref = R.norm_grads(*_f64(v, "r", "u", "w", "p", "g", "dr", "dx"), 0.7, 1e-5, unit)
    bounds = _grad_bounds(v, ref, unit, T, D)
    assert set(got) == set(ref)
    for name, g in got.items():
        want = {"dresidual": DT[res], "dblock": DT[blk]}.get(name, torch.float32)
        assert g.dtype == want and g.shape == ref[name].shape, name
        b = bounds[name] + R.half_step(want) * (ref[name].abs() + bounds[name]) + R.smallest(want)
        err = (g.cpu().double() - ref[name]).abs()
        assert bool((err <= b).all()), (name, float((err / b).max()))


def test_backward_against_differences():
    """Central differences of the f32 forward, along random directions."""
    v = _inputs(6, 264, "f32", "f32", "f32", True, "channel", False, seed=11)
    dev = {n: _dev(t) for n, t in v.items()}

    def forward(t):
        out, x = moe.moe_norm(t["r"], t["u"], t["w"], t["p"], t["g"], alpha=0.7, eps=1e-5,
                              x_dtype=torch.float32)
        return (out.double() * dev["dr"].double()).sum() + (x.double() * dev["dx"].double()).sum(), out

    _, out = forward(dev)
    got = moe.moe_norm_backward(out, dev["u"], dev["dx"], dev["dr"], dev["w"], dev["p"], dev["g"],
                                alpha=0.7, eps=1e-5)
    step = 2.0 ** -7
    for n, name in (("r", "dresidual"), ("u", "dblock"), ("w", "dweight"), ("p", "dpost_weight"),
                    ("g", "dgate")):
        d = torch.randn(dev[n].shape, generator=torch.Generator().manual_seed(3)).cuda()
        hi, _ = forward(dict(dev, **{n: dev[n] + step * d}))
        lo, _ = forward(dict(dev, **{n: dev[n] - step * d}))
        slope = float(hi - lo) / (2 * step)
        want = float((got[name].double() * d.double()).sum())
        # step^2 curvature terms against the gradient's own norm
        size = float(got[name].double().norm() * d.double().norm())
        assert abs(slope - want) <= 4 * step * step * size + 1e-3 * size / 16, (name, slope, want)


def test_backward_parts_and_determinism():
    v = _inputs(300, 520, "f32", "bf16", "bf16", True, "channel", False, seed=4)
    a, b = _grads(v, False, torch.bfloat16), _grads(v, False, torch.bfloat16)
    assert all(torch.equal(a[n], b[n]) for n in a)
    r, u, w, dx = (_dev(v[n]) for n in ("r", "u", "w", "dx"))
    only = moe.moe_norm_backward(r, None, dx, weight=w, eps=1e-5)      # before the first block
    assert set(only) == {"dresidual", "dweight"}
    ref = R.norm_grads(*_f64(v, "r"), None, *_f64(v, "w"), None, None, None, *_f64(v, "dx"), 1.0, 1e-5, False)
    for n in only:
        e = (only[n].cpu().double() - ref[n]).norm() / ref[n].norm()
        assert float(e) < 1e-5, n     # sums of 300 rows: under 400 u in the norm
    last = moe.moe_norm_backward(r, u, None, _dev(v["dr"]), post_weight=_dev(v["p"]))
    assert set(last) == {"dresidual", "dblock", "dpost_weight"}
    assert torch.equal(last["dresidual"], _dev(v["dr"]))
    none = moe.moe_norm_backward(torch.empty(0, 64, device="cuda"), None,
                                 torch.empty(0, 64, device="cuda"), weight=torch.ones(64, device="cuda"))
    assert none["dresidual"].shape == (0, 64) and bool((none["dweight"] == 0).all())


@pytest.mark.parametrize("par", ["bf16", "f16", "f32"])
def test_backward_token_gate_to_the_last_byte(par):
    """A gate a token whose values end where the tensor's pages do: each
    token's own value, none read past the last."""
    T, D = 1 << 20, 8
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[par]
    u = torch.ones(T, D, device="cuda")
    gate = (torch.arange(T, device="cuda") % 251 + 1).to(dt)[:, None]
    out = moe.moe_norm_backward(u, u, None, u, gate=gate, alpha=0.5)
    assert torch.equal(out["dblock"], 0.5 * gate.float().expand(T, D))
    assert torch.equal(out["dgate"], torch.full_like(gate, 4.0, dtype=torch.float32))


def test_layer_step_together():
    """Norm, router, experts on 8-bit weights, norm with the next
    projection's quantised rows, product; then captured and replayed."""
    T, D, F, E, k = 96, 256, 128, 8, 2
    g = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = torch.bfloat16
    r, wr = rn(T, D).cuda(), (rn(E, D) * D ** -0.5).to(bf).cuda()
    w1, w2, p, gate = ((1 + 0.1 * rn(D)).to(bf).cuda() for _ in range(4))
    weights = [moe.moe_quant_f8_weights((rn(E, *s) * s[1] ** -0.5).to(bf).cuda())
               for s in ((F, D), (F, D), (D, F))]
    proj = moe.moe_quant_f8_weights((rn(320, D) * D ** -0.5).to(bf).cuda())

    def step():
        _, x = moe.moe_norm(r, weight=w1)
        plan, _, _ = moe.moe_route(x, wr, k)
        y = moe.moe_forward(plan, x, *weights)
        r2, xq = moe.moe_norm(r, y, w2, p, gate, alpha=0.5, x_dtype=R.F8)
        return plan, x, y, r2, xq, moe.moe_gemm_f8(xq, proj)

    plan, x, y, r2, xq, z = step()
    v = moe.moe_plan_get_views(plan)
    cpu = lambda t: tuple(a.cpu() for a in t)  # noqa: E731
    ref_y, ey = R.layer(x.cpu(), *(cpu(t) for t in weights), v["topk_id"].cpu().long(), v["topk_w"].cpu(),
                        v["tok2pair"].cpu() >= 0, E, 0, 7.0, torch.float32, torch.float32)
    assert bool(((y.cpu().double() - ref_y).abs() <= ey).all())
    ref_r, ref_x, er, ex = R.norm(r.cpu().double(), y.cpu().double(), w2.cpu().double(), p.cpu().double(),
                                  gate.cpu().double(), 0.5, 1e-6, False)
    assert bool(((r2.cpu().double() - ref_r).abs() <= er + 2 * R.U * ref_r.abs()).all())
    deq = R.rows_f64(*cpu(xq))
    step8 = xq[1].cpu().double().repeat_interleave(128, 1)
    assert bool(((deq - ref_x).abs() <= R.half_step(R.F8) * (ref_x.abs() + ex) + step8 * 2.0 ** -10 + 2 * ex).all())
    wf = R.weights_f64(*cpu(proj))
    ref_z = deq @ wf.t()
    assert bool(((z.cpu().double() - ref_z).abs() <= R.product_bound(deq, wf, bf, ref_z, units8=True)).all())

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(3):
        r.copy_(torch.randn(T, D, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        rz, rr = kept[5].clone(), kept[3].clone()
        eager = step()
        assert torch.equal(rz, eager[5]) and torch.equal(rr, eager[3])
