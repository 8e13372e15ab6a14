"""
Views and empty batches in the 8-bit and norm calls: tensors that start off a
16-byte boundary, as slices of rows, experts, tokens and flat parameter buffers
do, give what their copies give; no rows give empty rows and zero sums.
"""

import pytest
import torch

import f8_ref as R
import mixture_experts_routed_route_amd as moe

pytestmark = pytest.mark.gpu


def _off(t):
    """The same values in a view that starts one element into its storage."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    flat[1:] = t.cuda().flatten()
    v = flat[1:].view(t.shape)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


def _randn(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed))


def test_product_of_slices():
    """23 scales a row of 2880 values, 9 a matrix of 384 x 384."""
    q, s = moe.moe_quant_f8(_randn(9, 2880).cuda())
    w = moe.moe_quant_f8_weights(_randn(100, 2880, seed=1).cuda())
    whole = moe.moe_gemm_f8((q, s), w, out_dtype=torch.float32)
    for i in range(1, 5):
        assert torch.equal(moe.moe_gemm_f8((q[i:], s[i:]), w, out_dtype=torch.float32), whole[i:])
    a = moe.moe_quant_f8(_randn(70, 384, seed=2).cuda())
    stack = moe.moe_quant_f8_weights(_randn(3, 384, 384, seed=3).cuda())
    for i in range(3):
        one = tuple(t[i] for t in stack)
        assert torch.equal(moe.moe_gemm_f8(a, one), moe.moe_gemm_f8(a, tuple(t.clone() for t in one)))


def test_quantisers_of_views():
    for dt in (torch.float32, torch.bfloat16):
        v = _randn(5, 136).to(dt)
        for f in (moe.moe_quant_f8, moe.moe_quant_f8_weights):
            for got, ref in zip(f(_off(v)), f(v.cuda())):
                assert torch.equal(got.float(), ref.float())


def test_layer_on_some_of_the_experts():
    """Experts 1 .. 4 of five: 9 scales a matrix."""
    ws = [moe.moe_quant_f8_weights((0.05 * _randn(5, 384, 384, seed=i)).cuda()) for i in range(3)]
    x, logits = _randn(50, 384).to(torch.bfloat16).cuda(), _randn(50, 4, seed=9).cuda()
    plan = moe.moe_plan_create(logits, 2)
    got = moe.moe_forward(plan, x, *(tuple(t[1:] for t in w) for w in ws))
    assert torch.equal(got, moe.moe_forward(plan, x, *(tuple(t[1:].clone() for t in w) for w in ws)))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_norm_of_views(dt):
    T, D = 21, 264
    v = dict(residual=_randn(T, D), block=_randn(T, D, seed=1), weight=_randn(D, seed=2),
             post_weight=_randn(D, seed=3), gate=_randn(T, 1, seed=4))
    v = {n: t.to(dt).cuda() for n, t in v.items()}
    for views in ({n: _off(t) for n, t in v.items()}, dict(v, gate=_off(v["gate"])), dict(v, weight=_off(v["weight"]))):
        out, x = moe.moe_norm(**v)
        for got, ref in zip(moe.moe_norm(**views), (out, x)):
            assert torch.equal(got, ref)
        dx, dr = _randn(T, D, seed=5).to(dt).cuda(), _randn(T, D, seed=6).to(dt).cuda()
        par = lambda a: {n: a[n] for n in ("weight", "post_weight", "gate")}  # noqa: E731
        ref = moe.moe_norm_backward(out, v["block"], dx, dr, **par(v))
        got = moe.moe_norm_backward(_off(out), views["block"], _off(dx), _off(dr), **par(views))
        assert all(torch.equal(got[n], ref[n]) for n in ref)


def test_norm_of_some_of_the_tokens():
    """Rows t .. of a batch with their gates."""
    r, u, g = _randn(40, 64).cuda(), _randn(40, 64, seed=1).cuda(), _randn(40, 1, seed=2).to(torch.bfloat16).cuda()
    w = torch.ones(64, device="cuda")
    out, x = moe.moe_norm(r, u, w, gate=g)
    for t in (1, 3, 7):
        o2, x2 = moe.moe_norm(r[t:], u[t:], w, gate=g[t:])
        assert torch.equal(o2, out[t:]) and torch.equal(x2, x[t:])
        back = moe.moe_norm_backward(out, u, x, r, w, gate=g)
        part = moe.moe_norm_backward(out[t:], u[t:], x[t:], r[t:], w, gate=g[t:])
        for n in ("dresidual", "dblock", "dgate"):
            assert torch.equal(part[n], back[n][t:]), n


@pytest.mark.parametrize("D", [64, 8200])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_norm_of_no_rows(gate, D):
    rows = lambda: torch.empty(0, D, device="cuda")  # noqa: E731
    one = torch.ones(D, device="cuda")
    g = None if gate is None else one if gate == "channel" else torch.empty(0, 1, device="cuda")
    out, (q, s) = moe.moe_norm(rows(), rows(), one, one, g, x_dtype=R.F8)
    assert out.shape == q.shape == (0, D) and s.shape == (0, -(-D // 128))
    out, x = moe.moe_norm(rows(), rows(), None, one, g)
    assert out.shape == (0, D) and x is None
    got = moe.moe_norm_backward(rows(), rows(), rows(), rows(), one, one, g)
    assert got["dresidual"].shape == got["dblock"].shape == (0, D)
    for n in ("dweight", "dpost_weight") + (("dgate",) if gate == "channel" else ()):
        assert torch.equal(got[n], torch.zeros(D, device="cuda")), n
    assert gate != "token" or got["dgate"].shape == (0, 1)
    got = moe.moe_norm_backward(rows(), rows(), None, rows(), None, one, g)
    assert set(got) == {"dresidual", "dblock", "dpost_weight"} | ({"dgate"} if gate else set())
    assert bool((got["dpost_weight"] == 0).all())
