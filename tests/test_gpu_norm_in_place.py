"""
The norms over their own inputs, as the C entry points allow (x over block,
dresidual over dresidual_out, dblock over block), and the backward captured and
replayed: the bits of separate buffers and of eager calls.
"""

import ctypes

import pytest
import torch

import mixture_experts_routed_route_amd as moe

pytestmark = pytest.mark.gpu

MOE = {torch.float32: moe.MOE_F32, torch.bfloat16: moe.MOE_BF16}
# one turn of the backward's rows and more, its columns whole and in two parts
SHAPES = [(5, 72), (2100, 1000), (600, 4096), (261, 16384)]


def _inputs(T, D, dt):
    g = torch.Generator().manual_seed(T + D)
    rn = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
    return dict(r=rn(T, D), u=rn(T, D), w=rn(D), p=rn(D), g=rn(D), dr=rn(T, D), dx=rn(T, D))


def _desc(T, D, dt):
    n = MOE[dt]
    return ctypes.byref(moe.NormDesc(T, D, n, n, n, n, n, moe.MOE_GATE_CHANNEL, 0, 0.5, 1e-6))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,D", SHAPES)
def test_forward_over_block(T, D, dt):
    v = _inputs(T, D, dt)
    out, x = moe.moe_norm(v["r"], v["u"], v["w"], v["p"], v["g"], alpha=0.5, x_dtype=dt)
    ptr = {n: t.data_ptr() for n, t in v.items()}
    st = moe.library().moe_norm_forward(
        _desc(T, D, dt), ptr["r"], ptr["u"], ptr["p"], ptr["g"], ptr["w"], ptr["r"], ptr["u"], None,
        torch.cuda.current_stream().cuda_stream)
    assert st == moe.MOE_OK and torch.equal(v["r"], out) and torch.equal(v["u"], x)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,D", SHAPES)
def test_backward_over_inputs(T, D, dt):
    v = _inputs(T, D, dt)
    ref = moe.moe_norm_backward(v["r"], v["u"], v["dx"], v["dr"], v["w"], v["p"], v["g"], alpha=0.5)
    L, d = moe.library(), _desc(T, D, dt)
    ws = torch.empty(L.moe_norm_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    dp, dg, dw = (torch.empty(D, device="cuda") for _ in range(3))
    ptr = {n: t.data_ptr() for n, t in v.items()}
    st = L.moe_norm_backward(d, ptr["r"], ptr["u"], ptr["p"], ptr["g"], ptr["w"], ptr["dr"], ptr["dx"],
                             ptr["dr"], ptr["u"], dp.data_ptr(), dg.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                             ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == moe.MOE_OK
    for got, name in ((v["dr"], "dresidual"), (v["u"], "dblock"), (dp, "dpost_weight"), (dg, "dgate"), (dw, "dweight")):
        assert torch.equal(got, ref[name]), name


@pytest.mark.parametrize("T,D", SHAPES)
def test_backward_captured(T, D):
    v = _inputs(T, D, torch.bfloat16)

    def step():
        return moe.moe_norm_backward(v["r"], v["u"], v["dx"], v["dr"], v["w"], v["p"], v["g"], alpha=0.5)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(3):
        for i, n in enumerate(("r", "u", "dx", "dr")):
            g = torch.Generator().manual_seed(10 * seed + i)
            v[n].copy_(torch.randn(T, D, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in kept.items()}
        eager = step()
        assert all(torch.equal(got[n], eager[n]) for n in eager)
