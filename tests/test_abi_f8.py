"""
Refusals of the 8-bit and norm entry points, on the host before any launch:
the C ABI with made-up pointers that no call may reach, and the binding with
CPU tensors.
"""

import ctypes

import pytest
import torch

import mixture_experts_routed_route_amd as moe

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    return moe.library()


def _quant(lib, x=0x1000, dt=moe.MOE_BF16, rows=4, K=128, q=0x2000, s=0x3000):
    return lib.moe_quant_f8(x, dt, rows, K, q, s, None)


def _quant_w(lib, w=0x1000, dt=moe.MOE_BF16, mats=2, N=64, K=128, q=0x2000, s=0x3000):
    return lib.moe_quant_f8_weights(w, dt, mats, N, K, q, s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=moe.MOE_F8B128), moe.MOE_EUNSUPPORTED), (dict(dt=moe.MOE_Q4B32), moe.MOE_EUNSUPPORTED),
    (dict(K=0), moe.MOE_EINVAL), (dict(K=12), moe.MOE_EINVAL), (dict(x=None), moe.MOE_EINVAL),
    (dict(x=0x1008), moe.MOE_EINVAL), (dict(q=0x2004), moe.MOE_EINVAL), (dict(s=None), moe.MOE_EINVAL),
    (dict(s=0x3004), moe.MOE_EINVAL)])
def test_quantisers_refuse(lib, kw, want):
    assert _quant(lib, **kw) == want and moe.moe_last_error()
    if "x" in kw:
        kw = dict(w=kw["x"])
    assert _quant_w(lib, **kw) == want


def test_quantiser_sizes(lib):
    assert _quant(lib, rows=-1) == moe.MOE_EINVAL
    assert _quant(lib, rows=1 << 31) == moe.MOE_EUNSUPPORTED
    assert _quant(lib, rows=1 << 30, K=512) == moe.MOE_EUNSUPPORTED
    assert _quant(lib, x=None, q=None, s=None, rows=0) == moe.MOE_OK
    assert _quant_w(lib, mats=-1) == moe.MOE_EINVAL
    assert _quant_w(lib, N=-1) == moe.MOE_EINVAL
    assert _quant_w(lib, mats=1 << 40) == moe.MOE_EUNSUPPORTED
    assert _quant_w(lib, w=None, q=None, s=None, mats=0) == moe.MOE_OK
    assert _quant_w(lib, w=None, q=None, s=None, N=0) == moe.MOE_OK


def _gemm(lib, x=0x1000, xs=0x2000, w=0x3000, ws=0x4000, M=4, N=64, K=128, out=0x5000,
          odt=moe.MOE_BF16):
    return lib.moe_gemm_f8(x, xs, w, ws, M, N, K, out, odt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(odt=moe.MOE_F8B128), moe.MOE_EUNSUPPORTED), (dict(M=-1), moe.MOE_EINVAL),
    (dict(N=-1), moe.MOE_EINVAL), (dict(K=0), moe.MOE_EINVAL), (dict(K=136), moe.MOE_EINVAL),
    (dict(M=1 << 31), moe.MOE_EUNSUPPORTED), (dict(x=None), moe.MOE_EINVAL),
    (dict(xs=None), moe.MOE_EINVAL), (dict(w=None), moe.MOE_EINVAL), (dict(ws=None), moe.MOE_EINVAL),
    (dict(out=None), moe.MOE_EINVAL), (dict(x=0x1008), moe.MOE_EINVAL), (dict(xs=0x2004), moe.MOE_EINVAL),
    (dict(w=0x3001), moe.MOE_EINVAL), (dict(ws=0x4008), moe.MOE_EINVAL), (dict(out=0x5002), moe.MOE_EINVAL),
    (dict(K=(1 << 22) + 16), moe.MOE_EINVAL)])
def test_product_refuses(lib, kw, want):
    assert _gemm(lib, **kw) == want and moe.moe_last_error()


def test_product_empty(lib):
    assert _gemm(lib, M=0, x=None, xs=None, out=None) == moe.MOE_OK
    assert _gemm(lib, N=0, w=None, ws=None, out=None) == moe.MOE_OK


def _desc(**kw):
    d = dict(T=4, D=64, residual_dtype=moe.MOE_F32, block_dtype=moe.MOE_BF16, x_dtype=moe.MOE_BF16,
             weight_dtype=moe.MOE_BF16, gate_dtype=moe.MOE_F32, gate_kind=0, flags=0, alpha=1.0, eps=1e-6)
    d.update(kw)
    return moe.NormDesc(*(d[n] for n, _ in moe.NormDesc._fields_))


def _norm(lib, d, r=0x1000, u=0x2000, p=0x3000, g=None, w=0x4000, ro=0x5000, x=0x6000, xs=None):
    return lib.moe_norm_forward(ctypes.byref(d) if d else None, r, u, p, g, w, ro, x, xs, None)


def _back(lib, d, r=0x1000, u=0x2000, p=0x3000, g=None, w=0x4000, dro=0x5000, dx=0x6000, dr=0x7000,
          du=0x8000, dp=0x9000, dg=None, dw=0xA000, work=0x10000, nbytes=1 << 40):
    return lib.moe_norm_backward(ctypes.byref(d) if d else None, r, u, p, g, w, dro, dx, dr, du, dp, dg,
                                 dw, work, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), moe.MOE_EINVAL), (dict(D=0), moe.MOE_EINVAL), (dict(D=12), moe.MOE_EINVAL),
    (dict(D=moe.MOE_NORM_MAX_D + 8), moe.MOE_EUNSUPPORTED), (dict(residual_dtype=9), moe.MOE_EUNSUPPORTED),
    (dict(block_dtype=moe.MOE_Q4B32), moe.MOE_EUNSUPPORTED), (dict(weight_dtype=-1), moe.MOE_EUNSUPPORTED),
    (dict(gate_dtype=moe.MOE_F8B128), moe.MOE_EUNSUPPORTED), (dict(x_dtype=moe.MOE_Q4A64), moe.MOE_EUNSUPPORTED),
    (dict(gate_kind=3), moe.MOE_EINVAL), (dict(gate_kind=-1), moe.MOE_EINVAL), (dict(flags=2), moe.MOE_EINVAL),
    (dict(alpha=float("nan")), moe.MOE_EINVAL), (dict(eps=-1e-6), moe.MOE_EINVAL),
    (dict(eps=float("inf")), moe.MOE_EINVAL)])
def test_norm_desc_refused(lib, kw, want):
    d = _desc(**kw)
    assert _norm(lib, d) == want
    assert _back(lib, d) == want
    assert lib.moe_norm_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_norm_pointers_refused(lib):
    E = moe.MOE_EINVAL
    assert _norm(lib, None) == E and _back(lib, None) == E
    for kw in (dict(r=None), dict(ro=None), dict(x=None), dict(u=None), dict(u=None, p=None, w=None),
               dict(r=0x1004), dict(u=0x2008), dict(p=0x3002), dict(w=0x4004), dict(ro=0x5008), dict(x=0x6001)):
        assert _norm(lib, _desc(), **kw) == E, kw
    assert _norm(lib, _desc(gate_kind=1)) == E                        # no gate
    assert _norm(lib, _desc(gate_kind=2), u=None, p=None, g=0xB000) == E
    assert _norm(lib, _desc(x_dtype=moe.MOE_F8B128)) == E             # no scales
    assert _norm(lib, _desc(T=0), r=None, u=0x2000, ro=None, x=None) == moe.MOE_OK
    for kw in (dict(r=None), dict(dx=None), dict(dr=None), dict(du=None), dict(dp=None), dict(dw=None),
               dict(u=None), dict(w=None, dro=None), dict(dro=0x5004), dict(dx=0x6008), dict(dr=0x7002),
               dict(du=0x8004), dict(dw=0xA004), dict(work=None), dict(work=0x10080)):
        assert _back(lib, _desc(), **kw) == E, kw
    assert _back(lib, _desc(gate_kind=1), g=0xB000) == E              # no dgate
    assert _back(lib, _desc(x_dtype=moe.MOE_F8B128)) == moe.MOE_EUNSUPPORTED
    need = lib.moe_norm_backward_workspace_bytes(ctypes.byref(_desc()))
    assert need > 0 and need % 256 == 0
    assert _back(lib, _desc(), nbytes=need - 1) == moe.MOE_EWORKSPACE


def test_layer_on_8bit_weights_refused(lib):
    d = moe.PlanDesc(4, 8, 2, 0, 0.0)
    assert lib.moe_plan_workspace_bytes(ctypes.byref(d)) > 0
    w = moe.Weight(moe.MOE_F8B128, 0x1000, 0x2000)
    assert lib.moe_forward(None, 0x1000, moe.MOE_BF16, w, w, w, 128, 128, 0x2000, moe.MOE_F32, 0x10000,
                           1 << 30, None, None) == moe.MOE_EINVAL


class _FakePlan:
    def __init__(self, T, E, k, n_shared=0):
        self.T, self.E, self.k, self.n_shared = T, E, k, n_shared
        self.handle = None


@pytest.mark.parametrize("case", ["codes_shape", "scales_shape", "scales_dtype", "mixed", "experts"])
def test_binding_refuses_8bit_weights(case):
    T, D, F, E = 4, 256, 128, 8
    x = torch.zeros(T, D, dtype=torch.bfloat16)

    def f8(N, K, n=E):
        return (torch.zeros(n, N, K, dtype=F8), torch.zeros(n, -(-N // 128), -(-K // 128)))

    wg, wu, wd = f8(F, D), f8(F, D), f8(D, F)
    if case == "codes_shape":
        wu = (torch.zeros(E, F, D + 16, dtype=F8), wu[1])
    elif case == "scales_shape":
        wd = (wd[0], torch.zeros(E, 2, 2))
    elif case == "scales_dtype":
        wg = (wg[0], wg[1].half())
    elif case == "mixed":
        wd = torch.zeros(E, D, F, dtype=torch.bfloat16)
    else:
        wu = f8(F, D, E - 1)
    with pytest.raises(ValueError):
        moe.moe_forward(_FakePlan(T, E, 2), x, wg, wu, wd)
    with pytest.raises(ValueError):
        moe.moe_backward(_FakePlan(T, E, 2), x, f8(F, D), f8(F, D), f8(D, F), torch.zeros(T, D))


def test_binding_refuses_tensors():
    z = torch.zeros
    for bad in (z(4, 12), z(4, 64, dtype=torch.float64), z(4, 64)):     # K, type, on the CPU
        with pytest.raises(ValueError):
            moe.moe_quant_f8(bad)
        with pytest.raises(ValueError):
            moe.moe_quant_f8_weights(bad)
    with pytest.raises(ValueError):
        moe.moe_quant_f8_weights(z(64))
    a, s = z(4, 256, dtype=F8), z(4, 2)
    w, ws = z(130, 256, dtype=F8), z(2, 2)
    for x, y in (((a, z(4, 3)), (w, ws)), ((a, s), (w, z(1, 2))), ((a, s), (w[:, :128], ws)),
                 ((a.float(), s), (w, ws)), ((a, s.half()), (w, ws)), ((a, s), (w[None], ws[None])),
                 ((a[:, :24], s[:, :1]), (w[:, :24], ws[:, :1])), ((a, s), (w, ws))):
        with pytest.raises(ValueError):
            moe.moe_gemm_f8(x, y)
    r, u, v = z(4, 64), z(4, 64, dtype=torch.bfloat16), torch.ones(64)
    for kw in (dict(residual=z(4, 64, dtype=torch.int32), weight=v), dict(residual=z(64), weight=v),
               dict(residual=z(4, 20), weight=torch.ones(20)), dict(residual=r), dict(residual=r, block=u[:3], weight=v),
               dict(residual=r, block=u, weight=v[:32]), dict(residual=r, block=u, weight=v, post_weight=v.half()),
               dict(residual=r, block=u, weight=v, gate=z(4)), dict(residual=r, post_weight=v, weight=v),
               dict(residual=r, weight=v, gate=v), dict(residual=r, block=u, weight=v, x_dtype=torch.int8),
               dict(residual=r, block=u, weight=v)):
        with pytest.raises(ValueError):
            moe.moe_norm(**kw)
    for args, kw in (((r, u, None), dict(weight=v)), ((r, u, r), dict()), ((r, u, r[:2]), dict(weight=v)),
                     ((r, u, r, u), dict(weight=v)), ((r, u, r, r), dict(weight=v))):
        with pytest.raises(ValueError):
            moe.moe_norm_backward(*args, **kw)


def test_binding_refuses_sizes_past_an_int():
    """Sizes of 2^31 and more, which the C call would read modulo 2^32."""
    n = 2 ** 31
    wide = torch.zeros(1).expand(1, n + 16)
    tall = torch.zeros(8).expand(n, 8)
    for call in (lambda: moe.moe_quant_f8(wide), lambda: moe.moe_quant_f8_weights(wide),
                 lambda: moe.moe_quant_f8_weights(tall), lambda: moe.moe_norm(tall, weight=torch.ones(8)),
                 lambda: moe.moe_norm_backward(tall, None, tall, weight=torch.ones(8))):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()
    q, s = torch.zeros(1, dtype=F8), torch.zeros(1)
    a, sa = q.expand(4, 2 ** 32 + 16), s.expand(4, 2 ** 25 + 1)
    w, sw = q.expand(2, 2 ** 32 + 16), s.expand(1, 2 ** 25 + 1)
    with pytest.raises(ValueError, match="below 2\\^31"):
        moe.moe_gemm_f8((a, sa), (w, sw))
    with pytest.raises(ValueError, match="below 2\\^31"):
        moe.moe_gemm_f8((q.expand(4, 16), s.expand(4, 1)), (q.expand(n, 16), s.expand(2 ** 24, 1)))


def test_constants_match_the_header():
    import os
    import re
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "moe.h")).read()
    defs = dict(re.findall(r"#define\s+(MOE_\w+)\s+\(?(-?\d+)\)?\s*(?:/\*.*)?$", hdr, re.M))
    for name in ("MOE_GATE_NONE", "MOE_GATE_CHANNEL", "MOE_GATE_TOKEN", "MOE_NORM_UNIT_OFFSET",
                 "MOE_NORM_MAX_D"):
        assert getattr(moe, name) == int(defs[name]), name
    assert re.search(r"MOE_F8B128 = (\d+)", hdr).group(1) == str(moe.MOE_F8B128)
