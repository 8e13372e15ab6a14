"""Refusals of the 4-bit quantiser, the product on 4-bit weights and the layer for
a few tokens, on the host before any launch: the C ABI with made-up pointers
that no call may reach, and the binding with CPU tensors."""

import ctypes

import pytest
import torch

import mixture_experts_routed_route_amd as moe

Q4 = (moe.MOE_Q4B32, moe.MOE_Q4A32, moe.MOE_Q4A64)
E, U = moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return moe.library()


def _quant(lib, w=0x1000, dt=moe.MOE_BF16, wdt=moe.MOE_Q4B32, rows=4, K=128, data=0x2000, s=0x3000):
    return lib.moe_quant_q4_weights(w, dt, wdt, rows, K, data, s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=moe.MOE_Q4B32), U), (dict(dt=moe.MOE_F8B128), U), (dict(wdt=moe.MOE_F16), U), (dict(wdt=7), U),
    (dict(K=0), E), (dict(K=48), E), (dict(wdt=moe.MOE_Q4A64, K=96), E), (dict(K=-32), E), (dict(rows=-1), E),
    (dict(w=None), E), (dict(data=None), E), (dict(s=None), E), (dict(w=0x1008), E), (dict(data=0x2004), E),
    (dict(s=0x3002), E), (dict(rows=1 << 36), U)])
def test_quantiser_refuses(lib, kw, want):
    assert _quant(lib, **kw) == want and moe.moe_last_error()


def test_nothing_to_do(lib):
    for f in Q4:
        assert _quant(lib, wdt=f, rows=0, w=None, data=None, s=None) == moe.MOE_OK
        assert _gemm(lib, wdt=f, M=0, x=None, out=None) == moe.MOE_OK
        assert _gemm(lib, wdt=f, N=0, w=None, s=None, out=None) == moe.MOE_OK


def _gemm(lib, x=0x1000, xdt=moe.MOE_F16, wdt=moe.MOE_Q4A32, w=0x2000, s=0x3000, M=4, N=64, K=128, out=0x4000,
          odt=moe.MOE_F32):
    return lib.moe_gemm_q4(x, xdt, moe.Weight(wdt, w, s), M, N, K, out, odt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(wdt=moe.MOE_F16), U), (dict(wdt=moe.MOE_F8B128), U), (dict(xdt=moe.MOE_F32), U), (dict(xdt=moe.MOE_Q4B32), U),
    (dict(odt=moe.MOE_Q4B32), U), (dict(M=-1), E), (dict(N=-1), E), (dict(K=0), E), (dict(K=144), E),
    (dict(wdt=moe.MOE_Q4A64, K=96), E), (dict(K=(1 << 22) + 32), E), (dict(M=1 << 31), U), (dict(N=(1 << 26) + 1), U), (dict(N=2 ** 31 - 1), U),
    (dict(x=None), E), (dict(w=None), E), (dict(s=None), E), (dict(out=None), E), (dict(x=0x1008), E),
    (dict(w=0x2008), E), (dict(s=0x3004), E), (dict(out=0x4002), E)])
def test_product_refuses(lib, kw, want):
    assert _gemm(lib, **kw) == want and moe.moe_last_error()


def _decode(lib, T=4, n_exp=8, k=2, shared=0, cf=0.0, x=0x1000, xdt=moe.MOE_F16, router=None, logits=0x2000,
            wdt=moe.MOE_Q4B32, w=0x3000, s=0x4000, up=None, D=256, F=128, y=0x5000, ydt=moe.MOE_F32, ws=0x10000,
            nbytes=1 << 40, opt=None):
    d = moe.PlanDesc(T, n_exp, k, shared, cf)
    wt = moe.Weight(wdt, w, s)
    return lib.moe_decode(ctypes.byref(d), x, xdt, router, logits, wt, up or wt, wt, D, F, y, ydt, ws, nbytes,
                          opt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), E), (dict(T=17), U), (dict(n_exp=0), E), (dict(n_exp=1025), E), (dict(k=0), E), (dict(k=9), E),
    (dict(shared=2), E), (dict(cf=-1.0), E), (dict(cf=float("nan")), E), (dict(D=0), U), (dict(D=192), U),
    (dict(F=64), U), (dict(D=(1 << 20) + 128), U), (dict(xdt=moe.MOE_F32), U), (dict(xdt=moe.MOE_F32, wdt=moe.MOE_F32), U),
    (dict(wdt=moe.MOE_BF16), U), (dict(wdt=moe.MOE_F8B128), U), (dict(up=moe.Weight(moe.MOE_Q4A32, 0x3000, 0x4000)), E),
    (dict(x=None), E), (dict(logits=None), E), (dict(w=None), E), (dict(s=None), E), (dict(y=None), E), (dict(ws=None), E),
    (dict(x=0x1008), E), (dict(router=0x1004), E), (dict(logits=0x2004), E), (dict(w=0x3008), E), (dict(s=0x4002), E),
    (dict(y=0x5004), E), (dict(ws=0x10080), E), (dict(ydt=moe.MOE_BF16), U)])
def test_decode_refuses(lib, kw, want):
    assert _decode(lib, **kw) == want and moe.moe_last_error()


def test_decode_workspace(lib):
    d = moe.PlanDesc(4, 8, 2, 0, 0.0)
    need = lib.moe_decode_workspace_bytes(ctypes.byref(d), 256, 128, moe.MOE_F16, moe.MOE_Q4B32)
    assert need > 0 and need % 256 == 0
    assert _decode(lib, nbytes=need - 1) == moe.MOE_EWORKSPACE
    assert lib.moe_decode_workspace_bytes(ctypes.byref(d), 200, 128, moe.MOE_F16, moe.MOE_Q4B32) == 0
    assert lib.moe_decode_workspace_bytes(None, 256, 128, moe.MOE_F16, moe.MOE_Q4B32) == 0
    assert moe.moe_decode_workspace_bytes(4, 8, 2, 256, 128, moe.MOE_F16, moe.MOE_Q4B32) == need
    bad = moe.make_options(swiglu_limit=float("nan"))
    assert _decode(lib, opt=ctypes.byref(bad)) == E
    none = moe.PlanDesc(0, 8, 2, 0, 0.0)
    assert lib.moe_decode_workspace_bytes(ctypes.byref(none), 256, 128, moe.MOE_F16, moe.MOE_Q4B32) >= 0
    assert _decode(lib, T=0, x=None, logits=None, y=None) == moe.MOE_OK


def test_header_constant():
    import os
    import re
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "moe.h")).read()
    assert int(re.search(r"#define MOE_DECODE_MAX_T (\d+)", hdr).group(1)) == moe.MOE_DECODE_MAX_T


def test_binding_refuses_tensors():
    z, h, u8 = torch.zeros, torch.float16, torch.uint8
    for w, f in ((z(4, 48), moe.MOE_Q4B32), (z(4, 96), moe.MOE_Q4A64), (z(64), moe.MOE_Q4B32), (z(4, 0), moe.MOE_Q4B32),
                 (z(4, 64, dtype=torch.float64), moe.MOE_Q4B32), (z(4, 64), moe.MOE_F16), (z(4, 64), moe.MOE_Q4B32)):
        with pytest.raises(ValueError):     # the last one is on the CPU
            moe.moe_quant_q4_weights(w, f)
    x, w = z(3, 128, dtype=h), (z(8, 64, dtype=u8), z(8, 4, dtype=h))
    for a, b in ((x.float(), w), (x[:, :64], w), (x, (w[0].to(torch.int8), w[1])), (x, (w[0], w[1].float())),
                 (x, (w[0][None], w[1][None])), (x, (w[0], z(7, 4, dtype=h))), (x, (w[0], z(8, 3, dtype=h))),
                 (z(3, 0, dtype=h), (z(8, 0, dtype=u8), z(8, 0, dtype=h))), (x, w)):
        with pytest.raises(ValueError):
            moe.moe_gemm_q4(a, b)
    with pytest.raises(ValueError):
        moe.moe_gemm_q4(x, w, out=z(3, 9))


def test_binding_refuses_decode():
    z, bf = torch.zeros, torch.bfloat16
    T, D, F, n = 2, 128, 256, 4
    x, lg, rt = z(T, D, dtype=bf), z(T, n), z(n, D, dtype=bf)
    wg, wd = z(n, F, D, dtype=bf), z(n, D, F, dtype=bf)
    for kw in (dict(), dict(logits=lg, w_router=rt), dict(logits=lg.double()), dict(logits=lg[:1]), dict(logits=lg[0]),
               dict(w_router=rt.half()), dict(w_router=rt[:, :64]), dict(logits=lg)):
        with pytest.raises(ValueError):     # the last one is on the CPU
            moe.moe_decode(x, wg, wg, wd, 2, **kw)
    for a in ((x.float(), wg, wg, wd), (x[0], wg, wg, wd), (x, wg[:, :, :64], wg, wd), (x, wg, wg[:3], wd),
              (x, wg, wg, wd[:, :64]), (x, wg, wg.half(), wd)):
        with pytest.raises(ValueError):
            moe.moe_decode(*a, 2, logits=lg)
    with pytest.raises(ValueError):
        moe.moe_decode(x, wg, wg, wd, 2, logits=lg, n_shared=1)
