"""Products of few rows on 4-bit weights where K passes what LDS holds of the rows
(turns of K, in one and in several rounds of strips), rows of an odd number of
scales, and the shortest rows."""

import math

import pytest
import torch

import mixture_experts_routed_route_amd as moe
from helpers import say
from q4_ref import DT, FORMATS, GROUP, product_tolerance, random_weights, rel, values

pytestmark = pytest.mark.gpu

TYPES = [("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")]


def _check(x, w, fmt, out_dtype, columns=None):
    got = moe.moe_gemm_q4(x, w, out_dtype=out_dtype)
    N = w[0].shape[0]
    assert got.shape == (x.shape[0], N) and got.dtype == out_dtype and got.isfinite().all()
    for at in columns or (slice(0, N),):
        part = (w[0][at], w[1][at])
        ref = torch.matmul(x.double(), values(part, fmt).t().contiguous())
        tol = product_tolerance(x, part, fmt, out_dtype)
        assert rel(got[:, at], ref) <= tol, (rel(got[:, at], ref), tol)
        scale = ref.square().mean().sqrt()
        far = (got[:, at].double() - ref).abs() - torch.finfo(out_dtype).eps / 2 * ref.abs()
        assert (far <= 8 * tol * scale + torch.finfo(out_dtype).tiny).all()
    assert torch.equal(got, moe.moe_gemm_q4(x, w, out_dtype=out_dtype))


# turns of K: from 39808 values at 1 row, 15872 at 4, 8576 at 8, 4224 at 16; then odd
# numbers of scales, and rows of one group
SHAPES = [(16, 100, 14336), (8, 64, 14336), (4, 21, 16384), (1, 48, 45056), (9, 5, 4128), (16, 33, 4256), (1, 17, 32),
          (3, 40, 96), (16, 33, 1056), (5, 77, 160), (17, 50, 32), (130, 40, 32), (1, 1, 64), (2, 300, 64)]


@pytest.mark.parametrize("shape,fmt", [(s, f) for s in SHAPES for f in FORMATS if s[2] % GROUP[f] == 0],
                         ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(t))
def test_turns_and_odd_rows(shape, fmt, types):
    M, N, K = shape
    say(f"product {shape} {fmt} {types}")
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randn(M, K, generator=g).to(DT[types[0]]).cuda()
    _check(x, random_weights(g, (N,), K, fmt, "cuda"), fmt, DT[types[1]])


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
def test_turns_in_rounds(fmt, xdt):
    """13 rows of 8192 values by 70000: two turns in each of two rounds of strips, no strip shared."""
    M, N, K, G = 13, 70000, 8192, GROUP[fmt]
    say(f"turns in rounds {fmt} {xdt}")
    g = torch.Generator("cuda").manual_seed(7)
    data = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = 0.005 + 0.015 * torch.rand(N, K // G, device="cuda", generator=g)
    params = s.half() if fmt == "b32" else torch.stack([s, -7.5 * s], -1).half()
    x = torch.randn(M, K, device="cuda", generator=g).to(DT[xdt])
    _check(x, (data, params), fmt, torch.float32, [slice(0, 130), slice(N // 2, N // 2 + 130), slice(N - 130, N)])


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("M", [1, 6, 16])
@pytest.mark.parametrize("K", [160, 4224, 14336])
def test_rows_and_surroundings(fmt, M, K):
    """A NaN stays in its row or column; what lies around the operands is never used; outputs stop at M and N."""
    if K % GROUP[fmt]:
        K += 32
    say(f"surroundings {fmt} {M} {K}")
    g, N = torch.Generator().manual_seed(M + K), 77
    x = torch.randn(M, K, generator=g).half().cuda()
    d, p = random_weights(g, (N,), K, fmt, "cuda")
    clean = moe.moe_gemm_q4(x, (d, p), out_dtype=torch.float32)
    wide = torch.full((M + 16, K), math.nan, dtype=torch.float16, device="cuda")
    wide[8:8 + M] = x
    data = torch.full((N + 40, K // 2), 255, dtype=torch.uint8, device="cuda")
    data[8:8 + N] = d
    params = torch.full((N + 40, *p.shape[1:]), math.nan, dtype=torch.float16, device="cuda")
    params[8:8 + N] = p
    buf = torch.full((M * N + 4096,), 3.5, device="cuda")
    out = buf[1024:1024 + M * N].view(M, N)
    got = moe.moe_gemm_q4(wide[8:8 + M], (data[8:8 + N], params[8:8 + N]), out=out)
    assert got is out and torch.equal(got, clean)
    assert (buf[:1024] == 3.5).all() and (buf[1024 + M * N:] == 3.5).all()
    bad = x.clone()
    bad[M - 1, K - 1] = math.nan
    got = moe.moe_gemm_q4(bad, (d, p), out_dtype=torch.float32)
    assert torch.equal(got[:M - 1], clean[:M - 1]) and got[M - 1].isnan().all()
    p = p.clone()
    p.view(N, -1)[N - 1, -1] = math.nan
    got = moe.moe_gemm_q4(x, (d, p), out_dtype=torch.float32)
    assert torch.equal(got[:, :N - 1], clean[:, :N - 1]) and got[:, N - 1].isnan().all()
