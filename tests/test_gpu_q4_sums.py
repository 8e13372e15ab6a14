"""Sums of products on 4-bit weights: exact on whole numbers as long as 40 times the
sum of a group's x fits 24 bits, close on rows of one sign, and independent of x's
power of two."""

import math

import pytest
import torch

import mixture_experts_routed_route_amd as moe
from helpers import say
from q4_ref import DT, FORMATS, GROUP, U, codes, half_step, random_weights, rel, values

pytestmark = pytest.mark.gpu

# few rows; slices; tiles (above 768 slices of 64 x 64)
SHAPES = [(1, 100), (5, 48), (16, 77), (20, 64), (100, 130), (300, 1000), (900, 4000)]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_whole_numbers_are_exact(M, N, fmt, xdt):
    """Positive whole numbers x up to 13312, half of them small and odd: a group's sum of (24 + q) x stays below
    31 * 32 * 13312 < 2^24, and so do all others (K of 64, scales of 1, biases of -8)."""
    K, G = 64, GROUP[fmt]
    say(f"whole numbers {M} x {N} {fmt} {xdt}")
    g = torch.Generator().manual_seed(M)
    unit, odd = (8, 2048) if xdt == "f16" else (64, 256)
    small = torch.randint(0, odd // 2, (M, K), generator=g) * 2 + 1
    large = torch.randint(8192 // unit, 13312 // unit + 1, (M, K), generator=g) * unit
    x = torch.where(torch.rand(M, K, generator=g) < 0.5, small, large)
    x16 = x.to(DT[xdt])
    assert torch.equal(x16.long(), x)
    data = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    p = torch.ones(N, K // G, dtype=torch.float16, device="cuda")
    if fmt != "b32":
        p = torch.stack([p, -8 * p], -1)
    ref = torch.matmul(x.double().cuda(), values((data, p), fmt).t().contiguous())
    got = moe.moe_gemm_q4(x16.cuda(), (data, p), out_dtype=torch.float32)
    wrong = got.double() != ref
    say(f"  {int(wrong.sum())} of {wrong.numel()} differ")
    assert not wrong.any()


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_rows_of_one_sign(M, N, fmt, xdt):
    """Rows as a ReLU or a gate leaves them. A step of 32 values adds at most 33 numbers to minus off times the sum S of
    its x, itself a sum of 32, off 24 (signed codes) or 16: partial sums up to off S, falling or rising evenly (a third of
    it in the mean square), each off by at most a step, 2 u (a third of that squared): sqrt(65) 2 / 3 u off S a step, of
    either sign. The scaled sums add u a piece and their number's square root."""
    K = 4096
    say(f"one sign {M} x {N} {fmt} {xdt}")
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).abs().to(DT[xdt]).cuda()
    w = random_weights(g, (N,), K, fmt, "cuda")
    ref = torch.matmul(x.double(), values(w, fmt).t().contiguous())
    got = moe.moe_gemm_q4(x, w, out_dtype=torch.float32)
    off, n = (24.0 if fmt == "b32" else 16.0), K // 32
    s = w[1].double() if fmt == "b32" else w[1][..., 0].double()
    s = s.repeat_interleave(n // s.shape[1], 1)
    S = x.double().view(M, n, 32).sum(2)
    per = torch.matmul(S.square(), s.square().t().contiguous()).mean().sqrt()
    terms = torch.matmul(x.double().square(), values(w, fmt).square().t().contiguous()).mean().sqrt()
    rms = ref.square().mean().sqrt()
    tol = ((math.sqrt(65) * 2 / 3 * off * per + math.sqrt(4 * n) * torch.maximum(rms, terms)) / rms).item() * U
    err = rel(got, ref)
    say(f"  error {err:.2e} of {tol:.2e}")
    assert err <= tol + half_step(torch.float32)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("M,N", SHAPES)
def test_powers_of_two(M, N, fmt):
    """bf16 rows times 2^108: sums of a group of 64 stay below 2^120, and nothing but the exponent changes."""
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()
    w = random_weights(g, (N,), 256, fmt, "cuda")
    a = moe.moe_gemm_q4(x, w, out_dtype=torch.float32)
    b = moe.moe_gemm_q4(x * 2.0 ** 108, w, out_dtype=torch.float32)
    assert b.isfinite().all() and torch.equal(a * 2.0 ** 108, b)
