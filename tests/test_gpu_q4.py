"""The 4-bit quantiser (bit for bit) and products on 4-bit weights against f64,
over formats, types, one row to hundreds, odd widths, K of whole blocks and not,
views, NaN and infinities, long matrices; captured in a graph, on two streams."""

import math

import pytest
import torch

import mixture_experts_routed_route_amd as moe
from helpers import say
from q4_ref import (DT, FORMATS, GROUP, codes, product_tolerance, quantise, random_weights, rel, values)

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(g, M, K, xdt):
    return torch.randn(M, K, generator=g).to(DT[xdt]).cuda()


# ---- quantiser ------------------------------------------------------------------

@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 64), (3, 128), (5, 7, 192), (130, 1088), (1025, 64)])
def test_quantiser_bit_for_bit(fmt, dt, shape):
    say(f"quantise {shape} {dt} to {fmt}")
    g = _gen(sum(shape))
    v = (torch.randn(*shape, generator=g) * torch.exp(torch.randn(*shape[:-1], 1, generator=g))).to(DT[dt])
    data, p = moe.moe_quant_q4_weights(v.cuda(), FORMATS[fmt])
    q, want, _ = quantise(v, fmt)
    assert torch.equal(p.cpu(), want)
    assert torch.equal(codes(data.cpu(), fmt), q)
    got = moe.moe_dequant_weights(data, p)
    assert torch.equal(got.cpu(), values((data.cpu(), p.cpu()), fmt).half())


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_quantiser_edges(fmt, dt):
    """Groups of zeros, of one value, of values whose scale is a subnormal fp16 or none, ties of a code, of a NaN, of
    infinities, and (not in fp16) of values past fp16's range; a group beside is not touched by them."""
    say(f"quantiser edges {dt} {fmt}")
    G, big = GROUP[fmt], 6e5 if dt != "f16" else 6e4
    step = torch.arange(G).float() - G // 2
    rows = [torch.zeros(G), torch.full((G,), -0.75), step * 2.0 ** -27, step * 2.0 ** -40, step / 4.0, step * 0.5 + 0.25,
            torch.where(step == 3, math.nan, step), torch.where(step == 3, math.inf, step),
            torch.where(step == 3, -math.inf, step), step * big / G, torch.full((G,), -0.0)]
    v = torch.stack(rows).to(DT[dt])
    v = torch.cat([v, torch.randn(len(rows), G, generator=_gen(1)).to(DT[dt])], 1)
    data, p = moe.moe_quant_q4_weights(v.cuda(), FORMATS[fmt])
    q, want, nan = quantise(v, fmt)
    ok = ~want.isnan() if fmt == "b32" else ~want.isnan().any(-1)
    assert torch.equal(torch.nan_to_num(p.cpu().float(), 7.5), torch.nan_to_num(want.float(), 7.5))
    got = values((data.cpu(), p.cpu()), fmt).unflatten(-1, (-1, G))
    ref = (q.unflatten(-1, (-1, G)) * (want if fmt == "b32" else want[..., 0]).double()[..., None]
           + (0.0 if fmt == "b32" else want[..., 1].double()[..., None]))
    finite = ok & (want.isfinite() if fmt == "b32" else want.isfinite().all(-1))
    assert torch.equal(got[finite], ref[finite])
    assert not got[~finite].isfinite().any()
    bad = v.double().unflatten(-1, (-1, G))
    assert (~got[bad.isnan().any(-1)].isfinite()).all() and (~got[bad.isinf().any(-1)].isfinite()).all()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_quantiser_codes_beside_infinite_parameters(fmt):
    """Where a scale or a bias leaves fp16's range the codes are still the formula's: quotients of infinity, of an
    infinite scale, and of the largest f32 values."""
    G = GROUP[fmt]
    step = torch.arange(G).float()
    rows = [-7e4 - step, -7e4 + step * 4e3, step * 1e5, -step * 1e5, step * 1e37, step * 1e-3 - 6.5e4, step * 2e-7,
            (step - G // 2) * 1e-7]
    for dt in (torch.float32, torch.bfloat16):
        v = torch.stack(rows).to(dt)
        data, p = moe.moe_quant_q4_weights(v.cuda(), FORMATS[fmt])
        q, want, _ = quantise(v, fmt)
        assert torch.equal(p.cpu(), want)
        fixed = ~want.isnan() if fmt == "b32" else ~want.isnan().any(-1)
        got, q = (t.unflatten(-1, (-1, G)) for t in (codes(data.cpu(), fmt), q))
        # a NaN quotient (infinity minus or over itself) has any code: its group's values are infinite or NaN
        s = (want if fmt == "b32" else want[..., 0]).float()[..., None]
        b = 0.0 if fmt == "b32" else want[..., 1].float()[..., None]
        fixed = fixed[..., None] & ~((v.float().unflatten(-1, (-1, G)) - b) / s).isnan()
        assert torch.equal(got[fixed], q[fixed])


def test_quantiser_views():
    v = torch.randn(6, 300, generator=_gen(2)).cuda()
    a = v[:, 4:260]                       # strided, off 16 bytes
    d, p = moe.moe_quant_q4_weights(a, moe.MOE_Q4A64)
    e, q = moe.moe_quant_q4_weights(a.contiguous().clone(), moe.MOE_Q4A64)
    assert torch.equal(d, e) and torch.equal(p, q)
    d, p = moe.moe_quant_q4_weights(v.new_zeros(0, 4, 64))
    assert d.shape == (0, 4, 32) and p.shape == (0, 4, 2)


# ---- product ----------------------------------------------------------------------

SHAPES = [(1, 1, 64), (1, 17, 128), (2, 48, 192), (4, 16, 512), (5, 33, 1024), (8, 130, 2048), (9, 1001, 2112),
          (13, 64, 4096), (16, 31, 4160), (17, 48, 4224), (31, 96, 640), (33, 257, 512), (64, 100, 1088), (65, 64, 2048),
          (100, 300, 1056), (129, 130, 256), (257, 513, 192), (300, 1000, 1024)]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("types", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("bf16", "f16")],
                         ids=lambda t: "-".join(t))
def test_product(fmt, shape, types):
    M, N, K = shape
    if K % GROUP[fmt]:
        pytest.skip("K is no multiple of the group")
    say(f"product {shape} {fmt} {types}")
    g = _gen(M + N + K)
    x, w = _rows(g, M, K, types[0]), random_weights(g, (N,), K, fmt, "cuda")
    ref = torch.matmul(x.double(), values(w, fmt).t().contiguous())
    got = moe.moe_gemm_q4(x, w, out_dtype=DT[types[1]])
    assert got.shape == (M, N) and got.dtype == DT[types[1]]
    tol = product_tolerance(x, w, fmt, got.dtype)
    assert rel(got, ref) <= tol, (rel(got, ref), tol)
    # no element is far: 8 times the norm's share, and its own rounding
    scale = ref.square().mean().sqrt()
    far = (got.double() - ref).abs() - torch.finfo(got.dtype).eps / 2 * ref.abs()
    assert (far <= 8 * tol * scale + torch.finfo(got.dtype).tiny).all(), (far.max() / scale).item()
    assert torch.equal(got, moe.moe_gemm_q4(x, w, out_dtype=DT[types[1]]))


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("M", [1, 7, 40, 200])
def test_rows_do_not_mix(fmt, M):
    """A NaN or an infinity in a row of x, or in a weight row's parameters, stays in its row or column."""
    say(f"rows do not mix {fmt} {M}")
    g, N, K = _gen(M), 100, 704 if fmt != "a64" else 704
    x, w = _rows(g, M, K, "bf16"), random_weights(g, (N,), K, fmt, "cuda")
    clean = moe.moe_gemm_q4(x, w, out_dtype=torch.float32)
    bad = x.clone()
    bad[M // 2, 5] = math.nan
    bad[M - 1, K - 1] = math.inf
    got = moe.moe_gemm_q4(bad, w, out_dtype=torch.float32)
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[M // 2] = rows[M - 1] = False
    assert torch.equal(got[rows], clean[rows]) and not got[~rows].isfinite().any()
    p = w[1].clone()
    p.view(N, -1)[N - 1, -2:] = math.nan       # the last group's parameters
    p.view(N, -1)[3, 0] = math.inf
    got = moe.moe_gemm_q4(x, (w[0], p), out_dtype=torch.float32)
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[N - 1] = cols[3] = False
    assert torch.equal(got[:, cols], clean[:, cols]) and not got[:, ~cols].isfinite().any()


@pytest.mark.parametrize("M", [1, 3, 20, 150])
def test_rows_behind_are_left(M):
    """Outputs stop at M rows and N columns; inputs around the operands are never used."""
    g, N, K, fmt = _gen(M), 77, 160, "a32"
    wide = torch.full((M + 40, K), math.nan, dtype=torch.float16, device="cuda")
    wide[8:8 + M] = _rows(g, M, K, "f16")
    x = wide[8:8 + M]
    d, p = random_weights(g, (N,), K, fmt, "cuda")
    data = torch.full((N + 40, K // 2), 255, dtype=torch.uint8, device="cuda")
    data[8:8 + N] = d
    params = torch.full((N + 40, K // 32, 2), math.nan, dtype=torch.float16, device="cuda")
    params[8:8 + N] = p
    buf = torch.full((M * N + 4096,), 3.5, device="cuda")
    out = buf[1024:1024 + M * N].view(M, N)
    got = moe.moe_gemm_q4(x, (data[8:8 + N], params[8:8 + N]), out=out)
    want = moe.moe_gemm_q4(x.clone(), (d, p), out_dtype=torch.float32)
    assert got is out and torch.equal(got, want)
    assert (buf[:1024] == 3.5).all() and (buf[1024 + M * N:] == 3.5).all()


def test_product_shapes_and_views():
    g, N, K = _gen(5), 40, 256
    w = random_weights(g, (N,), K, "b32", "cuda")
    x = torch.randn(2, 3, 2 * K, generator=g).half().cuda()
    a = x[..., 1:1 + K]                     # strided, off 16 bytes
    got = moe.moe_gemm_q4(a, w)
    assert got.shape == (2, 3, N) and got.dtype == torch.float16
    assert torch.equal(got, moe.moe_gemm_q4(a.contiguous().view(6, K), w).view(2, 3, N))
    assert torch.equal(moe.moe_gemm_q4(a[0, 0], w), got[0, 0])
    d2 = torch.stack([w[0], w[0]], 1)[:, 1]     # strided weights
    p2 = torch.cat([w[1].new_zeros(1), w[1].flatten()])[1:].view_as(w[1])
    assert torch.equal(moe.moe_gemm_q4(a, (d2, p2)), got)
    assert moe.moe_gemm_q4(a[:0], w).shape == (0, 3, N)
    assert moe.moe_gemm_q4(a, (w[0][:0], w[1][:0])).shape == (2, 3, 0)


@pytest.mark.parametrize("M", [2, 70])
def test_weights_past_31_bits(M):
    """Codes of more than 2^31 bytes: the last rows against f64."""
    N, K = 1050000, 4096
    say(f"long weights {N} x {K}, {M} rows")
    data = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    params = torch.full((N, K // 32), 0.01, dtype=torch.float16, device="cuda")
    x = _rows(_gen(M), M, K, "f16")
    got = moe.moe_gemm_q4(x, (data, params), out_dtype=torch.float32)
    for at in (0, N // 2, N - 64):
        w = (data[at:at + 64], params[at:at + 64])
        ref = torch.matmul(x.double(), values(w, "b32").t().contiguous())
        assert rel(got[:, at:at + 64], ref) <= product_tolerance(x, w, "b32", torch.float32)


def test_output_past_31_bits():
    """An output of more than 2^31 values."""
    M, N, K = 70000, 31000, 64
    say(f"output {M} x {N}")
    g = _gen(9)
    w = random_weights(g, (N,), K, "a64", "cuda")
    x = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    got = moe.moe_gemm_q4(x, w, out_dtype=torch.bfloat16)
    for at in (0, M // 2, M - 100):
        ref = torch.matmul(x[at:at + 100].double(), values(w, "a64").t().contiguous())
        assert rel(got[at:at + 100], ref) <= product_tolerance(x[at:at + 100], w, "a64", torch.bfloat16)


@pytest.mark.parametrize("M", [1, 24, 140])
def test_graph_and_streams(M):
    """Captured and replayed on new inputs, and on two streams at once, as the eager call."""
    say(f"graph and streams {M}")
    g, N, K = _gen(M), 520, 1056
    w = random_weights(g, (N,), K, "a32", "cuda")
    xs = [_rows(g, M, K, "f16") for _ in range(4)]
    want = [moe.moe_gemm_q4(x, w) for x in xs]
    buf, out = xs[0].clone(), torch.empty(M, N, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_gemm_q4(buf, w, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_gemm_q4(buf, w, out=out)
    for i in (1, 2, 3, 0):
        buf.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        assert torch.equal(moe.moe_gemm_q4(xs[i], w), want[i])
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append(moe.moe_gemm_q4(x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
