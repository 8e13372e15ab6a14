"""The layer for a few tokens holds its SwiGLU output as f32: layers whose sums are
exact (small whole numbers, a down product that picks one value a column) leave
nothing else to see, at ordinary, small and large outputs; 4-bit layers of small
outputs."""

import math

import pytest
import torch

import mixture_experts_routed_route_amd as moe
from helpers import say
from q4_ref import DT, U, layer, random_weights, rel, route

pytestmark = pytest.mark.gpu

TOKENS = [1, 2, 3, 5, 8, 9, 16]


def _picked(T, D, xdt, gate, up, E=3, F=256):
    """x and weights of whole numbers times powers of two; the f64 sums of gate and up; h to y's columns."""
    g = torch.Generator().manual_seed(T + D)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()
    x = ints(-1, 1, T, D)
    wg, wu = ints(-2, 2, E, F, D) * gate, ints(-2, 2, E, F, D) * up
    at = torch.randint(0, F, (E, D), generator=g)
    factor = torch.exp2(ints(-2, 2, E, D))
    wd = torch.zeros(E, D, F).scatter_(2, at[..., None], factor[..., None])
    e = torch.arange(T) % E
    logits = torch.zeros(T, E)
    logits[torch.arange(T), e] = 9.0
    sums = lambda w: torch.stack([w[e[t]].double() @ x[t].double() for t in range(T)])
    assert all(torch.equal(t.to(DT[xdt]).float(), t) for t in (x, wg, wu, wd))
    x_, wg_, wu_, wd_ = (t.to(DT[xdt]).cuda() for t in (x, wg, wu, wd))
    return x_, wg_, wu_, wd_, logits.cuda(), sums(wg), sums(wu), at[e], factor[e].double()


@pytest.mark.parametrize("xdt,gate,up", [("bf16", 2.0 ** -4, 2.0 ** -4), ("f16", 2.0 ** -4, 2.0 ** -4),
                                         ("bf16", 2.0 ** -4, 2.0 ** -16), ("f16", 2.0 ** -4, 2.0 ** -16),
                                         ("bf16", 2.0 ** -4, 2.0 ** 40), ("f16", 1.0, 4.0)])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("D", [256, 4096])
def test_h_is_f32(T, D, xdt, gate, up):
    """Both column widths of the down launch (D of 4096 and more fills the units with 16 columns)."""
    if D == 4096:
        gate, up = gate / 4, up / 4     # the sums' size as at 256
    say(f"h of {T} tokens {D} {xdt} gate {gate} up {up}")
    x, wg, wu, wd, lg, pre, u, at, factor = _picked(T, D, xdt, gate, up)
    h = pre * torch.sigmoid(pre) * u
    y, _ = moe.moe_decode(x, wg, wu, wd, 1, logits=lg, options=moe.make_options(swiglu_limit=0.0))
    ref = h.gather(1, at) * factor
    # 2^x of g log2(e): the constant's and the product's rounding, half a step of each, |g| u both; 2^x and the
    # reciprocal one step (2 u) each, 1 + e, two products and the weight's 1 half a step: 10 u. Two fp16 parts: 2^-23 = 2 u
    # of the value, and half of fp16's last step, 2^-25, of the second part, which stands 2^12 higher: 2^-37
    bound = ((12 + 2 * pre.abs().gather(1, at)) * U * ref.abs() + (2.0 ** -37 if xdt == "f16" else 0.0) * factor + 1e-30)
    far = (y.cpu().double() - ref).abs() / bound
    say(f"  {far.max().item():.3f} of the bound, h to {h.abs().max().item():.1e}")
    assert y.isfinite().all() and (far <= 1).all()


@pytest.mark.parametrize("T", [1, 7, 16])
def test_past_fp16_beside_fp16_weights(T):
    """Beside fp16 weights h past 65504 is infinite, as moe_forward's 16-bit h is, and not NaN; the largest below holds,
    and so do the other tokens."""
    D, F = 256, 128
    x = torch.zeros(T, D, dtype=torch.float16)
    x[:, 0] = torch.linspace(0.25, 1.0, T) if T > 1 else 1.0
    x[T - 1, 1] = 1.0
    wg, wu, wd = torch.zeros(1, F, D), torch.zeros(1, F, D), torch.zeros(1, D, F)
    wg[0, :, 0], wu[0, :, 0] = 32.0, 32.0            # h of 1024 and less
    wg[0, 5, 1], wu[0, 5, 1] = 224.0, 224.0          # the last token: 256 * 256 = 65536 at 5, the others' 1024
    wd[0, :, 5], wd[0, :, 6] = 1.0, 2.0 ** -4
    args = [t.half().cuda() for t in (x, wg, wu, wd)]
    lg, o = torch.zeros(T, 1, device="cuda"), moe.make_options(swiglu_limit=0.0)
    y, _ = moe.moe_decode(*args, 1, logits=lg, options=o)
    assert (y[T - 1] == math.inf).all()
    a = 32.0 * x[:T - 1, 0].double()
    assert rel(y[:T - 1].cpu(), (a * torch.sigmoid(a) * a * (1 + 2.0 ** -4))[:, None].expand(T - 1, D)) <= 16 * U
    wu[0, 5, 1] = 223.0                              # 256 * 255 = 65280
    args[2] = wu.half().cuda()
    y, _ = moe.moe_decode(*args, 1, logits=lg, options=o)
    assert (y[T - 1] == 65280.0 + 1024 / 16).all()


@pytest.mark.parametrize("fmt", ["b32", "a32", "a64"])
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 4, 8, 16])
@pytest.mark.parametrize("scale,limit", [(2.0 ** -8, 7.0), (2.0 ** 9, 0.0), (2.0 ** 9, 300.0), (2.0 ** 3, 100.0)])
def test_4_bit_layers_of_small_and_large_h(fmt, xdt, T, scale, limit):
    """h of about 1e-5, and past fp16's range."""
    D, F, E, k = 256, 384, 8, 2
    say(f"4-bit h {fmt} {xdt} {T} x {scale}")
    g = torch.Generator().manual_seed(T)
    w = [random_weights(g, (E, s[0]), s[1], fmt, "cuda") for s in ((F, D), (F, D), (D, F))]
    x = (torch.randn(T, D, generator=g).to(DT[xdt]) * scale).cuda()
    lg = torch.randn(T, E, generator=g).cuda()
    y, _ = moe.moe_decode(x, *w, k, logits=lg, options=moe.make_options(swiglu_limit=limit))
    ids, wt, keep = route(lg, k)
    ref = layer(x, *w, fmt, ids, wt, keep, E, 0, clamp=limit)
    # products as product_tolerance has them (the larger constant beside a code: 136 of bf16, 3 and more the codes' mean
    # square), g and u in h, whose slope is at most 1.1 and 1; h 2 u; exp and its factors 12 u, and 2 u |g| of e^-|g|, which
    # is below |g| e^-|g| < 1 where it counts: 2 u
    off = 136.0 if xdt == "bf16" else 72.0
    sums = math.sqrt(33) * 2 / math.sqrt(3) * off / 3.0 + math.sqrt(F / 16)
    tol = (1.1 + 1 + 1) * sums * U + 16 * U
    err = rel(y, ref)
    say(f"  error {err:.2e} of {tol:.2e}")
    assert y.isfinite().all() and err <= tol


@pytest.mark.parametrize("w,x", [("bf16", "bf16"), ("f16", "f16"), ("b32", "bf16"), ("a32", "f16")])
@pytest.mark.parametrize("T", [5, 12, 16])
@pytest.mark.parametrize("limit", [7.0, 0.0])
def test_groups_of_tokens_do_not_mix(w, x, T, limit):
    """A token of NaN or of infinities leaves the others' bits alone, in its own group of tokens and in the others; an
    expert whose down weights are NaN or infinite reaches its own tokens only; few tokens an expert, and all at one."""
    D, F, E, k = 256, 384, 24, 2
    say(f"groups {w} {x} {T} {limit}")
    g = torch.Generator().manual_seed(T)
    mk = lambda N, K: (random_weights(g, (E + 1, N), K, w, "cuda") if w not in DT
                       else (torch.randn(E + 1, N, K, generator=g) * K ** -0.5).to(DT[w]).cuda())
    wg, wu, wd = mk(F, D), mk(F, D), mk(D, F)
    xs = torch.randn(T, D, generator=g).to(DT[x]).cuda()
    lg = torch.randn(T, E, generator=g).cuda()
    kw = dict(logits=lg, n_shared=1, options=moe.make_options(swiglu_limit=limit))
    y, _ = moe.moe_decode(xs, wg, wu, wd, k, **kw)
    assert y.isfinite().all()
    for t in (0, T // 2, T - 1):
        for v in (math.nan, math.inf):
            bad = xs.clone()
            bad[t, 7] = v
            z, _ = moe.moe_decode(bad, wg, wu, wd, k, **kw)
            rows = torch.arange(T, device="cuda") != t
            assert torch.equal(z[rows], y[rows])
            assert z[t].isnan().all() if v != v else not z[t].isfinite().any()
    ids, _, _ = route(lg, k)
    e = int(ids[T - 1, 0])
    hit = (ids == e).any(1).cuda()
    for v in (math.nan, math.inf):
        if w in DT:
            broken = wd.clone()
            broken[e] = v
        else:
            broken = (wd[0], wd[1].clone())
            broken[1][e] = v
        z, _ = moe.moe_decode(xs, wg, wu, broken, k, **kw)
        assert torch.equal(z[~hit], y[~hit]) and not z[hit].isfinite().any()
