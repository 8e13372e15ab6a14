"""Plain f64 forms of the 8-bit block format, its products, the routed layer
on it and the norms around a block, with the error that f32 arithmetic may
add to each (u = 2^-24, half a step of f32)."""

import math

import torch

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
TINY = 2.0 ** -100


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half of the smallest step a type has near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def div32(a, b):
    """Correctly rounded f32 quotient, in f64 (one rounding of the f64
    quotient is the f32 quotient's: 53 >= 2 * 24 + 2 bits)."""
    return (a.double() / b.double()).float()


def quant_blocks(v, amax):
    """v and its blocks' largest magnitudes (f32) -> codes, scales, bit for bit."""
    amax = torch.clamp_min(amax, TINY)
    inv = div32(torch.full_like(amax, 448.0), amax)
    return (v.float() * inv).to(F8), div32(amax, torch.full_like(amax, 448.0))


def quant_rows(v):
    R, K = v.shape
    nb = -(-K // 128)
    f = torch.zeros(R, nb * 128)
    f[:, :K] = v.float()
    f = f.view(R, nb, 128)
    q, s = quant_blocks(f, f.abs().amax(-1, keepdim=True))
    return q.view(R, -1)[:, :K].contiguous(), s.view(R, nb)


def quant_weights(w):
    n, N, K = w.shape
    nn, nk = -(-N // 128), -(-K // 128)
    f = torch.zeros(n, nn * 128, nk * 128)
    f[:, :N, :K] = w.float()
    f = f.view(n, nn, 128, nk, 128)
    q, s = quant_blocks(f, f.abs().amax((2, 4), keepdim=True))
    return q.view(n, nn * 128, nk * 128)[:, :N, :K].contiguous(), s.view(n, nn, nk)


def rows_f64(q, s):
    return q.double() * s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]


def weights_f64(q, s):
    N, K = q.shape[-2:]
    s = s.double().repeat_interleave(128, -1)[..., :K]
    return q.double() * s.repeat_interleave(128, -2)[..., :N, :]


def _max8(v):
    """Largest magnitude of each eight neighbouring values of a row."""
    pad = torch.zeros(v.shape[0], -v.shape[1] % 8, dtype=v.dtype)
    return torch.cat([v.abs(), pad], 1).view(v.shape[0], -1, 8).amax(-1)


def product_bound(a, w, out_dtype=None, out=None, units8=False):
    """f32 error of a . w^T by blocks of 128: each of the 128 products of a
    block loses at most u of the block's largest term in the sum, and each
    block's scaled addition rounds three times. units8: the 8-bit matrix
    unit's sums, where of eight neighbouring products the seven that are not
    the largest may each lose 2^-13 of it."""
    K = a.shape[1]
    n = 128 + 3 * -(-K // 128)
    e = n * U * (a.abs() @ w.abs().t())
    if units8:
        e = e + 7 * 2.0 ** -13 * (_max8(a) @ _max8(w).t())
    if out_dtype is not None:
        e = e * (1 + half_step(out_dtype)) + half_step(out_dtype) * out.abs() + smallest(out_dtype)
    return e


def _codes_between(h, e, a, ea):
    """Least and largest value that quantised h may stand for, h within e and
    its block's largest magnitude within ea."""
    lo_a, hi_a = torch.clamp_min(a - ea, TINY), torch.clamp_min(a + ea, TINY)
    lo, hi = h - e, h + e
    pick = lambda v, up: torch.where((v > 0) == up, lo_a, hi_a)  # noqa: E731
    q = lambda v, d: (v * (448.0 / d) * (1 + 4 * U * torch.sign(v))).clamp(-448, 448).to(F8).double()  # noqa: E731
    qd = lambda v, d: (v * (448.0 / d) * (1 - 4 * U * torch.sign(v))).clamp(-448, 448).to(F8).double()  # noqa: E731
    up = torch.where(hi > 0, q(hi, pick(hi, True)), qd(hi, pick(hi, True)))
    dn = torch.where(lo > 0, qd(lo, pick(lo, False)), q(lo, pick(lo, False)))
    s_up = torch.where(up > 0, hi_a, lo_a) / 448.0
    s_dn = torch.where(dn > 0, lo_a, hi_a) / 448.0
    return dn * s_dn, up * s_up


def expert(x, wg, wu, wd, limit, up8=False, down8=False):
    """One expert on quantised rows x (f64): outputs and their f32 bound; up8,
    down8: the products' sums in the 8-bit matrix unit."""
    lim = limit if limit > 0 else math.inf
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = (product_bound(x, m, units8=up8) for m in (wg, wu))
    gc, uc = g.clamp(max=lim), u.clamp(-lim, lim)
    sig = torch.sigmoid(gc)
    h = gc * sig * uc
    # |silu'| <= 1.1; the hardware's exponential and reciprocal and the
    # products: a few steps each, 16 u of the value
    eh = 1.1 * uc.abs() * eg + (gc * sig).abs() * eu + 1.1 * eg * eu + 16 * U * h.abs()
    R, Fd = h.shape
    b = h.view(R, Fd // 128, 128)
    a = b.abs().amax(-1, keepdim=True)
    ea = eh.view_as(b).amax(-1, keepdim=True)
    lo, hi = _codes_between(b, eh.view_as(b), a, ea)
    aq = torch.clamp_min(a, TINY)
    val = (b * (448.0 / aq)).clamp(-448, 448).to(F8).double() * aq / 448.0
    off = torch.maximum(hi - val, val - lo).view(R, Fd).clamp_min(0)
    val = val.view(R, Fd)
    y = val @ wd.t()
    return y, off @ wd.abs().t() + product_bound(val.abs() + off, wd, units8=down8)


def layer(x, w_gate, w_up, w_down, ids, w, keep, E, n_shared, limit, out_dtype, pair_dtype):
    """The routed layer on 8-bit weights: y and its bound. x [T, D] as given;
    ids, w, keep [T, k] from the plan. Pair outputs are held in pair_dtype."""
    T, k = ids.shape
    xq = rows_f64(*quant_rows(x))
    y = torch.zeros(T, x.shape[1], dtype=torch.float64)
    e = torch.zeros_like(y)
    for ex in range(E + n_shared):
        if ex < E:
            t, j = torch.nonzero((ids == ex) & keep, as_tuple=True)
            pw = w[t, j].double()
        else:
            t, pw = torch.arange(T), torch.ones(T, dtype=torch.float64)
        if not t.numel():
            continue
        m = [weights_f64(q[ex], s[ex]) for q, s in (w_gate, w_up, w_down)]
        # experts of more than 16 rows may run on the tile, whose down products
        # may be summed in the 8-bit matrix unit; a bf16 layer's gate/up, summed
        # in f32, is given the bound of that unit's sums here too
        tile = t.numel() > 16
        o, b = expert(xq[t], *m, limit, tile and x.dtype == torch.bfloat16, tile)
        b = b + half_step(pair_dtype) * (o.abs() + b) + smallest(pair_dtype)
        y.index_add_(0, t, pw[:, None] * o)
        # the weight (a softmax in f32, 1e-6 relative), its product, the sum
        e.index_add_(0, t, pw[:, None] * (b + (1e-6 + (k + 2) * U) * (o.abs() + b)))
    return y, e + half_step(out_dtype) * (y.abs() + e) + smallest(out_dtype)


# ---- norms --------------------------------------------------------------------

# Relative error of 1 / sqrt(mean of squares + eps) in f32 over D values: each
# thread adds at most 16 squares in turn, then 6 + 4 levels and 16 waves' sums:
# under 64 roundings of positive terms, halved by the root, plus the root's own.
INV = 36 * U


def norm(r, u, w, p, g, alpha, eps, unit):
    """f64 (r', x) of f64 inputs (u, w, p, g may be None) and their f32 bounds."""
    one = 1.0 if unit else 0.0
    er = torch.zeros_like(r)
    if u is not None:
        z = u
        rel = 3 * U
        if p is not None:
            z = u / torch.sqrt(u.square().mean(1, keepdim=True) + eps) * (p + one)
            rel += INV + 4 * U
        z = alpha * z * (g if g is not None else 1.0)
        r = r + z
        er = rel * z.abs() + 2 * U * r.abs()
    if w is None:
        return r, None, er, None
    inv = 1.0 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    x = r * inv * (w + one)
    # r' itself is off by er; its norm by at most the rows' largest relative er
    ex = (INV + 4 * U) * x.abs() + er * inv * (w + one).abs()
    ex = ex + x.abs() * inv * torch.sqrt(er.square().mean(1, keepdim=True))
    return r, x, er, ex


def norm_grads(r, u, w, p, g, dr, dx, alpha, eps, unit):
    """f64 gradients by differentiating the definition, at a given r'."""
    one = 1.0 if unit else 0.0
    leaf = lambda v: None if v is None else v.detach().clone().requires_grad_(True)  # noqa: E731
    r, w, u, p, g = (leaf(v) for v in (r, w, u, p, g))
    got = {}
    d = dr if dr is not None else torch.zeros_like(r)
    if w is not None:
        x = r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * (w + one)
        (x * dx).sum().backward()
        d = d + r.grad
        got["dweight"] = w.grad
    got["dresidual"] = d
    if u is not None:
        z = u
        if p is not None:
            z = u / torch.sqrt(u.square().mean(1, keepdim=True) + eps) * (p + one)
        if g is not None:
            z = z * g
        (alpha * z * d).sum().backward()
        got["dblock"] = u.grad
        if p is not None:
            got["dpost_weight"] = p.grad
        if g is not None:
            got["dgate"] = g.grad
    return got
