"""Plain f64 forms of the 4-bit formats, products on them and the layer for a
few tokens, with the error that f32 arithmetic may add (u = 2^-24, half a step
of f32)."""

import math

import torch

import mixture_experts_routed_route_amd as moe

U = 2.0 ** -24
FORMATS = {"b32": moe.MOE_Q4B32, "a32": moe.MOE_Q4A32, "a64": moe.MOE_Q4A64}
GROUP = {"b32": 32, "a32": 32, "a64": 64}
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---- formats ----------------------------------------------------------------

def codes(data, fmt):
    """Codes [.., K] of packed bytes, f64."""
    n = torch.stack([data & 15, data >> 4], -1).flatten(-2).double()
    return torch.where(n > 7, n - 16, n) if fmt == "b32" else n


def values(w, fmt):
    data, p = w
    q, p = codes(data, fmt), p.double()
    if fmt == "b32":
        return q * p.repeat_interleave(GROUP[fmt], -1)
    p = p.repeat_interleave(GROUP[fmt], -2)
    return q * p[..., 0] + p[..., 1]


def random_weights(g, lead, K, fmt, dev="cpu"):
    """Uniform codes, scales of either sign, biases."""
    G = GROUP[fmt]
    data = torch.randint(0, 256, (*lead, K // 2), generator=g, dtype=torch.uint8)
    s = (0.005 + 0.015 * torch.rand(*lead, K // G, generator=g)) * torch.where(
        torch.rand(*lead, K // G, generator=g) < 0.1, -1.0, 1.0)
    if fmt == "b32":
        return data.to(dev), s.half().to(dev)
    b = -7.5 * s + 0.02 * torch.randn(*lead, K // G, generator=g)
    return data.to(dev), torch.stack([s, b], -1).half().to(dev)


def _f32(v):
    """An f64 value rounded to f32 (of quotients of f32 values: their f32 quotient, 53 >= 2 * 24 + 2 bits)."""
    return v.float().double()


def quantise(v, fmt):
    """Codes and fp16 parameters of rows (f32 or 16-bit values), bit for bit."""
    G = GROUP[fmt]
    b = v.double().unflatten(-1, (-1, G))
    nan = b.isnan().any(-1)
    if fmt == "b32":
        s = _f32(b.abs().amax(-1) / 7).half()
        q = torch.round(_f32(b / s.double()[..., None])).clamp(-8, 7)
        p = s
    else:
        lo, hi = b.amin(-1), b.amax(-1)
        s, bias = _f32(_f32(hi - lo) / 15).half(), lo.half()
        q = torch.round(_f32(_f32(b - bias.double()[..., None]) / s.double()[..., None])).clamp(0, 15)
        p = torch.stack([s, bias], -1)
    q = torch.where((s == 0)[..., None], 0.0, q)
    return q.flatten(-2), p, nan


# ---- product ----------------------------------------------------------------

def product_tolerance(x, w, fmt, out_dtype):
    """Relative error, in the norm, of a product whose groups' sums pass through
    f32 with a constant `off` beside each code (f16 64, bf16 128, 8 more for
    signed codes) and are scaled and added in f32. A group of G values: at most G
    + 1 additions, each off by at most a step (2 u) of a partial sum whose size
    is off sqrt(G) rms(x) against codes' c sqrt(G) rms(x); errors of either sign
    add in squares: sqrt(G + 1) 2 / sqrt(3) u off / c. The scaled sums add as many
    u as the square root of their number; the output is rounded once."""
    off = (64.0 if x.dtype == torch.float16 else 128.0) + (8.0 if fmt == "b32" else 0.0)
    q = codes(w[0], fmt)
    if fmt != "b32":
        q = q - 7.5
    c = q.square().mean().sqrt().item()
    G = GROUP[fmt]
    n = x.shape[-1] // G
    # an instruction sums 32 values: groups of 64 are two
    sums = math.sqrt(33) * 2 / math.sqrt(3) * off / max(c, 1.0) + math.sqrt(2 * n + 2)
    return sums * U + half_step(out_dtype)


def rel(got, ref):
    return ((got.double() - ref).square().sum().sqrt() / ref.square().sum().sqrt().clamp_min(1e-300)).item()


# ---- the layer ----------------------------------------------------------------

def route(logits, k, limit=None):
    """Experts [T, k] (ties to the lower index, NaN below -inf), weights (f64),
    kept pairs."""
    lg = logits.double().cpu()
    key = torch.where(lg.isnan(), torch.full_like(lg, -math.inf), lg)
    # NaN after every other value, -0 and +0 alike
    order = torch.argsort(-key + 0.0, dim=1, stable=True)
    T, E = lg.shape
    ids = torch.empty(T, k, dtype=torch.int64)
    for t in range(T):
        row = [e for e in order[t].tolist() if not lg[t, e].isnan()] + \
              [e for e in range(E) if lg[t, e].isnan()]
        ids[t] = torch.tensor(row[:k])
    top = lg.gather(1, ids)
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    keep = torch.ones(T, k, dtype=torch.bool)
    if limit is not None:
        seen = [0] * E
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j])
                keep[t, j] = seen[e] < limit
                seen[e] += 1
    return ids, w, keep


def capacity(T, E, k, cf):
    return None if cf == 0 else max(1, math.floor(float(torch.tensor(cf).float()) * T * k / E))


def dense(w, i, fmt):
    """Matrix i in f64 on its device."""
    return w[i].double() if fmt is None else values((w[0][i], w[1][i]), fmt)


def layer(x, wg, wu, wd, fmt, ids, w, keep, E, n_shared, clamp=7.0):
    """y [T, D] in f64 from f64 sums, nothing rounded on the way."""
    T = x.shape[0]
    xd = x.double()
    y = torch.zeros(T, x.shape[1], dtype=torch.float64, device=x.device)
    pairs = {}
    for t in range(T):
        for j in range(ids.shape[1]):
            if keep[t, j]:
                pairs.setdefault(int(ids[t, j]), []).append((t, float(w[t, j])))
    if n_shared:
        pairs[E] = [(t, 1.0) for t in range(T)]
    c = clamp if clamp > 0 else math.inf
    for e, lst in sorted(pairs.items()):
        rows = torch.tensor([t for t, _ in lst], device=x.device)
        wt = torch.tensor([v for _, v in lst], dtype=torch.float64, device=x.device)
        g = torch.matmul(xd[rows], dense(wg, e, fmt).t().contiguous()).clamp(max=c)
        u = torch.matmul(xd[rows], dense(wu, e, fmt).t().contiguous()).clamp(-c, c)
        o = torch.matmul(g * torch.sigmoid(g) * u, dense(wd, e, fmt).t().contiguous())
        y.index_add_(0, rows, o * wt[:, None])
    return y


def layer_tolerance(xdt, fmt, ydt, D, F):
    """Relative error, in the norm. h is held to 2^-17 (bf16, two parts of 8 bits:
    half a step of the second, 2^-9 of 2^-8) or 2^-22 (f16); the sums of either
    product as in product_tolerance, with codes of 3 and more in the mean square
    (16-bit weights: sqrt(K) steps); g and u both enter h, whose slope is below
    2 in each, exp and reciprocal add 4 u; y is rounded once."""
    if fmt is None:
        sums = 2 * (math.sqrt(D) + math.sqrt(F)) * 2 / math.sqrt(3)
    else:
        off = (64.0 if xdt == torch.float16 else 128.0) + (8.0 if fmt == "b32" else 0.0)
        sums = math.sqrt(33) * 2 / math.sqrt(3) * off / 3.0 + math.sqrt(max(D, F) / 16)
    h = 2.0 ** -22 if xdt == torch.float16 else 2.0 ** -17
    return (5 * sums + 8) * U + h + half_step(ydt)
