"""Cases and plain forms of the layer's 8-bit and norm operators.

Four operators that surround and carry a routed feed-forward layer whose
weights are held in 8-bit floating point (e4m3) with one f32 scale for each
block of 128 values:

* ``quant``    rows [R, K] to e4m3 with a scale per row and 128 values, or
  weights [n, N, K] with a scale per 128 x 128 block:
  s = max(amax, 2^-100) / 448, q = e4m3(v * (448 / max(amax, 2^-100))), the
  quotients and the product rounded to f32;
* ``product``  out[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] w[n, k];
* ``experts``  the routed feed-forward layer on such weights: logits to plan,
  rows quantised, gate/up products, clamped SwiGLU, its output quantised per
  128 features, down product, weighted sum over a token's kept experts;
* ``norm``     r' = r + alpha g (RMSnorm(u) p) and x' = RMSnorm(r') w: the
  norms after a block and before the next one with the block's gate and the
  residual's scale, forward (x' in 16 bits or quantised) and backward.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, with the package's entry points.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_F8 = torch.float8_e4m3fn
_BLOCK = 128
_TINY = 2.0 ** -100
_LIMIT = 7.0     # the layer's default SwiGLU limit
_EPS = 1e-6


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the row of one decoded token entering a product
        {"name": "quant token", "op": "quant", "kind": "rows", "R": 1, "K": 2048, "dtype": "bf16"},
        # a whole long prompt's rows
        {"name": "quant prompt", "op": "quant", "kind": "rows", "R": 13312, "K": 4096, "dtype": "f16"},
        # a projection of one decoded token: the weights' stream
        {"name": "product token", "op": "product", "M": 1, "N": 4096, "K": 2048, "out": "bf16"},
        # a short prompt, an odd output width and a last block of 16 values
        {"name": "product ragged", "op": "product", "M": 517, "N": 1001, "K": 1040, "out": "f32"},
        # a projection of a long prompt: bound by the matrix units
        {"name": "product prompt", "op": "product", "M": 13312, "N": 4096, "K": 4096, "out": "f16"},
        # one decoded token through the layer with a shared expert
        {"name": "experts token", "op": "experts", "T": 1, "D": 2048, "F": 768, "E": 128, "k": 8,
         "shared": 1, "cap": 0.0, "zipf": 0.0, "dtype": "bf16"},
        # a short prompt: every expert holds a few pairs
        {"name": "experts short prompt", "op": "experts", "T": 128, "D": 2048, "F": 768, "E": 128, "k": 8,
         "shared": 1, "cap": 0.0, "zipf": 0.0, "dtype": "bf16"},
        # prefill under a skewed router: a few experts hold most rows
        {"name": "experts prefill", "op": "experts", "T": 4096, "D": 2048, "F": 768, "E": 128, "k": 8,
         "shared": 0, "cap": 0.0, "zipf": 1.1, "dtype": "bf16"},
        # between two blocks of one decoded token, feeding an 8-bit product
        {"name": "norm token", "op": "norm", "way": "forward", "T": 1, "D": 2048, "res": "f32", "blk": "bf16",
         "x": "f8", "par": "bf16", "post": True, "gate": "token", "unit": False},
        # between two blocks of a long prompt, f32 residual stream
        {"name": "norm prompt", "op": "norm", "way": "forward", "T": 13312, "D": 4096, "res": "f32", "blk": "f16",
         "x": "f16", "par": "f16", "post": True, "gate": "channel", "unit": False},
        # a training step's short batch, all bf16, weights stored around zero
        {"name": "norm backward ragged", "op": "norm", "way": "backward", "T": 333, "D": 1000, "res": "bf16",
         "blk": "bf16", "x": "bf16", "par": "bf16", "post": True, "gate": "token", "unit": True},
        # a training step on the prefill layer's rows
        {"name": "norm backward", "op": "norm", "way": "backward", "T": 4096, "D": 2048, "res": "f32", "blk": "f32",
         "x": "f32", "par": "f32", "post": True, "gate": "channel", "unit": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in lo .. hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "experts", "experts", "norm", "norm"])
    if op == "quant":
        kind = rng.choice(["rows", "rows", "weights"])
        c = {"op": op, "kind": kind, "R": _log(rng, 1, 13312), "K": _log(rng, 64, 4096, 8),
             "dtype": rng.choice(["f32", "bf16", "f16"])}
        if kind == "weights":
            c["n"] = rng.randint(1, 4)
            c["R"] = _log(rng, 64, 2048)
        return c
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 13312), "N": _log(rng, 64, 4096), "K": _log(rng, 128, 4096, 16),
                "out": rng.choice(["f32", "bf16", "f16"])}
    if op == "experts":
        E = rng.choice([8, 16, 33, 64, 128])
        return {"op": op, "T": _log(rng, 1, 4096), "D": 128 * rng.randint(2, 16), "F": 128 * rng.randint(1, 6),
                "E": E, "k": rng.randint(1, min(8, E // 2)), "shared": rng.randint(0, 1),
                "cap": rng.choice([0.0, 0.0, 1.5]), "zipf": rng.choice([0.0, 1.1]),
                "dtype": rng.choice(["bf16", "f16"])}
    lay = rng.choice(["bf16", "f16"])
    way = rng.choice(["forward", "backward"])
    return {"op": op, "way": way, "T": _log(rng, 1, 13312 if way == "forward" else 8192), "D": _log(rng, 64, 4096, 8),
            "res": rng.choice(["f32", lay]), "blk": rng.choice(["f32", lay]),
            "x": rng.choice([lay, "f8"] if way == "forward" else ["f32", lay]), "par": rng.choice(["f32", lay]),
            "post": rng.random() < 0.75, "gate": rng.choice(["none", "channel", "token"]),
            "unit": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------

def _gen(seed, case):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + len(str(sorted(case.items()))))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows_scaled(g, R, K, dtype):
    """Rows as a residual stream has them: each with a size of its own, a few channels much wider than the rest."""
    v = _randn(g, R, K) * torch.exp(0.5 * _randn(g, R, 1))
    wide = torch.rand(1, K, generator=g, device="cuda") < 0.01
    return torch.where(wide, v * 20.0, v).to(_DT[dtype])


def _weights_f8(g, n, N, K):
    """[n, N, K] weights of a trained layer in blocks, one matrix at a time."""
    q = torch.empty(n, N, K, dtype=_F8, device="cuda")
    s = torch.empty(n, -(-N // _BLOCK), -(-K // _BLOCK), device="cuda")
    for i in range(n):
        q[i], s[i] = _quant_weights(_randn(g, N, K) * (K ** -0.5))
    return q, s


def prepare(case, seed):
    g = _gen(seed, case)
    st = dict(case)
    if case["op"] == "quant":
        if case["kind"] == "rows":
            st["v"] = _rows_scaled(g, case["R"], case["K"], case["dtype"])
        else:
            st["v"] = (_randn(g, case["n"], case["R"], case["K"]) * (case["K"] ** -0.5)).to(_DT[case["dtype"]])
    elif case["op"] == "product":
        st["a"] = _quant_rows(_rows_scaled(g, case["M"], case["K"], "bf16"))
        q, s = _weights_f8(g, 1, case["N"], case["K"])
        st["w"] = (q[0], s[0])
    elif case["op"] == "experts":
        T, E, n = case["T"], case["E"], case["E"] + case["shared"]
        logits = _randn(g, T, E)
        if case["zipf"]:
            rank = torch.randperm(E, generator=g, device="cuda").float()
            logits = logits - case["zipf"] * torch.log1p(rank)
        st["logits"] = logits
        st["rows"] = _randn(g, T, case["D"]).to(_DT[case["dtype"]])
        st["gate_w"] = _weights_f8(g, n, case["F"], case["D"])
        st["up_w"] = _weights_f8(g, n, case["F"], case["D"])
        st["down_w"] = _weights_f8(g, n, case["D"], case["F"])
    else:
        T, D, par = case["T"], case["D"], _DT[case["par"]]
        shift = 0.0 if case["unit"] else 1.0
        st["r"] = (_randn(g, T, D) * torch.exp(0.5 * _randn(g, T, 1))).to(_DT[case["res"]])
        st["u"] = _randn(g, T, D).to(_DT[case["blk"]])
        st["w"] = (shift + 0.1 * _randn(g, D)).to(par)
        st["p"] = (shift + 0.1 * _randn(g, D)).to(par) if case["post"] else None
        st["g"] = None
        if case["gate"] != "none":
            shape = (D,) if case["gate"] == "channel" else (T, 1)
            st["g"] = (0.5 + 0.2 * _randn(g, *shape)).to(par)
        st["alpha"] = 0.7
        if case["way"] == "backward":
            # st["r"] stands for the forward's new residual
            st["dx"] = _randn(g, T, D).to(_DT[case["x"]])
            st["dr"] = _randn(g, T, D).to(_DT[case["res"]])
    return st


# ---- plain forms ------------------------------------------------------------

def _quant_blocks(v, amax):
    """v f32 and its blocks' largest magnitudes (broadcastable): q and s. The
    quotient is a division of two tensors: number / tensor would be a
    reciprocal and a product, rounded twice, and values that lie halfway
    between two of the format's (frequent among 16-bit ones) would move."""
    amax = torch.clamp_min(amax, _TINY)
    return (v * torch.div(torch.full_like(amax, 448.0), amax)).to(_F8), amax / 448.0


def _quant_rows(v):
    R, K = v.shape
    nb = -(-K // _BLOCK)
    b = torch.nn.functional.pad(v.float(), (0, nb * _BLOCK - K)).view(R, nb, _BLOCK)
    q, s = _quant_blocks(b, b.abs().amax(-1, keepdim=True))
    return q.view(R, -1)[:, :K].contiguous(), s.view(R, nb)


def _quant_weights(v):
    *lead, N, K = v.shape
    nn, nk = -(-N // _BLOCK), -(-K // _BLOCK)
    b = torch.nn.functional.pad(v.float(), (0, nk * _BLOCK - K, 0, nn * _BLOCK - N))
    b = b.view(*lead, nn, _BLOCK, nk, _BLOCK)
    q, s = _quant_blocks(b, b.abs().amax((-3, -1), keepdim=True))
    q = q.view(*lead, nn * _BLOCK, nk * _BLOCK)[..., :N, :K].contiguous()
    return q, s.view(*lead, nn, nk)


def _rows_of(q, s):
    """The values that quantised rows stand for."""
    R, K = q.shape
    nb = s.shape[1]
    v = torch.nn.functional.pad(q.float(), (0, nb * _BLOCK - K)).view(R, nb, _BLOCK) * s.unsqueeze(-1)
    return v.view(R, -1)[:, :K]


def _weights_of(q, s):
    N, K = q.shape
    nn, nk = s.shape
    v = torch.nn.functional.pad(q.float(), (0, nk * _BLOCK - K, 0, nn * _BLOCK - N))
    v = v.view(nn, _BLOCK, nk, _BLOCK) * s.view(nn, 1, nk, 1)
    return v.view(nn * _BLOCK, nk * _BLOCK)[:N, :K]


def _route(logits, k, limit):
    """Experts and weights of each token (ties to the lower index) and which pairs are kept."""
    T, E = logits.shape
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, w = order.indices[:, :k], torch.softmax(order.values[:, :k], 1)
    if limit is None:
        return ids, w, torch.ones_like(ids, dtype=torch.bool)
    chosen = torch.zeros(T, E, dtype=torch.int32, device=logits.device).scatter_(1, ids, 1)
    earlier = torch.cumsum(chosen, 0) - chosen
    return ids, w, earlier.gather(1, ids) < limit


def _limit(case):
    if not case["cap"]:
        return None
    return max(1, math.floor(case["cap"] * case["T"] * case["k"] / case["E"]))


def _experts_plain(st):
    T, E, k = st["T"], st["E"], st["k"]
    ids, w, keep = _route(st["logits"], k, _limit(st))
    x = _rows_of(*_quant_rows(st["rows"]))
    pair_e = torch.where(keep, ids, E + 1).reshape(-1)
    if st["shared"]:
        pair_e = torch.cat([pair_e, torch.full((T,), E, dtype=pair_e.dtype, device=pair_e.device)])
    order = torch.sort(pair_e, stable=True).indices
    token = torch.where(order < T * k, order // k, order - T * k)
    counts = torch.bincount(pair_e, minlength=E + 2)[:E + 1].tolist()
    out = torch.zeros(pair_e.numel(), st["D"], device=x.device)
    at = 0
    for e, n in enumerate(counts):
        if n:
            rows = order[at:at + n]
            xe = x[token[at:at + n]]
            gate = xe @ _weights_of(st["gate_w"][0][e], st["gate_w"][1][e]).t()
            up = xe @ _weights_of(st["up_w"][0][e], st["up_w"][1][e]).t()
            gate = gate.clamp_max(_LIMIT)
            h = gate / (1.0 + torch.exp(-gate)) * up.clamp(-_LIMIT, _LIMIT)
            out[rows] = _rows_of(*_quant_rows(h)) @ _weights_of(st["down_w"][0][e], st["down_w"][1][e]).t()
            at += n
    y = (out[:T * k].view(T, k, -1) * torch.where(keep, w, 0.0).unsqueeze(-1)).sum(1)
    if st["shared"]:
        y = y + out[T * k:]
    return y.to(st["rows"].dtype)


def _vec(v, unit, dtype=torch.float32):
    return v.to(dtype) + 1.0 if unit else v.to(dtype)


def _norm_plain(st):
    u = st["u"].float()
    if st["p"] is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + _EPS) * _vec(st["p"], st["unit"])
    if st["g"] is not None:
        u = u * st["g"].float()
    r = st["r"].float() + st["alpha"] * u
    x = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS) * _vec(st["w"], st["unit"])
    x = _quant_rows(x) if st["x"] == "f8" else x.to(_DT[st["x"]])
    return r.to(st["r"].dtype), x


def _norm_back(v, dy, w):
    """Gradients of RMSnorm(v) w: for v, and for w before the sum over rows."""
    inv = torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)
    n = v * inv
    t = dy * w
    return inv * (t - n * (t * n).mean(-1, keepdim=True)), dy * n


def _norm_backward(st, dtype):
    r, u, unit = st["r"].to(dtype), st["u"].to(dtype), st["unit"]
    d, dw = _norm_back(r, st["dx"].to(dtype), _vec(st["w"], unit, dtype))
    d = d + st["dr"].to(dtype)
    got = {"dresidual": d, "dweight": dw.sum(0)}
    gate = st["g"].to(dtype) if st["g"] is not None else 1.0
    dz = st["alpha"] * d * gate
    z = u
    if st["p"] is not None:
        p = _vec(st["p"], unit, dtype)
        z = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + _EPS) * p
        dz, dp = _norm_back(u, dz, p)
        got["dpost_weight"] = dp.sum(0)
    got["dblock"] = dz
    if st["g"] is not None:
        dg = st["alpha"] * d * z
        got["dgate"] = dg.sum(0) if st["g"].dim() == 1 else dg.sum(1, keepdim=True)
    return got


def _rounded(st, got):
    """Gradients of rows in the rows' type, the parameters' in f32."""
    to = {"dresidual": st["r"].dtype, "dblock": st["u"].dtype}
    return {n: v.to(to.get(n, torch.float32)) for n, v in got.items()}


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "quant":
        return _quant_rows(st["v"]) if st["kind"] == "rows" else _quant_weights(st["v"])
    if st["op"] == "product":
        return (_rows_of(*st["a"]) @ _weights_of(*st["w"]).t()).to(_DT[st["out"]])
    if st["op"] == "experts":
        return _experts_plain(st)
    if st["way"] == "forward":
        return _norm_plain(st)
    return _rounded(st, _norm_backward(st, torch.float32))


def _run_own(st):
    import mixture_experts_routed_route_amd as moe

    if st["op"] == "quant":
        return moe.moe_quant_f8(st["v"]) if st["kind"] == "rows" else moe.moe_quant_f8_weights(st["v"])
    if st["op"] == "product":
        return moe.moe_gemm_f8(st["a"], st["w"], out_dtype=_DT[st["out"]])
    if st["op"] == "experts":
        plan = moe.moe_plan_create(st["logits"], st["k"], st["cap"], st["shared"])
        return moe.moe_forward(plan, st["rows"], st["gate_w"], st["up_w"], st["down_w"], y_dtype=st["rows"].dtype)
    kw = dict(weight=st["w"], post_weight=st["p"], gate=st["g"], alpha=st["alpha"], eps=_EPS, unit_offset=st["unit"])
    if st["way"] == "forward":
        return moe.moe_norm(st["r"], st["u"], x_dtype=_F8 if st["x"] == "f8" else _DT[st["x"]], **kw)
    return moe.moe_norm_backward(st["r"], st["u"], st["dx"], dresidual_out=st["dr"], **kw)


# ---- work -------------------------------------------------------------------

_SIZE = {"f32": 4, "bf16": 2, "f16": 2, "f8": 1}


def work(case):
    if case["op"] == "quant":
        n = case.get("n", 1)
        vals = n * case["R"] * case["K"]
        rows = case["R"] if case["kind"] == "rows" else -(-case["R"] // _BLOCK)
        return {"bytes": vals * (_SIZE[case["dtype"]] + 1) + 4 * n * rows * -(-case["K"] // _BLOCK), "flops": 3 * vals}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        nb = -(-K // _BLOCK)
        return {"bytes": (M + N) * K + 4 * nb * (M + -(-N // _BLOCK)) + M * N * _SIZE[case["out"]], "flops": 2 * M * N * K}
    if case["op"] == "experts":
        T, D, F, E, k, shared = (case[n] for n in ("T", "D", "F", "E", "k", "shared"))
        pop = [(1 + i) ** -case["zipf"] for i in range(E)]
        load = [k * p / sum(pop) for p in pop]
        touched = sum(1 - (1 - min(1.0, v)) ** T for v in load)
        limit = _limit(case)
        kept = sum(min(T * min(1.0, v), limit or T) for v in load) if limit else T * k
        weights = (touched + shared) * 3 * D * F * (1 + 4 / _BLOCK ** 2)
        return {"bytes": weights + T * E * 4 + 2 * T * D * _SIZE[case["dtype"]], "flops": 6 * D * F * (kept + shared * T)}
    vals = case["T"] * case["D"]
    size = {n: _SIZE[case[n]] for n in ("res", "blk", "x", "par")}
    if case["way"] == "forward":
        return {"bytes": vals * (2 * size["res"] + size["blk"] + size["x"]), "flops": 10 * vals}
    return {"bytes": vals * (3 * size["res"] + 2 * size["blk"] + size["x"]), "flops": 25 * vals}


# ---- exact ------------------------------------------------------------------

def _exact_scaled(v, amax):
    """q and s of f64 blocks by the definition: quotients and the product
    rounded to f32 (each exact in f64 before its one rounding), then e4m3."""
    amax = torch.clamp_min(amax, _TINY)
    inv = (448.0 / amax).float().double()
    return (v * inv).float().to(_F8).double(), (amax / 448.0).float().double()


def _exact_rows(v):
    """[R, K] f64 to (q, s), block by block over a zero-filled copy."""
    R, K = v.shape
    nb = -(-K // _BLOCK)
    full = v.new_zeros(R, nb * _BLOCK)
    full[:, :K] = v
    full = full.reshape(R, nb, _BLOCK)
    q, s = _exact_scaled(full, full.abs().max(-1, keepdim=True).values)
    return q.reshape(R, -1)[:, :K], s.squeeze(-1)


def _exact_matrices(v):
    n, N, K = v.shape
    nn, nk = -(-N // _BLOCK), -(-K // _BLOCK)
    full = v.new_zeros(n, nn * _BLOCK, nk * _BLOCK)
    full[:, :N, :K] = v
    full = full.reshape(n, nn, _BLOCK, nk, _BLOCK).transpose(2, 3).reshape(n, nn, nk, -1)
    q, s = _exact_scaled(full, full.abs().max(-1, keepdim=True).values)
    q = q.reshape(n, nn, nk, _BLOCK, _BLOCK).transpose(2, 3).reshape(n, nn * _BLOCK, nk * _BLOCK)
    return q[:, :N, :K], s.squeeze(-1)


def _spread(s, N, axis):
    """Block scales to one for each of N places of an axis."""
    return s.double().index_select(axis, torch.arange(N, device=s.device) // _BLOCK)


def _exact_w(q, s):
    return q.double() * _spread(_spread(s, q.shape[0], 0), q.shape[1], 1)


def _exact_experts(case, st):
    T, E, k, D = case["T"], case["E"], case["k"], case["D"]
    q, s = _exact_rows(st["rows"].double())
    x = q * _spread(s, D, 1)
    logits = st["logits"].double()
    y = torch.zeros(T, D, dtype=torch.float64, device=x.device)
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    top = logits.gather(1, ids)
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    limit = _limit(case) or T
    for e in range(E + case["shared"]):
        if e < E:
            t, j = torch.nonzero(ids == e, as_tuple=True)   # tokens in order
            t, j = t[:limit], j[:limit]
            if not t.numel():
                continue
            weight = p[t, j]
        else:
            t = torch.arange(T, device=x.device)
            weight = torch.ones(T, dtype=torch.float64, device=x.device)
        g = torch.matmul(x[t], _exact_w(st["gate_w"][0][e], st["gate_w"][1][e]).t().contiguous())
        u = torch.matmul(x[t], _exact_w(st["up_w"][0][e], st["up_w"][1][e]).t().contiguous())
        g = torch.minimum(g, torch.full_like(g, _LIMIT))
        h = g * torch.sigmoid(g) * torch.clamp(u, -_LIMIT, _LIMIT)
        hq, hs = _exact_rows(h)
        o = torch.matmul(hq * _spread(hs, case["F"], 1), _exact_w(st["down_w"][0][e], st["down_w"][1][e]).t().contiguous())
        y[t] += weight.unsqueeze(1) * o
    return y


def _exact_norm_of(v, w):
    ms = torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / v.shape[1]
    return v / torch.sqrt(ms + _EPS) * w


def _exact_norm(case, st):
    one = 1.0 if case["unit"] else 0.0
    z = st["u"].double()
    if st["p"] is not None:
        z = _exact_norm_of(z, st["p"].double() + one)
    gate = st["g"].double() if st["g"] is not None else torch.ones(1, dtype=torch.float64, device=z.device)
    r = st["r"].double() + st["alpha"] * gate * z
    x = _exact_norm_of(r, st["w"].double() + one)
    return r, _exact_rows(x) if case["x"] == "f8" else x


def _exact_norm_backward(case, st):
    """By differentiating the definition, f64."""
    one = 1.0 if case["unit"] else 0.0
    leaf = lambda v: v.detach().double().requires_grad_(True)  # noqa: E731
    with torch.enable_grad():
        r, w = leaf(st["r"]), leaf(st["w"])
        (_exact_norm_of(r, w + one) * st["dx"].double()).sum().backward()
        dr = r.grad + st["dr"].double()
        got = {"dresidual": dr, "dweight": w.grad}
        u = leaf(st["u"])
        p = leaf(st["p"]) if st["p"] is not None else None
        g = leaf(st["g"]) if st["g"] is not None else None
        z = _exact_norm_of(u, p + one) if p is not None else u
        if g is not None:
            z = z * g
        (st["alpha"] * z * dr).sum().backward()
        got["dblock"] = u.grad
        if p is not None:
            got["dpost_weight"] = p.grad
        if g is not None:
            got["dgate"] = g.grad
    return got


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_rows(st["v"].double()) if case["kind"] == "rows" else _exact_matrices(st["v"].double())
    if case["op"] == "product":
        a = st["a"][0].double() * _spread(st["a"][1], case["K"], 1)
        return torch.matmul(a, _exact_w(*st["w"]).t().contiguous())
    if case["op"] == "experts":
        return _exact_experts(case, st)
    return _exact_norm(case, st) if case["way"] == "forward" else _exact_norm_backward(case, st)
