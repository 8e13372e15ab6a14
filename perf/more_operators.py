"""Cases and plain forms of the operators on 4-bit weights and of the whole
layer for a few tokens.

A 4-bit weight row [K] is cut into groups of 32 or 64 values with fp16
parameters. ``b32``: codes q in -8..7 and a scale s a group of 32, value q s;
``a32`` and ``a64``: codes q in 0..15, a scale s and a bias b a group of 32 or
64, value q s + b.

* ``quant``    rows of weights to codes and parameters; b32: s = fp16(max|v| /
  7), q = clamp(round(v / s), -8, 7); a32, a64: s = fp16((max - min) / 15), b =
  fp16(min), q = clamp(round((v - b) / s), 0, 15); quotients and differences
  rounded to f32, a scale of zero has codes of zero;
* ``product``  out[m, n] = sum_k x[m, k] value(w[n, k]) on such weights;
* ``decode``   the routed feed-forward layer on 1 to 16 tokens, from router
  logits, or from x and the router's map, to its output: top-k experts of each
  token (ties to the lower index), softmax over the k, an optional limit of
  pairs an expert, gate and up products, clamped SwiGLU, down product, weighted
  sum over the kept experts and an optional shared one; on 16-bit or 4-bit
  weights.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, with the package's entry points.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_GROUP = {"b32": 32, "a32": 32, "a64": 64}
_CLAMP = 7.0     # the layer's default SwiGLU limit


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one expert's gate matrix of a 16-bit checkpoint taken to 4 bits
        {"name": "quant matrix", "op": "quant", "rows": 768, "K": 2048, "fmt": "a64", "dtype": "bf16"},
        # the gate matrices of 32 experts at load time
        {"name": "quant experts", "op": "quant", "rows": 65536, "K": 4096, "fmt": "b32", "dtype": "f16"},
        # a projection of one decoded token: latency
        {"name": "product token", "op": "product", "M": 1, "N": 4096, "K": 2048, "fmt": "b32", "x": "f16", "out": "f16"},
        # the head of one decoded token: a long weight stream, f32 logits
        {"name": "product head", "op": "product", "M": 1, "N": 65536, "K": 4096, "fmt": "a64", "x": "bf16", "out": "f32"},
        # a few tokens' rows, an odd width, 65 groups a row
        {"name": "product few ragged", "op": "product", "M": 13, "N": 1001, "K": 2080, "fmt": "a32", "x": "f16", "out": "f32"},
        # a short prompt's projection
        {"name": "product short prompt", "op": "product", "M": 186, "N": 4096, "K": 4096, "fmt": "b32", "x": "bf16",
         "out": "bf16"},
        # a long prompt's projection: bound by the matrix units
        {"name": "product prompt", "op": "product", "M": 13312, "N": 4096, "K": 4096, "fmt": "b32", "x": "f16", "out": "f16"},
        # one decoded token through a 16-bit layer with a shared expert
        {"name": "decode token", "op": "decode", "T": 1, "D": 2048, "F": 768, "E": 128, "k": 8, "shared": 1, "cap": 0.0,
         "w": "bf16", "x": "bf16", "router": False},
        # one decoded token through a 4-bit layer, router included
        {"name": "decode token 4-bit", "op": "decode", "T": 1, "D": 4096, "F": 2048, "E": 256, "k": 8, "shared": 0, "cap": 0.0,
         "w": "b32", "x": "f16", "router": True},
        # three users' tokens on a small layer of odd sizes, a limit that drops pairs
        {"name": "decode ragged", "op": "decode", "T": 3, "D": 640, "F": 384, "E": 33, "k": 3, "shared": 0, "cap": 1.5,
         "w": "a64", "x": "bf16", "router": False},
        # a step of eight users on the 4-bit layer
        {"name": "decode batch 4-bit", "op": "decode", "T": 8, "D": 4096, "F": 2048, "E": 256, "k": 8, "shared": 0, "cap": 0.0,
         "w": "b32", "x": "f16", "router": False},
        # a step of sixteen users on the 16-bit layer with a shared expert
        {"name": "decode batch", "op": "decode", "T": 16, "D": 2048, "F": 768, "E": 128, "k": 8, "shared": 1, "cap": 0.0,
         "w": "bf16", "x": "bf16", "router": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in lo .. hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "product", "decode", "decode", "decode"])
    fmt = rng.choice(["b32", "a32", "a64"])
    if op == "quant":
        return {"op": op, "rows": _log(rng, 64, 65536), "K": _log(rng, 128, 4096, _GROUP[fmt]), "fmt": fmt,
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "product":
        M = _log(rng, 1, 13312)
        return {"op": op, "M": M, "N": _log(rng, 64, 65536 if M <= 64 else 4096), "K": _log(rng, 128, 4096, _GROUP[fmt]),
                "fmt": fmt, "x": rng.choice(["f16", "bf16"]), "out": rng.choice(["f32", "bf16", "f16"])}
    E = rng.choice([8, 16, 33, 64, 128])
    x = rng.choice(["f16", "bf16"])
    w = rng.choice([x, x, fmt])
    wide = 1 if w == x else 2   # 4-bit layers are the larger ones
    return {"op": op, "T": rng.randint(1, 16), "D": 128 * rng.randint(1, 16 * wide), "F": 128 * rng.randint(1, 8 * wide),
            "E": E, "k": rng.randint(1, min(8, E // 2)), "shared": rng.randint(0, 1), "cap": rng.choice([0.0, 0.0, 1.5]),
            "w": w, "x": x, "router": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------

def _gen(seed, case):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + len(str(sorted(case.items()))))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, R, K, dtype):
    """Rows as a norm gives them: a few channels much wider than the rest."""
    v = _randn(g, R, K)
    wide = torch.rand(1, K, generator=g, device="cuda") < 0.01
    return torch.where(wide, v * 10.0, v).to(_DT[dtype])


def _trained(g, N, K):
    """A trained matrix: rows of somewhat different sizes."""
    return _randn(g, N, K) * torch.exp(0.2 * _randn(g, N, 1)) * (K ** -0.5)


def _matrices(g, n, N, K, kind):
    """n matrices [N, K] in 16 bits, or 4-bit codes and parameters, made one at a time."""
    if kind in _DT:
        w = torch.empty(n, N, K, dtype=_DT[kind], device="cuda")
        for i in range(n):
            w[i] = _trained(g, N, K)
        return w
    G = _GROUP[kind]
    data = torch.empty(n, N, K // 2, dtype=torch.uint8, device="cuda")
    params = torch.empty(*((n, N, K // G) if kind == "b32" else (n, N, K // G, 2)), dtype=torch.float16, device="cuda")
    for i in range(n):
        q, params[i] = _quantise(_trained(g, N, K), kind)
        data[i] = _pack(q)
    return data, params


def prepare(case, seed):
    g = _gen(seed, case)
    st = dict(case)
    if case["op"] == "quant":
        v = torch.empty(case["rows"], case["K"], dtype=_DT[case["dtype"]], device="cuda")
        for at in range(0, case["rows"], 8192):
            v[at:at + 8192] = _trained(g, min(8192, case["rows"] - at), case["K"])
        st["v"] = v
    elif case["op"] == "product":
        st["rows_x"] = _rows(g, case["M"], case["K"], case["x"])
        data, params = _matrices(g, 1, case["N"], case["K"], case["fmt"])
        st["weight"] = (data[0], params[0])
    else:
        T, D, F, E, n = case["T"], case["D"], case["F"], case["E"], case["E"] + case["shared"]
        st["rows_x"] = _rows(g, T, D, case["x"])
        st["logits"] = st["map"] = None
        if case["router"]:
            st["map"] = (_randn(g, E, D) * (D ** -0.5)).to(_DT[case["x"]])
        else:
            st["logits"] = _randn(g, T, E)
        st["gate_w"] = _matrices(g, n, F, D, case["w"])
        st["up_w"] = _matrices(g, n, F, D, case["w"])
        st["down_w"] = _matrices(g, n, D, F, case["w"])
    return st


# ---- plain forms ------------------------------------------------------------

def _over(a, b):
    """a / b for a tensor b: a quotient by a number may become a product with its reciprocal, rounded twice."""
    return torch.div(a, torch.full_like(a, b) if not torch.is_tensor(b) else b)


def _quantise(v, fmt):
    """Codes (f32, [.., K]) and fp16 parameters of rows."""
    G = _GROUP[fmt]
    b = v.float().reshape(*v.shape[:-1], v.shape[-1] // G, G)
    if fmt == "b32":
        s = _over(b.abs().amax(-1), 7.0).half()
        sf = s.float().unsqueeze(-1)
        q = torch.clamp(torch.round(torch.div(b, sf.expand_as(b))), -8.0, 7.0)
        return torch.where(sf == 0, 0.0, q).reshape(v.shape), s
    lo, hi = b.amin(-1), b.amax(-1)
    s, bias = _over(hi - lo, 15.0).half(), lo.half()
    sf = s.float().unsqueeze(-1)
    q = torch.clamp(torch.round(torch.div(b - bias.float().unsqueeze(-1), sf.expand_as(b))), 0.0, 15.0)
    return torch.where(sf == 0, 0.0, q).reshape(v.shape), torch.stack([s, bias], -1)


def _pack(q):
    """Codes to bytes, the even K index in the low nibble."""
    n = q.to(torch.int16) & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)


def _codes(data, signed, dtype):
    n = torch.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1)
    if signed:
        n = n ^ 8
        return n.to(dtype) - 8.0
    return n.to(dtype)


def _values(w, dtype=torch.float32):
    """The values [.., N, K] that weights stand for."""
    if torch.is_tensor(w):
        return w.to(dtype)
    data, params = w
    signed = params.dim() == data.dim()
    q = _codes(data, signed, dtype)
    groups = params.shape[-1] if signed else params.shape[-2]
    q = q.reshape(*q.shape[:-1], groups, -1)
    if signed:
        q = q * params.to(dtype).unsqueeze(-1)
    else:
        q = q * params[..., 0].to(dtype).unsqueeze(-1) + params[..., 1].to(dtype).unsqueeze(-1)
    return q.flatten(-2)


def _limit(case):
    if not case["cap"]:
        return None
    return max(1, math.floor(case["cap"] * case["T"] * case["k"] / case["E"]))


def _chosen(logits, k, limit):
    """Experts [T, k], their weights and which pairs are kept (in token order)."""
    T, E = logits.shape
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, w = order.indices[:, :k], torch.softmax(order.values[:, :k], 1)
    if limit is None:
        return ids, w
    taken = torch.zeros(T, E, dtype=torch.int32, device=logits.device).scatter_(1, ids, 1)
    earlier = torch.cumsum(taken, 0) - taken
    return ids, torch.where(earlier.gather(1, ids) < limit, w, torch.zeros_like(w))


def _pick(w, ids):
    return w[ids] if torch.is_tensor(w) else (w[0][ids], w[1][ids])


def _decode_plain(st):
    x = st["rows_x"].float()
    logits = st["logits"] if st["map"] is None else x @ st["map"].float().t()
    ids, w = _chosen(logits, st["k"], _limit(st))
    y = []
    for t in range(st["T"]):
        e, we = ids[t], w[t]
        if st["shared"]:
            e, we = torch.cat([e, torch.full_like(e[:1], st["E"])]), torch.cat([we, torch.ones_like(we[:1])])
        g = (_values(_pick(st["gate_w"], e)) @ x[t]).clamp_max(_CLAMP)
        u = (_values(_pick(st["up_w"], e)) @ x[t]).clamp(-_CLAMP, _CLAMP)
        h = g / (1.0 + torch.exp(-g)) * u
        o = (_values(_pick(st["down_w"], e)) * h.unsqueeze(1)).sum(-1)
        y.append((o * we.unsqueeze(1)).sum(0))
    y = torch.stack(y).to(st["rows_x"].dtype)
    return y if st["map"] is None else (y, logits)


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "quant":
        q, params = _quantise(st["v"], st["fmt"])
        G = _GROUP[st["fmt"]]
        q = q.reshape(q.shape[0], -1, G)
        if st["fmt"] == "b32":
            q = q * params.float().unsqueeze(-1)
        else:   # the code's product is exact, the sum rounded once to f64, then to fp16
            q = (q * params[..., :1].float()).double() + params[..., 1:].double()
        return q.flatten(1).half(), params
    if st["op"] == "product":
        return (st["rows_x"].float() @ _values(st["weight"]).t()).to(_DT[st["out"]])
    return _decode_plain(st)


def _run_own(st):
    import mixture_experts_routed_route_amd as moe

    if st["op"] == "quant":
        kind = {"b32": moe.MOE_Q4B32, "a32": moe.MOE_Q4A32, "a64": moe.MOE_Q4A64}[st["fmt"]]
        data, params = moe.moe_quant_q4_weights(st["v"], kind)
        return moe.moe_dequant_weights(data, params), params
    if st["op"] == "product":
        return moe.moe_gemm_q4(st["rows_x"], st["weight"], out_dtype=_DT[st["out"]])
    y, logits = moe.moe_decode(st["rows_x"], st["gate_w"], st["up_w"], st["down_w"], st["k"], logits=st["logits"],
                               w_router=st["map"], capacity_factor=st["cap"], n_shared=st["shared"],
                               y_dtype=st["rows_x"].dtype)
    return y if st["map"] is None else (y, logits)


# ---- work -------------------------------------------------------------------

_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_PER = {"bf16": 2.0, "f16": 2.0, "b32": 0.5 + 2 / 32, "a32": 0.5 + 4 / 32, "a64": 0.5 + 4 / 64}   # bytes a weight


def work(case):
    if case["op"] == "quant":
        # codes are read again for the values that they stand for
        vals = case["rows"] * case["K"]
        return {"bytes": vals * (_SIZE[case["dtype"]] + 2 * _PER[case["fmt"]] + 2), "flops": 5 * vals}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K * _PER[case["fmt"]] + M * N * _SIZE[case["out"]], "flops": 2 * M * N * K}
    T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "k"))
    touched = E * (1 - (1 - k / E) ** T) + case["shared"]
    limit = _limit(case)
    pairs = T * (k + case["shared"]) if limit is None else min(T * k, E * limit) + T * case["shared"]
    small = 4 * T * E + 2 * T * D * 2 + (2 * E * D if case["router"] else 0)
    return {"bytes": touched * 3 * D * F * _PER[case["w"]] + small, "flops": 6 * D * F * pairs}


# ---- exact ------------------------------------------------------------------

def _exact_quant(v, fmt):
    """Values and parameters by the definition; each rounding to f32 or fp16 of an f64 value is written out."""
    rows, K = v.shape
    G = _GROUP[fmt]
    v = v.double().view(rows, K // G, G)
    if fmt == "b32":
        top = torch.maximum(v.max(-1).values, -v.min(-1).values)
        s = (top / 7.0).float().half().double()
        safe = torch.where(s == 0, torch.ones_like(s), s).unsqueeze(-1)
        q = torch.round((v / safe).float().double()).clamp(-8, 7) * (s != 0).unsqueeze(-1)
        return (q * s.unsqueeze(-1)).reshape(rows, K), s
    lo, hi = v.min(-1).values, v.max(-1).values
    s = ((hi - lo).float().double() / 15.0).float().half().double()
    b = lo.half().double()
    safe = torch.where(s == 0, torch.ones_like(s), s).unsqueeze(-1)
    d = (v - b.unsqueeze(-1)).float().double()
    q = torch.round((d / safe).float().double()).clamp(0, 15) * (s != 0).unsqueeze(-1)
    return (q * s.unsqueeze(-1) + b.unsqueeze(-1)).reshape(rows, K), torch.stack([s, b], -1)


def _exact_matrix(w, i=None):
    """One weight matrix in f64, byte by byte."""
    if torch.is_tensor(w):
        return w[i].double()
    data, params = (w[0], w[1]) if i is None else (w[0][i], w[1][i])
    N, half = data.shape
    q = torch.empty(N, 2 * half, dtype=torch.float64, device=data.device)
    q[:, 0::2] = torch.remainder(data, 16).double()
    q[:, 1::2] = torch.div(data, 16, rounding_mode="floor").double()
    if params.dim() == 2:
        q = torch.where(q > 7, q - 16, q)
        return q * params.double().repeat_interleave(2 * half // params.shape[1], 1)
    p = params.double().repeat_interleave(2 * half // params.shape[1], 1)
    return q * p[..., 0] + p[..., 1]


def _exact_decode(case, st):
    T, E, k = case["T"], case["E"], case["k"]
    x = st["rows_x"].double()
    logits = st["logits"].double() if st["map"] is None else torch.matmul(x, st["map"].double().t().contiguous())
    # by value, then by index
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    top = logits.gather(1, ids)
    p = torch.exp(top - top[:, :1])
    p = (p / p.sum(1, keepdim=True)).tolist()
    ids = ids.tolist()
    limit = _limit(case) or T
    y = torch.zeros(T, case["D"], dtype=torch.float64, device=x.device)
    users = {}
    for t in range(T):
        for j, e in enumerate(ids[t]):
            users.setdefault(e, []).append((t, p[t][j]))
    if case["shared"]:
        users[E] = [(t, 1.0) for t in range(T)]
    for e, pairs in users.items():
        kept = pairs if e == E else pairs[:limit]
        wg, wu, wd = (_exact_matrix(st[n], e) for n in ("gate_w", "up_w", "down_w"))
        for t, weight in kept:
            g = torch.mv(wg, x[t])
            g = torch.minimum(g, torch.full_like(g, _CLAMP))
            u = torch.mv(wu, x[t])
            u = torch.maximum(torch.minimum(u, torch.full_like(u, _CLAMP)), torch.full_like(u, -_CLAMP))
            y[t] += weight * torch.mv(wd, g * torch.sigmoid(g) * u)
    return y if st["map"] is None else (y, logits)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(st["v"], case["fmt"])
    if case["op"] == "product":
        w = _exact_matrix(st["weight"])
        return torch.matmul(st["rows_x"].double(), w.t().contiguous())
    return _exact_decode(case, st)
