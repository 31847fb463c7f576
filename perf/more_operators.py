"""More operators of a training step on this package: their cases, inputs, plain forms and definitions.

  clip             the norm of all gradients of a model and their clipping: N = sqrt(sum g^2) over
                   every tensor, c = min(1, max_norm / (N + eps)), g <- c g
  residual norm    the norm behind a block and the one before the next, with the block's gate and
                   scales: p = norm1(u), h = alpha x + rho act(z) p, y = norm2(h); and its gradients
  FP8 layer        8-bit floating point with an fp32 scale for each run of 128 values or each block
                   of 128 x 128: s = max(amax / qmax, 2^-126), q = rne(x (1 / s)); quantization along
                   rows and columns, from bf16 or from the INT8 weights; the linear layer
                   Y = q(X) W^T and its gradients dX = q(dY) W, G = qT(dY)^T qT(X), where q() takes runs
                   along a row and qT() runs along a column

`own` chooses between the plain form in elementary torch operations and this package's entry points.
"""
import math

import torch

own = False

GROUP = 256                     # INT8 weights per scale
BLOCK = 128                     # FP8 values per scale, along the inner dimension of a product
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 57344.0, 2, -14)}
S_MIN = 2.0 ** -126
NORM_EPS = 1e-5
CLIP_EPS = 1e-6


# ------------------------------------------------------------------------------- cases ---
def listed():
    return [
        # all gradients of the 60M set: launches and latency
        {"name": "clip_60m", "op": "clip", "blocks": 8, "d": 512, "f": 1376, "max_norm": 1.0},
        # the gradients of four blocks of the 1B set (one of six pipeline stages), with odd rows
        {"name": "clip_1b_stage", "op": "clip", "blocks": 4, "d": 2048, "f": 5461, "max_norm": 1.0},
        # one generated token between two blocks of the 7B set
        {"name": "resnorm_token", "op": "rnf", "T": 1, "n": 4096, "dtype": "bf16", "center": False,
         "post": True, "gate": "", "per": 1, "rho": False, "alpha": 1.0},
        # a training batch of the 7B set with a gate for every value
        {"name": "resnorm_batch", "op": "rnf", "T": 8192, "n": 4096, "dtype": "bf16",
         "center": False, "post": True, "gate": "sigmoid", "per": 1, "rho": True, "alpha": 1.0},
        # its backward pass
        {"name": "resnorm_bwd", "op": "rnb", "T": 8192, "n": 4096, "dtype": "bf16",
         "center": False, "post": True, "gate": "sigmoid", "per": 1, "rho": True, "alpha": 1.0},
        # backward of sequences that each share one gate (four of 1000 tokens, width of the 1B set)
        {"name": "resnorm_bwd_shared", "op": "rnb", "T": 4000, "n": 2048, "dtype": "bf16",
         "center": True, "post": True, "gate": "none", "per": 1000, "rho": False, "alpha": 1.0},
        # activations before the down projection of the 7B set, for both of their products
        {"name": "quant_batch", "op": "quant", "T": 4096, "n": 11008, "fmt": "e4m3"},
        # a down projection of the 1B set: INT8 weights with rows of 5461
        {"name": "quant_weight", "op": "weight", "m": 2048, "n": 5461},
        # one generated token through a gate projection of the 7B set
        {"name": "fp8_token", "op": "fwd", "T": 1, "m": 11008, "n": 4096},
        # a training batch through it
        {"name": "fp8_batch", "op": "fwd", "T": 4096, "m": 11008, "n": 4096},
        # its backward pass, with gradients in the format of the wider range
        {"name": "fp8_bwd_batch", "op": "bwd", "T": 4096, "m": 11008, "n": 4096, "fmt": "e5m2"},
        # a ragged batch of the 60M set's gate projection
        {"name": "fp8_bwd_ragged", "op": "bwd", "T": 1000, "m": 1376, "n": 512, "fmt": "e4m3"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["clip", "rnf", "rnb", "quant", "weight", "fwd", "bwd"])
    if op == "clip":
        return {"op": op, "blocks": _log(rng, 1, 4), "d": _log(rng, 64, 2048),
                "f": _log(rng, 128, 5461), "max_norm": rng.choice([0.1, 1.0, 1e6])}
    if op in ("rnf", "rnb"):
        T = _log(rng, 1, 8192)
        gate = rng.choice(["", "none", "sigmoid", "tanh"])
        return {"op": op, "T": T, "n": _log(rng, 32, 8192), "dtype": rng.choice(["bf16", "fp32"]),
                "center": rng.random() < 0.5, "post": rng.random() < 0.7, "gate": gate,
                "per": rng.choice([1, _log(rng, 1, T), T]) if gate else 1,
                "rho": rng.random() < 0.5, "alpha": rng.choice([1.0, 1.5])}
    if op == "quant":
        return {"op": op, "T": _log(rng, 1, 4096), "n": _log(rng, 64, 11008),
                "fmt": rng.choice(["e4m3", "e5m2"])}
    if op == "weight":
        return {"op": op, "m": _log(rng, 64, 8192), "n": _log(rng, 64, 4096)}
    c = {"op": op, "T": _log(rng, 1, 4096), "m": _log(rng, 64, 11008), "n": _log(rng, 64, 4096)}
    if op == "bwd":
        c["fmt"] = rng.choice(["e4m3", "e5m2"])
    return c


# ------------------------------------------------------------------------------ inputs ---
def _quantize(x, fmt, rows):
    """FP8 codes of a matrix, as values in fp32, and their scales: runs of 128 along a row
    (rows = 1), or blocks of 128 x 128 (rows = 128). Scales as (runs along the row, rows or blocks)."""
    r, c = x.shape
    rb, cb = -(-r // rows), -(-c // BLOCK)
    qdt, qmax = FP8[fmt][:2]
    p = torch.zeros(rb * rows, cb * BLOCK, device=x.device)
    p[:r, :c] = x
    p = p.view(rb, rows, cb, BLOCK)
    amax = p.abs().amax((1, 3)).double()
    s = (amax / torch.full_like(amax, qmax)).float().clamp(min=S_MIN)
    inv = s.double().reciprocal().float()
    q = (p * inv[:, None, :, None]).to(qdt).float()
    return q.view(rb * rows, cb * BLOCK)[:r, :c], s.t().contiguous()


def _codes(q, fmt):
    """The codes as they are stored: rows padded with zeros to a multiple of 16."""
    r, c = q.shape
    out = torch.zeros(r, -(-c // 16) * 16, dtype=torch.uint8, device=q.device)
    out[:, :c] = q.to(FP8[fmt][0]).view(torch.uint8)
    return out.view(FP8[fmt][0])


def _act(z, gate):
    return torch.sigmoid(z) if gate == "sigmoid" else torch.tanh(z) if gate == "tanh" else z


def _stats64(v, center):
    mean = v.mean(1) if center else torch.zeros_like(v[:, 0])
    return mean, ((v - mean[:, None]).square().mean(1) + NORM_EPS).rsqrt()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if op == "clip":
        d, f = case["d"], case["f"]
        shapes = [(d, d)] * 4 + [(f, d)] * 2 + [(d, f)]
        st["G"] = []
        for _ in range(case["blocks"]):
            st["G"] += [(1e-3 * randn(*s)).to(torch.bfloat16) for s in shapes]
        # the gradients of all norms lie in one fp32 tensor
        st["G"].append(1e-2 * randn(2 * case["blocks"] * d))
        st["out"] = [torch.empty_like(t) for t in st["G"]]
    elif op in ("rnf", "rnb"):
        T, n, center = case["T"], case["n"], case["center"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a block's output with a spread of its own in every row, onto a larger stream
        st["U"] = (randn(T, n) * (0.5 + torch.rand(T, 1, generator=g, device=dev)) + 0.1).to(dt)
        st["X"] = (2 * randn(T, n) + 0.3).to(dt)
        st["Z"] = randn(-(-T // case["per"]), n).to(dt) if case["gate"] else None
        for k in (("g1", "g2") if case["post"] else ("g2",)):
            st[k] = 1 + 0.2 * randn(n)
            st["b" + k[1]] = 0.2 * randn(n) if center else None
        st["rho"] = 0.5 + 0.2 * randn(n) if case["rho"] else None
        if op == "rnb":
            st["dH"], st["dY"] = randn(T, n).to(dt), randn(T, n).to(dt)
            h, s1 = _residual(st, torch.float64)
            s2 = _stats64(h, center)
            st["H"] = h.to(dt)
            st["stats"] = torch.stack([*s1, *s2]).float()
    elif op == "quant":
        # activations: a few columns that are much larger than the rest
        x = randn(case["T"], case["n"]) * torch.exp(randn(case["n"]))
        st["X"] = x.to(torch.bfloat16)
    elif op == "weight":
        m, n = case["m"], case["n"]
        st["Wq"] = torch.randint(-127, 128, (m, n), generator=g, device=dev, dtype=torch.int8)
        s = 0.5 + 1.5 * torch.rand(-(-m * n // GROUP), generator=g, device=dev)
        st["Ws"] = s * 1e-3
    else:
        T, m, n = case["T"], case["m"], case["n"]
        q, st["S"] = _quantize(randn(m, n) / math.sqrt(n), "e4m3", BLOCK)
        st["X"] = randn(T, n).to(torch.bfloat16)
        if op == "fwd":
            st["W"] = _codes(q, "e4m3")
        else:
            # what the forward pass kept: the weight's transpose and the inputs' columns
            st["W"], st["S"] = _codes(q.t().contiguous(), "e4m3"), st["S"].t().contiguous()
            st["dY"] = (1e-2 * randn(T, m)).to(torch.bfloat16)
            xt, st["Xs"] = _quantize(st["X"].float().t().contiguous(), "e4m3", 1)
            st["Xt"] = _codes(xt, "e4m3")
            st["X"] = None
    return st


# ------------------------------------------------------------------------- plain forms ---
def _plain_clip(st):
    total = torch.zeros((), dtype=torch.float64, device=st["G"][0].device)
    for t in st["G"]:
        total += t.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    c = (st["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    return {"norm": norm.float(), "G": [(t.float() * c).to(t.dtype) for t in st["G"]]}


def _per_row(v, st):
    """One row of v for each token: row t // per."""
    T, per = st["case"]["T"], st["case"]["per"]
    return v if per == 1 else v.repeat_interleave(per, 0)[:T]


def _residual(st, dt):
    """h in `dt`, and the first norm's mean and rstd."""
    c = st["case"]
    p = st["U"].to(dt)
    stats = (torch.zeros_like(p[:, 0]), torch.zeros_like(p[:, 0]))
    if c["post"]:
        mean = p.mean(1) if c["center"] else stats[0]
        p = p - mean[:, None]
        rstd = torch.rsqrt(p.square().mean(1) + NORM_EPS)
        stats = (mean, rstd)
        p = p * rstd[:, None] * st["g1"].to(dt)
        if st["b1"] is not None:
            p = p + st["b1"].to(dt)
    if c["gate"]:
        p = p * _per_row(_act(st["Z"].to(dt), c["gate"]), st)
    if st["rho"] is not None:
        p = p * st["rho"].to(dt)
    return c["alpha"] * st["X"].to(dt) + p, stats


def _plain_rnf(st):
    c = st["case"]
    h, (mean1, rstd1) = _residual(st, torch.float32)
    mean2 = h.mean(1) if c["center"] else torch.zeros_like(mean1)
    d = h - mean2[:, None]
    rstd2 = torch.rsqrt(d.square().mean(1) + NORM_EPS)
    y = d * rstd2[:, None] * st["g2"]
    if st["b2"] is not None:
        y = y + st["b2"]
    dt = st["X"].dtype
    return {"H": h.to(dt), "Y": y.to(dt), "stats": torch.stack([mean1, rstd1, mean2, rstd2])}


def _norm_grad(dh, h, rstd, center):
    """Through h = (v - mean) rstd, from dh to dv."""
    r = dh - h * (dh * h).mean(1, keepdim=True)
    if center:
        r = r - dh.mean(1, keepdim=True)
    return r * rstd[:, None]


def _plain_rnb(st):
    c = st["case"]
    dt, center = st["U"].dtype, c["center"]
    mean1, rstd1, mean2, rstd2 = st["stats"]
    out = {}
    dy = st["dY"].float()
    hn = (st["H"].float() - mean2[:, None]) * rstd2[:, None]
    out["dg2"] = (dy * hn).sum(0)
    if center:
        out["db2"] = dy.sum(0)
    D = st["dH"].float() + _norm_grad(dy * st["g2"], hn, rstd2, center)
    out["dX"] = (c["alpha"] * D).to(dt)
    u = st["U"].float()
    if c["post"]:
        un = (u - mean1[:, None]) * rstd1[:, None]
        u = un * st["g1"]
        if st["b1"] is not None:
            u = u + st["b1"]
    gate = 1.0
    if c["gate"]:
        a = _act(st["Z"].float(), c["gate"])
        gate = _per_row(a, st)
    if st["rho"] is not None:
        out["drho"] = (D * u * gate).sum(0)
        D = D * st["rho"]
    if c["gate"]:
        dz = D * u
        if c["per"] > 1:
            whole = torch.zeros(len(a) * c["per"], c["n"], device=dz.device)
            whole[:c["T"]] = dz
            dz = whole.view(len(a), c["per"], c["n"]).sum(1)
        der = {"none": lambda: 1.0, "sigmoid": lambda: a * (1 - a), "tanh": lambda: 1 - a * a}
        out["dZ"] = (dz * der[c["gate"]]()).to(dt)
    dp = D * gate
    if c["post"]:
        out["dg1"] = (dp * un).sum(0)
        if center:
            out["db1"] = dp.sum(0)
        dp = _norm_grad(dp * st["g1"], un, rstd1, center)
    out["dU"] = dp.to(dt)
    return out


def _spread(s, rows, cols, per_rows):
    """One scale for each value of a rows x cols matrix."""
    s = s.t()
    if per_rows > 1:
        s = s.repeat_interleave(per_rows, 0)[:rows]
    return s.repeat_interleave(BLOCK, 1)[:, :cols]


def _values(x, fmt, rows):
    """What quantization makes of a matrix, in fp32."""
    q, s = _quantize(x, fmt, rows)
    return q * _spread(s, *x.shape, rows), s


def _plain_quant(st):
    fmt = st["case"]["fmt"]
    x = st["X"].float()
    v, s = _values(x, fmt, 1)
    vt, sc = _values(x.t().contiguous(), fmt, 1)
    bf16 = torch.bfloat16
    return {"V": v.to(bf16), "S": s, "Vt": vt.to(bf16), "St": sc}


def _int8(st):
    m, n = st["Wq"].shape
    s = st["Ws"].repeat_interleave(GROUP)[: m * n].view(m, n)
    return st["Wq"].float() * s


def _plain_weight(st):
    v, s = _values(_int8(st), "e4m3", BLOCK)
    v = v.to(torch.bfloat16)
    return {"V": v, "S": s, "Vt": v.t().contiguous(), "St": s.t().contiguous()}


def _weight(st):
    """W (fwd: m x n) or W^T (bwd: n x m) in fp32."""
    c = st["case"]
    m, n = (c["m"], c["n"]) if c["op"] == "fwd" else (c["n"], c["m"])
    return st["W"][:, :n].float() * _spread(st["S"], m, n, BLOCK)


def _plain_fwd(st):
    x = _values(st["X"].float(), "e4m3", 1)[0]
    return {"Y": torch.matmul(x, _weight(st).t()).to(torch.bfloat16)}


def _plain_bwd(st):
    c = st["case"]
    dy = st["dY"].float()
    dx = torch.matmul(_values(dy, c["fmt"], 1)[0], _weight(st).t())
    dyt = _values(dy.t().contiguous(), c["fmt"], 1)[0]
    xt = st["Xt"][:, :c["T"]].float() * _spread(st["Xs"], c["n"], c["T"], 1)
    return {"dX": dx.to(torch.bfloat16), "G": torch.matmul(dyt, xt.t()).to(torch.bfloat16)}


# --------------------------------------------------------------- this package's calls ---
def _own(st):
    from quantized_rank_gradient_amd import binding as B

    c = st["case"]
    op = c["op"]
    if op == "clip":
        if "set" not in st:      # the table of tensors that a training program keeps
            st["set"] = B.GradSet(st["G"], out=st["out"], eps=CLIP_EPS)
        return {"norm": st["set"].clip(c["max_norm"]), "G": st["out"]}
    if op in ("rnf", "rnb"):
        kw = dict(post=(st["g1"], st["b1"]) if c["post"] else None, pre=(st["g2"], st["b2"]),
                  gate=st["Z"], gate_act=c["gate"] or "none", per=c["per"], rho=st["rho"],
                  alpha=c["alpha"], center=c["center"])
        if op == "rnf":
            H, Y, stats = B.residual_norm_fwd(st["U"], st["X"], eps=NORM_EPS, **kw)
            return {"H": H, "Y": Y, "stats": stats}
        r = B.residual_norm_bwd(st["dH"], st["dY"], st["U"], st["H"], st["stats"], **kw)
        out = {"dX": r.dX, "dU": r.dU, "dg2": r.dpre[0]}
        if c["center"]:
            out["db2"] = r.dpre[1]
        if c["post"]:
            out["dg1"] = r.dpost[0]
            if c["center"]:
                out["db1"] = r.dpost[1]
        if c["gate"]:
            out["dZ"] = r.dgate
        if c["rho"]:
            out["drho"] = r.drho
        return out
    if op in ("quant", "weight"):
        if op == "quant":
            Q, S, Qt, St = B.fp8_quantize(st["X"], fmt=c["fmt"], columns=True)
            m, n, rows = c["T"], c["n"], 1
        else:
            Q, S, Qt, St = B.fp8_quantize(st["Wq"], scales=st["Ws"], block=True, columns=True)
            m, n, rows = c["m"], c["n"], BLOCK
        # the values that the codes stand for
        return {"V": B.fp8_dequantize(Q, S, n, block=rows > 1), "S": S,
                "Vt": B.fp8_dequantize(Qt, St, m, block=rows > 1), "St": St}
    if op == "fwd":
        return {"Y": B.fp8_linear_fwd(st["X"], st["W"], st["S"])}
    dX, G = B.fp8_linear_bwd(st["dY"], st["W"], st["S"], st["Xt"], st["Xs"], fmt=c["fmt"])
    return {"dX": dX, "G": G}


def run(state):
    if own:
        return _own(state)
    return {"clip": _plain_clip, "rnf": _plain_rnf, "rnb": _plain_rnb, "quant": _plain_quant,
            "weight": _plain_weight, "fwd": _plain_fwd, "bwd": _plain_bwd}[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- work ---
def work(case):
    op = case["op"]
    if op == "clip":
        d, f = case["d"], case["f"]
        w = case["blocks"] * (4 * d * d + 3 * d * f)
        v = case["blocks"] * 2 * d
        return {"bytes": 2 * (2 * w + 4 * v), "flops": 3 * (w + v)}
    if op in ("rnf", "rnb"):
        T, n = case["T"], case["n"]
        e = 2 if case["dtype"] == "bf16" else 4
        gate = -(-T // case["per"]) if case["gate"] else 0
        vec = (1 + case["center"]) * (1 + case["post"]) + case["rho"]
        stats = 4 * (1 + case["center"]) * (1 + case["post"]) * T
        if op == "rnf":
            return {"bytes": (4 * T + gate) * n * e + 4 * vec * n + stats, "flops": 20 * T * n}
        return {"bytes": (6 * T + 2 * gate) * n * e + 8 * vec * n + stats, "flops": 40 * T * n}
    if op in ("quant", "weight"):
        m, n = (case["T"], case["n"]) if op == "quant" else (case["m"], case["n"])
        if op == "quant":        # values in; both sets of values out
            scales = m * -(-n // BLOCK) + n * -(-m // BLOCK)
            return {"bytes": 6 * m * n + 4 * scales, "flops": 6 * m * n}
        scales = 2 * -(-m // BLOCK) * -(-n // BLOCK) + -(-m * n // GROUP)
        return {"bytes": 5 * m * n + 4 * scales, "flops": 6 * m * n}
    T, m, n = case["T"], case["m"], case["n"]
    w = m * n + 4 * -(-m // BLOCK) * -(-n // BLOCK)
    if op == "fwd":
        return {"bytes": w + 2 * T * (m + n), "flops": 2 * T * m * n}
    xt = T * n + 4 * n * -(-T // BLOCK)
    return {"bytes": w + xt + 2 * T * (m + n) + 2 * m * n, "flops": 4 * T * m * n}


# ------------------------------------------------------------------- exact definitions ---
def _round64(y, fmt):
    """Half to even onto the format's values, in float64: steps of 2^(e - digits) from the smallest
    exponent on. |y| <= qmax (1 + 2^-22) rounds to qmax at most."""
    _, _, digits, emin = FP8[fmt]
    e = torch.frexp(y)[1] - 1
    step = torch.pow(2.0, (e.clamp(min=emin) - digits).double())
    return torch.round(y / step) * step


def _fp8_64(x, fmt, rows):
    """Values and scales of quantized x (fp32 values held in float64). The scale, its reciprocal and
    x (1 / s) are fp32 numbers by definition; each is rounded from its 64-bit value."""
    m, n = x.shape
    cb, rb = math.ceil(n / BLOCK), math.ceil(m / rows)
    big = torch.nn.functional.pad(x.abs(), (0, cb * BLOCK - n, 0, rb * rows - m))
    amax = big.reshape(rb, rows, cb, BLOCK).transpose(1, 2).reshape(rb, cb, -1).max(2).values
    qmax = torch.tensor([FP8[fmt][1]], dtype=torch.float64, device=x.device)
    s = torch.maximum((amax / qmax).float(), torch.tensor(S_MIN, device=x.device)).double()
    one = torch.ones_like(s)
    inv = (one / s).float().double()
    ri = torch.arange(m, device=x.device) // rows
    ci = torch.arange(n, device=x.device) // BLOCK
    v = torch.empty_like(x)
    for a in range(0, m, 1024):          # rows at a time
        r = ri[a:a + 1024]
        y = (x[a:a + 1024] * inv[r][:, ci]).float().double()
        v[a:a + 1024] = _round64(y, fmt) * s[r][:, ci]
    return v, s.t()


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "clip":
        sq = sum(float(torch.dot(t.double().view(-1), t.double().view(-1))) for t in st["G"])
        norm = math.sqrt(sq)
        c = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "G": [t.double() * c for t in st["G"]]}
    if op in ("rnf", "rnb"):
        return _exact_residual(case, st)
    if op in ("quant", "weight"):
        if op == "quant":
            x = st["X"].double()
            v, s = _fp8_64(x, case["fmt"], 1)
            vt, sc = _fp8_64(x.T.contiguous(), case["fmt"], 1)
            return {"V": v, "S": s, "Vt": vt, "St": sc}
        i = torch.arange(case["m"] * case["n"], device=st["Ws"].device) // GROUP
        # the weight is the fp32 product of code and scale
        x = (st["Wq"].double() * st["Ws"].double()[i].view(case["m"], -1)).float().double()
        v, s = _fp8_64(x, "e4m3", BLOCK)
        return {"V": v, "S": s, "Vt": v.T, "St": s.T}
    T, m, n = case["T"], case["m"], case["n"]
    r, k = (m, n) if op == "fwd" else (n, m)
    dev = st["W"].device
    ri, ki = torch.arange(r, device=dev) // BLOCK, torch.arange(k, device=dev) // BLOCK
    w = st["W"].view(torch.uint8)[:, :k].view(torch.float8_e4m3fn).double()
    w = w * st["S"].double().T[ri][:, ki]
    if op == "fwd":
        return {"Y": _fp8_64(st["X"].double(), "e4m3", 1)[0] @ w.T}
    dy = st["dY"].double()
    xt = st["Xt"][:, :T].double() * st["Xs"].double().T[:, torch.arange(T, device=dev) // BLOCK]
    return {"dX": _fp8_64(dy, case["fmt"], 1)[0] @ w.T,
            "G": _fp8_64(dy.T.contiguous(), case["fmt"], 1)[0] @ xt.T}


def _exact_residual(case, st):
    center, per = case["center"], case["per"]
    f64 = {k: v.double() if torch.is_tensor(v) else v for k, v in st.items()}
    T, n = f64["U"].shape
    row = torch.arange(T, device=f64["U"].device) // per
    zero = torch.zeros(T, dtype=torch.float64, device=f64["U"].device)

    def stats(v):
        mu = v.sum(1) / n if center else zero
        return mu, 1 / torch.sqrt(((v - mu[:, None]) ** 2).sum(1) / n + NORM_EPS)

    def back(d, vh, r):
        proj = (d * vh).sum(1, keepdim=True) / n
        base = d.sum(1, keepdim=True) / n if center else 0.0
        return r[:, None] * (d - base - vh * proj)

    bias = lambda k: f64[k] if f64.get(k) is not None else 0.0  # noqa: E731
    fwd = case["op"] == "rnf"
    mu1, r1 = (zero, zero)
    if case["post"]:
        mu1, r1 = stats(f64["U"]) if fwd else f64["stats"][:2]
        uh = (f64["U"] - mu1[:, None]) * r1[:, None]
        p = uh * f64["g1"] + bias("b1")
    else:
        p = f64["U"]
    a, da = 1.0, None
    if case["gate"]:
        z = f64["Z"]
        if case["gate"] == "sigmoid":
            a = 1 / (1 + torch.exp(-z))
            da = torch.exp(-z) * a * a
        elif case["gate"] == "tanh":
            a = 1 - 2 / (torch.exp(2 * z) + 1)
            da = 1 / torch.cosh(z) ** 2
        else:
            a, da = z, torch.ones_like(z)
        a = a[row]
    rho = f64["rho"] if case["rho"] else 1.0
    if fwd:
        h = case["alpha"] * f64["X"] + rho * a * p
        mu2, r2 = stats(h)
        y = (h - mu2[:, None]) * r2[:, None] * f64["g2"] + bias("b2")
        return {"H": h, "Y": y, "stats": torch.stack([mu1, r1, mu2, r2])}
    mu2, r2 = f64["stats"][2:]
    hh = (f64["H"] - mu2[:, None]) * r2[:, None]
    D = f64["dH"] + back(f64["dY"] * f64["g2"], hh, r2)
    out = {"dX": case["alpha"] * D, "dg2": (f64["dY"] * hh).sum(0)}
    dp = D * rho * a
    if case["post"]:
        out["dU"], out["dg1"] = back(dp * f64["g1"], uh, r1), (dp * uh).sum(0)
        if center:
            out["db1"] = dp.sum(0)
    else:
        out["dU"] = dp
    if center:
        out["db2"] = f64["dY"].sum(0)
    if case["rho"]:
        out["drho"] = (D * a * p).sum(0)
    if case["gate"]:
        dz = D * rho * p
        groups = torch.zeros(len(f64["Z"]), n, dtype=torch.float64, device=dz.device)
        for k in range(0, T, 1024):
            groups.index_add_(0, row[k:k + 1024], dz[k:k + 1024])
        out["dZ"] = groups * da
    return out
