"""Operators of training on INT8 weights: their cases, inputs, plain forms and definitions.

Three operators that stand beside the Q-GaLore step and the products of a linear layer whose
weight is held in INT8 codes W_q with one fp32 scale per 256 flat elements:

  orthogonalize / muon_step   the momentum M <- mu M + G, N = G + mu M, its orthogonal part O by
                              Newton-Schulz products (X0 = N / (|N|_F + eps), A = X X^T,
                              X <- a X + (b A + c A A) X), and W <- W - lr alpha O with the
                              unbiased stochastic rounding of the INT8 weights
  linear_fwd / linear_bwd     Y = act(X W~^T + bias) + residual and its gradients
                              dZ = dY act'(Z), dbias = sum_t dZ, dX = dZ W~, G = dZ^T X
  norm_fwd / norm_bwd         layer norm (or with center = False the norm by the root mean
                              square) over the last dimension, and its gradients

`own` chooses between the plain form in elementary torch operations and this package's entry
points.
"""
import math

import numpy as np
import torch

own = False

GROUP = 256                                 # weights per INT8 scale
COEF = (3.4445, -4.7750, 2.0315)            # a, b, c of the Newton-Schulz polynomial
NS_STEPS = 5
NS_EPS = 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01
SEED = 1234                                 # of the stochastic rounding
NORM_EPS = 1e-5


# ------------------------------------------------------------------------------- cases ---
def listed():
    return [
        # one attention matrix of a small model: launches and dependent products, latency
        {"name": "orth_512", "op": "orth", "count": 1, "m": 512, "n": 512},
        # matrices that are no multiple of a tile, taller than wide
        {"name": "orth_ragged", "op": "orth", "count": 3, "m": 1360, "n": 1004},
        # the four attention matrices of one 7B block
        {"name": "orth_4096x4", "op": "orth", "count": 4, "m": 4096, "n": 4096},
        # gate and up of all blocks of the 60M set, in one call
        {"name": "muon_60m", "op": "muon", "count": 16, "m": 1376, "n": 512, "nesterov": True},
        # down of 1B blocks: rows of 5461 weights
        {"name": "muon_1b", "op": "muon", "count": 4, "m": 2048, "n": 5461, "nesterov": True},
        # down of 7B blocks
        {"name": "muon_7b", "op": "muon", "count": 2, "m": 4096, "n": 11008, "nesterov": True},
        # one token through the gate projection of a 7B block
        {"name": "fwd_token", "op": "fwd", "T": 1, "m": 11008, "n": 4096, "act": "silu",
         "bias": True, "residual": False, "keep": False},
        # a training batch through the up projection, keeping what the backward pass takes
        {"name": "fwd_batch", "op": "fwd", "T": 4096, "m": 11008, "n": 4096, "act": "gelu",
         "bias": True, "residual": False, "keep": True},
        # its backward pass
        {"name": "bwd_batch", "op": "bwd", "T": 4096, "m": 11008, "n": 4096, "act": "gelu",
         "bias": True},
        # a ragged batch of the 60M set's gate layer
        {"name": "bwd_ragged", "op": "bwd", "T": 1000, "m": 1376, "n": 512, "act": "silu",
         "bias": True},
        # the norm before a 7B block's products, forward and backward
        {"name": "norm_fwd_batch", "op": "nfwd", "T": 8192, "n": 4096, "center": True,
         "dtype": "bf16"},
        {"name": "norm_bwd_batch", "op": "nbwd", "T": 8192, "n": 4096, "center": True,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(round(v / mult)) * mult)


def draw(rng):
    op = rng.choice(["orth", "muon", "fwd", "bwd", "nfwd", "nbwd"])
    if op in ("orth", "muon"):
        count = rng.choice([1, 1, 2, 5])
        # several matrices lie behind one another, each on a 16-byte border
        m = _log(rng, 64, 4096, 16 if count > 1 else 1)
        n = _log(rng, 64, 4096)
        c = {"op": op, "count": count, "m": m, "n": n}
        if op == "muon":
            c["nesterov"] = rng.random() < 0.7
        return c
    if op in ("fwd", "bwd"):
        c = {"op": op, "T": _log(rng, 1, 4096), "m": _log(rng, 64, 8192, 8),
             "n": _log(rng, 64, 8192, 8),
             "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
             "bias": rng.random() < 0.7}
        if op == "fwd":
            c["residual"] = rng.random() < 0.5
            c["keep"] = rng.random() < 0.5
        return c
    return {"op": op, "T": _log(rng, 1, 8192), "n": _log(rng, 32, 8192),
            "center": rng.random() < 0.6, "dtype": rng.choice(["bf16", "fp32"])}


# ------------------------------------------------------------------------------ inputs ---
def _gradient(g, count, m, n, sigma, dev):
    """A few strong directions over a floor of noise, as a layer's gradient has them."""
    r = max(4, min(m, n) // 32)
    a = torch.randn(count, m, r, generator=g, device=dev)
    b = torch.randn(count, r, n, generator=g, device=dev)
    s = torch.linspace(1.5, 0.5, r, device=dev) / math.sqrt(r)
    return sigma * (torch.matmul(a * s, b)
                    + 0.3 * torch.randn(count, m, n, generator=g, device=dev))


def _weights(g, count, m, n, dev):
    q = torch.randint(-127, 128, (count, m, n), generator=g, device=dev, dtype=torch.int8)
    s = (0.5 + 1.5 * torch.rand(count, -(-m * n // GROUP), generator=g, device=dev)) * 1e-3
    return q, s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}

    def bf16(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g, device=dev)).to(torch.bfloat16)

    if op in ("orth", "muon"):
        count, m, n = case["count"], case["m"], case["n"]
        st["G"] = _gradient(g, count, m, n, 1e-3, dev).to(torch.bfloat16)
        if op == "muon":
            st["M"] = _gradient(g, count, m, n, 5e-3, dev)
            st["Wq"], st["Ws"] = _weights(g, count, m, n, dev)
            st["W"] = torch.empty(count, m, n, dtype=torch.bfloat16, device=dev)
            st["t"] = 7
    elif op in ("fwd", "bwd"):
        T, m, n = case["T"], case["m"], case["n"]
        q, s = _weights(g, 1, m, n, dev)
        st["Wq"], st["Ws"] = q[0], s[0]
        st["X"] = bf16(T, n)
        if op == "fwd":
            st["bias"] = (torch.randn(m, generator=g, device=dev) if case["bias"] else None)
            st["residual"] = bf16(T, m) if case["residual"] else None
        else:
            st["Z"] = bf16(T, m, scale=2.0) if case["act"] != "none" else None
            st["dY"] = bf16(T, m)
    else:
        T, n = case["T"], case["n"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # activations: a spread of their own in every row, and a mean away from zero
        x = torch.randn(T, n, generator=g, device=dev)
        x = x * (0.5 + 2 * torch.rand(T, 1, generator=g, device=dev)) + 0.5
        st["X"] = x.to(dt)
        st["gamma"] = 1 + 0.2 * torch.randn(n, generator=g, device=dev)
        st["beta"] = 0.2 * torch.randn(n, generator=g, device=dev) if case["center"] else None
        if op == "nbwd":
            st["dY"] = torch.randn(T, n, generator=g, device=dev).to(dt)
            x = st["X"].double()
            mean = x.mean(1) if case["center"] else torch.zeros(T, device=dev).double()
            var = (x - mean[:, None]).square().mean(1)
            st["mean"] = mean.float() if case["center"] else None
            st["rstd"] = (var + NORM_EPS).rsqrt().float()
    return st


# ------------------------------------------------------------------------- plain forms ---
def _uniform(seed, step, layers, m, n, dev):
    """The rounding's uniforms: 16-bit halves of Philox4x32-10 with key = seed and counter =
    (column >> 3, row, step, layer); word (column >> 1) & 3, low half for even columns."""
    lo32 = 0xFFFFFFFF
    n8 = -(-n // 8)
    shape = (layers, m, n8)
    c0 = torch.arange(n8, device=dev).expand(shape)
    c1 = torch.arange(m, device=dev)[:, None].expand(shape)
    c2 = torch.full(shape, step, device=dev, dtype=torch.int64)
    c3 = torch.arange(layers, device=dev)[:, None, None].expand(shape)
    k0, k1 = seed & lo32, (seed >> 32) & lo32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57     # 64-bit products, wrapping
        c0, c1, c2, c3 = (((p1 >> 32) & lo32) ^ c1 ^ k0, p1 & lo32,
                          ((p0 >> 32) & lo32) ^ c3 ^ k1, p0 & lo32)
        k0, k1 = (k0 + 0x9E3779B9) & lo32, (k1 + 0xBB67AE85) & lo32
    w = torch.stack((c0, c1, c2, c3), -1)
    bits = torch.stack((w & 0xFFFF, w >> 16), -1).reshape(layers, m, n8 * 8)[:, :, :n]
    return bits.float() * 2.0 ** -16


def _scales(s, m, n):
    """One scale for each weight."""
    return s.repeat_interleave(GROUP, -1)[..., : m * n].reshape(*s.shape[:-1], m, n)


def _newton_schulz(N):
    a, b, c = COEF
    x = N / (N.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(NS_STEPS):
        A = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * A + c * torch.matmul(A, A), x)
    return x.transpose(1, 2).contiguous() if tall else x


def _alpha(case):
    return math.sqrt(max(1.0, case["m"] / case["n"]))


def _plain_muon(st):
    c = st["case"]
    m, n = c["m"], c["n"]
    g = st["G"].float()
    st["M"].mul_(MOMENTUM).add_(g)
    N = g + MOMENTUM * st["M"] if c["nesterov"] else st["M"]
    U = (-LR * _alpha(c)) * _newton_schulz(N)
    s = _scales(st["Ws"], m, n)
    w = st["Wq"].float()
    d = w + (U * (1 / s) - (LR * DECAY) * w) + _uniform(SEED, st["t"], c["count"], m, n, g.device)
    q = d.floor().clamp(-127, 127)
    st["Wq"].copy_(torch.where(torch.isfinite(d), q, w))
    return {"M": st["M"], "W": (st["Wq"].float() * s).to(torch.bfloat16)}


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _dequant(st, m, n):
    """W~ = bf16(q s), the weight that the products of a linear layer take."""
    return (st["Wq"].float() * _scales(st["Ws"], m, n)).to(torch.bfloat16)


def _plain_fwd(st):
    c = st["case"]
    z = torch.matmul(st["X"].float(), _dequant(st, c["m"], c["n"]).float().t())
    if st["bias"] is not None:
        z = z + st["bias"]
    y = _act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = {"Y": y.to(torch.bfloat16)}
    if c["keep"]:
        out["Z"] = z.to(torch.bfloat16)
    return out


def _plain_bwd(st):
    c = st["case"]
    dz = st["dY"].float()
    if st["Z"] is not None:
        dz = dz * _act_grad(st["Z"].float(), c["act"])
    out = {"dX": torch.matmul(dz, _dequant(st, c["m"], c["n"]).float()).to(torch.bfloat16),
           "G": torch.matmul(dz.t(), st["X"].float()).to(torch.bfloat16)}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def _plain_norm_fwd(st):
    c = st["case"]
    x = st["X"].float()
    out = {}
    if c["center"]:
        mean = x.mean(1, keepdim=True)
        out["mean"] = mean[:, 0]
        x = x - mean
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + NORM_EPS)
    y = x * rstd * st["gamma"]
    if st["beta"] is not None:
        y = y + st["beta"]
    out["Y"], out["rstd"] = y.to(st["X"].dtype), rstd[:, 0]
    return out


def _plain_norm_bwd(st):
    c = st["case"]
    x, dy = st["X"].float(), st["dY"].float()
    h = (x - st["mean"][:, None] if c["center"] else x) * st["rstd"][:, None]
    dh = dy * st["gamma"]
    dx = dh - h * (dh * h).mean(1, keepdim=True)
    if c["center"]:
        dx = dx - dh.mean(1, keepdim=True)
    out = {"dX": (dx * st["rstd"][:, None]).to(st["X"].dtype), "dgamma": (dy * h).sum(0)}
    if c["center"]:
        out["dbeta"] = dy.sum(0)
    return out


# --------------------------------------------------------------- this package's calls ---
def _own(st):
    from quantized_rank_gradient_amd import binding as B

    c = st["case"]
    op = c["op"]
    if op == "orth":
        return B.orthogonalize(list(st["G"].unbind(0)), steps=NS_STEPS, coef=COEF, eps=NS_EPS)
    if op == "muon":
        if "muon" not in st:     # the layer table that a training program builds once
            layers = [B.MuonLayer(k, st["G"][k], st["Wq"][k], st["Ws"][k], st["M"][k])
                      for k in range(c["count"])]
            st["muon"] = B.Muon(layers, dict(lr=LR, momentum=MOMENTUM, nesterov=c["nesterov"],
                                             weight_decay=DECAY, alpha=_alpha(c), eps=NS_EPS,
                                             ns_steps=NS_STEPS, coef=COEF))
        st["muon"].step(st["t"], SEED)
        # the weights that the codes stand for
        size = c["m"] * c["n"]
        if size % GROUP == 0:
            torch.mul(st["Wq"].view(c["count"], -1, GROUP), st["Ws"][:, :, None],
                      out=st["W"].view(c["count"], -1, GROUP))
        else:
            torch.mul(st["Wq"], _scales(st["Ws"], c["m"], c["n"]), out=st["W"])
        return {"M": st["M"], "W": st["W"]}
    if op == "fwd":
        r = B.int8_linear_act_fwd(st["X"], st["Wq"], st["Ws"], bias=st["bias"],
                                  residual=st["residual"], act=c["act"], keep_z=c["keep"])
        return {"Y": r[0], "Z": r[1]} if c["keep"] else {"Y": r}
    if op == "bwd":
        dX, G, dbias = B.int8_linear_act_bwd(st["dY"], st["X"], st["Wq"], st["Ws"], Z=st["Z"],
                                             act=c["act"], bias=c["bias"])
        return {"dX": dX, "G": G, "dbias": dbias} if c["bias"] else {"dX": dX, "G": G}
    if op == "nfwd":
        Y, mean, rstd = B.norm_fwd(st["X"], st["gamma"], st["beta"], eps=NORM_EPS,
                                   center=c["center"])
        return {"Y": Y, "mean": mean, "rstd": rstd} if c["center"] else {"Y": Y, "rstd": rstd}
    dX, dgamma, dbeta = B.norm_bwd(st["dY"], st["X"], st["gamma"], st["mean"], st["rstd"],
                                   center=c["center"])
    out = {"dX": dX, "dgamma": dgamma}
    if c["center"]:
        out["dbeta"] = dbeta
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "orth":
        return list(_newton_schulz(state["G"].float()).to(torch.bfloat16).unbind(0))
    return {"muon": _plain_muon, "fwd": _plain_fwd, "bwd": _plain_bwd, "nfwd": _plain_norm_fwd,
            "nbwd": _plain_norm_bwd}[op](state)


# -------------------------------------------------------------------------------- work ---
def work(case):
    op = case["op"]
    if op in ("orth", "muon"):
        m, n, k = case["m"], case["n"], case["count"]
        p, q = min(m, n), max(m, n)
        # X X^T and A A are symmetric: half of each product
        flops = k * NS_STEPS * (p * p * q + p * p * p + 2 * p * p * q)
        io = m * n * 4                                    # G in, O out
        if op == "muon":
            io = m * n * (2 + 8 + 2) + -(-m * n // GROUP) * 4   # G, M in and out, W in and out
        return {"bytes": k * io, "flops": flops}
    if op in ("fwd", "bwd"):
        T, m, n = case["T"], case["m"], case["n"]
        w = m * n + -(-m * n // GROUP) * 4
        if op == "fwd":
            io = 2 * T * n + 2 * T * m * (1 + case["residual"] + case["keep"]) + 4 * m * case["bias"]
            return {"bytes": w + io, "flops": 2 * T * m * n}
        z = 1 if case["act"] != "none" else 0
        io = 2 * T * m * (1 + z) + 2 * T * n * 2 + 2 * m * n + 4 * m * case["bias"]
        return {"bytes": w + io, "flops": 4 * T * m * n}
    T, n = case["T"], case["n"]
    e = 2 if case["dtype"] == "bf16" else 4
    k = 2 if case["center"] else 1
    if op == "nfwd":
        return {"bytes": 2 * T * n * e + 4 * k * (T + n), "flops": 8 * T * n}
    return {"bytes": 3 * T * n * e + 4 * (k * T + n + k * n), "flops": 14 * T * n}


# ------------------------------------------------------------------- exact definitions ---
def _philox_numpy(seed, step, layer, m, n):
    """The uniforms of one layer, word by word as the generator is defined."""
    u64, mask = np.uint64, np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    n8 = -(-n // 8)
    ctr = [np.broadcast_to(np.arange(n8, dtype=u64)[None, :], (m, n8)),
           np.broadcast_to(np.arange(m, dtype=u64)[:, None], (m, n8)),
           np.full((m, n8), step, u64), np.full((m, n8), layer, u64)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = ctr[0] * u64(0xD2511F53), ctr[2] * u64(0xCD9E8D57)
        ctr = [(b >> sh) ^ ctr[1] ^ u64(key[0]), b & mask,
               (a >> sh) ^ ctr[3] ^ u64(key[1]), a & mask]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    out = np.empty((m, n8, 8))
    for w in range(4):
        out[:, :, 2 * w] = (ctr[w] & u64(0xFFFF)).astype(np.float64)
        out[:, :, 2 * w + 1] = (ctr[w] >> u64(16)).astype(np.float64)
    return out.reshape(m, n8 * 8)[:, :n] / 65536.0


def _polar64(N):
    """p_5(...p_1(N / (|N| + eps))) for the odd polynomial p(x) = a x + b x^3 + c x^5."""
    a, b, c = COEF
    x = N / (torch.linalg.norm(N) + NS_EPS)
    wide = x.shape[0] <= x.shape[1]
    for _ in range(NS_STEPS):
        if wide:
            g = x @ x.T
            x = a * x + b * (g @ x) + c * (g @ (g @ x))
        else:
            g = x.T @ x
            x = a * x + b * (x @ g) + c * ((x @ g) @ g)
    return x


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "orth":
        return [_polar64(g.double()) for g in st["G"]]
    if op == "muon":
        m, n = case["m"], case["n"]
        M = MOMENTUM * st["M"].double() + st["G"].double()
        W = torch.empty(case["count"], m, n, dtype=torch.float64, device=M.device)
        idx = torch.arange(m * n, device=M.device).div(GROUP, rounding_mode="floor")
        for k in range(case["count"]):
            N = st["G"][k].double() + MOMENTUM * M[k] if case["nesterov"] else M[k]
            s = st["Ws"][k].double()[idx].view(m, n)
            u = torch.from_numpy(_philox_numpy(SEED, st["t"], k, m, n)).to(M.device)
            q = st["Wq"][k].double()
            d = q * (1 - LR * DECAY) - LR * _alpha(case) * _polar64(N) / s + u
            W[k] = torch.clamp(torch.floor(d), -127, 127) * s
        return {"M": M, "W": W}
    if op in ("fwd", "bwd"):
        m, n, act = case["m"], case["n"], case["act"]
        idx = torch.arange(m * n, device=st["X"].device).div(GROUP, rounding_mode="floor")
        # the weight is defined in bf16, from the code and its scale in fp32
        W = (st["Wq"].float() * st["Ws"][idx].view(m, n)).to(torch.bfloat16).double()
        phi = lambda z: 0.5 * torch.special.erfc(-z / math.sqrt(2.0))  # noqa: E731
        tz = lambda z: torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))  # noqa: E731
        if op == "fwd":
            z = st["X"].double() @ W.T
            if st["bias"] is not None:
                z = z + st["bias"].double()[None, :]
            y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
                 "gelu": lambda: z * phi(z), "gelu_tanh": lambda: z * (1 + tz(z)) / 2,
                 "silu": lambda: z / (1 + torch.exp(-z))}[act]()
            if st["residual"] is not None:
                y = y + st["residual"].double()
            return {"Y": y, "Z": z} if case["keep"] else {"Y": y}
        dz = st["dY"].double()
        if act != "none":
            z = st["Z"].double()
            e = 1 / (1 + torch.exp(-z))
            t = tz(z)
            dz = dz * {"relu": lambda: (z > 0).double(),
                       "gelu": lambda: phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                       "gelu_tanh": lambda: (1 + t) / 2 + z / 2 * (1 - t ** 2)
                       * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2),
                       "silu": lambda: e + z * e * (1 - e)}[act]()
        out = {"dX": dz @ W, "G": dz.T @ st["X"].double()}
        if case["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    x = st["X"].double()
    n = x.shape[1]
    gamma = st["gamma"].double()
    if op == "nfwd":
        mean = x.sum(1) / n if case["center"] else torch.zeros_like(x[:, 0])
        rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / n + NORM_EPS)
        y = (x - mean[:, None]) * rstd[:, None] * gamma
        if not case["center"]:
            return {"Y": y, "rstd": rstd}
        return {"Y": y + st["beta"].double(), "mean": mean, "rstd": rstd}
    dy, rstd = st["dY"].double(), st["rstd"].double()[:, None]
    h = (x - st["mean"].double()[:, None]) * rstd if case["center"] else x * rstd
    dh = dy * gamma
    proj = (dh * h).sum(1, keepdim=True) / n
    base = dh.sum(1, keepdim=True) / n if case["center"] else 0.0
    out = {"dX": rstd * (dh - base - h * proj), "dgamma": torch.einsum("tn,tn->n", dy, h)}
    if case["center"]:
        out["dbeta"] = dy.sum(0)
    return out
