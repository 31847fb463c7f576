"""The linear layer with bias, activation and residual, forward and backward, against float64.

Tolerances. Both sides hold the same bf16 W~, X, dY and Z. fp32 sums of K products are off by
less than 2^-20 of the sum of their magnitudes (K <= 4096 here; the error grows like sqrt(K) 2^-24);
an activation and its derivative are at most 1.2 steep, evaluated in fp32 to a few units of 2^-23
of (1 + |z|), 2^-20 with room. Outputs are rounded to bf16: 2^-8 of the value. In the backward
pass dZ is rounded to bf16 before its products: at most 2^-8 of the sum of magnitudes, and, the
roundings of different terms being independent, no more than 2^-8 / sqrt(3) of the whole in the
2-norm, beside the output's own 2^-8 / sqrt(3): together 3.2e-3, 4e-3 with room for small sizes."""
import numpy as np
import pytest

from oracle import qgalore_oracle as O

torch = pytest.importorskip("torch")

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
U16, U20 = 2.0 ** -8, 2.0 ** -20


def B():
    from quantized_rank_gradient_amd import binding
    return binding


def bf16_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def bits(x):
    return O.f32_to_bf16_bits(np.asarray(x, np.float32))


def make(T, m, n, seed):
    rng = np.random.default_rng(seed)
    d = dict(Wq=rng.integers(-127, 128, size=(m, n)).astype(np.int8),
             Ws=(rng.uniform(0.5, 2.0, O.n_groups(m * n)) * 1e-3).astype(np.float32),
             X=bits(rng.standard_normal((T, n))), dY=bits(rng.standard_normal((T, m))),
             Z=bits(3 * rng.standard_normal((T, m))), res=bits(rng.standard_normal((T, m))),
             bias=rng.standard_normal(m).astype(np.float32))
    d["Wd"], d["Sd"] = torch.from_numpy(d["Wq"]).cuda(), torch.from_numpy(d["Ws"]).cuda()
    return d


def check_fwd(d, T, m, n, act, bias, res, keep):
    out = B().int8_linear_act_fwd(
        bf16_dev(d["X"]), d["Wd"], d["Sd"],
        bias=torch.from_numpy(d["bias"]).cuda() if bias else None,
        residual=bf16_dev(d["res"]) if res else None, act=act, keep_z=keep)
    Y, Z = O.linear_act_forward(d["X"], d["Wq"], d["Ws"], m, n, d["bias"] if bias else None,
                                d["res"] if res else None, act)
    mags = np.abs(O.bf16_bits_to_f32(d["X"]).astype(np.float64)) @ \
        np.abs(O.dequant_weight(d["Wq"], d["Ws"], m, n).astype(np.float64)).T
    err = 1.2 * U20 * (mags + np.abs(Z) + 1) + U20 * np.abs(Y)
    got = out if not keep else out[0]
    bad = np.abs(f64(got) - Y) > U16 * (np.abs(Y) + err) + err
    assert not bad.any(), (act, int(bad.sum()), float(np.abs(f64(got) - Y).max()))
    if keep:
        assert (np.abs(f64(out[1]) - Z) <= U16 * (np.abs(Z) + err) + err).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 200])
@pytest.mark.parametrize("m,n", [(8, 8), (24, 40), (136, 264), (264, 1376), (520, 512)])
def test_forward_sizes(T, m, n):
    d = make(T, m, n, T + 3 * m + n)
    check_fwd(d, T, m, n, "gelu", True, True, True)
    check_fwd(d, T, m, n, "none", False, False, False)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 40, 130])
@pytest.mark.parametrize("bias,res,keep", [(True, False, True), (False, True, False),
                                           (True, True, False)])
def test_forward_epilogues(act, T, bias, res, keep):
    check_fwd(make(T, 136, 200, T), T, 136, 200, act, bias, res, keep)


@pytest.mark.gpu
@pytest.mark.parametrize("T,m,n", [(300, 11008, 4096), (1, 4096, 11008), (64, 4096, 4096)])
def test_forward_7b_shapes(T, m, n):
    d = make(T, m, n, 1)
    check_fwd(d, T, m, n, "silu", True, False, False)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [17, 33, 63, 64, 65, 100, 127, 129, 250])
@pytest.mark.parametrize("m,n", [(2048, 1024), (4104, 192), (72, 2112)])
def test_forward_some_tokens(T, m, n):
    """Between few tokens and many, where the form of the product changes with the sizes."""
    d = make(T, m, n, T + m)
    check_fwd(d, T, m, n, "silu", True, True, True)
    check_fwd(d, T, m, n, "gelu_tanh", False, False, False)


@pytest.mark.gpu
@pytest.mark.parametrize("T,m,n", [(4090, 4344, 72), (1030, 4096, 200), (4090, 1032, 136)])
def test_forward_large_tiles(T, m, n):
    """Outputs of tiles of 256, the first with a last round of quarters."""
    check_fwd(make(T, m, n, 7), T, m, n, "gelu", True, True, True)


def check_bwd(d, T, m, n, act, bias=True, **kw):
    dX, G, db = B().int8_linear_act_bwd(
        bf16_dev(d["dY"]), bf16_dev(d["X"]), d["Wd"], d["Sd"],
        Z=bf16_dev(d["Z"]) if act != "none" else None, act=act, bias=bias, **kw)
    dZ, rdX, rG, rdb = O.linear_act_backward(d["dY"], d["Z"], d["X"], d["Wq"], d["Ws"], m, n, act)
    W = np.abs(O.dequant_weight(d["Wq"], d["Ws"], m, n).astype(np.float64))
    X = np.abs(O.bf16_bits_to_f32(d["X"]).astype(np.float64))
    za = np.abs(O.bf16_bits_to_f32(d["Z"]).astype(np.float64)) if act != "none" else 0.0
    # dZ: its rounding, and the derivative's evaluation
    ez = np.abs(O.bf16_bits_to_f32(d["dY"]).astype(np.float64)) * 1.2 * U20 * (1 + za)
    rel = 0.0 if act == "none" else U16
    for got, want, mags, emag in ((dX, rdX, np.abs(dZ) @ W, ez @ W),
                                  (G, rG, np.abs(dZ).T @ X, ez.T @ X)):
        if got is None:
            continue
        err = (rel + U20) * mags + 2 * emag
        g = f64(got)
        assert (np.abs(g - want) <= U16 * (np.abs(want) + err) + err).all(), act
        assert np.linalg.norm(g - want) <= 4e-3 * np.linalg.norm(want) + np.linalg.norm(emag), act
    if bias:
        assert (np.abs(f64(db) - rdb) <= U20 * np.abs(dZ).sum(0) + ez.sum(0)).all(), act
    return dX, G, db


@pytest.mark.gpu
@pytest.mark.parametrize("T,m,n", [(1, 8, 8), (7, 24, 40), (64, 136, 264), (129, 264, 136),
                                   (200, 520, 512), (300, 264, 1376), (515, 1376, 520)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_sizes(T, m, n, act):
    check_bwd(make(T, m, n, T + m + n), T, m, n, act)


@pytest.mark.gpu
@pytest.mark.parametrize("T,m,n", [(4090, 72, 4344), (72, 4096, 4344), (1500, 2000, 2048)])
def test_backward_large_tiles(T, m, n):
    check_bwd(make(T, m, n, 7), T, m, n, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_backward_activations(act):
    check_bwd(make(150, 136, 200, 5), 150, 136, 200, act)


@pytest.mark.gpu
def test_backward_7b_shape():
    check_bwd(make(256, 4096, 11008, 2), 256, 4096, 11008, "silu")


@pytest.mark.gpu
def test_backward_parts_equal_the_whole():
    d = make(130, 136, 72, 6)
    whole = check_bwd(d, 130, 136, 72, "gelu")
    b, dY, Z = B(), bf16_dev(d["dY"]), bf16_dev(d["Z"])
    dX, g, db = b.int8_linear_act_bwd(dY, None, d["Wd"], d["Sd"], Z=Z, act="gelu", need_G=False)
    assert g is None and db is None and torch.equal(dX, whole[0])
    dX, G, db = b.int8_linear_act_bwd(dY, bf16_dev(d["X"]), Z=Z, act="gelu", need_dX=False)
    assert dX is None and db is None and torch.equal(G, whole[1])
    dX, G, db = b.int8_linear_act_bwd(dY, Z=Z, act="gelu", bias=True, need_dX=False, need_G=False)
    assert dX is None and G is None and torch.equal(db, whole[2])


@pytest.mark.gpu
@pytest.mark.parametrize("T,m,n", [(1, 4104, 72), (5, 5000, 264), (64, 2056, 520), (3001, 72, 136),
                                   (40, 11008, 1024)])
def test_backward_long_sums_of_few_tiles(T, m, n):
    """Products of few tiles are cut along their inner dimension: the order in which the parts come
    does not show, nor a workspace's old content, nor what else is asked for."""
    b, d = B(), make(T, m, n, 9)
    whole = check_bwd(d, T, m, n, "silu")
    dY, X, Z = bf16_dev(d["dY"]), bf16_dev(d["X"]), bf16_dev(d["Z"])
    ws = b.alloc_workspace(b.lib().qgalore_int8_linear_act_bwd_workspace_bytes(T, m, n))
    out = [torch.empty_like(t) for t in whole]

    def run():
        b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], Z=Z, act="silu", dX=out[0], G=out[1],
                              dbias=out[2], workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for k in range(6):
        ws.fill_(0xFF)
        for t in out:
            t.zero_()
        g.replay() if k % 2 else run()
        assert all(torch.equal(x, y) for x, y in zip(out, whole)), k
    plain = check_bwd(d, T, m, n, "none")
    ws.fill_(0xFF)
    G = b.int8_linear_act_bwd(dY, X, need_dX=False, workspace=ws)[1]
    assert torch.equal(G, plain[1])
    ws.fill_(0xFF)
    dX = b.int8_linear_act_bwd(dY, None, d["Wd"], d["Sd"], need_G=False, workspace=ws)[0]
    assert torch.equal(dX, plain[0])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_extreme_values(act):
    """Z over all magnitudes of bf16: finite derivatives that go to their limits; a NaN in Z stays
    in its row and column."""
    T, m, n = 16, 64, 8
    d = make(T, m, n, 8)
    z = np.array([0.0, -0.0, 1e-38, -1e-38, 1e-20, 0.5, -0.5, 8, -8, 12.5, -12.5, 39, -39, 41, -41,
                  100, -100, 1e4, -1e4, 1e15, -1e15, 1e20, -1e20, 3e38, -3e38], np.float32)
    d["Z"] = bits(np.resize(z, (T, m)))
    check_bwd(d, T, m, n, act)
    if act == "none":
        return
    d["Z"][3, 5] = 0x7FC0
    dX, G, db = B().int8_linear_act_bwd(bf16_dev(d["dY"]), bf16_dev(d["X"]), d["Wd"], d["Sd"],
                                        Z=bf16_dev(d["Z"]), act=act, bias=True)
    assert np.isnan(f64(dX)[3]).all() and np.isfinite(np.delete(f64(dX), 3, 0)).all()
    assert np.isnan(f64(G)[5]).all() and np.isfinite(np.delete(f64(G), 5, 0)).all()
    assert np.isnan(f64(db)[5]) and np.isfinite(np.delete(f64(db), 5)).all()


def derivative64(z, act):
    """act'(z) in float64, accurate relative to its own size in the left tails too."""
    from scipy.special import expit, ndtr
    z = np.clip(np.asarray(z, np.float64), -200, 200)   # at its limits long before
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    if act == "silu":
        return expit(z) * (1 + z * expit(-z))
    u, w = tanh_argument(z)
    return expit(u) + z * expit(u) * expit(-u) * w


def tanh_argument(z):
    """2 u and its derivative for u = sqrt(2 / pi) (z + 0.044715 z^3)."""
    k = np.sqrt(2 / np.pi)
    return 2 * k * (z + 0.044715 * z ** 3), 2 * k * (1 + 3 * 0.044715 * z * z)


def derivative_error(z, act):
    """How far an fp32 derivative may be off. An exponential's argument y is rounded a few times, which
    moves its value by 2^-23 |y| of itself, and the exponential, reciprocal and polynomial by 2^-23 x 16:
    left of zero that is relative to the terms of the derivative, right of zero to what is missing to 1
    and 2^-22 of the terms. Values below 2^-126 count as zero, times |z| and the polynomial's slope."""
    from scipy.special import expit, ndtr
    z = np.clip(np.asarray(z, np.float64), -200, 200)
    zc = np.minimum(np.abs(z), 40)
    if act == "relu":
        return np.zeros_like(z)
    if act == "gelu":
        tail = ndtr(-np.abs(z)) + zc * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
        e = tail * 2.0 ** -23 * (z * z + 16)
    elif act == "silu":
        e = expit(z) * (1 + np.abs(z)) * 2.0 ** -23 * (np.abs(z) + 16) * (z < 0)
        e += 2.0 ** -22 * (1 + zc) * (z > 0)
    else:
        u, w = tanh_argument(z)
        e = (expit(u) + np.abs(z) * expit(u) * expit(-u) * w) * 2.0 ** -20 * (np.abs(u) + 1) * (z < 0)
        zc = np.minimum(zc, 6)       # s is 1 from there on
        e += 2.0 ** -22 * (1 + zc * tanh_argument(zc)[1]) * (z > 0)
    return e + 2.0 ** -22 * np.abs(derivative64(z, act)) + 2.0 ** -118


def every_magnitude():
    """bf16 values of both signs: dense about the transitions, their tails, and every power of ten."""
    z = np.concatenate([np.linspace(0, 15, 901), np.linspace(15, 130, 460),
                        [0.0, 1e-38, 1e-20, 1e-3, 1e3, 1e4, 1e15, 1e20, 3e38]])
    return O.bf16_bits_to_f32(bits(np.concatenate([z, -z, np.zeros((-2 * len(z)) % 8)])))


@pytest.mark.gpu
@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_activation_derivatives_one_by_one(act):
    """One token with dY = 1: dbias is the derivative at each z by itself, and with an identity for the
    weight dX is the same rounded to bf16 twice (the second time exactly)."""
    z = np.concatenate([every_magnitude(), np.float32([np.inf, -np.inf] * 4)])
    m = len(z)
    want, err = derivative64(z, act), derivative_error(z, act)
    dY, Z = torch.ones(1, m, dtype=torch.bfloat16).cuda(), bf16_dev(bits(z)).view(1, m)
    got = f64(B().int8_linear_act_bwd(dY, Z=Z, act=act, bias=True, need_dX=False, need_G=False)[2])
    bad = np.abs(got - want) > err
    assert not bad.any(), (act, z[bad][:8], got[bad][:8], want[bad][:8])
    eye = 64 * torch.eye(m, dtype=torch.int8).cuda()
    scale = torch.full((O.n_groups(m * m),), 2.0 ** -6).cuda()
    dX = f64(B().int8_linear_act_bwd(dY, None, eye, scale, Z=Z, act=act, need_G=False)[0])[0]
    # a value below bf16's smallest normal may lose bits or be zero
    assert (np.abs(dX - want) <= err + U16 * (np.abs(want) + err) + 2.0 ** -126).all(), act


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_a_wrong_derivative_is_outside_the_bound(act):
    z = every_magnitude()
    want, err = derivative64(z, act), derivative_error(z, act)
    far = np.abs(z) > 41
    for wrong in (1000.0, 1.0, 0.0, 1.5e-16, -1.5e-16):
        assert (np.abs(wrong - want) > err)[far].any(), wrong
    for wrong in (derivative64(np.clip(z, -30, 30), act) + 1e-5 * (z < -41), want * (1 + 1e-3)):
        assert (np.abs(wrong - want) > err).any()
    assert (err <= 1e-4).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 100])
def test_nan_of_one_token_stays_in_its_row(T):
    d = make(T, 72, 136, 3)
    d["X"][2, 9] = 0x7FC0
    Y = f64(B().int8_linear_act_fwd(bf16_dev(d["X"]), d["Wd"], d["Sd"], act="relu"))
    assert np.isnan(Y[2]).all() and np.isfinite(np.delete(Y, 2, 0)).all()


@pytest.mark.gpu
def test_outputs_behind_the_last_row_stay_as_they_were():
    """Y, Z, dX, G and dbias are views of larger buffers: nothing outside them is written."""
    b = B()
    for T, m, n in ((5, 40, 72), (70, 136, 40)):
        d = make(T, m, n, T)
        pad = 64

        def buf(rows, cols, dt=torch.bfloat16):
            t = torch.full(((rows + 2) * cols + 2 * pad,), 7.0, dtype=dt, device="cuda")
            return t, t[pad:pad + rows * cols].view(rows, cols)
        bufs = {"Y": buf(T, m), "Z": buf(T, m), "dX": buf(T, n), "G": buf(m, n),
                "db": buf(1, m, torch.float32)}
        v = {k: x[1] for k, x in bufs.items()}
        b.int8_linear_act_fwd(bf16_dev(d["X"]), d["Wd"], d["Sd"], act="gelu", out=v["Y"],
                              z_out=v["Z"])
        b.int8_linear_act_bwd(bf16_dev(d["dY"]), bf16_dev(d["X"]), d["Wd"], d["Sd"],
                              Z=bf16_dev(d["Z"]), act="gelu", dX=v["dX"], G=v["G"],
                              dbias=v["db"][0])
        for k, (whole, view) in bufs.items():
            end = pad + view.numel()
            assert (whole[:pad] == 7).all() and (whole[end:] == 7).all(), k
            assert not (view == 7).all()


@pytest.mark.gpu
def test_linear_captured_and_replayed():
    b = B()
    for T in (2, 96):
        d = make(T, 136, 264, T)
        X, dY, Z = bf16_dev(d["X"]), bf16_dev(d["dY"]), bf16_dev(d["Z"])
        bias = torch.from_numpy(d["bias"]).cuda()

        def both():
            Y = b.int8_linear_act_fwd(X, d["Wd"], d["Sd"], bias=bias, act="silu")
            return (Y, *b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], Z=Z, act="silu", bias=True))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = both()
        for k in range(4):
            X.copy_(bf16_dev(make(T, 136, 264, 50 + k)["X"]))
            g.replay()
            want = both()
            torch.cuda.synchronize()
            for x, y in zip(got, want):
                assert torch.equal(x, y)


@pytest.mark.gpu
def test_linear_on_a_stream_of_its_own():
    b = B()
    d = make(90, 136, 264, 1)
    X, dY = bf16_dev(d["X"]), bf16_dev(d["dY"])
    want = (b.int8_linear_act_fwd(X, d["Wd"], d["Sd"], act="relu"),
            *b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], bias=True))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (b.int8_linear_act_fwd(X, d["Wd"], d["Sd"], act="relu", stream=s),
           *b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], bias=True, stream=s))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


# ---------------------------------------------------------------------- on the CPU ---
@pytest.mark.parametrize("act", ACTS)
def test_oracle_derivative_against_differences(act):
    z = np.concatenate([np.linspace(-9, 9, 401) + 1e-3, [60.0, -60.0]])
    h = 1e-5
    num = (O.activation(z + h, act)[0] - O.activation(z - h, act)[0]) / (2 * h)
    # central differences: h^2 / 6 of the third derivative (below 3), and 2^-52 |act| / h
    assert np.allclose(num, O.activation(z, act)[1], rtol=0, atol=h * h + 2.0 ** -50 * 64 / h)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_oracle_backward_against_differences(act):
    T, m, n = 5, 16, 24
    rng = np.random.default_rng(3)
    Wq = rng.integers(-127, 128, size=(m, n)).astype(np.int8)
    Ws = (rng.uniform(0.5, 2.0, O.n_groups(m * n)) * 1e-2).astype(np.float32)
    W = O.dequant_weight(Wq, Ws, m, n).astype(np.float64)
    X = O.bf16_bits_to_f32(bits(rng.standard_normal((T, n)))).astype(np.float64)
    dY = O.bf16_bits_to_f32(bits(rng.standard_normal((T, m)))).astype(np.float64)
    bias = rng.standard_normal(m)

    def f(x, w, b):
        return float((dY * O.activation(x @ w.T + b, act)[0]).sum())
    dZ = dY * O.activation(X @ W.T + bias, act)[1]
    dX, G, db = dZ @ W, dZ.T @ X, dZ.sum(0)
    h = 1e-6
    for _ in range(4):
        u, v, w = (rng.standard_normal(s) for s in (X.shape, W.shape, bias.shape))
        num = (f(X + h * u, W + h * v, bias + h * w) - f(X - h * u, W - h * v, bias - h * w)) / 2 / h
        ana = (dX * u).sum() + (G * v).sum() + (db * w).sum()
        assert abs(num - ana) <= 1e-5 * (np.abs(dX * u).sum() + np.abs(G * v).sum()
                                         + np.abs(db * w).sum())


FAKE = 0x10000


def desc(T=128, m=64, n=32, act=2, **kw):
    d = B().LinearDesc(T, m, n, act, FAKE, 1 << 40, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fwd(d, X=FAKE, Wq=FAKE, Ws=FAKE, bias=FAKE, res=FAKE, Y=FAKE, Z=FAKE):
    import ctypes
    return B().lib().qgalore_int8_linear_act_fwd(ctypes.byref(d), X, Wq, Ws, bias, res, Y, Z)


def bwd(d, dY=FAKE, Z=FAKE, X=FAKE, Wq=FAKE, Ws=FAKE, dX=FAKE, G=FAKE, db=FAKE):
    import ctypes
    return B().lib().qgalore_int8_linear_act_bwd(ctypes.byref(d), dY, Z, X, Wq, Ws, dX, G, db)


def test_linear_refusals_come_before_any_device_call():
    for k in ("X", "Wq", "Ws", "Y"):
        assert fwd(desc(), **{k: None}) == 1, k
    for k in ("X", "Wq", "res", "Y", "Z"):
        assert fwd(desc(), **{k: FAKE + 8}) == 3, k
    for k in ("Ws", "bias"):
        assert fwd(desc(), **{k: FAKE + 2}) == 3, k
    for bad in (dict(T=0), dict(m=12), dict(n=12), dict(m=0), dict(n=-8),
                dict(T=1 << 20, m=1 << 10, n=8), dict(m=1 << 16, n=1 << 16)):
        assert fwd(desc(**bad)) == 2 and bwd(desc(**bad)) == 2, bad
    for act in (-1, 5):
        assert fwd(desc(act=act)) == 5 and bwd(desc(act=act)) == 5
    assert fwd(desc(workspace=None)) == 1 and bwd(desc(workspace=None)) == 1
    assert fwd(desc(workspace=FAKE + 8)) == 3 and bwd(desc(workspace=FAKE + 8)) == 3
    assert fwd(desc(workspace_bytes=64)) == 4 and bwd(desc(workspace_bytes=64)) == 4
    assert bwd(desc(), dY=None) == 1
    assert bwd(desc(), Z=None) == 1
    assert bwd(desc(), X=None) == 1
    assert bwd(desc(), Wq=None) == 1
    assert bwd(desc(), Ws=None) == 1
    assert bwd(desc(), dX=None, G=None, db=None) == 1
    for k in ("dY", "Z", "X", "Wq", "dX", "G"):
        assert bwd(desc(), **{k: FAKE + 8}) == 3, k
    assert bwd(desc(), db=FAKE + 1) == 3
    q = B().lib().qgalore_int8_linear_act_fwd_workspace_bytes
    assert q(1, 64, 32) == 0 and q(64, 64, 32) == 0 and q(4096, 64, 32) >= 64 * 32 * 2
    assert q(0, 64, 32) == 0 and q(128, 12, 32) == 0
    w = B().lib().qgalore_int8_linear_act_bwd_workspace_bytes
    assert w(128, 64, 32) >= 64 * 32 * 2 + 128 * 64 * 2 + 64 * 4
    assert w(128, 64, 31) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    b = B()
    X, Wq, Ws = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.int8), \
        torch.ones(1)
    with pytest.raises(ValueError):
        b.int8_linear_act_fwd(X, Wq, Ws, act="swish")
    with pytest.raises(ValueError):
        b.int8_linear_act_fwd(X, Wq, Ws)
    with pytest.raises(ValueError):
        b.int8_linear_act_bwd(X, None, Wq, Ws)
    with pytest.raises(ValueError):
        b.int8_linear_act_bwd(X, X)


def workspace_sizes(which, T, m, n):
    return getattr(B().lib(), f"qgalore_int8_linear_act_{which}_workspace_bytes")(T, m, n)


@pytest.mark.parametrize("m,n", [(11008, 4096), (4096, 11008), (4096, 4096), (1376, 512), (512, 1376),
                                 (512, 512), (64, 64), (8, 64), (64, 4096), (8192, 64), (72, 40),
                                 (2048, 5440), (25600, 128), (128, 25600)])
def test_workspace_of_the_largest_batch_serves_the_smaller_ones(m, n):
    top = min(70000, 2 ** 29 // max(m, n))
    tokens = sorted(set(range(1, 3000)) | set(range(3000, top, 509)))
    apart = [FAKE + (k << 32) for k in range(9)]
    for which, call in (("fwd", lambda d: fwd(d, *apart[:7])), ("bwd", lambda d: bwd(d, *apart[:8]))):
        sizes = [workspace_sizes(which, T, m, n) for T in tokens]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (which, m, n)
        if torch.cuda.is_available():
            continue
        # accepted at every T: the next thing that the call asks for is a device
        for T in tokens[::7]:
            for have in (workspace_sizes(which, T, m, n), sizes[-1]):
                assert call(desc(T, m, n, workspace_bytes=have)) == 7, (which, T)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(4096, 1024), (1376, 512), (136, 264)])
def test_one_workspace_for_batches_of_any_size(m, n):
    b, top = B(), 2600
    ws = b.alloc_workspace(max(workspace_sizes("fwd", top, m, n), workspace_sizes("bwd", top, m, n)))
    for T in (2600, 2496, 500, 192, 100, 64, 17, 1):
        d = make(T, m, n, T)
        X, dY, Z = bf16_dev(d["X"]), bf16_dev(d["dY"]), bf16_dev(d["Z"])

        def both(ws):
            Y = b.int8_linear_act_fwd(X, d["Wd"], d["Sd"], act="silu", workspace=ws)
            return (Y, *b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], Z=Z, act="silu", bias=True,
                                              workspace=ws))
        for x, y in zip(both(ws), both(None)):
            assert torch.equal(x, y), T


def test_outputs_over_what_a_call_still_reads_are_refused():
    T, m = 128, 64                                   # m = n: all of X, Y, Z, dY and dX are T x m
    rows, far = 2 * T * m, 1 << 30
    d = desc(T, m, m)
    a = dict(X=FAKE, Wq=FAKE + far, Ws=FAKE + 2 * far, bias=FAKE + 3 * far, res=FAKE + 4 * far,
             Y=FAKE + 5 * far, Z=FAKE + 6 * far)
    for out in ("Y", "Z"):
        for other, size in (("X", rows), ("Wq", m * m), ("res", rows), ("Ws", 4 * 16), ("bias", 4 * m)):
            assert fwd(d, **{**a, out: a[other] + size - 16}) == 5, (out, other)
            assert fwd(d, **{**a, other: a[out] + rows - 16}) == 5, (out, other)
        assert fwd(d, **{**a, out: a["X"]}) == 5
    assert fwd(d, **{**a, "Z": a["Y"]}) == 5 and fwd(d, **{**a, "Z": a["res"]}) == 5
    g = dict(dY=FAKE, Z=FAKE + far, X=FAKE + 2 * far, Wq=FAKE + 3 * far, Ws=FAKE + 4 * far,
             dX=FAKE + 5 * far, G=FAKE + 6 * far, db=FAKE + 7 * far)
    none = desc(T, m, m, act=0)
    for out, size in (("dX", rows), ("G", 2 * m * m), ("db", 4 * m)):
        assert bwd(none, **{**g, "dY": g[out] + size - 16}) == 5, out
        assert bwd(none, **{**g, "X": g[out] + size - 16}) == 5, out
        assert bwd(d, **{**g, "X": g[out] + size - 16}) == 5, out
        for other in ("dX", "G", "db"):
            if other != out:
                assert bwd(d, **{**g, other: g[out] + size - 16}) == 5, (out, other)
    assert bwd(none, **{**g, "dX": g["dY"]}) == 5 and bwd(d, **{**g, "dX": g["X"]}) == 5
    if not torch.cuda.is_available():                # accepted: the next thing it needs is a device
        assert fwd(d, **a) == 7 and fwd(d, **{**a, "Y": a["res"]}) == 7
        assert bwd(d, **g) == 7 and bwd(none, **g) == 7
        assert bwd(d, **{**g, "dX": g["dY"]}) == 7
        assert bwd(d, **{**g, "dX": g["X"], "G": None}) == 7


@pytest.mark.gpu
@pytest.mark.parametrize("T,m", [(3, 136), (40, 512), (100, 512), (700, 264), (2100, 1032)])
def test_linear_in_place(T, m):
    """Y over the residual in every form of the product; dX over dY where an activation stands between."""
    b, d = B(), make(T, m, m, T)
    X, res, dY, Z = (bf16_dev(d[k]) for k in ("X", "res", "dY", "Z"))
    want = b.int8_linear_act_fwd(X, d["Wd"], d["Sd"], residual=res, act="gelu")
    assert torch.equal(b.int8_linear_act_fwd(X, d["Wd"], d["Sd"], residual=res, act="gelu", out=res), want)
    want = b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], Z=Z, act="silu", bias=True)
    got = b.int8_linear_act_bwd(dY, X, d["Wd"], d["Sd"], Z=Z, act="silu", bias=True, dX=dY)
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_rows_behind_the_last_token_are_zeros_at_the_widest():
    """The most outputs (or inputs) that the limits allow: byte offsets of the rows that a tile has behind
    the last one pass 2^32. An infinity in the first row shows what is read there: times zero it is NaN."""
    b, T, wide = B(), 8, 1 << 26
    big = torch.ones(T, wide, dtype=torch.bfloat16, device="cuda")
    big[0, 5] = float("inf")
    small = torch.ones(T, 8, dtype=torch.bfloat16, device="cuda")
    G = b.int8_linear_act_bwd(big, small, need_dX=False)[1]
    assert torch.isinf(G[5]).all() and (G[:5] == T).all() and (G[6:] == T).all()
    del G, big
    Wq = torch.ones(8, wide, dtype=torch.int8, device="cuda")
    Ws = torch.ones(b.n_groups(8 * wide), device="cuda")
    Ws[0] = float("inf")                             # the first 256 inputs of output 0
    dX = b.int8_linear_act_bwd(small, None, Wq, Ws, need_G=False)[0]
    assert torch.isinf(dX[:, :256]).all() and (dX[:, 256:] == 8).all()
