"""The norms around a block with its gate and scales, forward and backward, against float64.

Tolerances. U = 2^-24 is one fp32 rounding. A centred and normed value h = (v - mean) rstd is off by
2^-21 (s + |h| (2 + s)) in the forward pass, with s = max over the row of (|v| + |mean|) rstd (the mean's sum
2^-20 of its magnitudes at most, the variance's half of that), and by 2^-22 (|v| + |mean|) rstd where mean
and rstd are given (backward). The gate's functions are off by 2^-20 of themselves (exp and tanh two ulp, the
sum, the quotient and the products one each). Sums over a row or over tokens are off by 2^-20 of the sum of
magnitudes. What a quantity's inputs are off by goes through the formula's first derivatives (`e` below).
Results in bf16 add 2^-8 of themselves, in fp32 2^-24."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import qgalore_oracle as O

torch = pytest.importorskip("torch")

U20, U21, U22, U23 = (2.0 ** -k for k in (20, 21, 22, 23))
BF16, FP32 = torch.bfloat16, torch.float32


def B():
    from quantized_rank_gradient_amd import binding
    return binding


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, n, dtype, seed, post=True, pre=True, beta=True, gate="", per=1, rho=False):
    """Tensors on the CPU, by name (None for what is not there)."""
    rng = np.random.default_rng(seed)

    def rows(k, scale=1.0, mean=0.0):
        v = rng.standard_normal((k, n)) * scale * rng.uniform(0.5, 2.0, (k, 1)) + mean
        return torch.from_numpy(v.astype(np.float32)).to(dtype)

    def vec(mean):
        return torch.from_numpy((mean + 0.2 * rng.standard_normal(n)).astype(np.float32))
    return dict(u=rows(T, 1.0, 0.2), x=rows(T, 2.0, 0.5), dh=rows(T), dy=rows(T),
                z=rows(-(-T // per), 1.5) if gate else None, rho=vec(0.5) if rho else None,
                g1=vec(1.0) if post else None, b1=vec(0.0) if post and beta else None,
                g2=vec(1.0) if pre else None, b2=vec(0.0) if pre and beta else None)


def options(t, gate, per, alpha, center):
    return dict(post=(t["g1"], t["b1"]) if t["g1"] is not None else None,
                pre=(t["g2"], t["b2"]) if t["g2"] is not None else None, per=per, rho=t["rho"],
                alpha=alpha, center=center), gate or "none"


def on(t, f):
    return {k: f(v) if v is not None else None for k, v in t.items()}


def gpu_forward(t, gate, per, alpha, center, **kw):
    o, act = options(t, gate, per, alpha, center)
    return B().residual_norm_fwd(t["u"], t["x"], gate=t["z"], gate_act=act, **o, **kw)


def gpu_backward(t, H, stats, gate, per, alpha, center, dh=True, **kw):
    o, act = options(t, gate, per, alpha, center)
    pre = t["g2"] is not None
    r = B().residual_norm_bwd(t["dh"] if dh else None, t["dy"] if pre else None, t["u"], H, stats,
                              gate=t["z"], gate_act=act, **o, **kw)
    return dict(du=r.dU, dx=r.dX, dz=r.dgate, drho=r.drho, dg1=r.dpost[0], db1=r.dpost[1],
                dg2=r.dpre[0], db2=r.dpre[1])


def near(got, want, err, out_eps, name):
    got = f64(got)
    bad = np.abs(got - want) > err + out_eps * (np.abs(want) + err) + 1e-37
    assert not bad.any(), (name, float(np.abs(got - want)[bad].max()), int(bad.sum()))


def nan0(v):
    return 0.0 if v is None else v


def check(T, n, dtype, seed=0, gate="", per=1, alpha=1.0, center=False, dh=True, t=None, **kw):
    t = make(T, n, dtype, seed, gate=gate, per=per, **kw) if t is None else t
    w, d = on(t, f64), on(t, lambda v: v.cuda())
    out_eps = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    post, pre = t["g1"] is not None, t["g2"] is not None
    o, act = options(w, gate, per, alpha, center)
    eps = float(np.float32(1e-5))
    H, Y, stats = gpu_forward(d, gate, per, alpha, center)
    h, y, st = O.residual_norm_forward(w["u"], w["x"], z=w["z"], act=act, eps=eps, **o)

    # forward
    rows = np.arange(T) // per
    a, da = O.gate(w["z"], act) if gate else (np.ones((1, n)), None)
    ag = np.abs(a[rows]) if gate else np.ones((T, n))
    rho = np.abs(nan0(w["rho"])) if w["rho"] is not None else 1.0
    p, ep = w["u"], np.zeros((T, n))
    if post:
        m1, r1 = st[0][:, None], st[1][:, None]
        s = ((np.abs(w["u"]) + np.abs(m1)).max(1) * st[1])[:, None]
        uh = (w["u"] - m1) * r1
        p = uh * w["g1"] + nan0(w["b1"])
        ep = U21 * (s + np.abs(uh) * (2 + s)) * np.abs(w["g1"]) + U23 * (np.abs(p) + np.abs(nan0(w["b1"])))
    eh = rho * ag * (ep + U20 * np.abs(p)) + U23 * (np.abs(alpha * w["x"]) + rho * ag * np.abs(p))
    near(H, h, eh, out_eps, "h")
    got = f64(stats)
    if post:
        assert (np.abs(got[0] - st[0]) <= U20 * np.abs(w["u"]).mean(1)).all()
        assert (np.abs(got[1] - st[1]) <= st[1] * (U20 + U21 * s[:, 0])).all()
    else:
        assert (got[:2] == 0).all()
    if not center:
        assert (got[[0, 2]] == 0).all()
    if pre:
        m2, r2 = st[2][:, None], st[3][:, None]
        s2 = ((np.abs(h) + np.abs(m2)).max(1) * st[3])[:, None]
        hh = (h - m2) * r2
        rms = r2 * np.sqrt((eh * eh).mean(1, keepdims=True))
        ehh = U21 * (s2 + np.abs(hh) * (2 + s2)) + r2 * (eh + eh.mean(1, keepdims=True)) \
            + np.abs(hh) * 1.01 * rms
        near(Y, y, ehh * np.abs(w["g2"]) + U23 * (np.abs(y) + np.abs(nan0(w["b2"]))), out_eps, "y")
        assert (np.abs(got[2] - st[2]) <= U20 * np.abs(h).mean(1) + eh.mean(1)).all()
        assert (np.abs(got[3] - st[3]) <= st[3] * (U20 + U21 * s2[:, 0] + 1.01 * rms[:, 0])).all()
    else:
        assert Y is None and (got[2:] == 0).all()

    # backward, from the forward pass's own h and statistics
    g = gpu_backward(d, H, stats, gate, per, alpha, center, dh)
    h, st = f64(H), f64(stats)
    want = O.residual_norm_backward(w["dh"] if dh else None, w["dy"], w["u"], h, st, z=w["z"], act=act,
                                    **o)
    D = want["dx"] / alpha
    eD = U23 * np.abs(w["dh"])

    def mean(v):
        return v.mean(1, keepdims=True)
    if pre:
        r2 = st[3][:, None]
        hh = (h - st[2][:, None]) * r2
        ehh = U22 * (np.abs(h) + np.abs(st[2])[:, None]) * r2
        e = np.abs(w["dy"] * w["g2"])
        eD = eD + r2 * (2 * U20 * (e + mean(e) + np.abs(hh) * mean(e * np.abs(hh)))
                        + ehh * mean(e * np.abs(hh)) + np.abs(hh) * mean(e * ehh)) + U23 * np.abs(D)
        near(g["dg2"], want["dg2"], U20 * np.abs(w["dy"] * hh).sum(0) + (np.abs(w["dy"]) * ehh).sum(0),
             2.0 ** -24, "dg2")
        if w["b2"] is not None:
            near(g["db2"], want["db2"], U20 * np.abs(w["dy"]).sum(0), 2.0 ** -24, "db2")
        else:
            assert g["db2"] is None
    near(g["dx"], want["dx"], abs(alpha) * eD + U23 * np.abs(want["dx"]), out_eps, "dx")
    p, ep, uh, euh = w["u"], np.zeros((T, n)), w["u"], np.zeros((T, n))
    if post:
        m1, r1 = st[0][:, None], st[1][:, None]
        uh = (w["u"] - m1) * r1
        euh = U22 * (np.abs(w["u"]) + np.abs(m1)) * r1
        p = uh * w["g1"] + nan0(w["b1"])
        ep = euh * np.abs(w["g1"]) + U22 * (np.abs(p) + np.abs(nan0(w["b1"])))
    tt = np.abs(D * p)
    et = eD * np.abs(p) + np.abs(D) * ep + U23 * tt
    if gate:
        ez = np.zeros(w["z"].shape)
        np.add.at(ez, rows, rho * (et + U20 * tt))
        near(g["dz"], want["dz"], np.abs(da) * ez + U20 * np.abs(want["dz"]), out_eps, "dz")
    else:
        assert g["dz"] is None
    if w["rho"] is not None:
        near(g["drho"], want["drho"], (ag * (et + 2 * U20 * tt)).sum(0), 2.0 ** -24, "drho")
    else:
        assert g["drho"] is None
    v = np.abs(D) * rho * ag
    ev = rho * ag * eD + U20 * v
    if post:
        near(g["dg1"], want["dg1"], (ev * np.abs(uh) + v * euh + U20 * v * np.abs(uh)).sum(0),
             2.0 ** -24, "dg1")
        if w["b1"] is not None:
            near(g["db1"], want["db1"], (ev + U20 * v).sum(0), 2.0 ** -24, "db1")
        f, ef = v * np.abs(w["g1"]), (ev + U23 * v) * np.abs(w["g1"])
        au = np.abs(uh)
        ev = r1 * (ef + mean(ef) + au * mean(ef * au) + 2 * U20 * (f + mean(f) + au * mean(f * au))
                   + euh * mean(f * au) + au * mean(f * euh))
    near(g["du"], want["du"], ev, out_eps, "du")


SIZES = [(1, 1), (3, 2), (2, 7), (5, 64), (7, 100), (2, 511), (9, 512), (4, 513), (33, 1000), (3, 1024),
         (6, 1376), (2, 2056), (5, 4096), (3, 5461), (2, 8200), (1, 16384), (2, 20001), (1, 32768),
         (3001, 40), (600, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,n", SIZES)
def test_resnorm(T, n, dtype):
    """A gate for every value, both norms by the root mean square, rho; and layer norms of a shared
    gate."""
    check(T, n, dtype, T + n, gate="sigmoid", rho=True, beta=False, alpha=1.25)
    check(T, n, dtype, T + n + 1, gate="tanh", per=max(1, T // 3), center=True)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["", "none", "sigmoid", "tanh"])
@pytest.mark.parametrize("post,pre,rho,center,beta", [
    (False, False, False, False, False), (False, False, True, False, False),
    (True, False, True, True, True), (False, True, False, True, False), (True, True, False, False, True),
    (False, True, True, False, True), (True, False, False, False, False), (True, True, True, True, True)])
def test_resnorm_parts(post, pre, rho, center, beta, gate):
    for T, n in ((70, 264), (13, 1100), (5, 4100)):
        check(T, n, BF16, T, gate=gate, per=4 if gate else 1, post=post, pre=pre, rho=rho, center=center,
              beta=beta, alpha=-0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T,per", [(1, 1), (64, 64), (1000, 1000), (1001, 1000), (999, 1000 // 3),
                                   (4000, 7), (515, 512), (2100, 2), (5000, 4999),
                                   (7, 1000)])
@pytest.mark.parametrize("n", [24, 1376])
def test_resnorm_of_shared_gates(T, per, n):
    check(T, n, FP32, T + per, gate="none", per=per, rho=True)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,per", [(300, 8200, 1), (261, 8193, 40), (140, 10000, 139), (40, 12288, 7),
                                     (40, 12289, 1), (90, 16390, 90),
                                     (77, 32768, 2), (1, 8200, 1)])
def test_resnorm_of_long_rows(T, n, per):
    for dtype in (BF16, FP32):
        check(T, n, dtype, T, gate="sigmoid", per=per, rho=True, alpha=0.75)
        check(T, n, dtype, T + 1, gate="tanh", per=per, center=True, dh=False)


@pytest.mark.gpu
@pytest.mark.parametrize("post,pre,rho,center", [
    (False, False, False, False), (False, False, True, True), (True, False, True, True),
    (False, True, False, True), (True, False, False, False), (False, True, True, False)])
def test_resnorm_of_long_rows_parts(post, pre, rho, center):
    for n in (8200, 12345):
        for gate, per in (("", 1), ("none", 1), ("sigmoid", 30)):
            check(70, n, BF16, n, gate=gate, per=per, post=post, pre=pre, rho=rho, center=center)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1025, 1536, 1537, 2049, 2560, 2561, 4097, 6143, 6144, 6145])
def test_resnorm_at_the_borders_of_row_shapes(n):
    for dtype in (BF16, FP32):
        check(261, n, dtype, n, gate="sigmoid", rho=True)
        check(9, n, dtype, n, gate="tanh", per=4, center=True, pre=False)


@pytest.mark.gpu
@pytest.mark.parametrize("T,per,n", [(37, 3, 520), (37, 3, 1032), (37, 7, 2052), (300, 3, 4104), (300, 1, 8195),
                                     (70, 70, 12000), (9, 2, 30001)])
def test_resnorm_of_strands_that_differ_in_length(T, per, n):
    """Workgroups of several strands, the last of which have fewer tokens, and rows that fill one chunk, two
    and four."""
    for dtype in (BF16, FP32):
        check(T, n, dtype, T, gate="sigmoid", per=per, rho=True, center=True)


def most_strands(n, dtype):
    """No fewer than the strands that the backward pass deals many tokens of n <= 4096 to: the slabs of which the
    workspace keeps five sums of n, with as many rows side by side as fill eight waves."""
    slabs = B().lib().qgalore_resnorm_bwd_workspace_bytes(
        ctypes.byref(desc(T=1 << 18, n=n, per=1, dtype=0 if dtype == BF16 else 1))) // (5 * 4 * n)
    waves = next(w for most, w in ((512, 1), (1024, 2), (1536, 3), (2048, 4), (2560, 5), (4096, 8)) if n <= most)
    return slabs * max(1, 8 // waves)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,tokens", [(2056, 3), (2051, 4), (2056, 5), (2051, 7), (2056, 17), (264, 5), (1376, 7),
                                      (1027, 4), (4096, 4), (4091, 3)])
def test_resnorm_of_many_tokens_a_strand(n, tokens, dtype):
    """Strands of at least `tokens` tokens, the last ones shorter: more than the values of the next tokens that
    are on their way, so that their registers go round. Gradients of every token, and sums over all."""
    T = most_strands(n, dtype) * tokens - 3
    check(T, n, dtype, tokens, gate="sigmoid", rho=True, alpha=1.25, beta=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,per,tokens", [(2056, 2, 3), (2051, 3, 4), (2056, 7, 7), (1376, 2, 5), (2051, 1000, 9),
                                          (1376, 1501, 5), (264, 1200, 4), (2056, 5, 6)])
def test_resnorm_of_shared_gates_with_many_tokens_a_strand(n, per, tokens, dtype):
    """Whole groups, several to a strand, and groups in parts: the gate's row changes, or does not, between the
    tokens that are on their way."""
    T = most_strands(n, dtype) * tokens - 1
    check(T, n, dtype, per, gate="tanh", per=per, center=True)
    check(T, n, dtype, per + 1, gate="none", per=per, rho=True, pre=False)


@pytest.mark.gpu
def test_gradient_through_y_alone():
    check(40, 264, FP32, 4, gate="sigmoid", dh=False)
    check(1, 4096, BF16, 4, dh=False)


@pytest.mark.gpu
def test_gates_far_from_zero():
    """Logits to both ends: the logistic function and its derivative go to their limits."""
    T, n = 6, 300
    for gate in ("sigmoid", "tanh"):
        t = make(T, n, FP32, 9, gate=gate)
        t["z"] = torch.linspace(-95, 95, T * n).view(T, n)
        check(T, n, FP32, gate=gate, t=t)
        t["z"][2, 5], t["z"][3, 7] = float("inf"), -float("inf")
        d = on(t, lambda v: v.cuda())
        H, Y, stats = gpu_forward(d, gate, 1, 1.0, False)
        g = gpu_backward(d, H, stats, gate, 1, 1.0, False)
        assert torch.isfinite(H).all() and all(torch.isfinite(v).all() for v in g.values() if v is not None)
        assert g["dz"][2, 5] == 0 and g["dz"][3, 7] == 0


@pytest.mark.gpu
def test_a_nan_stays_in_its_token():
    t = on(make(6, 300, BF16, 1, gate="sigmoid", rho=True), lambda v: v.cuda())
    t["u"][1, 299], t["x"][3, 0], t["z"][4, 17] = float("nan"), float("inf"), float("nan")
    H, Y, stats = gpu_forward(t, "sigmoid", 1, 1.0, True)
    assert (~torch.isfinite(Y)).any(1).tolist() == [False, True, False, True, True, False]
    assert (~torch.isfinite(H)).sum(1).tolist() == [0, 300, 0, 1, 1, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["", "sigmoid"])
@pytest.mark.parametrize("rho", [False, True])
@pytest.mark.parametrize("n", [7, 264, 1100, 4101, 5461, 8200, 8201])
def test_du_without_the_first_norm_has_no_part_of_u(n, rho, gate):
    """du = rho a(z) D whatever u is: infinite and NaN values of it reach the gradients of z and rho
    alone."""
    for pre in (False, True):
        t = on(make(6, n, BF16, n, gate=gate, post=False, pre=pre, rho=rho), lambda v: v.cuda())
        H, Y, stats = gpu_forward(t, gate, 1, 1.0, True)
        want = gpu_backward(t, H, stats, gate, 1, 1.0, True)
        for k, v in enumerate((float("inf"), -float("inf"), float("nan"))):
            t["u"][k + 1, n // 2 + k], t["u"][k + 2, n - 1] = v, v
        got = gpu_backward(t, H, stats, gate, 1, 1.0, True)
        assert torch.isfinite(want["du"]).all()
        for k in ("du", "dx", "dg2", "db2"):
            assert want[k] is None and got[k] is None or torch.equal(got[k], want[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,n", [(1, 1), (5, 7), (1030, 264), (40, 1100), (300, 4096), (300, 5461), (40, 8200),
                                 (9, 20001)])
def test_resnorm_backward_without_u(T, n, dtype):
    """h = alpha x + u alone: the gradients are those of a call that has u, in place too."""
    for pre in (False, True):
        t = on(make(T, n, dtype, T, post=False, pre=pre), lambda v: v.cuda())
        H, Y, stats = gpu_forward(t, "", 1, 1.5, True)
        for dh in (True, False) if pre else (True,):
            want = gpu_backward(t, H, stats, "", 1, 1.5, True, dh=dh)
            c = dict(on(t, torch.clone), u=None)
            kw = dict(dX=c["dh"], dU=c["dy"] if pre else None) if dh else {}
            got = gpu_backward(c, H if pre else None, stats, "", 1, 1.5, True, dh=dh, **kw)
            for k, v in want.items():
                assert v is None and got[k] is None or torch.equal(got[k], v), k


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,per", [(1030, 264, 1), (1030, 264, 400), (300, 5000, 300), (37, 40, 9)])
def test_resnorm_equal_calls_give_equal_bits_and_write_nothing_else(T, n, per):
    t = on(make(T, n, BF16, 3, gate="sigmoid", per=per, rho=True), lambda v: v.cuda())
    H, Y, stats = gpu_forward(t, "sigmoid", per, 1.0, True)
    first = gpu_backward(t, H, stats, "sigmoid", per, 1.0, True)

    def room(k):
        whole = torch.full((k * n + 128,), 7.0, dtype=BF16, device="cuda")
        return whole, whole[64:64 + k * n].view(k, n)
    groups = -(-T // per)
    outs = {k: room(groups if k == "dgate" else T) for k in ("dU", "dX", "dgate")}
    second = gpu_backward(t, H, stats, "sigmoid", per, 1.0, True, **{k: v[1] for k, v in outs.items()})
    for k, v in first.items():
        assert torch.equal(v, second[k]), k
    h, y = room(T), room(T)
    H2, Y2, s2 = gpu_forward(t, "sigmoid", per, 1.0, True, out=h[1], y_out=y[1])
    assert torch.equal(H, H2) and torch.equal(Y, Y2) and torch.equal(stats, s2)
    for whole, _ in [*outs.values(), h, y]:
        assert (whole[:64] == 7).all() and (whole[-64:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(1, 8), (3, 7), (1030, 264), (40, 8200)])
def test_resnorm_gradients_of_parameters_into_one_tensor(T, n):
    """The vectors' gradients as slices of a program's flat tensor, with nothing written between them; and a
    beta's without its beta."""
    t = on(make(T, n, BF16, 5, gate="sigmoid", rho=True), lambda v: v.cuda())
    H, Y, stats = gpu_forward(t, "sigmoid", 1, 1.0, True)
    want = gpu_backward(t, H, stats, "sigmoid", 1, 1.0, True)
    step = -(-n // 4) * 4 + 4
    flat = torch.full((5 * step,), 3.0, device="cuda")
    v = [flat[k * step:k * step + n] for k in range(5)]
    got = gpu_backward(t, H, stats, "sigmoid", 1, 1.0, True, drho=v[0], dpost=(v[1], v[2]), dpre=(v[3], v[4]))
    for k, (name, at) in enumerate(zip(("drho", "dg1", "db1", "dg2", "db2"), v)):
        assert got[name] is at and torch.equal(at, want[name]), name
        assert (flat[k * step + n:(k + 1) * step] == 3).all()
    for k in ("du", "dx", "dz"):
        assert torch.equal(got[k], want[k])
    flat.fill_(3.0)
    t["b1"] = None
    got = gpu_backward(t, H, stats, "sigmoid", 1, 1.0, True, dpost=(None, v[2]), dpre=(v[3], None))
    assert got["db1"] is v[2] and got["dg2"] is v[3] and torch.equal(v[2], want["db1"])
    assert torch.equal(got["dg1"], gpu_backward(t, H, stats, "sigmoid", 1, 1.0, True)["dg1"])
    assert torch.equal(got["db2"], want["db2"])


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(5, 7), (1030, 264), (300, 4096), (40, 8200), (9, 20001)])
@pytest.mark.parametrize("norms", [True, False])
def test_resnorm_in_place(T, n, norms):
    t = on(make(T, n, BF16, 3, gate="none", post=norms, pre=norms), lambda v: v.cuda())
    H, Y, stats = gpu_forward(t, "none", 1, 1.5, False)
    for over, other in (("u", "x"), ("x", "u")):
        c = on(t, torch.clone)
        kw = {"y_out": c[other]} if norms else {}
        gpu_forward(c, "none", 1, 1.5, False, out=c[over], **kw)
        assert torch.equal(c[over], H) and (not norms or torch.equal(c[other], Y))
    want = gpu_backward(t, H, stats, "none", 1, 1.5, False)
    for over in ("u", "dy") if norms else ("u",):
        c = on(t, torch.clone)
        gpu_backward(c, H, stats, "none", 1, 1.5, False, dX=c["dh"], dU=c[over])
        assert torch.equal(c["dh"], want["dx"]) and torch.equal(c[over], want["du"])


@pytest.mark.gpu
@pytest.mark.parametrize("per", [1, 30])
def test_resnorm_captured_and_replayed_on_another_stream(per):
    T, n = 70, 264
    t = on(make(T, n, BF16, 4, gate="sigmoid", per=per, rho=True), lambda v: v.cuda())

    def both(stream=None):
        H, Y, stats = gpu_forward(t, "sigmoid", per, 1.0, False, stream=stream)
        g = gpu_backward(t, H, stats, "sigmoid", per, 1.0, False, stream=stream)
        return [H, Y, stats, *(v for v in g.values() if v is not None)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = both()
    s = torch.cuda.Stream()
    for k in range(4):
        new = make(T, n, BF16, 20 + k, gate="sigmoid", per=per, rho=True)
        for name in ("u", "x", "dh", "dy", "z"):
            t[name].copy_(new[name])
        graph.replay()
        s.wait_stream(torch.cuda.current_stream())
        want = both(s)
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(524287, 4095), (65535, 32768)])
def test_resnorm_of_nearly_2_31_values(T, n):
    """Rows around every 2^30 values (tensors of 4 GiB), the first and the last ones are those of a call of their
    own; dbeta2, the sum of dy, is that in 64 bits."""
    g = torch.Generator("cuda").manual_seed(1)

    def rows():
        return torch.randn((T, n), generator=g, device="cuda", dtype=BF16)
    t = dict(u=rows(), x=rows(), dh=rows(), dy=rows(), z=rows(), rho=torch.rand(n, generator=g, device="cuda"))
    t.update({k: torch.rand(n, generator=g, device="cuda") for k in ("g1", "b1", "g2", "b2")})
    H, Y, stats = gpu_forward(t, "sigmoid", 1, 1.0, True)
    got = gpu_backward(t, H, stats, "sigmoid", 1, 1.0, True)
    for mid in (2, 2 ** 30 // n, T - 2):
        at = slice(mid - 2, mid + 2)
        part = {k: v[at].clone() if k in ("u", "x", "dh", "dy", "z") else v for k, v in t.items()}
        h, y, st = gpu_forward(part, "sigmoid", 1, 1.0, True)
        assert torch.equal(h, H[at]) and torch.equal(y, Y[at]) and torch.equal(st, stats[:, at])
        want = gpu_backward(part, h, st, "sigmoid", 1, 1.0, True)
        for k in ("du", "dx", "dz"):
            assert torch.equal(want[k], got[k][at]), (mid, k)
    total, size = torch.zeros(2, n, dtype=torch.float64, device="cuda")
    for k in range(0, T, 8192):
        d = t["dy"][k:k + 8192].double()
        total += d.sum(0)
        size += d.abs().sum(0)
    near(got["db2"], f64(total), U20 * f64(size), 2.0 ** -24, "db2")
    del t, H, Y, stats, got
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------- on the CPU ---
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("act", ["none", "sigmoid", "tanh"])
def test_oracle_gradients_against_differences(act, center):
    rng = np.random.default_rng(2)
    T, n, per, alpha = 7, 19, 3, 0.75
    v = {k: rng.standard_normal((T, n)) for k in ("u", "x", "dh", "dy")}
    v["z"] = rng.standard_normal((3, n))
    v.update({k: rng.standard_normal(n) for k in ("g1", "b1", "g2", "b2", "rho")})

    def run(p):
        return O.residual_norm_forward(p["u"], p["x"], (p["g1"], p["b1"]), (p["g2"], p["b2"]), p["z"],
                                       act, per, p["rho"], alpha, 1e-3, center)

    def loss(p):
        h, y, _ = run(p)
        return float((h * v["dh"]).sum() + (y * v["dy"]).sum())
    h, _, stats = run(v)
    got = O.residual_norm_backward(v["dh"], v["dy"], v["u"], h, stats, (v["g1"], v["b1"]),
                                   (v["g2"], v["b2"]), v["z"], act, per, v["rho"], alpha, center)
    for k in ("u", "x", "z", "rho", "g1", "b1", "g2", "b2"):
        d, step = rng.standard_normal(v[k].shape), 1e-6
        num = (loss({**v, k: v[k] + step * d}) - loss({**v, k: v[k] - step * d})) / (2 * step)
        assert abs(num - (got["d" + k] * d).sum()) <= 1e-6 * np.abs(got["d" + k] * d).sum() + 1e-8, k


FAKE, FAR = 0x10000, 1 << 30
NAMES = ("u", "x", "h", "y", "stats", "g1", "b1", "g2", "b2", "rho", "z")
GRADS = ("du", "dx", "dz", "drho", "dg1", "db1", "dg2", "db2")


def places(names):
    return {k: FAKE + FAR * i for i, k in enumerate(names)}


def desc(**kw):
    d = B().ResnormDesc(16, 64, 4, 0, 1, 1, 1.0, 1e-5, FAKE + 40 * FAR, 1 << 40, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fwd(d=None, **kw):
    b = B()
    a = {**places(NAMES), **kw}
    p = b.ResnormParams(a["g1"], a["b1"], a["g2"], a["b2"], a["rho"], a["z"])
    return b.lib().qgalore_resnorm_fwd(ctypes.byref(d or desc()), ctypes.byref(p), a["u"], a["x"],
                                       a["h"], a["y"], a["stats"])


def bwd(d=None, **kw):
    b = B()
    a = {**places(NAMES + ("dh", "dy") + GRADS), **kw}
    p = b.ResnormParams(a["g1"], a["b1"], a["g2"], a["b2"], a["rho"], a["z"])
    g = b.ResnormGrads(*(a[k] for k in GRADS))
    return b.lib().qgalore_resnorm_bwd(ctypes.byref(d or desc()), ctypes.byref(p), a["dh"], a["dy"],
                                       a["u"], a["h"], a["stats"], ctypes.byref(g))


def test_resnorm_refusals_come_before_any_device_call():
    for k in ("u", "x", "h", "y", "stats"):
        assert fwd(**{k: None}) == 1, k
    assert fwd(g2=None) == 1                      # y without its norm
    for k in ("u", "h", "dy", "stats", "du", "dx", "dz", "drho", "dg1", "dg2", "z", "rho", "g1", "g2"):
        assert bwd(**{k: None}) == 1, k
    at = {**places(NAMES + ("dh", "dy") + GRADS)}
    for k in NAMES:
        off = 2 if k == "stats" else 4
        assert fwd(**{k: at[k] + off}) == 3, k
        if k not in ("x", "y", "b2"):
            assert bwd(**{k: at[k] + off}) == 3, k
    for k in ("dh", "dy") + GRADS:
        assert bwd(**{k: at[k] + 4}) == 3, k
    for bad in (dict(T=0), dict(n=0), dict(n=32769), dict(T=1 << 30), dict(T=-1), dict(per=0)):
        assert fwd(desc(**bad)) == 2 and bwd(desc(**bad)) == 2, bad
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("inf")), dict(center=2),
                dict(dtype=2), dict(gate_act=3), dict(gate_act=-1)):
        assert fwd(desc(**bad)) == 5 and bwd(desc(**bad)) == 5, bad
    assert bwd(g1=None, dg1=None) == 5            # dbeta1 without its norm
    assert bwd(desc(workspace=None)) == 1
    assert bwd(desc(workspace=FAKE + 40 * FAR + 8)) == 3
    assert bwd(desc(workspace_bytes=16)) == 4
    q = B().lib().qgalore_resnorm_bwd_workspace_bytes
    assert q(ctypes.byref(desc())) >= 5 * 64 * 4
    assert q(ctypes.byref(desc(T=0))) == 0 and q(None) == 0


def test_resnorm_backward_needs_u_for_the_first_norm_the_gate_and_rho_alone():
    off = {"g1": dict(g1=None, dg1=None, db1=None), "z": dict(z=None, dz=None), "rho": dict(rho=None, drho=None)}
    for k in off:   # any one of them
        rest = {a: b for o in off if o != k for a, b in off[o].items()}
        assert bwd(u=None, **rest) == 1, k
    none = {a: b for o in off.values() for a, b in o.items()}
    at = places(NAMES + ("dh", "dy") + GRADS)
    # past its checks of null pointers, to a result over another
    assert bwd(u=None, **{**none, "du": at["dx"]}) == 5
    if not torch.cuda.is_available():   # accepted: the next thing it needs is a device
        assert bwd(u=None, **none) == 7
        assert bwd(u=None, **{**none, "g2": None, "dg2": None, "db2": None, "dy": None, "h": None}) == 7
    b, X = B(), torch.zeros(4, 8)
    for kw in (dict(post=(X[0], None)), dict(gate=X), dict(rho=X[0])):
        with pytest.raises(ValueError):
            b.residual_norm_bwd(X, None, None, None, X, **kw)
    with pytest.raises(ValueError):
        b.residual_norm_bwd(None, None, None, None, X)


def test_resnorm_outputs_over_what_a_call_still_reads_are_refused():
    rows = 2 * 16 * 64
    at = places(NAMES + ("dh", "dy") + GRADS)
    sizes = dict(h=rows, y=rows, stats=4 * 4 * 16, du=rows, dx=rows, dz=2 * 4 * 64, drho=256, dg1=256,
                 db1=256, dg2=256, db2=256)
    for o in ("h", "y", "stats"):
        for k in NAMES:
            if k != o:
                assert fwd(**{k: at[o] + sizes[o] - 16}) == 5, (o, k)
    for o in GRADS:
        for k in at:
            if k != o and k not in ("x", "y", "b2"):
                assert bwd(**{k: at[o] + sizes[o] - 16}) == 5, (o, k)
    assert fwd(h=at["y"]) == 5 and fwd(h=at["z"]) == 5 and bwd(dx=at["u"]) == 5
    assert bwd(du=at["dh"]) == 5 and bwd(du=at["dx"]) == 5 and bwd(dz=at["z"]) == 5
    assert bwd(desc(workspace=at["u"] + 16)) == 5
    if not torch.cuda.is_available():   # accepted: the next thing it needs is a device
        assert fwd() == 7 and bwd() == 7
        assert fwd(h=at["u"], y=at["x"]) == 7 and fwd(h=at["x"], y=at["u"]) == 7
        assert bwd(dx=at["dh"], du=at["dy"]) == 7 and bwd(du=at["u"]) == 7
        assert bwd(dh=None) == 7 and bwd(db1=None, db2=None) == 7
        assert bwd(g2=None, dg2=None, db2=None, dy=None, h=None) == 7


def test_resnorm_workspace_serves_calls_with_and_without_a_gate():
    """The query knows T, n and per, and what it gives is enough whether the call has a gate or not."""
    q = B().lib().qgalore_resnorm_bwd_workspace_bytes
    for T in (1, 2, 100, 1000, 5000):
        for per in (1, 3, T):
            for n in (8, 700, 4096):
                d = desc(T=T, per=per, n=n)
                d.workspace_bytes = q(ctypes.byref(d))
                wide = FAR * 8
                a = {k: FAKE + wide * i for i, k in enumerate(NAMES + ("dh", "dy") + GRADS)}
                d.workspace = FAKE + wide * 30
                for kw in ({}, dict(z=None, dz=None), dict(z=None, dz=None, rho=None, drho=None)):
                    assert bwd(d, **{**a, **kw}) in (0, 7) if not torch.cuda.is_available() else True


def test_resnorm_workspace_is_enough_whatever_the_call_has():
    """A call with the queried workspace comes past that check, to the one of results that overlap; with less
    than it needs it does not."""
    q = B().lib().qgalore_resnorm_bwd_workspace_bytes
    wide = FAR * 8
    a = {k: FAKE + wide * i for i, k in enumerate(NAMES + ("dh", "dy") + GRADS)}
    a["du"] = a["dx"]
    for T in (1, 2, 100, 1000, 5000, 60000):
        for per in (1, 3, 257, T):
            for n in (8, 700, 2051, 4096, 12345):
                d = desc(T=T, per=per, n=n, workspace=FAKE + wide * 30)
                d.workspace_bytes = need = q(ctypes.byref(d))
                calls = ({}, dict(z=None, dz=None), dict(z=None, dz=None, rho=None, drho=None))
                for kw in calls:
                    assert bwd(d, **{**a, **kw}) == 5, (T, per, n, kw)
                if need:
                    d.workspace_bytes = need - 1
                    assert 4 in [bwd(d, **{**a, **kw}) for kw in calls], (T, per, n)


def test_resnorm_workspace_without_a_gate_ignores_per():
    """A call without a gate may leave `per` as it likes, in the query too."""
    q = B().lib().qgalore_resnorm_bwd_workspace_bytes
    for T, n in ((16, 64), (1000, 700), (5000, 4096)):
        want = q(ctypes.byref(desc(T=T, n=n, per=1)))
        for per in (0, -5):
            d = desc(T=T, n=n, per=per)
            d.workspace_bytes = q(ctypes.byref(d))
            assert 0 < d.workspace_bytes <= want
            wide = FAR * 8
            a = {k: FAKE + wide * i for i, k in enumerate(NAMES + ("dh", "dy") + GRADS)}
            d.workspace = FAKE + wide * 30
            if not torch.cuda.is_available():
                assert bwd(d, **{**a, "z": None, "dz": None}) == 7


def test_resnorm_binding_refuses_other_calls():
    b = B()
    X, g = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(TypeError):
        b.residual_norm_fwd(X.half(), X.half())
    with pytest.raises(ValueError):
        b.residual_norm_fwd(X, X)                                    # not on a GPU
    with pytest.raises(ValueError):
        b.residual_norm_fwd(X, X, gate=X, per=0)
    with pytest.raises(ValueError):
        b.residual_norm_fwd(X, X, gate=X, gate_act="relu")
    with pytest.raises(ValueError):
        b.residual_norm_bwd(X, None, X, X, X, pre=(g, None))


def test_resnorm_binding_refuses_results_of_what_is_not_there():
    X, g = torch.zeros(4, 8), torch.ones(8)
    for kw in (dict(drho=g), dict(dpost=(g, None)), dict(dpre=(g, g)), dict(dgate=X)):
        with pytest.raises(ValueError, match="needs"):
            B().residual_norm_bwd(X, None, X, X, X, **kw)


def layouts(tmp_path, types):
    """The ctypes structs have the size and field offsets the C compiler gives the header's."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, want = ['#include <stdio.h>', '#include <stddef.h>', '#include "qgalore.h"',
                 "int main(void) {"], []
    for name, cls in types.items():
        src.append(f'  printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            src.append(f'  printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    (tmp_path / "s.c").write_text("\n".join(src + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(tmp_path / "s.c"),
                    "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True)
    assert [int(v) for v in got.stdout.split()] == want


def test_resnorm_struct_layouts_match_the_header(tmp_path):
    b = B()
    layouts(tmp_path, {"qg_resnorm_desc": b.ResnormDesc, "qg_resnorm_params": b.ResnormParams,
                       "qg_resnorm_grads": b.ResnormGrads})
