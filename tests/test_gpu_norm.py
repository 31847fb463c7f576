"""Layer norm and root-mean-square norm, forward and backward, against float64.

Tolerances. fp32 sums over n values, split over lanes and joined in a tree, are off by less than
2^-20 of the sum of magnitudes. The centred values are off by 2^-23 of (|x| + |mean|), which is
relative to the spread where the mean is large: with s = max over the row of (|x| + |mean|) rstd,
h is off by at most 2^-21 (s + |h|). Outputs in bf16 add 2^-8 of the value. dx is a difference of
terms of the size of rstd (|dh| + |h| mean|dh h| + mean|dh|): 2^-19 of that with the errors of h."""
import numpy as np
import pytest

from oracle import qgalore_oracle as O

torch = pytest.importorskip("torch")

U20 = 2.0 ** -20


def B():
    from quantized_rank_gradient_amd import binding
    return binding


def f64(t):
    return t.double().cpu().numpy()


def make(T, n, dtype, seed, mean=0.5, scale=1.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, n)) * scale * rng.uniform(0.5, 2.0, (T, 1)) + mean)
                         .astype(np.float32)).to(dtype)
    dy = torch.from_numpy(rng.standard_normal((T, n)).astype(np.float32)).to(dtype)
    g = (1 + 0.2 * rng.standard_normal(n)).astype(np.float32)
    b = (0.2 * rng.standard_normal(n)).astype(np.float32)
    return x, dy, g, b


def check(x, dy, g, b, center, eps=1e-5):
    out_eps = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    xd, gd = x.cuda(), torch.from_numpy(g).cuda()
    bd = torch.from_numpy(b).cuda() if b is not None else None
    Y, mean, rstd = B().norm_fwd(xd, gd, bd, eps=eps, center=center)
    x64 = x.double().numpy()
    y, rm, rr = O.norm_forward(x64, g, b, eps, center)
    n = x64.shape[1]
    ax = np.abs(x64)
    if center:
        assert (np.abs(f64(mean) - rm) <= U20 * ax.mean(1) + 1e-38).all()
    else:
        assert mean is None
    s = ((ax + np.abs(rm)[:, None]).max(1) * rr)[:, None]
    # rstd: the squares' sum is 2^-20 off, and each centred value 2^-23 s off its own
    assert (np.abs(f64(rstd) - rr) <= rr * (U20 + 2.0 ** -21 * s[:, 0])).all()
    h = (x64 - rm[:, None]) * rr[:, None]
    eh = 2.0 ** -21 * (s + np.abs(h) * (2 + s))
    ey = eh * np.abs(g) + 2.0 ** -23 * (np.abs(y) + np.abs(b if b is not None else 0))
    assert (np.abs(f64(Y) - y) <= ey + out_eps * (np.abs(y) + ey)).all()

    # backward, from the forward pass's own statistics
    dX, dg, db = B().norm_bwd(dy.cuda(), xd, gd, mean, rstd, center=center)
    m32 = f64(mean) if center else np.zeros(len(rm))
    d64 = dy.double().numpy()
    dx, rdg, rdb = O.norm_backward(d64, x64, g, m32, f64(rstd), center)
    r = f64(rstd)[:, None]
    h = (x64 - m32[:, None]) * r
    dh = np.abs(d64 * g)
    eh = 2.0 ** -22 * ((ax + np.abs(m32)[:, None]) * r)
    mags = r * (dh + np.abs(h) * (dh * np.abs(h)).mean(1, keepdims=True)
                + dh.mean(1, keepdims=True))
    ed = 2.0 ** -19 * mags + r * (eh * (dh * np.abs(h)).mean(1, keepdims=True)
                                  + np.abs(h) * (dh * eh).mean(1, keepdims=True))
    assert (np.abs(f64(dX) - dx) <= ed + out_eps * (np.abs(dx) + ed) + 1e-37).all()
    assert (np.abs(f64(dg) - rdg) <= U20 * np.abs(d64 * h).sum(0) + (np.abs(d64) * eh).sum(0)).all()
    if center:
        assert (np.abs(f64(db) - rdb) <= U20 * np.abs(d64).sum(0)).all()
    else:
        assert db is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("T,n", [(1, 1), (3, 2), (1, 7), (5, 64), (7, 100), (2, 511), (9, 512),
                                 (4, 513), (33, 1000), (3, 1024), (6, 1376), (2, 2056), (5, 4096),
                                 (3, 5461), (2, 8200), (1, 16384), (2, 20001), (1, 32768),
                                 (4099, 40)])
def test_norm(T, n, center, dtype):
    x, dy, g, b = make(T, n, dtype, T + n)
    check(x, dy, g, b if center else None, center)


@pytest.mark.gpu
@pytest.mark.parametrize("mean,scale", [(1000.0, 1.0), (0.0, 1e-6), (0.0, 1e6), (-30.0, 0.1)])
def test_norm_of_rows_far_from_zero(mean, scale):
    x, dy, g, b = make(17, 777, torch.float32, 5, mean, scale)
    check(x, dy, g, b, True)
    check(x, dy, g, None, False)


@pytest.mark.gpu
def test_norm_of_equal_values_and_zeros():
    """A row without spread: y = beta exactly where the values are equal (and 0 for zeros without
    center); its rstd is 1 / sqrt(eps)."""
    b = B()
    x = torch.zeros(3, 96)
    x[1] = 2.5
    g, beta = torch.full((96,), 3.0), torch.linspace(-1, 1, 96)
    for dt in (torch.float32, torch.bfloat16):
        Y, mean, rstd = b.norm_fwd(x.to(dt).cuda(), g.cuda(), beta.cuda())
        assert torch.equal(Y.cpu(), beta.to(dt).expand(3, 96))
        assert torch.equal(mean.cpu(), torch.tensor([0.0, 2.5, 0.0]))
        assert torch.allclose(rstd.cpu(), torch.tensor(1e-5 ** -0.5), rtol=2.0 ** -20)
        Y, _, rstd = b.norm_fwd(x.to(dt).cuda(), g.cuda(), center=False)
        assert (Y[0] == 0).all() and (Y[2] == 0).all()


@pytest.mark.gpu
def test_a_nan_stays_in_its_row():
    x, dy, g, b = make(6, 300, torch.bfloat16, 1)
    x[2, 17] = float("nan")
    x[4, 299] = float("inf")
    Y, mean, rstd = B().norm_fwd(x.cuda(), torch.from_numpy(g).cuda(), torch.from_numpy(b).cuda())
    bad = ~np.isfinite(f64(Y)).all(1)
    assert bad.tolist() == [False, False, True, False, True, False]
    assert np.isnan(f64(Y)[2]).all()


@pytest.mark.gpu
def test_norm_equal_calls_give_equal_bits_and_write_nothing_else():
    b = B()
    x, dy, g, beta = make(1030, 264, torch.bfloat16, 3)
    xd, dyd, gd = x.cuda(), dy.cuda(), torch.from_numpy(g).cuda()
    _, mean, rstd = b.norm_fwd(xd, gd)
    first = b.norm_bwd(dyd, xd, gd, mean, rstd)
    for _ in range(3):
        for p, q in zip(first, b.norm_bwd(dyd, xd, gd, mean, rstd)):
            assert torch.equal(p, q)
    whole = torch.full((1030 * 264 + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    view = whole[64:64 + 1030 * 264].view(1030, 264)
    b.norm_bwd(dyd, xd, gd, mean, rstd, dX=view)
    assert torch.equal(view, first[0]) and (whole[:64] == 7).all() and (whole[-64:] == 7).all()


@pytest.mark.gpu
def test_norm_captured_and_replayed_on_another_stream():
    b = B()
    x, dy, g, beta = make(70, 264, torch.bfloat16, 4)
    xd, dyd, gd, bd = x.cuda(), dy.cuda(), torch.from_numpy(g).cuda(), torch.from_numpy(beta).cuda()

    def both(stream=None):
        Y, mean, rstd = b.norm_fwd(xd, gd, bd, stream=stream)
        return (Y, *b.norm_bwd(dyd, xd, gd, mean, rstd, stream=stream))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    s = torch.cuda.Stream()
    for k in range(4):
        xd.copy_(make(70, 264, torch.bfloat16, 20 + k)[0])
        graph.replay()
        s.wait_stream(torch.cuda.current_stream())
        want = both(s)
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


# ---------------------------------------------------------------------- on the CPU ---
@pytest.mark.parametrize("center", [True, False])
def test_oracle_norm_gradients_against_differences(center):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((4, 31)), rng.standard_normal((4, 31))
    g, b = rng.standard_normal(31), rng.standard_normal(31)
    _, mean, rstd = O.norm_forward(x, g, b, 1e-3, center)
    dx, dg, db = O.norm_backward(dy, x, g, mean, rstd, center)
    h = 1e-6
    for _ in range(4):
        u, v, w = (rng.standard_normal(t.shape) for t in (x, g, b))
        f = lambda s: float((dy * O.norm_forward(x + s * u, g + s * v, b + s * w, 1e-3, center)[0]).sum())  # noqa: E731
        num, ana = (f(h) - f(-h)) / (2 * h), (dx * u).sum() + (dg * v).sum() + (db * w).sum()
        assert abs(num - ana) <= 1e-6 * (np.abs(dx * u).sum() + np.abs(dg * v).sum()
                                         + np.abs(db * w).sum())


FAKE = 0x10000


def desc(**kw):
    d = B().NormDesc(16, 64, 0, 1, 1e-5, FAKE, 1 << 40, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fwd(d, x=FAKE, g=FAKE, b=FAKE, y=FAKE, mean=FAKE, rstd=FAKE):
    import ctypes
    return B().lib().qgalore_norm_fwd(ctypes.byref(d), x, g, b, y, mean, rstd)


def bwd(d, dy=FAKE, x=FAKE, g=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dg=FAKE, db=FAKE):
    import ctypes
    return B().lib().qgalore_norm_bwd(ctypes.byref(d), dy, x, g, mean, rstd, dx, dg, db)


def test_norm_refusals_come_before_any_device_call():
    for k in ("x", "g", "y", "rstd"):
        assert fwd(desc(), **{k: None}) == 1, k
    for k in ("dy", "x", "g", "mean", "rstd", "dx", "dg"):
        assert bwd(desc(), **{k: None}) == 1, k
    for k in ("x", "g", "b", "y"):
        assert fwd(desc(), **{k: FAKE + 4}) == 3, k
    for k in ("mean", "rstd"):
        assert fwd(desc(), **{k: FAKE + 2}) == 3 and bwd(desc(), **{k: FAKE + 2}) == 3, k
    for k in ("dy", "x", "g", "dx", "dg", "db"):
        assert bwd(desc(), **{k: FAKE + 4}) == 3, k
    for bad in (dict(T=0), dict(n=0), dict(n=32769), dict(T=1 << 30, n=64), dict(T=-1)):
        assert fwd(desc(**bad)) == 2 and bwd(desc(**bad)) == 2, bad
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(center=2), dict(dtype=2),
                dict(dtype=-1)):
        assert fwd(desc(**bad)) == 5 and bwd(desc(**bad)) == 5, bad
    assert bwd(desc(workspace=None)) == 1
    assert bwd(desc(workspace=FAKE + 8)) == 3
    assert bwd(desc(workspace_bytes=16)) == 4
    q = B().lib().qgalore_norm_bwd_workspace_bytes
    assert q(16, 64) >= 2 * 64 * 4 and q(0, 64) == 0 and q(16, 40000) == 0


def test_norm_outputs_over_what_a_call_still_reads_are_refused():
    rows, far = 2 * 16 * 64, 1 << 30
    a = dict(x=FAKE, g=FAKE + far, b=FAKE + 2 * far, y=FAKE + 3 * far, mean=FAKE + 4 * far,
             rstd=FAKE + 5 * far)
    for out, size in (("y", rows), ("mean", 64), ("rstd", 64)):
        for other in a:
            if other != out:
                assert fwd(desc(), **{**a, other: a[out] + size - 16}) == 5, (out, other)
    g = dict(dy=FAKE, x=FAKE + far, g=FAKE + 2 * far, mean=FAKE + 3 * far, rstd=FAKE + 4 * far,
             dx=FAKE + 5 * far, dg=FAKE + 6 * far, db=FAKE + 7 * far)
    for other in g:
        if other != "dx":
            assert bwd(desc(), **{**g, other: g["dx"] + rows - 16}) == 5, other
    for out in ("dg", "db"):
        for other in ("dx", "dg", "db", "g"):
            if other != out:
                assert bwd(desc(), **{**g, other: g[out] + 4 * 64 - 16}) == 5, (out, other)
    assert bwd(desc(), **{**g, "db": g["dg"]}) == 5
    if not torch.cuda.is_available():                # accepted: the next thing it needs is a device
        assert fwd(desc(), **a) == 7 and fwd(desc(), **{**a, "y": a["x"]}) == 7
        assert bwd(desc(), **g) == 7
        assert bwd(desc(), **{**g, "dx": g["x"]}) == 7 and bwd(desc(), **{**g, "dx": g["dy"]}) == 7


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(5, 7), (1030, 264), (600, 1000), (300, 4096), (40, 8200), (9, 20001)])
@pytest.mark.parametrize("center", [True, False])
def test_norm_in_place(T, n, center):
    b = B()
    x, dy, g, beta = make(T, n, torch.bfloat16, 3)
    gd = torch.from_numpy(g).cuda()
    y, mean, rstd = b.norm_fwd(x.cuda(), gd, center=center)
    xd = x.cuda()
    assert torch.equal(b.norm_fwd(xd, gd, center=center, out=xd)[0], y)
    want = b.norm_bwd(dy.cuda(), x.cuda(), gd, mean, rstd, center=center)[0]
    for over in (0, 1):
        t = [dy.cuda(), x.cuda()]
        assert torch.equal(b.norm_bwd(*t, gd, mean, rstd, center=center, dX=t[over])[0], want)


def test_binding_refuses_other_types_and_host_tensors():
    b = B()
    with pytest.raises(TypeError):
        b.norm_fwd(torch.zeros(2, 8, dtype=torch.float16), torch.ones(8))
    with pytest.raises(ValueError):
        b.norm_fwd(torch.zeros(2, 8), torch.ones(8))


def test_struct_layouts_of_the_operators_match_the_header(tmp_path):
    """The ctypes structs have the size and field offsets the C compiler gives the header's."""
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    b = B()
    types = {"qg_linear_desc": b.LinearDesc, "qg_norm_desc": b.NormDesc,
             "qg_muon_desc": b.MuonDesc, "qg_muon_layer": b.MuonLayerDesc}
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
