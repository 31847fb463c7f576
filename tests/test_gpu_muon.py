"""The orthogonalised update against the 64-bit iteration.

Tolerances. The products take operands rounded to fp16 (half a step: 2^-11 of a value) and the
result is rounded to bf16 (2^-8). Norm-wise: rounding to bf16 is off by at most 2^-8 of each
value, 2^-8 / sqrt(3) in the mean square if errors spread evenly over the step; a step rounds A, B
and X, each off by 2^-11 / sqrt(3) in the mean square with a gain of at most a = 3.44, over s steps
sqrt(3 s) * 3.44 * 2^-11 / sqrt(3) at worst (five: 3.8e-3) and independent of the first: the whole
stays below sqrt((2^-8)^2 / 3 + s (3.44 * 2^-11)^2) (five: 4.4e-3). Element-wise: 2^-8 of the value
and eight times the steps' part of the root mean square. INT8 codes: the rounding input differs by the update's
element-wise error (without the bf16 rounding: the codes come from the fp32 result), times
lr alpha / s, and by fp32 roundings of numbers below 2^8; a code may be another only within that of
a border."""
import math

import numpy as np
import pytest

from oracle import qgalore_oracle as O

torch = pytest.importorskip("torch")

NORM_TOL = 4.4e-3        # five steps
ELEM_TOL = 8 * 3.8e-3


def B():
    from quantized_rank_gradient_amd import binding
    return binding


def bf16_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def matrix(m, n, seed, kind="gauss"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, n))
    if kind == "lowrank":      # a few directions, the others a hundred times smaller
        r = max(1, min(m, n) // 16)
        x = rng.standard_normal((m, r)) @ rng.standard_normal((r, n)) / math.sqrt(r) + 1e-2 * x
    elif kind == "rows":       # rows of very different sizes, some of zeros
        x = x * rng.random((m, 1)) ** 8 * (rng.random((m, 1)) > 0.2)
    return O.f32_to_bf16_bits(x.astype(np.float32))


def check_update(got, want, what="", steps=5):
    rms = np.sqrt(np.mean(want * want))
    part = math.sqrt(steps) * 3.44 * 2.0 ** -11
    assert np.linalg.norm(got - want) <= math.hypot(2.0 ** -8 / math.sqrt(3), part) \
        * np.linalg.norm(want), (what, np.linalg.norm(got - want) / np.linalg.norm(want))
    bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + 8 * part * rms
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want).max() / rms))


SHAPES = [(1, 1), (1, 300), (300, 1), (7, 13), (64, 64), (128, 128), (129, 127), (127, 130),
          (200, 512), (512, 200), (257, 640), (1000, 72), (384, 1021), (513, 515)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("kind", ["gauss", "lowrank", "rows"])
def test_orthogonalize(m, n, kind):
    bits = [matrix(m, n, 17 * m + n + k, kind) for k in range(2)]
    outs = B().orthogonalize([bf16_dev(b) for b in bits])
    for b, o in zip(bits, outs):
        check_update(f64(o), O.orthogonalize(O.bf16_bits_to_f32(b)), (m, n, kind))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(2048, 520), (700, 2500), (2304, 2304)])
def test_orthogonalize_many_tiles(m, n):
    bits = matrix(m, n, m + n)
    check_update(f64(B().orthogonalize([bf16_dev(bits)])[0]),
                 O.orthogonalize(O.bf16_bits_to_f32(bits)))


def orthogonalize_torch(bits, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """O.orthogonalize in float64 on the GPU, for sizes that take numpy too long."""
    a, b, c = (float(np.float32(x)) for x in coef)
    X = bf16_dev(bits).double()
    X = X / (X.norm() + float(np.float32(eps)))
    tall = X.shape[0] > X.shape[1]
    X = X.t().contiguous() if tall else X
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.t() if tall else X).cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("count,m,n,looked_at", [
    (13, 1500, 1540, (0, 6, 11, 12)), (13, 1540, 1500, (0, 12)), (5, 2000, 2041, (0, 3, 4)),
    (5, 2041, 2000, (0, 4)), (2, 4096, 4000, (0, 1)), (1, 1030, 5000, (0,)), (1, 5000, 1030, (0,))])
def test_orthogonalize_large_tiles(count, m, n, looked_at):
    """Sizes with tiles of 256 and, where the last round would be mostly empty, quarters of them."""
    bits = [matrix(m, n, k, ["gauss", "lowrank", "rows"][k % 3]) for k in range(count)]
    outs = B().orthogonalize([bf16_dev(b) for b in bits])
    for k in looked_at:
        check_update(f64(outs[k]), orthogonalize_torch(bits[k]), (count, m, n, k))


@pytest.mark.gpu
@pytest.mark.parametrize("count,m,n", [(1, 150, 3001), (1, 3001, 150), (3, 200, 1290), (2, 2333, 321),
                                       (1, 513, 8200)])
def test_orthogonalize_long_and_narrow(count, m, n):
    """Products of few tiles are cut along their inner dimension: the parts' order of arrival does not
    show, and a workspace's old content does not matter."""
    b = B()
    bits = [matrix(m, n, 5 + k, ["gauss", "lowrank", "rows"][k % 3]) for k in range(count)]
    G = [bf16_dev(x) for x in bits]
    outs = b.orthogonalize(G)
    for x, o in zip(bits, outs):
        check_update(f64(o), orthogonalize_torch(x), (count, m, n))
    ws = b.alloc_workspace(b.muon_workspace_bytes(m, n, count))
    g, cap = torch.cuda.CUDAGraph(), [torch.empty_like(o) for o in outs]
    with torch.cuda.graph(g):
        b.orthogonalize(G, out=cap, workspace=ws)
    for k in range(6):
        ws.fill_(0xFF)
        for o in cap:
            o.zero_()
        g.replay() if k % 2 else b.orthogonalize(G, out=cap, workspace=ws)
        assert all(torch.equal(o, c) for o, c in zip(outs, cap)), k


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(1100, 1301), (1304, 1100)])
def test_muon_step_large_tiles(m, n):
    b = B()
    G, M, Wq, Ws = state(m, n, 4)
    L = b.MuonLayer(3, bf16_dev(G), torch.from_numpy(Wq).cuda(), torch.from_numpy(Ws).cuda(),
                    torch.from_numpy(M).cuda())
    b.muon_step(L, 9, 123456789123, dict(lr=0.03, weight_decay=0.02))
    M1 = O.muon_momentum(M, G, 0.95)
    assert np.array_equal(L.M.cpu().numpy(), M1)
    X = O.orthogonalize(O.muon_direction(M1, G, 0.95, True).astype(np.float64))
    lr = float(np.float32(0.03))
    check_weights(L.Wq.cpu().numpy(), Wq, Ws, X, lr * math.sqrt(max(1, m / n)),
                  lr * float(np.float32(0.02)), 9, 123456789123, 3)


@pytest.mark.gpu
def test_orthogonalize_more_layers_than_one_launch_takes():
    bits = [matrix(96, 160, k) for k in range(35)]
    outs = B().orthogonalize([bf16_dev(b) for b in bits])
    for k, (b, o) in enumerate(zip(bits, outs)):
        check_update(f64(o), O.orthogonalize(O.bf16_bits_to_f32(b)), k)


@pytest.mark.gpu
@pytest.mark.parametrize("steps,coef", [(1, (3.4445, -4.7750, 2.0315)), (2, (1.875, -1.25, 0.375)),
                                        (7, (1.5, -0.5, 0.0))])
def test_orthogonalize_other_polynomials(steps, coef):
    bits = matrix(150, 260, 3)
    got = f64(B().orthogonalize([bf16_dev(bits)], steps=steps, coef=coef)[0])
    check_update(got, O.orthogonalize(O.bf16_bits_to_f32(bits), steps, coef), "", steps)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(100, 130), (40, 1000), (3000, 60), (128, 128)])
@pytest.mark.parametrize("steps,coef", [(1, (3.4445, -4.7750, 2.0315)), (3, (1.875, -1.25, 0.375)),
                                        (7, (3.4445, -4.7750, 2.0315)), (7, (1.5, -0.5, 0.0))])
def test_orthogonalize_small_matrices(m, n, steps, coef):
    """One side of at most 128: the steps' product in one workgroup, or step by step where they would
    multiply its rounding by too much."""
    for kind in ("gauss", "lowrank"):
        bits = [matrix(m, n, 3 + k, kind) for k in range(2)]
        outs = B().orthogonalize([bf16_dev(b) for b in bits], steps=steps, coef=coef)
        for b, o in zip(bits, outs):
            check_update(f64(o), O.orthogonalize(O.bf16_bits_to_f32(b), steps, coef), kind, steps)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-36, 1e-20, 1e20, 1e36])
def test_orthogonalize_does_not_depend_on_scale(scale):
    bits = O.f32_to_bf16_bits((O.bf16_bits_to_f32(matrix(96, 200, 5)) * np.float32(scale)))
    got = f64(B().orthogonalize([bf16_dev(bits)], eps=0.0)[0])
    check_update(got, O.orthogonalize(O.bf16_bits_to_f32(bits).astype(np.float64), eps=0.0))


@pytest.mark.gpu
@pytest.mark.parametrize("below", [1e-1, 1e-3, 1e-5, 1e-6, 1e-8, 1e-14, 1e-25])
@pytest.mark.parametrize("steps,coef", [(5, (3.4445, -4.7750, 2.0315)), (7, (1.5, -0.5, 0.0)),
                                        (1, (3.4445, -4.7750, 2.0315))])
def test_orthogonalize_matrices_smaller_than_eps(below, steps, coef):
    """A norm far below eps makes X small, not less exact."""
    for m, n, kind in ((150, 260, "gauss"), (300, 140, "lowrank"), (40, 100, "gauss")):
        x = O.bf16_bits_to_f32(matrix(m, n, 12, kind)).astype(np.float64)
        bits = O.f32_to_bf16_bits((x * (1e-7 * below / np.linalg.norm(x))).astype(np.float32))
        got = f64(B().orthogonalize([bf16_dev(bits)], steps=steps, coef=coef, eps=1e-7)[0])
        want = O.orthogonalize(O.bf16_bits_to_f32(bits).astype(np.float64), steps, coef, 1e-7)
        check_update(got, want, (m, n, kind), steps)


@pytest.mark.gpu
def test_orthogonalize_zero_and_non_finite_matrices():
    """Each matrix of a call stands for itself: zeros give zeros, an infinity or a NaN gives NaN."""
    bits = [matrix(70, 90, k) for k in range(4)]
    bits[0][:] = 0
    bits[1][3, 4] = 0x7F80
    bits[2][69, 89] = 0x7FC0
    for eps in (1e-7, 0.0):
        outs = [f64(o) for o in B().orthogonalize([bf16_dev(b) for b in bits], eps=eps)]
        assert (outs[0] == 0).all()
        assert np.isnan(outs[1]).all() and np.isnan(outs[2]).all()
        check_update(outs[3], O.orthogonalize(O.bf16_bits_to_f32(bits[3]), eps=eps))


def state(m, n, seed, k=0):
    rng = np.random.default_rng([seed, k])
    G = matrix(m, n, seed + 1000 * k)
    M = (3 * rng.standard_normal((m, n))).astype(np.float32)
    Wq = rng.integers(-127, 128, size=(m, n)).astype(np.int8)
    Ws = (rng.uniform(0.5, 2.0, O.n_groups(m * n)) * 1e-3).astype(np.float32)
    return G, M, Wq, Ws


def check_weights(got, Wq, Ws, X, lr_alpha, lr_decay, t, seed, layer_id):
    m, n = Wq.shape
    d = O.muon_rounding_input(Wq, Ws, X, lr_alpha, lr_decay, t, seed, layer_id)
    want = np.clip(np.floor(d), -127, 127)
    s = np.repeat(Ws.astype(np.float64), 256)[: m * n].reshape(m, n)
    reach = lr_alpha * ELEM_TOL * np.sqrt(np.mean(X * X)) / s + 6 * 2.0 ** -24 * 256
    off = got != want
    assert (np.abs(got - want)[off] == 1).all()
    assert (np.abs(d - np.round(d))[off] <= reach[off]).all()
    # on average a code is another with the probability of the mean error, a few times 1e-3 of the
    # update's root mean square
    mean = np.mean(lr_alpha * NORM_TOL * np.sqrt(np.mean(X * X)) / s + 2.0 ** -16)
    assert off.sum() <= 2 * mean * off.size + 4, (off.mean(), mean)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,nesterov,decay", [
    (64, 64, True, 0.0), (256, 200, False, 0.1), (129, 517, True, 0.1), (333, 40, True, 0.0),
    (1, 700, True, 0.0), (515, 512, False, 0.0)])
def test_muon_step(m, n, nesterov, decay):
    b = B()
    hp = dict(lr=0.02, momentum=0.95, nesterov=nesterov, weight_decay=decay)
    G, M, Wq, Ws = state(m, n, m + n)
    L = b.MuonLayer(11, bf16_dev(G), torch.from_numpy(Wq).cuda(), torch.from_numpy(Ws).cuda(),
                    torch.from_numpy(M).cuda())
    b.muon_step(L, 3, 77, hp)
    M1 = O.muon_momentum(M, G, 0.95)
    assert np.array_equal(L.M.cpu().numpy(), M1)
    X = O.orthogonalize(O.muon_direction(M1, G, 0.95, nesterov).astype(np.float64))
    lr = float(np.float32(0.02))
    check_weights(L.Wq.cpu().numpy(), Wq, Ws, X, lr * math.sqrt(max(1, m / n)),
                  lr * float(np.float32(decay)), 3, 77, 11)
    assert np.array_equal(L.G.view(torch.int16).cpu().numpy().view(np.uint16), G)


@pytest.mark.gpu
def test_muon_step_keeps_codes_where_nothing_is_defined():
    """A zero gradient and momentum move a weight by nothing (u < 1 keeps the floor); a gradient with
    a NaN keeps every code; a scale of zero keeps its group."""
    b = B()
    G, M, Wq, Ws = state(96, 128, 5)
    M[:] = 0
    zero = np.zeros_like(G)
    nan = G.copy()
    nan[1, 1] = 0x7FC0
    Ws0 = Ws.copy()
    Ws0[7] = 0
    layers = [b.MuonLayer(k, bf16_dev(g), torch.from_numpy(Wq).cuda(), torch.from_numpy(s).cuda(),
                          torch.from_numpy(M).cuda())
              for k, (g, s) in enumerate([(zero, Ws), (nan, Ws), (G, Ws0), (G, Ws)])]
    b.Muon(layers, dict(lr=0.5)).step(1, 5)
    out = [L.Wq.cpu().numpy() for L in layers]
    assert np.array_equal(out[0], Wq) and np.array_equal(out[1], Wq)
    assert np.array_equal(out[2].reshape(-1)[7 * 256: 8 * 256], Wq.reshape(-1)[7 * 256: 8 * 256])
    assert (out[2] != Wq).mean() > 0.3 and (out[3] != Wq).mean() > 0.3


@pytest.mark.gpu
def test_muon_set_of_shapes_equals_single_steps():
    """A set of layers of several shapes, two steps: bit for bit the layers stepped one by one, on a
    stream of its own with a shared workspace."""
    b = B()
    shapes = [(64, 200), (200, 64), (64, 200), (130, 130), (64, 200)]

    def make():
        return [b.MuonLayer(k, bf16_dev(G), torch.from_numpy(Wq).cuda(),
                            torch.from_numpy(Ws).cuda(), torch.from_numpy(M).cuda())
                for k, (G, M, Wq, Ws) in enumerate(state(m, n, 9, k)
                                                   for k, (m, n) in enumerate(shapes))]
    one, both = make(), make()
    opt = b.Muon(both, dict(lr=0.05, weight_decay=0.01))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (1, 2):
        opt.step(t, 3, stream=s)
        for L in one:
            b.muon_step(L, t, 3, dict(lr=0.05, weight_decay=0.01))
    torch.cuda.synchronize()
    for x, y in zip(one, both):
        assert torch.equal(x.M, y.M) and torch.equal(x.Wq, y.Wq)


@pytest.mark.gpu
def test_muon_captured_and_replayed():
    """A captured step replays as the eager one runs, with eager work of another object and
    synchronisations between the replays."""
    b = B()
    G, M, Wq, Ws = state(150, 264, 21)

    def make():
        return b.MuonLayer(2, bf16_dev(G), torch.from_numpy(Wq).cuda(),
                           torch.from_numpy(Ws).cuda(), torch.from_numpy(M).cuda())
    cap, eager, other = make(), make(), make()
    co, eo, oo = b.Muon([cap]), b.Muon([eager]), b.Muon([other])
    ws = b.alloc_workspace(co.workspace_bytes)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        co.step(4, 9, workspace=ws)
    for _ in range(4):
        g.replay()
        oo.step(1, 1)
        torch.cuda.synchronize()
        eo.step(4, 9)
        assert torch.equal(cap.M, eager.M) and torch.equal(cap.Wq, eager.Wq)


@pytest.mark.gpu
def test_two_sets_at_once_on_two_streams():
    b = B()
    data = [state(192, 320, 31, k) for k in range(2)]

    def make():
        return [b.MuonLayer(k, bf16_dev(G), torch.from_numpy(Wq).cuda(),
                            torch.from_numpy(Ws).cuda(), torch.from_numpy(M).cuda())
                for k, (G, M, Wq, Ws) in enumerate(data)]
    want, got = make(), make()
    for L in want:
        for t in (1, 2, 3):
            b.muon_step(L, t, 8)
    streams = [torch.cuda.Stream() for _ in got]
    sets = [b.Muon([L]) for L in got]
    torch.cuda.synchronize()
    for t in (1, 2, 3):
        for s, o in zip(streams, sets):
            o.step(t, 8, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x.M, y.M) and torch.equal(x.Wq, y.Wq)


@pytest.mark.gpu
def test_set_on_another_stream_than_its_workspace():
    b = B()
    G, M, Wq, Ws = state(192, 320, 33)

    def make():
        return b.MuonLayer(0, bf16_dev(G), torch.from_numpy(Wq).cuda(), torch.from_numpy(Ws).cuda(),
                           torch.from_numpy(M).cuda())
    one, two = make(), make()
    a, c = b.Muon([one]), b.Muon([two])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.step(1, 3)
    side.wait_stream(torch.cuda.current_stream())
    a.step(2, 3, stream=side)
    del a                       # its workspace is still in use on the other stream
    junk = torch.full((64 << 20,), -1, dtype=torch.int8, device="cuda")
    c.step(1, 3)
    c.step(2, 3)
    torch.cuda.synchronize()
    assert torch.equal(one.Wq, two.Wq) and torch.equal(one.M, two.M) and int(junk[0]) == -1


# ------------------------------------------------------------------------- refusals ---
FAKE = 0x10000


def desc(**kw):
    d = B()._muon_desc(64, 96, {})
    d.workspace, d.workspace_bytes = FAKE, 1 << 40
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def step_status(d, step=1, count=1, **kw):
    import ctypes
    L = B().MuonLayerDesc(FAKE, FAKE, FAKE, FAKE, 0)
    for k, v in kw.items():
        setattr(L, k, v)
    return B().lib().qgalore_muon_step(ctypes.byref(d), ctypes.byref(L), count, step, 1)


def test_muon_refusals_come_before_any_device_call():
    nan = float("nan")
    assert step_status(desc(), G=None) == 1
    assert step_status(desc(), M=None) == 1
    assert step_status(desc(), W_q=None) == 1
    assert step_status(desc(), W_scale=None) == 1
    assert step_status(desc(workspace=None)) == 1
    assert step_status(desc(m=0)) == 2
    assert step_status(desc(n=-1)) == 2
    assert step_status(desc(), count=0) == 2
    assert step_status(desc(m=1 << 30, n=1)) == 2             # rows of one padded to 64
    assert step_status(desc(m=30000, n=30000)) == 2
    assert step_status(desc(), G=FAKE + 2) == 3
    assert step_status(desc(), M=FAKE + 4) == 3
    assert step_status(desc(), W_q=FAKE + 8) == 3
    assert step_status(desc(), W_scale=FAKE + 2) == 3
    assert step_status(desc(workspace=FAKE + 8)) == 3
    assert step_status(desc(workspace_bytes=1000)) == 4
    for bad in (dict(lr=nan), dict(lr=float("inf")), dict(momentum=1.0), dict(momentum=-0.1),
                dict(weight_decay=-1.0), dict(weight_decay=nan), dict(alpha=nan),
                dict(lr=1e30, alpha=1e30), dict(nesterov=2), dict(ns_steps=0), dict(ns_steps=8), dict(ns_steps=16),
                dict(eps=-1.0), dict(eps=nan), dict(ns_a=nan), dict(ns_b=100.0),
                dict(ns_a=9.0, ns_b=0.0, ns_c=0.0)):
        assert step_status(desc(**bad)) == 5, bad
    for bad in (0, -1, 1 << 32):
        assert step_status(desc(), step=bad) == 5
    L = B().lib()
    assert L.qgalore_muon_step(None, None, 1, 1, 1) == 1
    assert L.qgalore_orthogonalize(None, None, None, 1) == 1
    assert L.qgalore_muon_workspace_bytes(0, 4, 1) == 0
    assert L.qgalore_muon_workspace_bytes(64, 96, 0) == 0
    assert L.qgalore_muon_workspace_bytes(64, 96, 3) > 3 * (4 * 64 * 128 * 2 + 2 * 64 * 64 * 2)
    # a call works through 16 layers at a time
    assert (L.qgalore_muon_workspace_bytes(64, 96, 16)
            == L.qgalore_muon_workspace_bytes(64, 96, 1000))


def test_a_layer_given_twice_is_refused():
    import ctypes
    b = B()
    two = (b.MuonLayerDesc * 2)(b.MuonLayerDesc(FAKE, FAKE, FAKE, FAKE, 0),
                                b.MuonLayerDesc(FAKE, FAKE + 4096, FAKE + 4096, FAKE, 1))

    def status():
        return b.lib().qgalore_muon_step(ctypes.byref(desc(workspace=None)), two, 2, 1, 1)
    assert status() == 1   # all but the workspace
    two[1].M = FAKE
    assert status() == 5
    two[1].M, two[1].W_q = FAKE + 4096, FAKE
    assert status() == 5
    src = (ctypes.c_void_p * 2)(FAKE, FAKE)
    dst = (ctypes.c_void_p * 2)(FAKE, FAKE)
    assert b.lib().qgalore_orthogonalize(ctypes.byref(desc(workspace=None)), src, dst, 2) == 5
    G = torch.zeros(8, 8, dtype=torch.bfloat16)
    Wq, Ws, M = torch.zeros(8, 8, dtype=torch.int8), torch.ones(1), torch.zeros(8, 8)
    with pytest.raises(ValueError):
        b.Muon([b.MuonLayer(0, G, Wq, Ws, M), b.MuonLayer(1, G, Wq, Ws, torch.zeros(8, 8))])


def test_outputs_that_overlap_are_refused():
    import ctypes
    b = B()
    size = 64 * 96                                   # of desc()'s matrices

    def step(dM, dW):
        two = (b.MuonLayerDesc * 2)(b.MuonLayerDesc(FAKE, FAKE, FAKE, FAKE, 0),
                                    b.MuonLayerDesc(FAKE, FAKE + dM, FAKE + dW, FAKE, 1))
        return b.lib().qgalore_muon_step(ctypes.byref(desc()), two, 2, 1, 1)
    assert step(4 * size - 16, size) == 5 and step(4 * size, size - 16) == 5
    assert step(16, 2 * size) == 5

    def orthogonalize(src, dst):
        n = len(src)
        return b.lib().qgalore_orthogonalize(ctypes.byref(desc()), (ctypes.c_void_p * n)(*src),
                                             (ctypes.c_void_p * n)(*dst), n)
    assert orthogonalize([FAKE, FAKE], [FAKE, FAKE + 2 * size - 16]) == 5
    # a result over a matrix that a later launch of 16 is still to read
    far = 1 << 30
    src = [FAKE + 2 * size * k for k in range(20)]
    dst = [far + 2 * size * k for k in range(20)]
    dst[3] = src[16]
    assert orthogonalize(src, dst) == 5
    dst[3] = src[19] + 2 * size - 16
    assert orthogonalize(src, dst) == 5
    if not torch.cuda.is_available():                # accepted: the next thing it needs is a device
        assert step(4 * size, size) == 7
        assert orthogonalize(src, src) == 7          # each over its own
        dst[3], dst[18] = src[15], src[2]            # read before, in the same launch or an earlier one
        assert orthogonalize(src, dst) == 7
    buf = torch.zeros(80, 8)
    G, Wq, Ws = torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(20, 8, dtype=torch.int8), \
        torch.ones(1)
    for M, W in (((buf[:8], buf[4:12]), (Wq[:8], Wq[8:16])), ((buf[:8], buf[8:16]), (Wq[:8], Wq[6:14])),
                 ((buf[:8], buf[2:4].view(2, 8)), (Wq[:8], Wq[8:10]))):
        with pytest.raises(ValueError, match="share"):
            b.Muon([b.MuonLayer(k, G[:m.shape[0]], w, Ws, m) for k, (m, w) in enumerate(zip(M, W))])


@pytest.mark.gpu
def test_orthogonalize_in_place():
    b = B()
    G = [bf16_dev(matrix(150, 72, k)) for k in range(18)]
    want = b.orthogonalize(G)
    b.orthogonalize(G, out=G)
    for x, y in zip(want, G):
        assert torch.equal(x, y)


def test_orthogonalize_refusals_come_before_any_device_call():
    import ctypes
    b = B()

    def status(d, g=FAKE, o=FAKE):
        src, dst = (ctypes.c_void_p * 1)(g), (ctypes.c_void_p * 1)(o)
        return b.lib().qgalore_orthogonalize(ctypes.byref(d), src, dst, 1)
    assert status(desc(), g=None) == 1
    assert status(desc(), o=None) == 1
    assert status(desc(), o=FAKE + 2) == 3
    assert status(desc(workspace_bytes=1)) == 4
    assert status(desc(ns_steps=0)) == 5
    assert status(desc(m=0)) == 2


def test_binding_refuses_host_tensors_and_wrong_types():
    b = B()
    G = torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.orthogonalize([G])
    with pytest.raises(ValueError):
        b.orthogonalize([])
    with pytest.raises(ValueError):
        b.Muon([])
    L = b.MuonLayer(0, G, torch.zeros(8, 8, dtype=torch.int8), torch.ones(1), torch.zeros(8, 8))
    with pytest.raises(ValueError):
        b.muon_step(L, 1, 1)
    with pytest.raises(ValueError):
        b.Muon([L])
