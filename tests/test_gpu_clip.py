"""The norm of a set of gradients and their clipping, against float64.

Tolerances. The sum of squares is formed in fp64 (each square exact to 2^-53 and each of fewer than 2^20
additions a lane and join off by 2^-53: below 2^-33 in all), so the norm is off by its rounding to fp32,
2^-24, and by no more than 2^-33 besides. The factor is rounded to fp32 (2^-24), the product to fp32 (2^-24)
and to the tensor's type (bf16 2^-8, fp32: the product's own); in the subnormal range each rounding is off by
half the type's smallest step."""
import ctypes

import numpy as np
import pytest

from oracle import qgalore_oracle as O

torch = pytest.importorskip("torch")

BF16, FP32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -134, FP32: 2.0 ** -150}   # half the smallest subnormal


def B():
    from quantized_rank_gradient_amd import binding
    return binding


def f64(t):
    return t.detach().double().cpu().numpy()


def grads(shapes, seed, scale=1.0):
    """Tensors of (shape, type)."""
    rng = np.random.default_rng(seed)
    return [torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).to(dt)
            for s, dt in shapes]


def check(ts, max_norm, kind="l2", eps=1e-6, inplace=False):
    dev = [t.cuda() for t in ts]
    out = dev if inplace else [torch.full_like(t, 9.0) for t in dev]
    s = B().GradSet(dev, out=None if inplace else out, kind=kind, eps=eps)
    norm, want = O.clip([f64(t) for t in ts], max_norm, float(np.float32(eps)), kind)
    got = float(s.norm())
    if norm >= 2.0 ** 128 - 2.0 ** 103:   # rounds to infinity in fp32; the factor comes from the fp64 norm
        assert got == float("inf")
    else:
        assert abs(got - norm) <= norm * 2.0 ** -23.9 + 2.0 ** -150
    assert float(s.clip(max_norm)) == got
    for g, w, o in zip(ts, want, out):
        rel = 2.0 ** -22.9 + (2.0 ** -8 if g.dtype == BF16 else 0.0)
        assert (np.abs(f64(o) - w) <= rel * np.abs(w) + 2 * STEP[g.dtype]).all()
    if not inplace:
        for t, d in zip(ts, dev):   # the gradients themselves stay
            assert torch.equal(t, d.cpu())


SETS = {
    "one value": [((1,), BF16)],
    "one fp32 value": [((1,), FP32)],
    "a vector": [((7,), FP32)],
    "mixed": [((3, 5), BF16), ((129,), FP32), ((64, 1000), BF16), ((1,), BF16), ((8192,), FP32)],
    "chunks": [((8191,), BF16), ((8192,), BF16), ((8193,), BF16), ((24577,), FP32)],
    "empty ones": [((0,), BF16), ((5, 0), FP32), ((33,), BF16), ((0,), FP32)],
    "many": [((17 + 13 * (k % 7),), BF16 if k % 3 else FP32) for k in range(301)],
    "one large": [((2049, 5461), BF16), ((11,), FP32)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("max_norm", [0.25, 1e9])
@pytest.mark.parametrize("name", list(SETS))
def test_clip(name, max_norm):
    check(grads(SETS[name], 3), max_norm)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["mixed", "many", "empty ones"])
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_clip_in_place_and_by_the_largest(name, kind):
    for max_norm in (0.01, 0.3, 1e9):
        check(grads(SETS[name], 5), max_norm, kind, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e20, 1e30, 1e37])
def test_clip_of_gradients_whose_squares_leave_fp32(scale):
    """Also where the sum of squares is beyond fp32's range; eps as large as the norm among them."""
    ts = grads(SETS["mixed"], 7, scale)
    check(ts, scale, eps=0.0)
    check(ts, scale, eps=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("scale,to", [(1e37, -3), (1e37, -10), (1e37, -30), (1e37, -60), (1e30, -40), (1e-20, -149)])
def test_clip_by_a_factor_below_fp32(scale, to, kind):
    """Norms from 2^126 times max_norm = 2^to on: the factor is subnormal in fp32 or 0, its products are not."""
    ts = grads(SETS["mixed"], 9, scale)
    for inplace in (False, True):
        check(ts, 2.0 ** to, kind, eps=0.0, inplace=inplace)


@pytest.mark.gpu
def test_views_at_any_address():
    """Tensors that begin at odd elements of a buffer, their results too; nothing beside them is written."""
    b = B()
    for dt in (BF16, FP32):
        whole = grads([((40000,), dt)], 1)[0].cuda()
        parts = [whole[1:1002], whole[1003:1004], whole[2007:2007 + 20003], whole[30001:]]
        into = torch.full((40000,), 5.0, dtype=dt, device="cuda")
        outs = [into[3:1004], into[1111:1112], into[2001:2001 + 20003], into[30001:]]
        norm = b.clip_gradients(parts, 1.0, out=outs)
        want, ref = O.clip([f64(p) for p in parts], 1.0, float(np.float32(1e-6)))
        assert abs(float(norm) - want) <= want * 2.0 ** -23.9
        for o, r in zip(outs, ref):
            assert (np.abs(f64(o) - r) <= (2.0 ** -22.9 + (2.0 ** -8 if dt == BF16 else 0)) * np.abs(r)).all()
        for gap in (into[:3], into[1004:1111], into[1112:2001], into[22004:30001]):
            assert (gap == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_zeros_nan_and_infinity(kind):
    b = B()
    zeros = [torch.zeros(100, device="cuda"), torch.zeros(7, dtype=BF16, device="cuda")]
    for max_norm in (0.0, 1.0):
        assert float(b.clip_gradients(zeros, max_norm, kind=kind, eps=0.0)) == 0
        assert all((z == 0).all() for z in zeros)
    for bad, at in ((float("nan"), 0), (float("inf"), 9999), (-float("inf"), 5)):
        ts = [t.cuda() for t in grads([((10000,), BF16), ((300,), FP32)], 2)]
        ts[0][at] = bad
        keep = [torch.empty_like(t) for t in ts]
        norm = float(b.clip_gradients(ts, 1.0, out=keep, kind=kind))
        if bad != bad:
            assert norm != norm and all(torch.isnan(t).all() for t in keep)
        else:
            assert norm == float("inf")
            assert torch.isnan(keep[0][at]) and (keep[1] == 0).all()
            rest = torch.ones_like(keep[0], dtype=torch.bool)
            rest[at] = False
            assert (keep[0][rest] == 0).all()
        b.clip_gradients(ts, 1.0, out=keep, kind=kind, nonfinite="zero")
        assert all((t == 0).all() for t in keep)
    # a norm that is finite is clipped the same with either setting
    ts = [t.cuda() for t in grads(SETS["mixed"], 2)]
    one, two = [torch.empty_like(t) for t in ts], [torch.empty_like(t) for t in ts]
    b.clip_gradients(ts, 1.0, out=one, kind=kind)
    b.clip_gradients(ts, 1.0, out=two, kind=kind, nonfinite="zero")
    assert all(torch.equal(p, q) for p, q in zip(one, two))


@pytest.mark.gpu
def test_shares_of_several_processes():
    """The totals of two shares, joined, clip each share as one set of both would."""
    b = B()
    ts = [t.cuda() for t in grads(SETS["many"], 11)]
    all_out = [torch.empty_like(t) for t in ts]
    whole = b.GradSet(ts, out=all_out)
    want = whole.clip(0.5)
    for kind, joined in (("l2", torch.add), ("max", torch.maximum)):
        outs = [torch.empty_like(t) for t in ts]
        halves = [b.GradSet(ts[:120], outs[:120], kind), b.GradSet(ts[120:], outs[120:], kind)]
        totals = [torch.zeros(1, dtype=torch.float64, device="cuda") for _ in halves]
        for h, t in zip(halves, totals):
            h.norm(total=t)
        total = joined(*totals)
        norms = [float(h.clip(0.5, total=total)) for h in halves]
        assert norms[0] == norms[1]
        if kind == "l2":
            assert abs(norms[0] - float(want)) <= 2.0 ** -23 * float(want)
            for p, q in zip(outs, all_out):
                assert (np.abs(f64(p) - f64(q)) <= 2.0 ** -7 * np.abs(f64(q))).all()
        else:
            assert norms[0] == max(float(t.abs().max()) for t in ts)


@pytest.mark.gpu
def test_the_same_tensor_twice_counts_twice():
    b = B()
    t = grads([((1000,), FP32)], 4)[0].cuda()
    outs = [torch.empty_like(t), torch.empty_like(t)]
    norm = float(b.clip_gradients([t, t], 1.0, out=outs))
    assert abs(norm - np.sqrt(2 * (f64(t) ** 2).sum())) <= norm * 2.0 ** -23
    assert torch.equal(*outs)


@pytest.mark.gpu
def test_clip_captured_and_replayed_between_eager_calls():
    b = B()
    ts = [t.cuda() for t in grads(SETS["many"], 1)]
    other = [t.cuda() for t in grads(SETS["mixed"], 1)]
    outs, twin = [torch.empty_like(t) for t in ts], [torch.empty_like(t) for t in ts]
    one, two, third = b.GradSet(ts, outs), b.GradSet(ts, twin), b.GradSet(other)
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one.clip(0.5, norm=norm)
    side = torch.cuda.Stream()
    for k in range(5):
        for t, n in zip(ts, grads(SETS["many"], 40 + k, 10.0 ** (k - 3))):
            t.copy_(n)
        graph.replay()
        third.clip(1.0)
        side.wait_stream(torch.cuda.current_stream())
        want = two.clip(0.5, stream=side)
        torch.cuda.synchronize()
        assert float(want) == float(norm)
        assert all(torch.equal(p, q) for p, q in zip(outs, twin))


@pytest.mark.gpu
def test_equal_calls_give_equal_bits():
    b = B()
    ts = [t.cuda() for t in grads(SETS["one large"], 1)]
    outs = [torch.empty_like(t) for t in ts]
    first = float(b.clip_gradients(ts, 1.0, out=outs))
    keep = [o.clone() for o in outs]
    for _ in range(5):
        assert float(b.clip_gradients(ts, 1.0, out=outs)) == first
        assert all(torch.equal(p, q) for p, q in zip(outs, keep))


# ---------------------------------------------------------------------- on the CPU ---
FAKE, FAR = 0x10000, 1 << 30


def call(fn, desc=None, arr=None, count=None, **kw):
    b = B()
    d = b.ClipDesc(0, 0, 1.0, 1e-6, FAKE + 8 * FAR, 1 << 20, None)
    for k, v in (desc or {}).items():
        setattr(d, k, v)
    if arr is None:
        arr = [(FAKE, FAKE + FAR, 100, 0), (FAKE + 2 * FAR, FAKE + 2 * FAR, 64, 1)]
    a = (b.Grad * len(arr))(*(b.Grad(*t) for t in arr))
    count = len(arr) if count is None else count
    if fn == "norm":
        return b.lib().qgalore_grad_norm(ctypes.byref(d), a, count, kw.get("norm", FAKE + 4 * FAR),
                                         kw.get("total", FAKE + 5 * FAR))
    return b.lib().qgalore_grad_clip(ctypes.byref(d), a, count, kw.get("total"),
                                     kw.get("norm", FAKE + 4 * FAR))


def test_clip_refusals_come_before_any_device_call():
    L = B().lib()
    assert L.qgalore_grad_norm(None, None, 1, FAKE, FAKE) == 1
    for fn in ("norm", "clip"):
        assert call(fn, arr=[(None, FAKE, 4, 0)]) == 1
        assert call(fn, dict(workspace=None)) == 1
        assert call(fn, arr=[(FAKE, FAKE, -1, 0)]) == 2
        assert call(fn, arr=[(FAKE, FAKE, (1 << 40) + 1, 0)]) == 2
        assert call(fn, arr=[(FAKE + 1, FAKE + 1, 4, 0)]) == 3
        assert call(fn, arr=[(FAKE + 2, FAKE + 2, 4, 1)]) == 3
        assert call(fn, dict(workspace=FAKE + 4)) == 3
        assert call(fn, dict(workspace_bytes=100)) == 4
        assert call(fn, count=0) == 5 and call(fn, count=65537) == 5 and call(fn, count=-1) == 5
        assert call(fn, dict(kind=2)) == 5 and call(fn, dict(zero_nonfinite=2)) == 5
        assert call(fn, arr=[(FAKE, FAKE, 4, 2)]) == 5
        assert call(fn, norm=FAKE + 2) == 3 and call(fn, total=FAKE + 4) == 3
    assert call("norm", norm=None, total=None) == 1
    assert call("clip", arr=[(FAKE, None, 4, 0)]) == 1
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")),
                dict(eps=-1.0), dict(eps=float("nan"))):
        assert call("clip", bad) == 5, bad
    assert L.qgalore_grad_workspace_bytes() >= 8 * 1024


def test_clip_results_over_other_memory_are_refused():
    g, o = FAKE, FAKE + FAR
    same = [(g, g, 100, 0), (g, g, 100, 0)]                     # scaled twice
    part = [(g, o, 100, 0), (g + 4096, o + 198, 100, 0)]        # two results share two bytes
    shift = [(g, g + 2, 100, 0)]                                # over its own gradient, moved
    cross = [(g, o, 100, 0), (o + 100, o + FAR, 100, 0)]        # over another's gradient
    for arr in (same, part, shift, cross):
        assert call("clip", arr=arr) == 5, arr
    ok = [(g, o, 100, 0), (g, o + 4096, 100, 0)]
    assert call("clip", arr=ok, norm=o + 10 * 4) == 5           # the norm over a result
    assert call("clip", arr=ok, norm=g + 20) == 5               # or over a gradient
    assert call("clip", arr=ok, total=o + 16) == 5              # the total under a result
    assert call("clip", dict(workspace=o + 64), arr=ok) == 5
    assert call("norm", dict(workspace=g + 64), arr=ok) == 5
    assert call("norm", arr=ok, norm=g + 20) == 5 and call("norm", arr=ok, total=g + 24) == 5
    assert call("norm", arr=ok, norm=FAKE + 4 * FAR, total=FAKE + 4 * FAR) == 5
    if not torch.cuda.is_available():   # accepted: the next thing it needs is a device
        assert call("clip", arr=ok) == 7 and call("norm", arr=ok) == 7 and call("norm", arr=same) == 7
        assert call("clip", arr=[(g, g, 100, 0), (g + 200, g + 200, 1, 0), (None, None, 0, 1)]) == 7


def test_binding_refuses_other_sets():
    b = B()
    for bad in ([], [torch.zeros(2)]):
        with pytest.raises(ValueError):
            b.GradSet(bad)


def test_clip_struct_layouts_match_the_header(tmp_path):
    from tests.test_gpu_resnorm import layouts
    b = B()
    layouts(tmp_path, {"qg_grad": b.Grad, "qg_clip_desc": b.ClipDesc})
