"""A training step as a program on these operators runs it: a block of two FP8 layers between the norms, its
backward pass, the gradients clipped by their joint norm, and the INT8 weights' updates.

    y0 = norm(x),  a = y0 W1^T,  u = a W2^T,  h = x + rho sigmoid(z) norm(u),  y = norm(h)

with loss sum(h dh + y dy), the weights in INT8 and their FP8 blocks made from them in every step.

Tolerances. The reference differentiates the same block in float64. An FP8 layer's gradients are by definition
those of its quantized operands, and a rounding to bf16 in front of a quantization may move a code by a whole
step; so the reference quantizes the very bf16 tensors that the block's layers were given (y0, a, and the
gradients behind them), and each of these is compared with the reference's own value at its place. What is left
between two such places are at most six roundings to bf16, 2^-8 / sqrt(3) of the whole in the 2-norm each,
stretched by no more than 1.5 through the maps between them (the products themselves are 1e-4 off):
1.5 sqrt(6) 2^-8 / sqrt(3) = 8.3e-3."""
import math

import numpy as np
import pytest

from oracle import qgalore_oracle as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TOL = 8.3e-3


def B():
    from quantized_rank_gradient_amd import binding
    return binding


class Step:
    def __init__(self, d, f, seed, optimizer="muon"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        b = B()

        def weight(m, n):
            q = torch.randint(-127, 128, (m, n), generator=g, device="cuda", dtype=torch.int8)
            s = (0.5 + torch.rand(b.n_groups(m * n), generator=g, device="cuda")) / 73 / math.sqrt(n)
            return q, s

        def vec(mean):
            return mean + 0.1 * torch.randn(d, generator=g, device="cuda")
        self.W = [weight(f, d), weight(d, f)]
        self.g0, self.g1, self.g2, self.rho = vec(1), vec(1), vec(1), vec(0.5)
        self.G = [torch.zeros(f, d, dtype=torch.bfloat16, device="cuda"),
                  torch.zeros(d, f, dtype=torch.bfloat16, device="cuda")]
        self.vecs = [torch.zeros(d, device="cuda") for _ in range(4)]   # of g0, g1, g2 and rho
        self.clip = b.GradSet(self.G + self.vecs)
        self.M = [torch.zeros(f, d, device="cuda"), torch.zeros(d, f, device="cuda")]
        self.opt = b.Muon([b.MuonLayer(k, self.G[k], *self.W[k], self.M[k]) for k in (0, 1)],
                          dict(lr=0.02, momentum=0.9))
        self.work = b.alloc_workspace(self.opt.workspace_bytes)

    def passes(self, x, z, dh, dy, per):
        b = B()
        q1, s1, q1t, s1t = b.fp8_quantize(self.W[0][0], scales=self.W[0][1], block=True, columns=True)
        q2, s2, q2t, s2t = b.fp8_quantize(self.W[1][0], scales=self.W[1][1], block=True, columns=True)
        y0, _, rstd = b.norm_fwd(x, self.g0, center=False)
        a = b.fp8_linear_fwd(y0, q1, s1)
        u = b.fp8_linear_fwd(a, q2, s2)
        kw = dict(post=(self.g1, None), pre=(self.g2, None), gate=z, gate_act="sigmoid", per=per,
                  rho=self.rho)
        h, y, stats = b.residual_norm_fwd(u, x, **kw)
        r = b.residual_norm_bwd(dh, dy, u, h, stats, **kw)
        at, sa = b.fp8_quantize(a, rows=False, columns=True)
        da, _ = b.fp8_linear_bwd(r.dU, q2t, s2t, at, sa, G=self.G[1])
        yt, sy = b.fp8_quantize(y0, rows=False, columns=True)
        dy0, _ = b.fp8_linear_bwd(da, q1t, s1t, yt, sy, G=self.G[0])
        dx, dg0, _ = b.norm_bwd(dy0, x, self.g0, None, rstd, center=False)
        for to, v in zip(self.vecs, (dg0, r.dpost[0], r.dpre[0], r.drho)):
            to.copy_(v)
        return dict(h=h, y=y, dx=dx + r.dX, dz=r.dgate, G1=self.G[0], G2=self.G[1], dg0=self.vecs[0],
                    dg1=self.vecs[1], dg2=self.vecs[2], drho=self.vecs[3], y0=y0, a=a, u=u, du=r.dU,
                    da=da, dy0=dy0)

    def step(self, x, z, dh, dy, per, t, max_norm, norm):
        out = self.passes(x, z, dh, dy, per)
        self.clip.clip(max_norm, norm=norm)
        self.opt.step(t, 77, workspace=self.work)
        return out


def data(T, d, per, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(k, d, generator=g, device="cuda").bfloat16() for k in (T, -(-T // per), T, T)]


def quantize64(v, fmt="e4m3", block=False):
    v32 = v.detach().float().numpy()
    q, s = O.fp8_quantize(v32, fmt, block)
    return torch.from_numpy(q * O.fp8_spread(s, *v32.shape))


class Fp8Product(torch.autograd.Function):
    """x w^T with the operands of each of its three products quantized as the layer does, from the tensors
    xg and dyg that it was given."""
    @staticmethod
    def forward(ctx, x, w, xg, dyg):
        ctx.xg, ctx.dyg = xg.double().cpu(), dyg.double().cpu()
        ctx.save_for_backward(w)
        return quantize64(ctx.xg) @ quantize64(w, block=True).t()

    @staticmethod
    def backward(ctx, dy):
        w, = ctx.saved_tensors
        return (quantize64(ctx.dyg, "e5m2") @ quantize64(w, block=True),
                quantize64(ctx.dyg.t(), "e5m2") @ quantize64(ctx.xg.t()).t(), None, None)


def reference(k, x, z, dh, dy, per, got):
    leaf = {n: v.double().cpu().requires_grad_() for n, v in
            dict(x=x, z=z, g0=k.g0, g1=k.g1, g2=k.g2, rho=k.rho).items()}
    for i, (q, s) in enumerate(k.W):
        w = q.float() * s.repeat_interleave(256)[:q.numel()].view(q.shape)
        leaf[f"W{i + 1}"] = w.double().cpu().requires_grad_()

    def norm(v, gamma):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + float(np.float32(1e-5))) * gamma
    y0 = norm(leaf["x"], leaf["g0"])
    a = Fp8Product.apply(y0, leaf["W1"], got["y0"], got["da"])
    u = Fp8Product.apply(a, leaf["W2"], got["a"], got["du"])
    for v in (y0, a, u):
        v.retain_grad()
    gate = torch.sigmoid(leaf["z"]).repeat_interleave(per, 0)[:len(x)]
    h = leaf["x"] + leaf["rho"] * gate * norm(u, leaf["g1"])
    y = norm(h, leaf["g2"])
    ((h * dh.double().cpu()).sum() + (y * dy.double().cpu()).sum()).backward()
    out = dict(h=h, y=y, y0=y0, a=a, u=u, G1=leaf["W1"].grad, G2=leaf["W2"].grad, du=u.grad, da=a.grad,
               dy0=y0.grad)
    out.update({"d" + n: leaf[n].grad for n in ("x", "z", "g0", "g1", "g2", "rho")})
    return {n: v.detach() for n, v in out.items()}


@pytest.mark.parametrize("T,d,f,per", [(300, 256, 688, 1), (33, 264, 136, 11), (1, 64, 128, 1),
                                       (520, 512, 1376, 130)])
def test_block_gradients(T, d, f, per):
    k = Step(d, f, T)
    args = data(T, d, per, T + 1)
    got = k.passes(*args, per)
    want = reference(k, *args, per, got)
    for name, w in want.items():
        g = got[name].double().cpu()
        err = float(torch.linalg.norm(g - w) / torch.linalg.norm(w))
        assert err <= TOL, (name, err)


def test_the_step_clips_all_gradients_by_one_norm_and_updates_the_weights():
    T, d, f = 200, 256, 392
    k, twin = Step(d, f, 3), Step(d, f, 3)
    args = data(T, d, 1, 9)
    norm = torch.empty(1, device="cuda")
    twin.passes(*args, 1)
    whole = [g.double() for g in twin.G + twin.vecs]
    total = math.sqrt(sum(float((g * g).sum()) for g in whole))
    before = [w[0].clone() for w in k.W]
    k.step(*args, 1, 1, 0.5 * total, norm)
    assert abs(float(norm) - total) <= 2.0 ** -23 * total
    for got, g in zip(k.G + k.vecs, whole):
        rel = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -22
        assert ((got.double() - 0.5 * g).abs() <= (rel + 2.0 ** -19) * 0.5 * g.abs() + 1e-38).all()
    assert all((w[0] != q).any() for w, q in zip(k.W, before))


def test_training_step_captured_beside_eager_steps():
    """A whole step captured once and replayed on new inputs, with eager steps of another block and
    synchronisations between the replays: bit for bit the eager steps of its twin."""
    T, d, f, per = 136, 256, 392, 34
    one, two, other = Step(d, f, 7), Step(d, f, 7), Step(d, f, 8)
    args = data(T, d, per, 1)
    norms = [torch.empty(1, device="cuda") for _ in range(3)]
    one.clip.norm()   # its workspace
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = one.step(*args, per, 5, 1.0, norms[0])
    for k in range(4):
        new = data(T, d, per, 30 + k)
        for t, v in zip(args, new):
            t.copy_(v)
        graph.replay()
        other.step(*new, per, 1, 1.0, norms[2])
        torch.cuda.synchronize()
        want = two.step(*new, per, 5, 1.0, norms[1])
        torch.cuda.synchronize()
        assert torch.equal(norms[0], norms[1])
        for n in want:
            assert torch.equal(got[n], want[n]), (k, n)
        for p, q in zip(one.W + one.M, two.W + two.M):
            p, q = (p[0], q[0]) if isinstance(p, tuple) else (p, q)
            assert torch.equal(p, q), k


def test_clipped_gradients_step_a_plan():
    """Clipping in place goes before a plan's step without a copy: the plan holds the gradient's address,
    and its weights are those of a layer that was given the scaled gradient."""
    from quantized_rank_gradient_amd import workloads as WL
    b = B()
    cfg = WL.CONFIGS["single256"]
    L = cfg.layers[0]

    def gpu(v):
        return torch.from_numpy(np.ascontiguousarray(v)).cuda()

    def state(G):
        Pq, Ps = b.quantize_proj(gpu(WL.orthonormal_f32(cfg, L, cfg.r)))
        return b.LayerTensors(L.layer_id, G, gpu(WL.weights_int8(cfg, L)), gpu(WL.weight_scales(cfg, L)),
                              Pq, Ps, *(gpu(v) for v in WL.zero_moments(cfg.r, L.n)), cfg.r)
    G = gpu(WL.gradient_f32(cfg, L, 1)).bfloat16()
    scaled = torch.empty_like(G)
    norm = float(b.clip_gradients([G], 0.01, out=[scaled]))
    c = 0.01 / (norm + 1e-6)
    assert c < 0.5 and float((scaled.double() - c * G.double()).norm()) <= 2.0 ** -8 * c * norm
    one, two = state(G), state(scaled)
    plan = b.Plan([one])
    b.clip_gradients([one.G], 0.01)
    plan.step(1, 5)
    b.step(two, 1, 5)
    assert torch.equal(one.Wq, two.Wq) and torch.equal(one.Mq, two.Mq)
