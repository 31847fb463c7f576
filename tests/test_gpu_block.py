"""The operators as a training program runs them: a pre-norm block on INT8 weights,
    h = norm(x),  a = gelu(h W1~^T + b1),  y = a W2~^T + b2 + x,
its backward pass from dy, and the orthogonalised update of both weights from the bf16 gradients.

Tolerances. y passes the roundings of h, a and y to bf16, the gradients up to three more (dZ, the
gradient between the layers, the result), each 2^-8 / sqrt(3) of the whole in the 2-norm; the maps
between them stretch an error by no more than they stretch the values, up to a factor of 1.5:
1.5 sqrt(6) 2^-8 / sqrt(3) = 8.3e-3."""
import math

import numpy as np
import pytest

from oracle import qgalore_oracle as O
from tests.test_gpu_muon import check_weights

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TOL = 8.3e-3
HP = dict(lr=0.02, momentum=0.9, weight_decay=0.01)


def B():
    from quantized_rank_gradient_amd import binding
    return binding


class Block:
    """Weights, their momentum, and one training step on the library's entry points."""

    def __init__(self, d, f, seed, center=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        b = B()
        self.d, self.f, self.center = d, f, center

        def weight(m, n):
            q = torch.randint(-127, 128, (m, n), generator=g, device="cuda", dtype=torch.int8)
            s = (0.5 + torch.rand(b.n_groups(m * n), generator=g, device="cuda")) / 73 / math.sqrt(n)
            return q, s
        self.W1, self.S1 = weight(f, d)
        self.W2, self.S2 = weight(d, f)
        self.b1 = 0.1 * torch.randn(f, generator=g, device="cuda")
        self.b2 = 0.1 * torch.randn(d, generator=g, device="cuda")
        self.gamma = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        self.beta = 0.1 * torch.randn(d, generator=g, device="cuda") if center else None
        self.G1 = torch.zeros(f, d, dtype=torch.bfloat16, device="cuda")
        self.G2 = torch.zeros(d, f, dtype=torch.bfloat16, device="cuda")
        self.M1, self.M2 = torch.zeros(f, d, device="cuda"), torch.zeros(d, f, device="cuda")
        self.opt = b.Muon([b.MuonLayer(0, self.G1, self.W1, self.S1, self.M1),
                           b.MuonLayer(1, self.G2, self.W2, self.S2, self.M2)], HP)

    def passes(self, x, dy):
        b = B()
        h, mean, rstd = b.norm_fwd(x, self.gamma, self.beta, center=self.center)
        a, z = b.int8_linear_act_fwd(h, self.W1, self.S1, bias=self.b1, act="gelu", keep_z=True)
        y = b.int8_linear_act_fwd(a, self.W2, self.S2, bias=self.b2, residual=x)
        da, _, db2 = b.int8_linear_act_bwd(dy, a, self.W2, self.S2, bias=True, G=self.G2)
        dh, _, db1 = b.int8_linear_act_bwd(da, h, self.W1, self.S1, Z=z, act="gelu", bias=True,
                                           G=self.G1)
        dx, dgamma, dbeta = b.norm_bwd(dh, x, self.gamma, mean, rstd, center=self.center)
        out = dict(y=y, dx=dx + dy, G1=self.G1, G2=self.G2, db1=db1, db2=db2, dgamma=dgamma)
        if self.center:
            out["dbeta"] = dbeta
        return out

    def step(self, x, dy, t, seed, workspace=None):
        out = self.passes(x, dy)
        self.opt.step(t, seed, workspace=workspace)
        return out


def reference(k, x, dy):
    """The same in float64 by torch's differentiation."""
    def dense(q, s):
        w = O.dequant_weight(q.cpu().numpy(), s.cpu().numpy(), *q.shape)
        return torch.from_numpy(w.astype(np.float64)).requires_grad_()
    W1, W2 = dense(k.W1, k.S1), dense(k.W2, k.S2)
    x64 = x.double().cpu().requires_grad_()
    b1, b2, gamma = (v.double().cpu().requires_grad_() for v in (k.b1, k.b2, k.gamma))
    beta = k.beta.double().cpu().requires_grad_() if k.center else None
    c = x64 - x64.mean(1, keepdim=True) if k.center else x64
    h = c / torch.sqrt((c * c).mean(1, keepdim=True) + float(np.float32(1e-5))) * gamma
    if k.center:
        h = h + beta
    z = h @ W1.t() + b1
    y = 0.5 * z * (1 + torch.erf(z / math.sqrt(2))) @ W2.t() + b2 + x64
    y.backward(dy.double().cpu())
    out = dict(y=y.detach(), dx=x64.grad, G1=W1.grad, G2=W2.grad, db1=b1.grad, db2=b2.grad,
               dgamma=gamma.grad)
    if k.center:
        out["dbeta"] = beta.grad
    return out


def data(T, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    return x, torch.randn(T, d, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("T,d,f,center", [(300, 256, 688, True), (33, 264, 136, False),
                                          (1, 64, 128, True), (520, 512, 1376, False)])
def test_block_gradients(T, d, f, center):
    k = Block(d, f, T + d, center)
    x, dy = data(T, d, T)
    got, want = k.passes(x, dy), reference(k, x, dy)
    for name, w in want.items():
        g = got[name].double().cpu()
        assert torch.linalg.norm(g - w) <= TOL * torch.linalg.norm(w), \
            (name, float(torch.linalg.norm(g - w) / torch.linalg.norm(w)))


def test_block_gradients_against_differences():
    """The gradients along random directions of the parameters against central differences of the
    float64 loss sum(y dy)."""
    T, d, f = 40, 64, 136
    k = Block(d, f, 3)
    x, dy = data(T, d, 5)
    got = k.passes(x, dy)
    P = {n: getattr(k, n).double().cpu() for n in ("b1", "b2", "gamma", "beta")}
    P["W1"] = torch.from_numpy(O.dequant_weight(k.W1.cpu().numpy(), k.S1.cpu().numpy(), f, d)).double()
    P["W2"] = torch.from_numpy(O.dequant_weight(k.W2.cpu().numpy(), k.S2.cpu().numpy(), d, f)).double()
    P["x"] = x.double().cpu()

    def loss(p):
        c = p["x"] - p["x"].mean(1, keepdim=True)
        h = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
        z = h @ p["W1"].t() + p["b1"]
        y = 0.5 * z * (1 + torch.erf(z / math.sqrt(2))) @ p["W2"].t() + p["b2"] + p["x"]
        return float((y * dy.double().cpu()).sum())
    name = dict(b1="db1", b2="db2", gamma="dgamma", beta="dbeta", W1="G1", W2="G2", x="dx")
    g = torch.Generator()
    g.manual_seed(1)
    eps = 1e-5
    for n, p in P.items():
        u = torch.randn(p.shape, generator=g, dtype=torch.float64)
        num = (loss({**P, n: p + eps * u}) - loss({**P, n: p - eps * u})) / (2 * eps)
        grad = got[name[n]].double().cpu()
        # along a random direction an error of TOL |grad| in the 2-norm shows as itself times a
        # standard normal number: four of them
        assert abs(num - float((grad * u).sum())) <= 4 * TOL * float(grad.norm()) + 1e-4, n


def test_block_updates_its_weights():
    """Two steps: the codes are those of the oracle's update of the gradients that the GPU formed."""
    T, d, f = 200, 256, 392
    k = Block(d, f, 11)
    lr, mu, wd = (float(np.float32(HP[n])) for n in ("lr", "momentum", "weight_decay"))
    for t in (1, 2):
        x, dy = data(T, d, 20 + t)
        before = [(w.cpu().numpy(), m.cpu().numpy()) for w, m in ((k.W1, k.M1), (k.W2, k.M2))]
        k.step(x, dy, t, 99)
        for i, (W, S, G, M) in enumerate(((k.W1, k.S1, k.G1, k.M1), (k.W2, k.S2, k.G2, k.M2))):
            bits = G.view(torch.int16).cpu().numpy().view(np.uint16)
            M1 = O.muon_momentum(before[i][1], bits, HP["momentum"])
            assert np.array_equal(M.cpu().numpy(), M1)
            X = O.orthogonalize(O.muon_direction(M1, bits, HP["momentum"], True).astype(np.float64))
            m, n = W.shape
            check_weights(W.cpu().numpy(), before[i][0], S.cpu().numpy(), X,
                          lr * math.sqrt(max(1, m / n)), lr * wd, t, 99, i)


def test_block_captured_beside_eager_steps():
    """A whole training step captured once and replayed on new inputs, with eager steps of another
    block and synchronisations between the replays: bit for bit the eager steps of its twin."""
    T, d, f = 136, 256, 392
    one, two, other = Block(d, f, 7), Block(d, f, 7), Block(d, f, 8)
    x, dy = data(T, d, 1)
    ws = B().alloc_workspace(one.opt.workspace_bytes)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = one.step(x, dy, 5, 3, workspace=ws)
    for k in range(4):
        nx, ndy = data(T, d, 30 + k)
        x.copy_(nx)
        dy.copy_(ndy)
        graph.replay()
        other.step(nx, ndy, 1, 1)
        torch.cuda.synchronize()
        want = two.step(nx, ndy, 5, 3)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (k, n)
        for n in ("W1", "W2", "M1", "M2"):
            assert torch.equal(getattr(one, n), getattr(two, n)), (k, n)
