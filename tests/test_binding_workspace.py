"""Workspaces that the binding allocates for a call, on the CPU: the library is stood in for by functions
that look at what the call holds while it runs."""
import contextlib
import weakref

import pytest

torch = pytest.importorskip("torch")


def B():
    from quantized_rank_gradient_amd import binding
    return binding


class Library:
    """Entry points that note whether the workspace in the descriptor is alive; size queries go to the
    library itself."""

    def __init__(self, real, allocated):
        self.real, self.allocated, self.calls = real, allocated, []

    def __getattr__(self, name):
        real = getattr(self.real, name)
        if name.endswith("_bytes"):
            return real

        def call(desc, *args):
            desc = desc._obj
            alive = [r() for r in self.allocated if r() is not None]
            self.calls.append((name, desc.workspace in [t.data_ptr() for t in alive]))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    b = B()
    allocated = []

    def alloc(nbytes, device="cuda"):
        t = torch.empty(max(int(nbytes), 16), dtype=torch.uint8)
        allocated.append(weakref.ref(t))
        return t

    def ptr(t, dtype, shape=None, name="tensor"):
        return None if t is None else t.data_ptr()
    stand_in = Library(b.lib(), allocated)
    monkeypatch.setattr(b, "alloc_workspace", alloc)
    monkeypatch.setattr(b, "_ptr", ptr)
    monkeypatch.setattr(b, "_arg", ptr)
    monkeypatch.setattr(b, "_on", lambda tensors, stream: contextlib.nullcontext(0))
    monkeypatch.setattr(b, "lib", lambda: stand_in)
    return stand_in


def test_a_workspace_lives_until_the_call_has_enqueued_its_kernels(library):
    """Freed earlier, its memory may go to another thread's tensor on the same stream while this call's
    kernels are still to be launched."""
    b = B()
    T, m, n = 512, 64, 64
    X, dY = torch.zeros(T, n, dtype=torch.bfloat16), torch.zeros(T, m, dtype=torch.bfloat16)
    Wq, Ws = torch.zeros(m, n, dtype=torch.int8), torch.ones(b.n_groups(m * n))
    gamma, stat = torch.ones(n), torch.ones(T)
    # a shape whose forward product writes the dequantized weight to the workspace
    Xt, Wt = torch.zeros(T, 40, dtype=torch.bfloat16), torch.zeros(m, 40, dtype=torch.int8)
    b.int8_linear_act_fwd(Xt, Wt, torch.ones(b.n_groups(m * 40)))
    b.int8_linear_act_bwd(dY, X, Wq, Ws)
    b.norm_bwd(X, X, gamma, stat, stat)
    b.muon_step(b.MuonLayer(0, torch.zeros(m, n, dtype=torch.bfloat16), Wq, Ws, torch.zeros(m, n)), 1, 1)
    b.orthogonalize([torch.zeros(m, n, dtype=torch.bfloat16)])
    assert library.calls == [(name, True) for name in (
        "qgalore_int8_linear_act_fwd", "qgalore_int8_linear_act_bwd", "qgalore_norm_bwd",
        "qgalore_muon_step", "qgalore_orthogonalize")]
    assert all(r() is None for r in library.allocated)   # and no longer


def test_a_workspace_of_the_caller_is_passed_on(library):
    b = B()
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    library.allocated.append(weakref.ref(ws))
    X = torch.zeros(16, 64, dtype=torch.bfloat16)
    b.norm_bwd(X, X, torch.ones(64), torch.ones(16), torch.ones(16), workspace=ws)
    assert library.calls == [("qgalore_norm_bwd", True)] and len(library.allocated) == 1
