"""The training calls together, and the ways a training program calls them.

A whole step of out = x + moe(layernorm(x)) against a 64-bit formula of it, by
its gradients and by differences along directions; captured into a graph;
two steps at once on two streams; and calls that are refused or contain
numbers that name no row.
"""
import time

import pytest
import torch

from moe_layer_gemm_b200 import abi

pytestmark = pytest.mark.gpu

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
EPS, AUX, ZC = 1e-5, 0.05, 0.02
# Relative 2-norm of a gradient's error: a chain of at most ten roundings to
# bf16 (norm, H, Y's operand, dY, dG and dU, dX, dL, each output), each at most
# half a step (2^-8) of its value.
TOL = 10 * 2.0 ** -8


class Step:
    """Buffers and calls of one training step."""

    def __init__(self, T, d, f, E, K, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s, std=1.0, dtype=BF16: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.dims = abi.Dims(T, d, f, E, K)
        A = T * K
        self.x, self.dout = rnd(T, d), rnd(T, d, std=0.1)
        self.gamma, self.beta = 1 + rnd(d, std=0.1, dtype=F32), rnd(d, std=0.1, dtype=F32)
        self.Wr = rnd(d, E, std=d ** -0.5)
        self.W1, self.W3, self.W2 = rnd(E, d, f, std=d ** -0.5), rnd(E, d, f, std=d ** -0.5), rnd(E, f, d, std=f ** -0.5)
        self.xn, self.mean, self.rstd = new(T, d), new(T, dtype=F32), new(T, dtype=F32)
        self.logits, self.idx, self.w, self.P = new(T, E, dtype=F32), new(T, K, dtype=I32), new(T, K, dtype=F32), new(E, dtype=F32)
        self.counts, self.kept, self.offsets = new(E, dtype=I32), new(E, dtype=I32), new(E + 1, dtype=I32)
        self.inv, self.src, self.x_perm = new(T, K, dtype=I32), new(A, dtype=I32), new(A, d)
        self.gu, self.h, self.y_perm, self.y = new(A, 2 * f), new(A, f), new(A, d, dtype=F32), new(T, d)
        self.dy_perm, self.dw, self.dgu, self.dx_perm, self.dxn = new(A, d), new(T, K, dtype=F32), new(A, 2 * f), new(A, d), new(T, d)
        self.grads = {"x": new(T, d), "gamma": new(d, dtype=F32), "beta": new(d, dtype=F32), "Wr": new(d, E, dtype=F32),
                      "W1": new(E, d, f), "W3": new(E, d, f), "W2": new(E, f, d)}
        self.ws, self.tws = abi.alloc_workspace(self.dims), abi.alloc_train_workspace(self.dims)

    def run(self):
        s, D, G = self, self.dims, self.grads
        abi.moe_layernorm(s.x, s.gamma, s.beta, EPS, s.xn, s.mean, s.rstd)
        abi.moe_route(D, s.xn, s.Wr, None, s.logits, s.idx, s.w, s.P, s.ws)
        abi.moe_permute(D, s.idx, s.xn, s.counts, s.kept, s.offsets, s.inv, s.src, s.x_perm, None, s.ws)
        abi.moe_ffn_train(D, s.x_perm, s.offsets, s.W1, s.W3, s.W2, s.gu, s.h, s.y_perm, s.tws)
        abi.moe_combine(D, s.y_perm, s.inv, s.w, s.y)
        abi.moe_combine_backward(D, s.dout, s.y_perm, s.inv, s.w, s.dy_perm, s.dw)
        abi.moe_ffn_backward(D, s.dy_perm, s.x_perm, s.offsets, s.W1, s.W3, s.W2, s.gu, s.h, s.dgu, s.dx_perm, G["W1"], G["W3"],
                             G["W2"], s.tws)
        abi.moe_route_backward(D, s.xn, s.Wr, s.logits, s.idx, s.w, s.dw, s.counts, AUX, ZC, s.dx_perm, s.inv, s.dxn, G["Wr"], None,
                               s.tws)
        abi.moe_layernorm_backward(s.dxn, s.x, s.gamma, s.mean, s.rstd, s.dout, G["x"], G["gamma"], G["beta"], s.tws)

    def params(self):
        return {k: getattr(self, k).to(F64) for k in self.grads}

    def results(self):
        n = int(self.offsets[-1])
        return [self.y, self.gu[:n], self.h[:n], self.dgu[:n], *self.grads.values()]

    def loss(self, p):
        """<out, dout> + AUX * aux + ZC * z_loss in 64 bits, with the step's expert choice."""
        D = self.dims
        xn = torch.nn.functional.layer_norm(p["x"], (D.d_model,), p["gamma"], p["beta"], EPS)
        logits = xn @ p["Wr"]
        idx = self.idx.long()
        w = torch.softmax(logits.gather(1, idx), 1)
        out = p["x"]
        for k in range(D.K):
            e = idx[:, k]
            h = torch.nn.functional.silu(torch.einsum("td,tdf->tf", xn, p["W1"][e])) * torch.einsum("td,tdf->tf", xn, p["W3"][e])
            out = out + w[:, k, None] * torch.einsum("tf,tfd->td", h, p["W2"][e])
        load = torch.bincount(idx.reshape(-1), minlength=D.E).to(F64) / (D.T * D.K)
        aux = D.E * (load * torch.softmax(logits, 1).mean(0)).sum()
        return (out * self.dout.to(F64)).sum() + AUX * aux + ZC * torch.logsumexp(logits, 1).square().mean()


@pytest.mark.parametrize("T,d,f,E,K", [(96, 256, 192, 6, 2), (1, 64, 48, 3, 2), (203, 528, 80, 12, 4)])
def test_step_against_formula_and_differences(T, d, f, E, K):
    s = Step(T, d, f, E, K, seed=T)
    s.run()
    assert abi.moe_get_device_status(s.ws) == (abi.MOE_OK, 0) and abi.moe_get_device_status(s.tws) == (abi.MOE_OK, 0)
    p = s.params()
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    s.loss(leaves).backward()
    for k, g in s.grads.items():
        g, want = g.to(F64), leaves[k].grad
        rel = float((g - want).norm() / want.norm())
        assert rel <= TOL, (k, rel)
        v = g / g.norm()  # the slope along the gradient itself is its length
        e = 1e-4 * float(p[k].norm()) / T ** 0.5
        with torch.no_grad():
            slope = float((s.loss({**p, k: p[k] + e * v}) - s.loss({**p, k: p[k] - e * v})) / (2 * e))
        assert abs(slope - float(g.norm())) <= TOL * float(g.norm()) + 1e-6, (k, slope, float(g.norm()))


def _bits(ts):
    return [t.clone().view(torch.int16 if t.dtype == BF16 else torch.int32) for t in ts]


def test_step_captured_and_replayed():
    s = Step(150, 272, 144, 5, 2, seed=3)
    s.run()
    want = _bits(s.results())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(3):
        for t in s.grads.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_bits(s.results()), want))


def test_two_steps_on_two_streams():
    steps = [Step(700, 512, 272, 8, 2, seed=k) for k in (1, 2)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(_bits(s.results()))
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        for t in s.grads.values():
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(_bits(s.results()), w))


def test_numbers_that_name_no_row():
    """Offsets, inv and topk_idx out of range are never addresses: the kept rows come out as without them."""
    T, d, f, E, K = 64, 128, 64, 4, 2
    s = Step(T, d, f, E, K, seed=9)
    s.run()
    D, A = s.dims, T * K
    off = torch.tensor([-5, 40, 30, 10 ** 9, 10 ** 9], dtype=I32, device="cuda")  # rows 0-39 to expert 0, 30-127 to expert 2
    gu, h, y = (torch.empty_like(t) for t in (s.gu, s.h, s.y_perm))
    abi.moe_ffn_train(D, s.x_perm, off, s.W1, s.W3, s.W2, gu, h, y, s.tws)
    dW = [torch.full_like(t, 7.0) for t in (s.W1, s.W3, s.W2)]
    abi.moe_ffn_backward(D, s.dy_perm, s.x_perm, off, s.W1, s.W3, s.W2, s.gu, s.h, s.dgu, s.dx_perm, *dW, s.tws)
    assert abi.moe_get_device_status(s.tws) == (abi.MOE_OK, 0)
    for t in dW:  # experts 1 (its end before its start) and 3 (behind all rows) have none
        assert (t[1] == 0).all() and (t[3] == 0).all() and (t[0] != 7).any()
    g0 = s.x_perm[:30].float() @ s.W1[0].float()
    assert (gu[:30, :f].float() - g0).abs().max() <= 2.0 ** -8 * g0.abs().max() + 1e-3
    inv = s.inv.clone()
    inv[3, 0], inv[5, 1] = 10 ** 9, -7
    dyp, dw = torch.zeros_like(s.dy_perm), torch.empty_like(s.dw)
    abi.moe_combine_backward(D, s.dout, s.y_perm, inv, s.w, dyp, dw)
    assert float(dw[3, 0]) == 0 and float(dw[5, 1]) == 0
    dx, dx2 = torch.empty(T, d, dtype=F32, device="cuda"), torch.empty(T, d, dtype=F32, device="cuda")
    abi.moe_permute_backward(D, s.dx_perm, inv, dx)
    ref = torch.where((inv >= 0) & (inv < A), inv, A).long()
    rows = torch.cat([s.dx_perm.float(), torch.zeros(1, d, device="cuda")])[ref]
    assert torch.equal(dx, rows[:, 0] + rows[:, 1])
    idx = s.idx.clone()
    idx[0, 0], idx[1, 0] = 1000, -3
    dl = torch.empty(T, E, dtype=F32, device="cuda")
    abi.moe_route_backward(D, None, s.Wr, None, idx, s.w, s.dw, None, 0.0, 0.0, s.dx_perm, inv, dx2, None, dl, s.tws)
    assert (dl[0] != 0).sum() <= 1 and (dl[1] != 0).sum() <= 1
    assert (dx2 - dx - dl.to(BF16).float() @ s.Wr.float().T).abs().max() <= 1e-5
    twice = s.idx.clone()
    twice[:, 1] = twice[:, 0]  # the same expert twice: both slots' terms
    abi.moe_route_backward(D, None, s.Wr, None, twice, s.w, s.dw, None, 0.0, 0.0, None, None, dx2, None, dl, s.tws)
    g = s.w * (s.dw - (s.w * s.dw).sum(1, keepdim=True))
    assert (dl.gather(1, twice[:, :1].long())[:, 0] - g.sum(1)).abs().max() <= 1e-6


def test_outputs_left_out():
    """Every subset of the wanted gradients comes out as with the others, and needs only its own inputs."""
    s = Step(120, 272, 144, 5, 2, seed=4)
    s.run()
    D, G, ws = s.dims, s.grads, s.tws
    n = int(s.offsets[-1])
    want = {k: G[k].clone() for k in ("W1", "W3", "W2", "gamma", "beta")}
    dgu, dx = s.dgu[:n].clone(), s.dx_perm[:n].clone()
    new = torch.empty_like
    a = new(s.dgu), new(s.dx_perm)
    abi.moe_ffn_backward(D, s.dy_perm, None, s.offsets, s.W1, s.W3, s.W2, s.gu, None, a[0], a[1], None, None, None, ws)
    assert torch.equal(a[0][:n], dgu) and torch.equal(a[1][:n], dx)
    b = new(s.dgu), new(s.W2)
    abi.moe_ffn_backward(D, s.dy_perm, None, s.offsets, None, None, s.W2, s.gu, s.h, b[0], None, None, None, b[1], ws)
    assert torch.equal(b[0][:n], dgu) and torch.equal(b[1], want["W2"])
    c = new(s.dgu), new(s.W1), new(s.W3)
    abi.moe_ffn_backward(D, s.dy_perm, s.x_perm, s.offsets, None, None, s.W2, s.gu, None, c[0], None, c[1], c[2], None, ws)
    assert torch.equal(c[1], want["W1"]) and torch.equal(c[2], want["W3"])
    db = new(s.beta)
    abi.moe_layernorm_backward(s.dxn, s.x, s.gamma, s.mean, s.rstd, s.dout, None, None, db, ws)
    assert torch.equal(db, want["beta"])
    dWr, dl = new(G["Wr"]), torch.empty(D.T, D.E, dtype=F32, device="cuda")
    abi.moe_route_backward(D, s.xn, None, s.logits, s.idx, s.w, s.dw, s.counts, AUX, ZC, None, None, None, dWr, dl, ws)
    assert torch.equal(dWr, G["Wr"])
    only = new(dl)
    abi.moe_route_backward(D, None, None, s.logits, s.idx, s.w, s.dw, s.counts, AUX, ZC, None, None, None, None, only, ws)
    assert torch.equal(only, dl)


def test_refused_tensors():
    s = Step(16, 64, 32, 4, 2, seed=1)
    D = s.dims
    with pytest.raises(ValueError, match="contiguous"):
        abi.moe_layernorm(s.x.t(), None, None, EPS, s.xn)
    with pytest.raises(TypeError):
        abi.moe_layernorm(s.x.half(), None, None, EPS, s.xn)
    with pytest.raises(TypeError):
        abi.moe_layernorm(s.x, s.gamma, s.beta.to(BF16), EPS, s.xn)
    with pytest.raises(ValueError, match="needed"):
        abi.moe_layernorm(s.x, s.gamma[:32], None, EPS, s.xn)
    with pytest.raises(ValueError, match="needed"):
        abi.moe_ffn_train(D, s.x_perm, s.offsets, s.W1, s.W3, s.W2, s.gu[:8], s.h, s.y_perm, s.tws)
    with pytest.raises(TypeError):
        abi.moe_ffn_backward(D, s.dy_perm, s.x_perm, s.offsets, s.W1, s.W3, s.W2, s.gu, s.h, s.dgu, s.dx_perm, s.grads["W1"],
                             s.grads["W3"].float(), s.grads["W2"], s.tws)
    with pytest.raises(ValueError):
        abi.moe_combine_backward(D, s.dout, s.y_perm.cpu(), s.inv, s.w, s.dy_perm, s.dw)
    with pytest.raises(abi.MoEError) as e:
        abi.moe_route_backward(D, s.xn, s.Wr, s.logits, s.idx, s.w, s.dw, s.counts, AUX, ZC, s.dx_perm, s.inv, s.dxn, s.grads["Wr"],
                               None, s.tws[:1024])
    assert e.value.status == abi.MOE_EWORKSPACE
    with pytest.raises(abi.MoEError) as e:
        abi.moe_permute_backward(abi.Dims(15, 64, 32, 4, 2), s.dx_perm.view(-1)[4:], s.inv, s.dxn)
    assert e.value.status == abi.MOE_EUNSUPPORTED  # 8 bytes off alignment


@pytest.mark.parametrize("T,d,f,E,K", [(64, 128, 256, 8, 2), (2500, 2112, 528, 3, 1)])
def test_timeouts_end_and_leave_the_context_usable(T, d, f, E, K):
    """Every epilogue waits for an event that never comes: each call returns MOE_ETIMEOUT, detail 4, after its abort and
    drain paths have run, and the same calls work afterwards."""
    s = Step(T, d, f, E, K, seed=2)
    s.run()
    want = _bits(s.results())
    torch.cuda.synchronize()
    try:
        abi.moe_test_set_wait_limits(1 << 14, 0, True)
        t0 = time.perf_counter()
        abi.moe_ffn_train(s.dims, s.x_perm, s.offsets, s.W1, s.W3, s.W2, s.gu, s.h, s.y_perm, s.tws)
        torch.cuda.synchronize()
        assert abi.moe_get_device_status(s.tws) == (abi.MOE_ETIMEOUT, 4)
        abi.moe_reset_device_status(s.tws)
        abi.moe_ffn_backward(s.dims, s.dy_perm, s.x_perm, s.offsets, s.W1, s.W3, s.W2, s.gu, s.h, s.dgu, s.dx_perm, s.grads["W1"],
                             s.grads["W3"], s.grads["W2"], s.tws)
        torch.cuda.synchronize()
        assert abi.moe_get_device_status(s.tws) == (abi.MOE_ETIMEOUT, 4)
        assert time.perf_counter() - t0 < 10.0
    finally:
        abi.moe_test_set_wait_limits(0, 0, False)
    abi.moe_reset_device_status(s.tws)
    s.run()
    assert abi.moe_get_device_status(s.tws) == (abi.MOE_OK, 0)
    assert all(torch.equal(a, b) for a, b in zip(_bits(s.results()), want))
