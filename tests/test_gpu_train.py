"""The training entry points against their formulas in 64 bits.

Each output is compared element by element.  Its bound counts roundings: half
a step of the output's type (bf16 2^-8, fp32 2^-24, relative), and one fp32
step (2^-23) of the sum of magnitudes for every term of an fp32 sum.  A product
of rounded intermediates (H, dG, dU, dL) is checked from the intermediates that
the kernel wrote, and those from the inputs.  Rows behind the last kept row
hold NaN on input and a mark on output: neither may be touched.
"""
import numpy as np
import pytest
import torch

from moe_layer_gemm_b200 import abi

pytestmark = pytest.mark.gpu

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
STEP = 2.0 ** -23
MARK = 77.0


def dev():
    return torch.device("cuda", 0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def marked(*shape, dtype=BF16):
    return torch.full(shape, MARK, dtype=dtype, device="cuda")


def check(got, want, slack, what):
    """|got - want| <= slack + half a step of got's type."""
    assert torch.isfinite(got).all(), what
    err = (got.to(F64) - want).abs()
    tol = slack + HALF[got.dtype] * (want.abs() + slack) + 1e-37
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.3g} of the bound"


class Rows:
    """Rows grouped by expert: distinct experts per token, given experts empty, some slots dropped."""

    def __init__(self, T, E, K, drop, seed, empty=()):
        rng = np.random.default_rng(seed)
        live = [e for e in range(E) if e not in empty]
        idx = np.stack([rng.permutation(live)[:K] for _ in range(T)])
        keep = rng.random((T, K)) >= drop
        flat = np.where(keep, idx, E).reshape(-1)
        order = np.argsort(flat, kind="stable")
        counts = np.bincount(flat, minlength=E + 1)[:E]
        self.n, self.T, self.E, self.K = int(counts.sum()), T, E, K
        inv = np.full(T * K, -1, np.int32)
        inv[order[: self.n]] = np.arange(self.n, dtype=np.int32)
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.idx = torch.from_numpy(idx.astype(np.int32)).to(dev())
        self.inv = torch.from_numpy(inv.reshape(T, K)).to(dev())
        self.offsets = torch.from_numpy(self.off).to(dev())
        self.counts = torch.from_numpy(np.bincount(idx.reshape(-1), minlength=E).astype(np.int32)).to(dev())

    def groups(self):
        return [(e, slice(int(self.off[e]), int(self.off[e + 1]))) for e in range(self.E)]


def behind_is_nan(t, n):
    t[n:] = float("nan")
    return t


def status_ok(ws):
    assert abi.moe_get_device_status(ws) == (abi.MOE_OK, 0)


# ---------------------------------------------------------------- layer norm

WIDTHS = [16, 64, 256, 272, 512, 768, 1024, 1040, 2048, 2064, 4096, 5120, 7168, 8192, 10000, 16384]


@pytest.mark.parametrize("xt,wt", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,d", [(1, 4096), (3, 16), (700, 128)] + [(37, d) for d in WIDTHS])
def test_layernorm(T, d, xt, wt):
    g = gen(T + d)
    x, dy, add = normal(g, (T, d), 1.5, xt) + 3.0, normal(g, (T, d), 0.5, xt), normal(g, (T, d), 0.5, xt)
    gamma, beta = 1 + normal(g, (d,), 0.2, wt), normal(g, (d,), 0.2, wt)
    y, dx = marked(T, d, dtype=xt), marked(T, d, dtype=xt)
    mean, rstd = marked(T, dtype=F32), marked(T, dtype=F32)
    dg, db = marked(d, dtype=wt), marked(d, dtype=wt)
    eps = 1e-5
    ws = torch.full((abi.moe_layernorm_workspace_size(T, d),), 255, dtype=torch.uint8, device=dev())
    abi.moe_layernorm(x, gamma, beta, eps, y, mean, rstd)
    abi.moe_layernorm_backward(dy, x, gamma, mean, rstd, add, dx, dg, db, ws)
    x64, dy64, w64 = x.to(F64), dy.to(F64), gamma.to(F64)
    m = x64.mean(1, keepdim=True)
    xc = x64 - m
    s = 1 / ((xc * xc).mean(1, keepdim=True) + eps).sqrt()
    xh = xc * s
    # the mean is an fp32 sum of d terms; it and x - mean carry that error into xh (times rstd), and rstd adds
    # the relative error of a sum of d squares and a square root
    em = d * STEP * x64.abs().mean(1, keepdim=True)
    check(mean[:, None], m, em, "mean")
    rel = d * STEP + 4 * STEP + 2 * em * s
    check(rstd[:, None], s, rel * s, "rstd")
    exh = em * s + (xh.abs() + STEP) * (rel + 4 * STEP)
    check(y, xh * w64 + beta.to(F64), exh * w64.abs() + 4 * STEP * (xh * w64).abs() + 2 * STEP, "y")
    q = dy64 * w64
    s1, s2 = q.mean(1, keepdim=True), (q * xh).mean(1, keepdim=True)
    e1 = (d + 2) * STEP * q.abs().mean(1, keepdim=True)
    e2 = (d + 4) * STEP * (q * xh).abs().mean(1, keepdim=True) + (q.abs() * exh).mean(1, keepdim=True)
    slack = s * (e1 + xh.abs() * e2 + exh * s2.abs() + (rel + 6 * STEP) * (q.abs() + s1.abs() + (xh * s2).abs()))
    check(dx, s * (q - s1 - xh * s2) + add.to(F64), slack + 2 * STEP * add.to(F64).abs(), "dx")
    check(dg, (dy64 * xh).sum(0), ((T + 4) * STEP * dy64 * xh).abs().sum(0) + (dy64.abs() * exh).sum(0), "dgamma")
    check(db, dy64.sum(0), (T + 2) * STEP * dy64.abs().sum(0), "dbeta")
    assert (ws[: abi.STATUS_BYTES] == 255).all()


def test_layernorm_without_weights_and_in_place():
    g = gen(5)
    T, d = 19, 1056
    x, dy = normal(g, (T, d), 2.0, F32), normal(g, (T, d), 1.0, F32)
    ref = torch.nn.functional.layer_norm(x.to(F64), (d,), eps=1e-6)
    mean, rstd = marked(T, dtype=F32), marked(T, dtype=F32)
    y = x.clone()
    abi.moe_layernorm(y, None, None, 1e-6, y, mean, rstd)
    assert (y.to(F64) - ref).abs().max() < 1e-5  # |xh| < 6, d 2^-23 = 1.3e-4 of the mean's magnitudes at the very worst
    dx = dy.clone()
    abi.moe_layernorm_backward(dx, x, None, mean, rstd, None, dx, None, None, None)
    x64 = x.to(F64).requires_grad_()
    torch.nn.functional.layer_norm(x64, (d,), eps=1e-6).backward(dy.to(F64))
    assert (dx.to(F64) - x64.grad).abs().max() < 1e-5
    dg = marked(d, dtype=F32)  # the weight's gradient alone
    ws = torch.zeros(abi.moe_layernorm_workspace_size(T, d), dtype=torch.uint8, device=dev())
    abi.moe_layernorm_backward(dy, x, None, mean, rstd, None, None, dg, None, ws)
    assert (dg.to(F64) - (dy.to(F64) * ref).sum(0)).abs().max() < 1e-4


def test_layernorm_of_constant_and_large_rows():
    """No variance: eps alone scales; a mean of 1e4 with deviations of 1 loses nothing to cancelled squares."""
    T, d = 4, 4096
    x = torch.full((T, d), 3.0, device=dev())
    x[2:] = 1e4 + torch.randn((2, d), generator=gen(1), device="cuda")
    y, mean, rstd = marked(T, d, dtype=F32), marked(T, dtype=F32), marked(T, dtype=F32)
    abi.moe_layernorm(x, None, None, 1e-5, y, mean, rstd)
    assert (y[:2] == 0).all() and (rstd[:2] - 1e-5 ** -0.5).abs().max() < 1e-4 * 316
    ref = torch.nn.functional.layer_norm(x.to(F64), (d,))
    # the mean of values of 1e4 is known to about 2^-24 * 1e4 per pairwise level of the sum (13 levels)
    assert (y[2:].to(F64) - ref[2:]).abs().max() < 13 * 2.0 ** -24 * 1e4 * 2


# ---------------------------------------------------------------- the experts

FFN = [  # T, d, f, E, K, drop, empty experts
    (1, 16, 16, 1, 1, 0.0, ()),
    (1, 128, 64, 8, 2, 0.0, ()),
    (5, 48, 80, 3, 2, 0.0, (1,)),
    (64, 128, 256, 8, 2, 0.0, ()),
    (300, 272, 336, 7, 3, 0.2, (0, 6)),
    (600, 64, 1040, 4, 1, 0.0, (3,)),
    (1000, 512, 144, 16, 4, 0.3, ()),
    (777, 1024, 528, 60, 4, 0.25, (5, 6, 59)),
    (2100, 320, 256, 1, 1, 0.0, ()),
    (500, 64, 64, 256, 8, 0.0, ()),
    # reductions long enough for tiles of two sub-tiles: the gate product's, the saved projections' gradient's, the weights'
    (40, 4112, 400, 2, 1, 0.0, ()),
    (30, 8208, 528, 1, 1, 0.0, ()),
    (4300, 320, 784, 2, 1, 0.0, ()),
    (4200, 800, 80, 2, 2, 0.3, ()),
]


@pytest.mark.parametrize("T,d,f,E,K,drop,empty", FFN)
def test_experts_forward(T, d, f, E, K, drop, empty):
    g, r = gen(T + d + f), Rows(T, E, K, drop, seed=T, empty=empty)
    n, A, dims = r.n, T * K, abi.Dims(T, d, f, E, K)
    x = behind_is_nan(normal(g, (A, d)), n)
    W1, W3, W2 = normal(g, (E, d, f), d ** -0.5), normal(g, (E, d, f), d ** -0.5), normal(g, (E, f, d), f ** -0.5)
    gu, h, y = marked(A, 2 * f), marked(A, f), marked(A, d, dtype=F32)
    ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device=dev())
    abi.moe_ffn_train(dims, x, r.offsets, W1, W3, W2, gu, h, y, ws)
    status_ok(ws)
    for e, s in r.groups():
        if s.start == s.stop:
            continue
        xe, w1, w3, w2 = x[s].to(F64), W1[e].to(F64), W3[e].to(F64), W2[e].to(F64)
        G, U = xe @ w1, xe @ w3
        eg, eu = d * STEP * (xe.abs() @ w1.abs()), d * STEP * (xe.abs() @ w3.abs())
        check(gu[s, :f], G, eg, f"G of {e}")
        check(gu[s, f:], U, eu, f"U of {e}")
        sig = torch.sigmoid(G)
        # |d silu| <= 1.1; the fast exponential and division: 2^-20 of the value
        check(h[s], G * sig * U, 1.1 * U.abs() * eg + (G * sig).abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * (G * sig * U).abs(), f"H of {e}")
        hk = h[s].to(F64)
        check(y[s], hk @ w2, f * STEP * (hk.abs() @ w2.abs()), f"Y of {e}")
    assert (gu[n:] == MARK).all() and (h[n:] == MARK).all() and (y[n:] == MARK).all()


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("T,d,f,E,K,drop,empty", FFN)
def test_experts_backward(T, d, f, E, K, drop, empty, dw):
    g, r = gen(T + d + f), Rows(T, E, K, drop, seed=T, empty=empty)
    n, A, dims = r.n, T * K, abi.Dims(T, d, f, E, K)
    x, dy = behind_is_nan(normal(g, (A, d)), n), behind_is_nan(normal(g, (A, d), 0.1), n)
    gu, h = behind_is_nan(normal(g, (A, 2 * f), 1.5), n), behind_is_nan(normal(g, (A, f)), n)
    W1, W3, W2 = normal(g, (E, d, f), d ** -0.5), normal(g, (E, d, f), d ** -0.5), normal(g, (E, f, d), f ** -0.5)
    dgu, dx = marked(A, 2 * f), marked(A, d)
    dW1, dW3, dW2 = marked(E, d, f, dtype=dw), marked(E, d, f, dtype=dw), marked(E, f, d, dtype=dw)
    ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device=dev())
    abi.moe_ffn_backward(dims, dy, x, r.offsets, W1, W3, W2, gu, h, dgu, dx, dW1, dW3, dW2, ws)
    status_ok(ws)
    for e, s in r.groups():
        if s.start == s.stop:
            assert (dW1[e] == 0).all() and (dW3[e] == 0).all() and (dW2[e] == 0).all()
            continue
        m = s.stop - s.start
        xe, dye, hk, w1, w3, w2 = (t.to(F64) for t in (x[s], dy[s], h[s], W1[e], W3[e], W2[e]))
        G, U = gu[s, :f].to(F64), gu[s, f:].to(F64)
        dH, eh = dye @ w2.T, d * STEP * (dye.abs() @ w2.T.abs())
        sig = torch.sigmoid(G)
        ds = sig * (1 + G * (1 - sig))
        # 1 + G (1 - s) cancels where it is near 0: its terms' magnitudes times the fast division's 2^-20
        eds = 2.0 ** -20 * sig * (1 + 2 * G.abs())
        check(dgu[s, :f], dH * U * ds, U.abs() * (eh * ds.abs() + (dH.abs() + eh) * eds), f"dG of {e}")
        check(dgu[s, f:], dH * G * sig, (G * sig).abs() * (eh + 2.0 ** -20 * (dH.abs() + eh)), f"dU of {e}")
        dG, dU = dgu[s, :f].to(F64), dgu[s, f:].to(F64)
        check(dx[s], dG @ w1.T + dU @ w3.T, 2 * f * STEP * (dG.abs() @ w1.T.abs() + dU.abs() @ w3.T.abs()), f"dX of {e}")
        check(dW1[e], xe.T @ dG, m * STEP * (xe.T.abs() @ dG.abs()), f"dW1 of {e}")
        check(dW3[e], xe.T @ dU, m * STEP * (xe.T.abs() @ dU.abs()), f"dW3 of {e}")
        check(dW2[e], hk.T @ dye, m * STEP * (hk.T.abs() @ dye.abs()), f"dW2 of {e}")
    assert (dgu[n:] == MARK).all() and (dx[n:] == MARK).all()


# ---------------------------------------------------------------- around the experts

@pytest.mark.parametrize("dyt", [BF16, F32])
@pytest.mark.parametrize("T,d,E,K,drop", [(1, 16, 1, 1, 0.0), (1, 4096, 8, 2, 0.0), (300, 272, 16, 16, 0.3), (513, 2048, 60, 4, 0.25),
                                          (64, 7168, 8, 3, 1.0)])
def test_combine_and_permute_backward(T, d, E, K, drop, dyt):
    g, r = gen(T + d), Rows(T, E, K, drop, seed=d)
    n, A, dims = r.n, T * K, abi.Dims(T, d, 16, E, K)
    dy, y = normal(g, (T, d), 1.0, dyt), behind_is_nan(normal(g, (A, d), 1.0, F32), n)
    w = torch.rand((T, K), generator=g, device="cuda")
    dyp, dw = marked(A, d), marked(T, K, dtype=F32)
    abi.moe_combine_backward(dims, dy, y, r.inv, w, dyp, dw)
    inv = r.inv.long()
    want_dw, mag = torch.zeros((T, K), dtype=F64, device=dev()), torch.zeros((T, K), dtype=F64, device=dev())
    for k in range(K):
        t = (inv[:, k] >= 0).nonzero()[:, 0]
        rows = inv[t, k]
        check(dyp[rows], w[t, k, None].to(F64) * dy[t].to(F64), STEP * (w[t, k, None] * dy[t].float()).to(F64).abs(), f"dy_perm of slot {k}")
        want_dw[t, k] = (dy[t].to(F64) * y[rows].to(F64)).sum(1)
        mag[t, k] = (dy[t].to(F64) * y[rows].to(F64)).abs().sum(1)
    check(dw, want_dw, d * STEP * mag, "dtopk_w")
    assert (dw[r.inv < 0] == 0).all() and (dyp[n:] == MARK).all()
    again = marked(A, d)
    abi.moe_combine_backward(dims, dy, None, r.inv, w, again)  # frozen weights: y_perm is not needed
    assert torch.equal(again.view(torch.int16), dyp.view(torch.int16))
    rows = behind_is_nan(normal(g, (A, d)), n)
    kept, take = (r.inv >= 0).to(F64)[..., None], inv.clamp(min=0)
    parts = torch.where(kept > 0, rows[take].to(F64), 0.0) if n else torch.zeros((T, K, d), dtype=F64, device=dev())
    for t in (BF16, F32):
        dx = marked(T, d, dtype=t)
        abi.moe_permute_backward(dims, rows, r.inv, dx)
        check(dx, parts.sum(1), K * STEP * parts.abs().sum(1), "dx")


@pytest.mark.parametrize("T,d,E,K,drop", [(1, 16, 1, 1, 0.0), (1, 4096, 8, 2, 0.0), (33, 272, 3, 2, 0.0), (700, 512, 17, 4, 0.25),
                                          (1500, 1040, 60, 4, 0.25), (513, 2048, 256, 8, 0.0), (3000, 128, 8, 2, 0.0)])
def test_route_backward(T, d, E, K, drop):
    g, r = gen(T + d + E), Rows(T, E, K, drop, seed=E)
    n, A, dims = r.n, T * K, abi.Dims(T, d, 16, E, K)
    x, Wr, logits = normal(g, (T, d)), normal(g, (d, E), d ** -0.5), normal(g, (T, E), 2.0, F32)
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    dw, rows = normal(g, (T, K), 0.1, F32), behind_is_nan(normal(g, (A, d), 0.1), n)
    aux, zc = 0.3, 0.05
    ws = torch.zeros(abi.moe_route_backward_workspace_size(dims), dtype=torch.uint8, device=dev())
    l64 = logits.to(F64)
    p, lse = torch.softmax(l64, 1), torch.logsumexp(l64, 1, keepdim=True)
    fe = r.counts.to(F64) / (T * K)
    bal = aux * E / T * p * (fe - (p * fe).sum(1, keepdim=True))
    zt = zc * 2 / T * lse * p
    w64, d64 = w.to(F64), dw.to(F64)
    top = torch.zeros_like(p).scatter_add(1, r.idx.long(), w64 * (d64 - (w64 * d64).sum(1, keepdim=True)))
    top_mag = torch.zeros_like(p).scatter_add(1, r.idx.long(), w64 * (d64.abs() + (w64 * d64).abs().sum(1, keepdim=True)))
    # expf, logf, sums of E and K terms and a handful of products
    slack = (E + K + 16) * STEP * (aux * E / T * p * (fe + (p * fe).sum(1, keepdim=True)) + zc * 2 / T * (lse.abs() + l64.abs().amax(1, keepdim=True) + 1) * p + top_mag)
    kept, take = (r.inv >= 0).to(F64)[..., None], r.inv.long().clamp(min=0)
    parts = torch.where(kept > 0, rows[take].to(F64), 0.0)
    for t in (BF16, F32):
        dx, dWr, dl = marked(T, d, dtype=t), marked(d, E, dtype=t), marked(T, E, dtype=F32)
        abi.moe_route_backward(dims, x, Wr, logits, r.idx, w, dw, r.counts, aux, zc, rows, r.inv, dx, dWr, dl, ws)
        status_ok(ws)
        check(dl, bal + zt + top, slack, "dlogits")
        dl16 = dl.to(BF16).to(F64)
        x64, wr64 = x.to(F64), Wr.to(F64)
        check(dx, dl16 @ wr64.T + parts.sum(1), (E + K) * STEP * (dl16.abs() @ wr64.T.abs() + parts.abs().sum(1)), "dx")
        check(dWr, x64.T @ dl16, (T + 16) * STEP * (x64.T.abs() @ dl16.abs()), "dWr")
    # a frozen expert path, no losses: the top-K softmax alone
    dx, dl = marked(T, d, dtype=F32), marked(T, E, dtype=F32)
    abi.moe_route_backward(dims, None, Wr, None, r.idx, w, dw, None, 0.0, 0.0, None, None, dx, None, dl, ws)
    check(dl, top, slack, "dlogits of the weights alone")
    dl16 = dl.to(BF16).to(F64)
    check(dx, dl16 @ Wr.to(F64).T, E * STEP * (dl16.abs() @ Wr.to(F64).T.abs()), "dx of the weights alone")
