"""Training products in tiles of two 256-column sub-tiles, many tiles to a CTA pair.

Groups are given by their sizes: ends inside a 64-row box and inside a tile,
groups without rows, of a few rows and of a whole number of tiles side by
side.  Widths leave a last tile of one sub-tile.  Bounds as in the tests of
the same calls at other sizes: half a step of the output's type and one fp32
step of the sum of magnitudes a term.
"""
import time

import pytest
import torch
from test_gpu_train import BF16, F32, F64, I32, MARK, STEP, behind_is_nan, check, gen, marked, normal, status_ok
from test_gpu_train_step import Step, _bits

from moe_layer_gemm_b200 import abi

pytestmark = pytest.mark.gpu


def groups_of(sizes, A):
    off = [0]
    for n in sizes:
        off.append(off[-1] + n)
    assert off[-1] <= A
    return torch.tensor(off, dtype=I32, device="cuda"), [slice(a, b) for a, b in zip(off, off[1:])], off[-1]


# rows, d, f, sizes of the groups, products in wide tiles
WIDE = [
    (9500, 4304, 4304, [4481, 0, 17, 4700], ("gate", "dx")),
    (7500, 4304, 4208, [2111, 1304, 64, 1600, 2001], ("gate", "dx")),
    (5000, 4304, 10256, [1111, 0, 70, 3600], ("gate", "down", "dx")),
    (3000, 4304, 10256, [70, 600, 0, 257, 1500, 500], ("gate", "down", "dx")),
    (3500, 4304, 10256, [3333], ("gate", "down", "dx")),
]


@pytest.mark.parametrize("A,d,f,sizes,wide", WIDE)
def test_forward(A, d, f, sizes, wide):
    E = len(sizes)
    g, (off, groups, n), dims = gen(A + d), groups_of(sizes, A), abi.Dims(A, d, f, E, 1)
    for p in ("gate", "down"):
        assert abi.moe_train_subtiles(dims, p) == (2 if p in wide else 1), p
    x = behind_is_nan(normal(g, (A, d)), n)
    W1, W3, W2 = normal(g, (E, d, f), d ** -0.5), normal(g, (E, d, f), d ** -0.5), normal(g, (E, f, d), f ** -0.5)
    gu, h, y = marked(A, 2 * f), marked(A, f), marked(A, d, dtype=F32)
    ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device="cuda")
    abi.moe_ffn_train(dims, x, off, W1, W3, W2, gu, h, y, ws)
    status_ok(ws)
    for e, s in enumerate(groups):
        if s.start == s.stop:
            continue
        xe, w1, w3, w2 = x[s].to(F64), W1[e].to(F64), W3[e].to(F64), W2[e].to(F64)
        G, U = xe @ w1, xe @ w3
        eg, eu = d * STEP * (xe.abs() @ w1.abs()), d * STEP * (xe.abs() @ w3.abs())
        check(gu[s, :f], G, eg, f"G of {e}")
        check(gu[s, f:], U, eu, f"U of {e}")
        sig = torch.sigmoid(G)
        # |d silu| <= 1.1; |G| < 8: 2^-20 of the value for the fast exponential and reciprocal
        assert float(G.abs().max()) < 8
        check(h[s], G * sig * U, 1.1 * U.abs() * eg + (G * sig).abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * (G * sig * U).abs(), f"H of {e}")
        hk = h[s].to(F64)
        check(y[s], hk @ w2, f * STEP * (hk.abs() @ w2.abs()), f"Y of {e}")
    assert (gu[n:] == MARK).all() and (h[n:] == MARK).all() and (y[n:] == MARK).all()


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("A,d,f,sizes,wide", WIDE)
def test_backward(A, d, f, sizes, wide, dw):
    E = len(sizes)
    g, (off, groups, n), dims = gen(A + d), groups_of(sizes, A), abi.Dims(A, d, f, E, 1)
    assert abi.moe_train_subtiles(dims, "dx") == (2 if "dx" in wide else 1)
    x, dy = behind_is_nan(normal(g, (A, d)), n), behind_is_nan(normal(g, (A, d), 0.1), n)
    gu, h = behind_is_nan(normal(g, (A, 2 * f), 1.5), n), behind_is_nan(normal(g, (A, f)), n)
    W1, W3, W2 = normal(g, (E, d, f), d ** -0.5), normal(g, (E, d, f), d ** -0.5), normal(g, (E, f, d), f ** -0.5)
    dgu, dx = marked(A, 2 * f), marked(A, d)
    dW1, dW3, dW2 = marked(E, d, f, dtype=dw), marked(E, d, f, dtype=dw), marked(E, f, d, dtype=dw)
    ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device="cuda")
    abi.moe_ffn_backward(dims, dy, x, off, W1, W3, W2, gu, h, dgu, dx, dW1, dW3, dW2, ws)
    status_ok(ws)
    for e, s in enumerate(groups):
        if s.start == s.stop:
            assert (dW1[e] == 0).all() and (dW3[e] == 0).all() and (dW2[e] == 0).all()
            continue
        m = s.stop - s.start
        xe, dye, hk, w1, w3 = (t.to(F64) for t in (x[s], dy[s], h[s], W1[e], W3[e]))
        dG, dU = dgu[s, :f].to(F64), dgu[s, f:].to(F64)
        check(dx[s], dG @ w1.T + dU @ w3.T, 2 * f * STEP * (dG.abs() @ w1.T.abs() + dU.abs() @ w3.T.abs()), f"dX of {e}")
        check(dW1[e], xe.T @ dG, m * STEP * (xe.T.abs() @ dG.abs()), f"dW1 of {e}")
        check(dW3[e], xe.T @ dU, m * STEP * (xe.T.abs() @ dU.abs()), f"dW3 of {e}")
        check(dW2[e], hk.T @ dye, m * STEP * (hk.T.abs() @ dye.abs()), f"dW2 of {e}")
    assert (dgu[n:] == MARK).all() and (dx[n:] == MARK).all()


def test_timeouts_of_wide_tiles_end_and_leave_the_context_usable():
    """As for narrow tiles: every epilogue waits for what never comes, in the middle of many tiles."""
    s = Step(3500, 4304, 10256, 2, 1, seed=6)
    assert [abi.moe_train_subtiles(s.dims, p) for p in ("gate", "down", "dx")] == [2, 2, 2]
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
