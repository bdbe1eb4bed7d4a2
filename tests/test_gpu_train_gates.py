"""The experts' activation and its derivative at gate values far from zero.

The logistic function is 1 / (1 + exp(-x)) from the fast exponential, whose
documented error is 2 + floor(1.173 |x|) units in the last place (2^-23 of the
value each), an addition (half a unit) and the approximate reciprocal (one
unit); below 2^-126 (x < -87.3) it is flushed to zero.  From x = 20 on,
1 + exp(-x) is 1 in 32 bits, so the function is 1 and silu's derivative is 1
within 20 exp(-20) < 2^-24.
"""
import pytest
import torch
from test_gpu_train import BF16, F32, F64, I32, STEP, check, gen, marked, normal, status_ok

from moe_layer_gemm_b200 import abi

pytestmark = pytest.mark.gpu

FLUSH = 2.0 ** -126
GATES = [-20, -40, -60, -80, -87, -87.5, -88.5, -89, -100, -1e4, -1e30, 20, 60, 90, 1e4, 1e30,
         0.0, -0.0, 1, -1, -1.28, -1.25, 5, -5, 10, -10, 15, -15, 1e-30, -1e-30, 0.01, -0.01]


def setup(T):
    gates = torch.tensor(GATES, dtype=BF16, device="cuda")
    off = torch.tensor([0, T], dtype=I32, device="cuda")
    ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device="cuda")
    G = gates.to(F64)
    e = (2 + 1.173 * G.abs() + 4) * STEP  # and two products, half a unit each, of G, s and the other factor
    return gates, off, ws, G, torch.sigmoid(G), torch.where(G >= 20, 6 * STEP, e)


def test_activation_of_large_gates():
    T, d, f = 65, 64, len(GATES)
    g = gen(1)
    gates, off, ws, G, sig, e = setup(T)
    x, W1, W3 = torch.zeros((T, d), dtype=BF16, device="cuda"), normal(g, (1, d, f)), normal(g, (1, d, f))
    x[:, 0] = 1  # G and U are row 0 of the weights, exactly
    W1[0, 0] = gates
    W2 = normal(g, (1, f, d))
    gu, h, y = marked(T, 2 * f), marked(T, f), marked(T, d, dtype=F32)
    abi.moe_ffn_train(abi.Dims(T, d, f, 1, 1), x, off, W1, W3, W2, gu, h, y, ws)
    status_ok(ws)
    U = W3[0, 0].to(F64)
    assert (gu[:, :f] == gates).all() and (gu[:, f:] == W3[0, 0]).all()
    want = G * sig * U
    check(h, want.expand(T, f), (e * want.abs() + G.abs() * U.abs() * FLUSH).expand(T, f), "H")


@pytest.mark.parametrize("T", [1, 65])
def test_derivative_of_large_gates(T):
    d, f = 64, len(GATES)
    g = gen(T)
    gates, off, ws, G, sig, e = setup(T)
    gu = normal(g, (T, 2 * f))
    gu[:, :f] = gates
    dy, W2 = normal(g, (T, d), 0.1), normal(g, (1, f, d), f ** -0.5)
    dgu = marked(T, 2 * f)
    abi.moe_ffn_backward(abi.Dims(T, d, f, 1, 1), dy, None, off, None, None, W2, gu, None, dgu, None, None, None, None, ws)
    status_ok(ws)
    U, w2 = gu[:, f:].to(F64), W2[0].to(F64)
    dH, eh = dy.to(F64) @ w2.T, d * STEP * (dy.to(F64).abs() @ w2.abs().T)
    ds = sig * (1 + G * (1 - sig))
    # s (1 + G (1 - s)): s's error in both factors where s is not 1, whose complement then costs one rounding of G
    eds = torch.where(G >= 20, 6 * STEP, e * sig * (1 + 2 * G.abs())) + FLUSH * (1 + G.abs()) * (G < -80)
    check(dgu[:, :f], dH * U * ds, U.abs() * (eh * ds.abs() + (dH.abs() + eh) * eds), "dG")
    check(dgu[:, f:], dH * G * sig, (G * sig).abs() * (eh + e * (dH.abs() + eh)) + (dH.abs() + eh) * G.abs() * FLUSH, "dU")
