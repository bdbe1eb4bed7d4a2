"""Host-side checks of the training entry points: no GPU needed, no kernel launched."""
import ctypes

import pytest
import torch

from moe_layer_gemm_b200 import abi, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


def fake(n=1):
    """A 16-byte aligned address that is never dereferenced: every call below is refused before a launch."""
    return ctypes.c_void_p(0x1000 * n)


ODD = ctypes.c_void_p(0x1008)


def test_layernorm_refusals(lib):
    p = fake()
    fwd = lambda T, d, x=p, y=p, g=p, eps=1e-5: lib.moe_layernorm(T, d, x, 1, g, None, 0, eps, y, None, None, None)  # noqa: E731
    assert fwd(0, 64) == abi.MOE_EINVAL and fwd((1 << 24) + 1, 64) == abi.MOE_EINVAL
    assert fwd(1, 8) == abi.MOE_EINVAL and fwd(1, 72) == abi.MOE_EUNSUPPORTED and fwd(1, 16400) == abi.MOE_EUNSUPPORTED
    assert fwd(1, 64, x=None) == abi.MOE_EINVAL and fwd(1, 64, y=None) == abi.MOE_EINVAL
    assert fwd(1, 64, eps=-1.0) == abi.MOE_EINVAL and fwd(1, 64, eps=float("nan")) == abi.MOE_EINVAL
    assert fwd(1, 64, x=ODD) == abi.MOE_EUNSUPPORTED and fwd(1, 64, g=ODD) == abi.MOE_EUNSUPPORTED

    def bwd(dy=p, x=p, mean=p, dx=p, dg=p, ws=p, n=1 << 30, T=4, d=64):
        return lib.moe_layernorm_backward(T, d, dy, x, 1, None, 0, mean, p, None, dx, dg, None, ws, n, None)

    assert bwd(dy=None) == abi.MOE_EINVAL and bwd(x=None) == abi.MOE_EINVAL and bwd(mean=None) == abi.MOE_EINVAL
    assert bwd(dx=None, dg=None) == abi.MOE_EINVAL and bwd(ws=None) == abi.MOE_EINVAL
    assert bwd(n=abi.moe_layernorm_workspace_size(4, 64) - 1) == abi.MOE_EWORKSPACE
    assert bwd(dx=ODD) == abi.MOE_EUNSUPPORTED and bwd(d=16400) == abi.MOE_EUNSUPPORTED
    with pytest.raises(abi.MoEError):
        abi.moe_layernorm_workspace_size(4, 72)


def test_expert_refusals(lib):
    d = abi.Dims(64, 128, 256, 8, 2).c()
    r, p, n = ctypes.byref(d), fake(), abi.STATUS_BYTES

    def fwd(dims=r, ws=p, size=n, **kw):
        a = {**dict(x=p, off=p, W1=p, W3=p, W2=p, gu=p, h=p, y=p), **kw}
        return lib.moe_ffn_train(dims, *a.values(), ws, size, None)

    for k in ("x", "off", "W1", "W3", "W2", "gu", "h", "y"):
        assert fwd(**{k: None}) == abi.MOE_EINVAL, k
    for k in ("x", "W1", "W3", "W2", "gu", "h", "y"):
        assert fwd(**{k: ODD}) == abi.MOE_EUNSUPPORTED, k
    assert fwd(ws=None) == abi.MOE_EINVAL and fwd(size=n - 1) == abi.MOE_EWORKSPACE and fwd(dims=None) == abi.MOE_EINVAL
    assert fwd(dims=ctypes.byref(abi.Dims(64, 136, 256, 8, 2).c())) == abi.MOE_EUNSUPPORTED
    assert fwd(dims=ctypes.byref(abi.Dims(64, 128, 256, 300, 2).c())) == abi.MOE_EINVAL

    def bwd(ws=p, size=n, **kw):
        a = {**dict(dy=p, x=p, off=p, W1=p, W3=p, W2=p, gu=p, h=p, dgu=p, dx=p, dW1=p, dW3=p, dW2=p), **kw}
        return lib.moe_ffn_backward(r, *a.values(), 1, ws, size, None)

    # what is wanted needs its inputs
    for k in ("dy", "x", "off", "W1", "W3", "W2", "gu", "h", "dgu", "dW1", "dW3"):
        assert bwd(**{k: None}) == abi.MOE_EINVAL, k
    assert bwd(dW2=ODD) == abi.MOE_EUNSUPPORTED and bwd(size=0) == abi.MOE_EWORKSPACE and bwd(ws=None) == abi.MOE_EINVAL


def test_rows_and_router_refusals(lib):
    d = abi.Dims(64, 128, 256, 8, 2)
    c, p = d.c(), fake()
    r = ctypes.byref(c)
    cb = lambda dy=p, y=p, inv=p, w=p, dyp=p, dw=p: lib.moe_combine_backward(r, dy, 1, y, inv, w, dyp, dw, None)  # noqa: E731
    for k in ("dy", "y", "inv", "w", "dyp"):
        assert cb(**{k: None}) == abi.MOE_EINVAL, k
    assert cb(dy=ODD) == abi.MOE_EUNSUPPORTED and cb(dyp=ODD) == abi.MOE_EUNSUPPORTED
    assert lib.moe_permute_backward(r, None, p, p, 1, None) == abi.MOE_EINVAL
    assert lib.moe_permute_backward(r, p, p, ODD, 1, None) == abi.MOE_EUNSUPPORTED
    n = abi.moe_route_backward_workspace_size(d)

    def rb(aux=0.1, z=0.1, ws=p, size=n, **kw):
        a = {**dict(x=p, Wr=p, logits=p, idx=p, w=p, dw=p, counts=p), **{k: v for k, v in kw.items() if k in ("x", "Wr", "logits", "idx", "w", "dw", "counts")}}
        b = {**dict(dxp=p, inv=p, dx=p, dWr=p, dl=p), **{k: v for k, v in kw.items() if k in ("dxp", "inv", "dx", "dWr", "dl")}}
        return lib.moe_route_backward(r, *a.values(), aux, z, b["dxp"], b["inv"], b["dx"], 1, b["dWr"], 1, b["dl"], ws, size, None)

    assert rb(dx=None, dWr=None, dl=None) == abi.MOE_EINVAL
    for k in ("x", "Wr", "logits", "idx", "w", "counts", "dxp", "inv", "dx"):
        assert rb(**{k: None}) == abi.MOE_EINVAL, k
    assert rb(size=n - 1) == abi.MOE_EWORKSPACE and rb(ws=None) == abi.MOE_EINVAL and rb(dx=ODD) == abi.MOE_EUNSUPPORTED


def test_wrappers_refuse_host_tensors():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        abi.moe_layernorm(t, None, None, 1e-5, t)
    with pytest.raises(ValueError):
        abi.moe_permute_backward(abi.Dims(4, 64, 64, 2, 1), t, t, t)


def test_workspace_covers_every_training_call():
    for T, d, E, K in [(1, 16, 1, 1), (4096, 7168, 256, 8), (100, 4096, 8, 2)]:
        dims = abi.Dims(T, d, 64, E, K)
        n = abi.alloc_train_workspace(dims, "cpu").numel()
        assert n >= abi.STATUS_BYTES and n >= abi.moe_route_backward_workspace_size(dims)
        assert n >= abi.moe_layernorm_workspace_size(T, d)
