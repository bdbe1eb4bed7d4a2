"""Which tiles the training products take: host-side choice, no GPU needed."""
import pytest

from moe_layer_gemm_b200 import abi, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


def tiles(product, T, d, f, E=1, K=1):
    return abi.moe_train_subtiles(abi.Dims(T, d, f, E, K), product)


def test_large_batches_take_wide_tiles():
    shape = (16384, 4096, 14336, 8, 2)
    assert [tiles(p, *shape) for p in abi.TRAIN_PRODUCTS] == [2, 2, 1, 2, 2]
    # short reductions do not
    assert [tiles(p, 16384, 1024, 512, 64, 2) for p in ("gate", "down", "dx", "dw")] == [1, 1, 1, 1]
    # nor outputs of one sub-tile
    assert tiles("down", 65536, 256, 14336) == 1 and tiles("gate", 65536, 8192, 128) == 1


@pytest.mark.parametrize("T,d,f,E,K", [(4096, 8192, 2048, 1, 1), (16384, 16384, 4096, 4, 2), (1 << 20, 65536, 16384, 1, 1)])
def test_saved_projections_gradient_takes_narrow_tiles(T, d, f, E, K):
    assert tiles("dgate", T, d, f, E, K) == 1


def test_refusals():
    with pytest.raises(abi.MoEError):
        tiles("gate", 0, 128, 128)
    with pytest.raises(ValueError):
        tiles("up", 64, 128, 128)
    assert abi.load().moe_train_subtiles(abi.ctypes.byref(abi.Dims(64, 128, 128, 1, 1).c()), 5) == abi.MOE_EINVAL
