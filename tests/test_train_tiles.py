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
    assert [tiles(p, *shape) for p in abi.TRAIN_PRODUCTS] == [2, 2, 1, 2, 1]
    # shorter reductions do not: the down projection's least of all
    assert [tiles(p, 16384, 1024, 512, 64, 2) for p in ("gate", "down", "dx", "dw")] == [1, 1, 1, 1]
    assert [tiles(p, 16384, 7168, 2048, 16, 2) for p in ("gate", "down", "dx")] == [2, 1, 1]
    assert [tiles(p, 16384, 4096, 4096, 8, 2) for p in ("gate", "down", "dx")] == [2, 1, 2]
    assert [tiles("down", 8192, 8192, f) for f in (4096, 8192, 10240, 14336)] == [1, 1, 2, 2]
    # nor outputs of one sub-tile
    assert tiles("down", 65536, 256, 14336) == 1 and tiles("gate", 65536, 8192, 128) == 1


@pytest.mark.parametrize("product", ["dgate", "dw"])
@pytest.mark.parametrize("T,d,f,E,K", [(4096, 8192, 2048, 1, 1), (16384, 16384, 4096, 4, 2), (1 << 20, 65536, 16384, 1, 1)])
def test_narrow_at_any_length(product, T, d, f, E, K):
    assert tiles(product, T, d, f, E, K) == 1


@pytest.mark.parametrize("product,T,d,f,E,K,want", [
    # 16 narrow tiles on 74 pairs, or 8 wide ones that take twice as long
    ("down", 256, 4096, 14336, 1, 1, 1), ("dx", 256, 4096, 14336, 1, 1, 1), ("gate", 768, 4096, 2048, 1, 1, 1),
    # rounds of narrow and wide tiles: (3, 2), (5, 3), (7, 4)
    ("down", 1024, 4096, 14336, 8, 2, 1), ("down", 2048, 4096, 14336, 8, 2, 1), ("dx", 1024, 4096, 8192, 8, 2, 1), ("dx", 4096, 8192, 4096, 1, 1, 1),
    # (2, 1), (4, 2), (14, 7) and more: wide
    ("down", 256, 4096, 14336, 8, 2, 2), ("gate", 256, 4096, 14336, 8, 2, 2), ("dx", 4096, 4096, 4096, 1, 1, 2), ("dx", 4096, 16384, 4096, 1, 1, 2)])
def test_few_tiles_are_not_halved(product, T, d, f, E, K, want):
    assert tiles(product, T, d, f, E, K) == want


def test_refusals():
    with pytest.raises(abi.MoEError):
        tiles("gate", 0, 128, 128)
    with pytest.raises(ValueError):
        tiles("up", 64, 128, 128)
    assert abi.load().moe_train_subtiles(abi.ctypes.byref(abi.Dims(64, 128, 128, 1, 1).c()), 5) == abi.MOE_EINVAL
