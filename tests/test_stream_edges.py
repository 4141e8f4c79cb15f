"""CPU checks of the streaming calls at the ends of what their documentation allows. No call here reaches the CUDA runtime."""
import ctypes

import pytest

import free_block_sparse_losa_b200 as L
from free_block_sparse_losa_b200 import build as B

FAKE = 0x10000  # aligned, never dereferenced
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def test_append_strides_of_single_extents(lib):
    """Nothing steps by the stride of an extent of one: such a call is refused for its head_dim only, which comes later."""
    def call(hk, total, strides):
        cache = L.make_cache(hk, 96, 128, 10, 1, 5)
        return lib.losa_cache_append(ctypes.byref(cache), None, 1, FAKE, strides[0], strides[1], FAKE, strides[2], strides[3],
                                     total, 1, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 0)

    assert call(1, 8, (96, 5, 96, -3)) == UNSUPPORTED
    assert call(4, 1, (7, 96, 1, 96)) == UNSUPPORTED
    for hk, total, strides in ((1, 8, (95, 8, 96, 8)), (4, 1, (8, 96, 8, 95)), (4, 1, (8, -96, 8, 96))):
        assert call(hk, total, strides) == INVALID
