"""Sizes that the calls over trees of drafted tokens take and refuse. Nothing
here is launched: a call whose sizes pass ends at a bad address that is
checked behind them, and the message says which of the two it was."""
import pytest

from linear_attention_chunk_gb300 import binding
from linear_attention_chunk_gb300.build import build

FAKE, ODD = 0x10000, 0x10008   # never dereferenced
BAD = binding.GLA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def why(L, status):
    assert status == BAD
    return L.gla_last_error().decode()


def conv(L, nseq, T, D, dt=0, ld=None, y=ODD):
    return why(L, L.gla_conv1d_tree(FAKE, ld or D, FAKE, None, FAKE, FAKE, FAKE, FAKE, max(nseq, 0), nseq, T, D, dt, y, None))


@pytest.mark.parametrize("nseq,T,D,dt", [(2560, 2560 * 64, 4096, 0), (1800, 1800 * 64, 6144, 0), (100000, 1 << 20, 2048, 1),
                                         (1, 1 << 15, 1 << 25, 0)])
def test_convolution_of_many_packed_trees(L, nseq, T, D, dt):
    """The tensors hold total_T rows, whatever the number of sequences."""
    assert conv(L, nseq, T, D, dt).startswith("y is not")


def test_convolution_sizes_refused(L):
    assert "too large" in conv(L, 1, (1 << 15) + 1, 1 << 25, y=2 * FAKE)
    assert "nseq*D" in conv(L, 1 << 16, 1 << 16, 1 << 15, y=2 * FAKE)
    assert "negative" in conv(L, -1, 8, 64, y=2 * FAKE) and "negative" in conv(L, 2, -1, 64, y=2 * FAKE)


def test_pools_without_pages(L):
    """They need no address; with pages they do."""
    import ctypes

    null, size = (ctypes.c_void_p * 2)(None, None), (ctypes.c_int64 * 2)(4, 4)
    assert "src" in why(L, L.gla_pages_copy(null, size, 2, 0, None, FAKE, 3, None))
    assert "slots" in why(L, L.gla_pages_clear(null, size, 2, 0, None, 3, None))
    assert "a pool" in why(L, L.gla_pages_copy(null, size, 2, 1, FAKE, FAKE, 3, None))
    assert L.gla_pages_copy(null, size, 2, 0, None, None, 0, None) == binding.GLA_OK
