"""Sizes that the paged calls count in 32 bits, through the C ABI without a GPU: refused before any launch."""
import pytest

from attention_quantized_kv_split_gb300 import _lib, build as qbuild

FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return _lib.lib()


@pytest.mark.parametrize("T,Hkv,D", [(1 << 30, 4, 64), (1 << 30, 4, 512), ((1 << 31) - 1, 3, 64), ((1 << 31) - 1, 8, 128),
                                     (1 << 29, 8, 256), (1 << 24, 256, 64)])
def test_append_refuses_rows_beyond_32_bits(L, T, Hkv, D):
    # token and head strides of 0 (an expanded row) make so many rows addressable
    p = [FAKE + 4096 * i for i in range(11)]
    assert L.qdecode_paged_append(p[0], p[1], 0, 0, 0, 0, *p[2:], T, Hkv, 4, 16, D, 64, 4, 1, None) == _lib.QDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("tstride,hstride,out", [
    (1024, 128, 0),                        # in place
    (1024, 128, 5 * 2048 - 16),            # from the last row's end on
    (1024, 128, -(5 * 2048) + 16),         # up to the first row's start
    (4096, 128, 3 * 8192 + 2048),          # between the rows of a wider tensor
    (0, 128, 2048 - 16),                   # behind an expanded row's start
    (-1024, 128, -2048),                   # rows in the other order
])
def test_attention_in_place_is_refused(L, tstride, hstride, out):
    # (no call here may be one that is not refused: its addresses do not exist)
    q = FAKE + (1 << 30)
    p = [FAKE + 4096 * i for i in range(6)]
    t = [FAKE + (1 << 33) + 4096 * i for i in range(3)]
    st = L.qdecode_paged_attn(q, tstride, hstride, *p, q + out, *t, 5, 2, 2, 8, 2, 9, 16, 4, 1, 128, 64, 4, 1, None)
    assert st == _lib.QDA_ERR_INVALID
