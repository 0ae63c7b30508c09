"""The paged calls' argument checks, through the C ABI without a GPU: every call below is refused before any launch."""
import ctypes

import pytest

from attention_quantized_kv_split_gb300 import _lib, build as qbuild

FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return _lib.lib()


def ptrs(n):
    return [FAKE + 4096 * i for i in range(n)]


INVALID, UNSUPPORTED, ALIGN = _lib.QDA_ERR_INVALID, _lib.QDA_ERR_UNSUPPORTED, _lib.QDA_ERR_ALIGN


def paged_map(L, p=None, B=4, max_pages=8, n_free=5, page=16, max_tokens=9):
    return L.qdecode_paged_map(*(p or ptrs(9)), B, max_pages, n_free, page, max_tokens, None)


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 5, 6, 8])   # positions (7) may be NULL
def test_map_null(L, i):
    p = ptrs(9)
    p[i] = None
    assert paged_map(L, p) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_free=-1), INVALID), (dict(max_tokens=-1), INVALID),
    (dict(page=0), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(B=_lib.QDA_MAX_B + 1), UNSUPPORTED),
])
def test_map_arguments(L, kw, status):
    assert paged_map(L, **kw) == status


def test_map_in_place_lengths_and_alignment(L):
    for i in (0, 1):
        p = ptrs(9)
        p[5] = p[i]   # kv_len written where other CTAs still read the lengths
        assert paged_map(L, p) == INVALID
    p = ptrs(9)
    p[6] += 2
    assert paged_map(L, p) == ALIGN


def append(L, p=None, strides=(1024, 128, 1024, 128), T=3, Hkv=8, num_pages=4, page=16, D=128, GS=64, bits=4, dtype=1):
    p = p or ptrs(11)
    return L.qdecode_paged_append(p[0], p[1], *strides, *p[2:], T, Hkv, num_pages, page, D, GS, bits, dtype, None)


@pytest.mark.parametrize("i", range(11))   # one of k_held (9) and v_held (10) alone is refused too
def test_append_null(L, i):
    p = ptrs(11)
    p[i] = None
    assert append(L, p) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(dtype=0), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=1 | 4 << 8), INVALID), (dict(dtype=1 | 1 << 16), INVALID),
    (dict(bits=3), UNSUPPORTED), (dict(GS=48), UNSUPPORTED), (dict(D=96, GS=32), UNSUPPORTED),
    (dict(D=64, GS=128), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED),
    (dict(strides=(1028, 128, 1024, 128)), ALIGN), (dict(strides=(1024, 128, 1024, 132)), ALIGN),
    (dict(strides=(1026, 128, 1024, 128), dtype=1 | 3 << 8), ALIGN),
    (dict(T=0), 0),
])
def test_append_arguments(L, kw, status):
    assert append(L, **kw) == status


@pytest.mark.parametrize("i", range(11))
def test_append_alignment(L, i):
    p = ptrs(11)
    p[i] += 2 if i == 2 else 8
    assert append(L, p) == ALIGN


def attn(L, p=None, strides=(1024, 128), total_q=5, max_q=2, B=2, H=8, Hkv=2, num_pages=9, page=16, max_pages=4, causal=1,
         D=128, GS=64, bits=4, dtype=1):
    p = p or ptrs(11)
    return L.qdecode_paged_attn(p[0], *strides, *p[1:], total_q, max_q, B, H, Hkv, num_pages, page, max_pages, causal, D,
                                GS, bits, dtype, None)


@pytest.mark.parametrize("i", range(11))
def test_attn_null(L, i):
    p = ptrs(11)
    p[i] = None
    assert attn(L, p) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(total_q=-1), INVALID), (dict(max_q=0), INVALID), (dict(B=0), INVALID), (dict(H=7), INVALID),
    (dict(Hkv=0), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=1 | 3 << 8), INVALID), (dict(bits=5), UNSUPPORTED), (dict(GS=16), UNSUPPORTED),
    (dict(D=192, GS=64), UNSUPPORTED), (dict(page=20), UNSUPPORTED), (dict(B=_lib.QDA_MAX_B + 1), UNSUPPORTED),
    (dict(H=65 * 2), UNSUPPORTED), (dict(num_pages=1 << 30, page=16), UNSUPPORTED),
    (dict(strides=(1025, 128)), ALIGN), (dict(strides=(1024, 4)), ALIGN), (dict(total_q=0), 0),
])
def test_attn_arguments(L, kw, status):
    assert attn(L, **kw) == status


@pytest.mark.parametrize("i", range(11))
def test_attn_alignment(L, i):
    p = ptrs(11)
    p[i] += 2 if i >= 8 else 8
    assert attn(L, p) == ALIGN


@pytest.mark.parametrize("args,status", [
    ((0, 8, 2, 1, 128, 64, 4), INVALID), ((1, 8, 3, 1, 128, 64, 4), INVALID), ((1, 8, 2, 0, 128, 64, 4), INVALID),
    ((1, 8, 2, 1, 128, 64, 5), UNSUPPORTED), ((1, 130, 2, 1, 128, 64, 4), UNSUPPORTED),
    ((_lib.QDA_MAX_B + 1, 8, 2, 1, 128, 64, 4), UNSUPPORTED),
])
def test_attn_workspace_arguments(L, args, status):
    n = ctypes.c_size_t()
    assert L.qdecode_paged_attn_workspace_bytes(*args, ctypes.byref(n)) == status
    assert L.qdecode_paged_attn_workspace_bytes(*args, None) == INVALID


def test_packed_calls(L):
    """The packed form makes the same calls: the same answers, and refusals of its own."""
    import struct
    P = lambda *a: struct.pack(f"={len(a)}q", *a)  # noqa: E731
    m = [*ptrs(9), 4, 8, 5, 16, 9, 0]
    a = [*ptrs(2), 1024, 128, 1024, 128, *ptrs(9), 3, 8, 4, 16, 128, 64, 4, 1, 0]
    t = [FAKE, 1024, 128, *ptrs(10), 5, 2, 2, 8, 2, 9, 16, 4, 1, 128, 64, 4, 1, 0]
    call = L.qdecode_paged_packed
    assert call(3, P(*m)) == call(-1, P(*m)) == call(0, None) == INVALID
    for op, args, i, v, status in [(0, m, 9, 0, INVALID), (0, m, 12, 24, UNSUPPORTED), (0, m, 0, 0, INVALID),
                                   (0, m, 13, 1 << 31, INVALID), (0, m, 6, FAKE + 2, ALIGN), (1, a, 7, 0, INVALID),
                                   (1, a, 2, 1028, ALIGN), (1, a, 15, 0, 0), (1, a, 21, 3, UNSUPPORTED),
                                   (2, t, 14, 0, INVALID), (2, t, 13, 0, 0), (2, t, 2, 4, ALIGN), (2, t, 24, 7, UNSUPPORTED),
                                   (2, t, 17, 3, INVALID), (2, t, 20, -(1 << 40), INVALID)]:
        x = list(args)
        x[i] = v
        assert call(op, P(*x)) == status, (op, i, v)


@pytest.mark.parametrize("total_q,H,Hkv", [((1 << 31) - 1, 8, 2), (1 << 25, 64, 1), ((1 << 31) - 200, 1, 1)])
def test_attn_refuses_query_rows_beyond_32_bits(L, total_q, H, Hkv):
    # rows are (token, query head of the KV head) pairs, counted in 32 bits by the kernels
    assert attn(L, total_q=total_q, H=H, Hkv=Hkv) == UNSUPPORTED
