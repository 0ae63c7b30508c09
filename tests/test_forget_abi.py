"""Argument checks of the calls behind a cache that forgets, without a GPU: every call below is refused before any launch."""
import contextlib
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda
from attention_quantized_kv_split_gb300 import _lib, build as qbuild

FAKE = 0x7F0000000000  # never dereferenced
INVALID, UNSUPPORTED, ALIGN = _lib.QDA_ERR_INVALID, _lib.QDA_ERR_UNSUPPORTED, _lib.QDA_ERR_ALIGN


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return _lib.lib()


def ptrs(n):
    return [FAKE + (1 << 20) * i for i in range(n)]


def edit(p, i, v):
    p = list(p)
    p[i] = v
    return p


# ------------------------------------------------------------------------------------------------------------ rotary


def rope(L, p=None, qs=(1024, 128), ks=(256, 128), qo=(1024, 128), ko=(256, 128), T=3, B=0, H=8, Hkv=2, D=128, rot=128,
         inter=0, inverse=0, dtype=1, scale=1.0):
    p = p or [*ptrs(6), None, None]
    return L.qdecode_rope(p[0], *qs, p[1], *ks, p[2], *qo, p[3], *ko, *p[4:], T, B, H, Hkv, D, rot, inter, inverse, dtype, scale,
                          None)


@pytest.mark.parametrize("i", range(6))
def test_rope_null(L, i):
    assert rope(L, edit([*ptrs(6), None, None], i, None)) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0, Hkv=0), INVALID), (dict(H=-1), INVALID), (dict(rot=0), INVALID), (dict(rot=7), INVALID),
    (dict(rot=130), INVALID), (dict(dtype=0), INVALID), (dict(dtype=4), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(D=96, rot=96), UNSUPPORTED), (dict(H=4096), UNSUPPORTED),
    (dict(T=(1 << 31) - 1), UNSUPPORTED), (dict(qs=(1028, 128)), ALIGN), (dict(ko=(256, 132)), ALIGN),
    (dict(ks=(258, 128), dtype=3), ALIGN), (dict(T=0), 0), (dict(qo=(1024, 64)), INVALID), (dict(ko=(64, 256)), INVALID),
])
def test_rope_arguments(L, kw, status):
    assert rope(L, **kw) == status


@pytest.mark.parametrize("i,off", [(0, 8), (1, 8), (2, 8), (3, 8), (4, 2), (5, 4), (6, 2), (7, 2)])
def test_rope_alignment(L, i, off):
    p = ptrs(8)
    p[i] += off
    assert rope(L, p, B=2) == ALIGN


def test_rope_shift_needs_its_starts(L):
    p = ptrs(8)
    assert rope(L, edit(p, 6, None), B=2) == rope(L, edit(p, 7, None), B=2) == rope(L, p, B=0) == INVALID
    assert rope(L, p, B=_lib.QDA_MAX_B + 1) == UNSUPPORTED


def test_rope_outputs_that_touch(L):
    """T = 3 tokens of 8 + 2 heads of 128 bf16 values; no launch is reached, so a call that is let through is not made here."""
    p = [*ptrs(6), None, None]
    assert rope(L, edit(p, 2, p[0] + 256)) == INVALID                       # over its own input, one head on
    assert rope(L, edit(p, 2, p[1] - 1024)) == INVALID                      # over the keys
    assert rope(L, edit(p, 3, p[2] + 3 * 2048 - 16)) == INVALID             # over the other output's end
    assert rope(L, edit(p, 2, p[0]), qo=(2048, 128)) == INVALID             # its own input by other strides
    fused = dict(qs=(1536, 128), ks=(1536, 128), qo=(1536, 128), ko=(1536, 128))
    q = edit(edit(edit(p, 2, p[0]), 1, p[0] + 2048 - 256), 3, p[0] + 2048 - 256)
    assert rope(L, q, **fused) == INVALID                                   # keys that begin in the queries' last head


def test_rope_freqs(L):
    out = (ctypes.c_double * 4)()
    call = lambda *a: L.qdecode_rope_freqs(*a, out)  # noqa: E731
    for bad in [(0, 1e4, 1, 0, 0, 0), (7, 1e4, 1, 0, 0, 0), (8, 0, 1, 0, 0, 0), (8, 1e4, 0, 0, 0, 0), (8, 1e4, -1, 0, 0, 0),
                (8, 1e4, 1, -1, 0, 0), (8, 1e4, 1, 100, 4, 4), (8, 1e4, 1, 100, 4, 1), (8, 1e4, 1, 100, -1, 1), (8, math.nan, 1, 0, 0, 0),
                (8, 1e4, 1, math.inf, 1, 4)]:
        assert call(*bad) == INVALID, bad
    assert L.qdecode_rope_freqs(8, 1e4, 1.0, 0.0, 0.0, 0.0, None) == INVALID
    assert call(8, 1e4, 1.0, 0.0, 0.0, 0.0) == 0
    np.testing.assert_allclose(list(out), [1, 0.1, 0.01, 0.001], rtol=1e-15)


def test_rope_freqs_stretched():
    f = qda.qdecode_rope_freqs(64, 500.0).numpy()
    np.testing.assert_allclose(qda.qdecode_rope_freqs(64, 500.0, 4.0).numpy(), f / 4, rtol=1e-15)
    g = qda.qdecode_rope_freqs(64, 500.0, 4.0, 1000.0, 2.0, 9.0).numpy()
    turns = f * 1000 / (2 * np.pi)
    assert (g[turns >= 9] == f[turns >= 9]).all() and (turns >= 9).any()
    np.testing.assert_allclose(g[turns <= 2], f[turns <= 2] / 4, rtol=1e-15)
    assert (turns <= 2).any()
    mid = (turns > 2) & (turns < 9)
    keep = (turns[mid] - 2) / 7
    np.testing.assert_allclose(g[mid], f[mid] * (keep + (1 - keep) / 4), rtol=1e-14)
    assert mid.any() and qda.qdecode_rope_freqs(64).dtype is torch.float64


# ------------------------------------------------------------------------------------------------------------ weights


def weights(L, p=None, strides=(1024, 128), total_q=5, max_q=2, window=0, B=2, H=8, Hkv=2, num_pages=9, page=16, max_pages=4,
            D=128, GS=64, bits=4, dtype=1, decay=1.0):
    p = p or ptrs(11)
    return L.qdecode_paged_weights(p[0], *strides, *p[1:], total_q, max_q, window, B, H, Hkv, num_pages, page, max_pages, D, GS,
                                   bits, dtype, decay, None)


@pytest.mark.parametrize("i", range(10))   # shift (10) may be NULL
def test_weights_null(L, i):
    assert weights(L, edit(ptrs(11), i, None)) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(total_q=-1), INVALID), (dict(max_q=0), INVALID), (dict(window=-1), INVALID), (dict(B=0), INVALID), (dict(H=7), INVALID),
    (dict(Hkv=0), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(dtype=3), INVALID),
    (dict(decay=math.nan), INVALID), (dict(decay=math.inf), INVALID), (dict(bits=5), UNSUPPORTED), (dict(GS=16), UNSUPPORTED),
    (dict(D=192), UNSUPPORTED), (dict(page=20), UNSUPPORTED), (dict(B=_lib.QDA_MAX_B + 1), UNSUPPORTED), (dict(H=130), UNSUPPORTED),
    (dict(num_pages=1 << 30), UNSUPPORTED), (dict(num_pages=1 << 26, page=16, Hkv=4, H=4), UNSUPPORTED),
    (dict(total_q=(1 << 31) - 1), UNSUPPORTED), (dict(strides=(1025, 128)), ALIGN), (dict(strides=(1024, 4)), ALIGN),
    (dict(total_q=0), 0),
])
def test_weights_arguments(L, kw, status):
    assert weights(L, **kw) == status


@pytest.mark.parametrize("i", range(11))
def test_weights_alignment(L, i):
    p = ptrs(11)
    p[i] += 8 if i < 4 else 2
    assert weights(L, p) == ALIGN


def test_weights_heads_beyond_a_grid(L):
    assert weights(L, H=65536, Hkv=65536, num_pages=9) == UNSUPPORTED


def test_weights_workspace(L):
    n = ctypes.c_size_t()
    call = lambda *a: L.qdecode_paged_weights_workspace_bytes(*a, ctypes.byref(n))  # noqa: E731
    assert call(64, 32, 8, 64, 1, 0, 128) == 0 and n.value == 0          # few rows need none
    assert call(1, 32, 8, 2048, 2048, 0, 128) == 0 and n.value >= 8 * 2048 * 4 * 128 * 2
    whole = n.value
    assert call(1, 32, 8, 2048, 2048, 64, 128) == 0 and 8 * 64 * 4 * 128 * 2 <= n.value < whole / 8
    assert call(1, 32, 8, 2048, 2048, 0, 512) == 0 and n.value == 0
    for bad in [(0, 32, 8, 1, 1, 0, 128), (1, 31, 8, 1, 1, 0, 128), (1, 32, 0, 1, 1, 0, 128), (1, 32, 8, -1, 1, 0, 128),
                (1, 32, 8, 1, 0, 0, 128), (1, 32, 8, 1, 1, -1, 128)]:
        assert call(*bad) == INVALID
    assert call(513, 32, 8, 1, 1, 0, 128) == call(1, 65, 1, 1, 1, 0, 128) == call(1, 32, 8, 1, 1, 0, 96) == UNSUPPORTED
    assert L.qdecode_paged_weights_workspace_bytes(1, 32, 8, 1, 1, 0, 128, None) == INVALID


def attn_lse(L, p=None, total_q=5):
    p = p or ptrs(12)
    return L.qdecode_paged_attn_lse(p[0], 1024, 128, *p[1:], total_q, 2, 2, 8, 2, 9, 16, 4, 1, 128, 64, 4, 1, None)


@pytest.mark.parametrize("i", range(12))
def test_attn_lse_null_and_alignment(L, i):
    p = ptrs(12)
    assert attn_lse(L, edit(p, i, None)) == INVALID
    assert attn_lse(L, edit(p, i, p[i] + (8 if i < 8 else 2))) == ALIGN
    assert attn_lse(L, total_q=0) == 0


# ------------------------------------------------------------------------------------------------------------ eviction


def evict(L, p=None, B=2, Hkv=2, num_pages=9, page=16, max_pages=4, max_freed=8, budget=20, limit=24, sinks=2, recent=4, D=128,
          GS=64, bits=4):
    return L.qdecode_paged_evict(*(p or ptrs(14)), B, Hkv, num_pages, page, max_pages, max_freed, budget, limit, sinks, recent, D,
                                 GS, bits, None)


@pytest.mark.parametrize("i", range(13))   # shift (13) may be NULL
def test_evict_null(L, i):
    assert evict(L, edit(ptrs(14), i, None)) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(max_freed=-1), INVALID),
    (dict(budget=0), INVALID), (dict(limit=19), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=10, recent=11), INVALID), (dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), INVALID), (dict(bits=3), UNSUPPORTED),
    (dict(GS=256, D=512), UNSUPPORTED), (dict(D=96, GS=32), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(B=513), UNSUPPORTED),
    (dict(Hkv=65), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED), (dict(num_pages=1 << 26, Hkv=4), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED),
])
def test_evict_arguments(L, kw, status):
    assert evict(L, **kw) == status


@pytest.mark.parametrize("i", range(14))
def test_evict_alignment(L, i):
    p = ptrs(14)
    p[i] += 8 if i < 6 else 2
    assert evict(L, p) == ALIGN


def test_evict_lengths_in_place(L):
    p = ptrs(14)
    assert evict(L, edit(p, 9, p[8])) == INVALID


def test_evict_workspace(L):
    n = ctypes.c_size_t()
    call = lambda *a: L.qdecode_paged_evict_workspace_bytes(*a, ctypes.byref(n))  # noqa: E731
    assert call(64, 8, 64, 100, 2048) == 0 and n.value >= 64 * 8 * 2048 * 8
    assert call(1, 1, 16, 4, 60) == 0 and n.value < 1024          # no more rows can move than lie behind the budget
    for bad in [(0, 8, 64, 100, 1), (1, 0, 64, 100, 1), (1, 8, 0, 100, 1), (1, 8, 64, 0, 1), (1, 8, 64, 100, 0)]:
        assert call(*bad) == INVALID
    assert call(513, 8, 64, 100, 1) == call(1, 65, 64, 100, 1) == call(1, 8, 48, 100, 1) == UNSUPPORTED
    assert L.qdecode_paged_evict_workspace_bytes(1, 8, 64, 100, 1, None) == INVALID


# ----------------------------------------------------------------------------------------------------- packed, Python


def test_packed_calls(L):
    P = lambda f, *a: struct.pack("=" + f, *a)  # noqa: E731
    lse = [FAKE, 1024, 128, *ptrs(11), 5, 2, 2, 8, 2, 9, 16, 4, 1, 128, 64, 4, 1, 0]
    r = [FAKE, 1024, 128, FAKE + 4096, 256, 128, *[x for p in ptrs(2) for x in (p + (1 << 24), 1024, 128)], *ptrs(4), 3, 2, 8, 2, 128,
         128, 0, 0, 1, 1.0, 0]
    w = [FAKE, 1024, 128, *ptrs(10), 5, 2, 0, 2, 8, 2, 9, 16, 4, 128, 64, 4, 1, 1.0, 0]
    e = [*ptrs(14), 2, 2, 9, 16, 4, 8, 20, 24, 2, 4, 128, 64, 4, 0]
    call = L.qdecode_paged_packed
    for op, f, args, i, v, status in [
            (4, "28q", lse, 10, 0, INVALID), (4, "28q", lse, 14, 0, 0), (4, "28q", lse, 24, 48, UNSUPPORTED),
            (4, "28q", lse, 22, 1 << 31, INVALID), (4, "28q", lse, 10, FAKE + 2, ALIGN),
            (5, "25qdq", r, 16, 0, 0), (5, "25qdq", r, 21, 7, INVALID), (5, "25qdq", r, 25, math.nan, INVALID), (5, "25qdq", r, 20, 96, INVALID),
            (5, "25qdq", r, 13, FAKE + 4, ALIGN), (5, "25qdq", r, 16, 1 << 40, INVALID), (5, "25qdq", r, 24, 9, INVALID),
            (6, "26qdq", w, 13, 0, 0), (6, "26qdq", w, 15, -1, INVALID), (6, "26qdq", w, 26, math.nan, INVALID),
            (6, "26qdq", w, 24, 7, UNSUPPORTED), (6, "26qdq", w, 12, FAKE + 2, ALIGN), (6, "26qdq", w, 25, 3, INVALID),
            (7, "28q", e, 20, 0, INVALID), (7, "28q", e, 26, 7, UNSUPPORTED), (7, "28q", e, 13, FAKE + 2, ALIGN),
            (7, "28q", e, 14, 1 << 33, INVALID)]:
        assert call(op, P(f, *edit(args, i, v))) == status, (op, i, v)
    assert call(3, P("28q", *e)) == call(8, P("28q", *e)) == INVALID


def tensors():
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    pool = qda.PagedKV(3, 2, 16, 64, 32, 4, torch.bfloat16, device="cpu", track=True)
    return pool, i32, torch.zeros(2, 4, 64, dtype=torch.bfloat16)


def test_python_checks():
    pool, i32, q = tensors()
    f = torch.ones(32, dtype=torch.float64)
    for bad in (dict(q=None, k=None), dict(freqs=f.float()), dict(positions=i32(3)), dict(positions=i32(2).long()), dict(k=q.float()),
                dict(k=q[:1]), dict(q_start=i32(3)), dict(q_start=i32(2), shift=i32(3)), dict(q=q[..., ::2], k=None), dict(k=None, k_out=q),
                dict(q=q.to(torch.int16), k=None), dict(q_out=q[:, :2])):
        kw = {**dict(q=q, k=q, positions=i32(2), freqs=f), **bad}
        with pytest.raises(ValueError):
            qda.qdecode_rope(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        qda.qdecode_rope(q, None, i32(2), f)
    ok = dict(q=q, lse=torch.zeros(2, 4), q_start=i32(2), kv_len=i32(1), block_table=i32(1, 2), max_q=2)
    for bad in (dict(lse=torch.zeros(2, 3)), dict(lse=torch.zeros(2, 4).double()), dict(q=q.half()), dict(kv_len=i32(2)),
                dict(shift=i32(2)), dict(q_start=i32(2).long())):
        with pytest.raises(ValueError):
            pool.weigh(**{**ok, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        pool.weigh(**ok)
    with pytest.raises(ValueError, match="CUDA"):
        pool.evict(i32(1), i32(1, 2), 4)
    for bad in (dict(kv_len=i32(2)), dict(kv_len=i32(1).long()), dict(shift=i32(2))):
        with pytest.raises(ValueError):
            pool.evict(**{**dict(kv_len=i32(1), block_table=i32(1, 2), budget=4), **bad})
    plain = qda.PagedKV(3, 2, 16, 64, 32, 4, torch.bfloat16, device="cpu")
    with pytest.raises(ValueError, match="track"):
        plain.evict(i32(1), i32(1, 2), 4)
    with pytest.raises(ValueError, match="track"):
        plain.weigh(**ok)
    with pytest.raises(ValueError):
        qda.qdecode_paged_attn(q, *pool.arrays(), q.clone(), i32(2), i32(1), i32(1, 2), 2, 32, 4, lse=torch.zeros(4, 2))


def test_evict_allocates_in_the_streams_context(monkeypatch):
    pool, i32, _ = tensors()
    inside, seen = [], []

    @contextlib.contextmanager
    def on(stream, device):
        inside.append(stream)
        yield
        inside.pop()

    monkeypatch.setattr(qda, "_on", on)
    monkeypatch.setattr(qda, "qdecode_paged_evict", lambda *a, **k: None)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(list(inside)), empty(*a, **k))[1])
    pool.evict(i32(1), i32(1, 2), 4, stream=77)
    assert len(seen) == 3 and all(s == [77] for s in seen)


# ------------------------------------------------------------------- outputs upon each other, numbers beyond fp32


@pytest.mark.parametrize("ts,hs", [(128, 128), (256, 128), (896, 128), (128, 256), (384, 256), (-128, 128), (256, -128)])
def test_rope_rows_of_an_output_that_collide(L, ts, hs):
    """Token and head strides of D or more each for itself, that bring two rows to one place or partly over each other (T = 3
    tokens of 8 heads of 128 values)."""
    assert rope(L, qo=(ts, hs)) == INVALID
    p = [*ptrs(6), None, None]
    assert rope(L, edit(p, 2, p[0]), qs=(ts, hs), qo=(ts, hs)) == INVALID


def test_rope_rows_that_collide_in_part(L):
    assert rope(L, qo=(128 * 9, 128 * 6 - 8)) == INVALID        # three tokens on, two heads back: 24 elements apart
    assert rope(L, qo=(128 + 8, 128), H=2, T=2) == INVALID      # the next token begins in the second head


def test_factors_beyond_fp32(L):
    """Finite in 64 bits, infinite in the 32 that the kernels hold them in."""
    for x in (1e39, -1e39, 3.5e38):
        assert rope(L, scale=x) == weights(L, decay=x) == INVALID


@pytest.mark.parametrize("other", [0, 7])
def test_attn_lse_over_queries_or_outputs(L, other):
    """lse [5, 8] of fp32 over q or out [5, 8, 128] of 16 bits: at their starts, their ends and in front."""
    p = ptrs(12)
    for off in (0, 160, 5 * 8 * 128 * 2 - 4, -156):
        assert attn_lse(L, edit(p, 8, p[other] + off)) == INVALID


def test_evict_lengths_that_overlap(L):
    p = ptrs(14)
    assert evict(L, edit(p, 9, p[8] + 4)) == evict(L, edit(p, 9, p[8] - 4)) == INVALID
    assert evict(L, edit(p, 9, p[13])) == evict(L, edit(p, 13, p[8])) == INVALID


def test_rope_takes_three_dimensions():
    _, i32, q = tensors()
    f = torch.ones(32, dtype=torch.float64)
    for x in (q[0], q[None], q[0, 0], q.reshape(-1)):
        for kw in (dict(q=x, k=None), dict(q=None, k=x), dict(q=q, k=x), dict(q=q, k=None, q_out=x)):
            with pytest.raises(ValueError):
                qda.qdecode_rope(**kw, positions=i32(2), freqs=f)
