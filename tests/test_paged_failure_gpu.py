"""A wait of the paged calls' chunk kernel that runs out (the checked build's testing aid holds back one block's pages): the
call ends by its bounded waits, says so in the device status, touches nothing but its own outputs, and the next call is
right."""
import ctypes
import time

import pytest
import torch

from attention_quantized_kv_split_gb300 import _lib, build

from paged_ref import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    handle = ctypes.CDLL(build.build(checked=True))
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = res, args
    yield handle
    handle.qdecode_attn_debug_stall_chunk(-1)


def status(L):
    v = ctypes.c_uint()
    assert L.qdecode_attn_device_status(ctypes.byref(v)) == 0
    return v.value


def run(L, c, out, causal):
    p = [t.data_ptr() for t in (*c.arrays, out, c.q_start, c.kv_len, c.table)]
    st = L.qdecode_paged_attn(c.q.data_ptr(), c.q.stride(0), c.q.stride(1), *p, c.total, max(c.q_lens), len(c.q_lens), c.H, c.Hkv,
                              c.arrays[0].shape[0], c.page, c.table.shape[1], causal, c.D, c.GS, c.bits,
                              {torch.bfloat16: 1, torch.float16: 2}[c.q.dtype], torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("q_lens,D,GS,bits", [([300], 128, 64, 4), ([40], 64, 32, 8), ([70, 200], 256, 64, 4), ([90], 512, 128, 4)])
@pytest.mark.parametrize("causal", [1, 0])
def test_a_stalled_block_ends_the_call(L, q_lens, D, GS, bits, causal):
    c = Case(q_lens, [4000 - 31 * b for b in range(len(q_lens))], 16, 8, D, bits, GS, "bf16", 32, seed=D)
    pad = 5   # rows behind the outputs, which nothing may touch
    buf = torch.full((c.total + 2 * pad, c.H, D), 7.0, dtype=c.q.dtype, device="cuda")
    out = buf[pad: pad + c.total]
    before = [a.clone() for a in c.arrays]
    status(L)
    for block in (0, 9):
        L.qdecode_attn_debug_stall_chunk(block)
        t0 = time.time()
        run(L, c, out, causal)
        L.qdecode_attn_debug_stall_chunk(-1)
        got = status(L)
        assert got & ~3 == 0 and (got & 1 or block == 9)   # (the first CTA may have fewer blocks than ten)
        assert time.time() - t0 < 10.0
        assert bool((buf[:pad] == 7.0).all()) and bool((buf[pad + c.total:] == 7.0).all())
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.arrays, before))
        run(L, c, out, causal)
        assert status(L) == 0
        c.check(out, bool(causal))
