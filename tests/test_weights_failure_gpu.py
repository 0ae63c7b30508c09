"""A wait of the weights' kernel for many rows that runs out (the checked build's testing aid holds back one slice of query rows
from the first CTA): the call ends by its bounded waits, says so in the device status, touches nothing but masses and tokens of
its sequences, and the next call is right."""
import ctypes
import time

import numpy as np
import pytest
import torch

from attention_quantized_kv_split_gb300 import _lib, build

import forget_ref as R
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


@pytest.mark.parametrize("q_lens,D,GS,bits", [([300], 128, 64, 4), ([70, 200], 256, 32, 8), ([90], 64, 32, 4)])
def test_a_stalled_slice_ends_the_call(L, q_lens, D, GS, bits):
    c = Case(q_lens, [4000 - 31 * b for b in range(len(q_lens))], 16, 8, D, bits, GS, "bf16", 32, seed=D)
    lse = torch.from_numpy(R.log_sums(c).astype(np.float32)).cuda()
    mass = torch.zeros(c.arrays[1].shape[:3], device="cuda")
    token = torch.full(mass.shape, -7, dtype=torch.int32, device="cuda")
    before = [a.clone() for a in c.arrays]

    def run():
        st = L.qdecode_paged_weights(c.q.data_ptr(), c.q.stride(0), c.q.stride(1), *(a.data_ptr() for a in c.arrays[:3]), lse.data_ptr(),
                                     mass.data_ptr(), token.data_ptr(), c.q_start.data_ptr(), c.kv_len.data_ptr(), c.table.data_ptr(),
                                     None, c.total, max(q_lens), 0, len(q_lens), c.H, c.Hkv, c.arrays[0].shape[0], c.page,
                                     c.table.shape[1], D, GS, bits, 1, 0.0, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()

    status(L)
    run()
    want = mass.clone()
    assert status(L) == 0
    for slice_ in (0, 3):
        L.qdecode_attn_debug_stall_chunk(slice_)
        t0 = time.time()
        run()
        L.qdecode_attn_debug_stall_chunk(-1)
        got = status(L)
        assert got & ~3 == 0 and got & 1
        assert time.time() - t0 < 20.0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.arrays, before))
        run()   # (nothing of the old masses is kept: decay 0)
        assert status(L) == 0 and torch.equal(mass, want)
