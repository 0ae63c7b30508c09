"""Rotary positions against the definition in 64 bits: layouts, partial heads, odd sizes, far positions, strides, places."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda

import forget_ref as R
from paged_ref import DT

pytestmark = pytest.mark.gpu


def data(T, H, Hkv, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H + 2 * Hkv, D, generator=g, dtype=torch.float64).to(DT[dtype])
    return x[:, :H], x[:, H: H + Hkv]


def check(got, x, positions, freqs, dtype, **kw):
    ref, tol = R.rope(x.double().numpy(), positions, freqs.numpy(), **kw)
    got = got.double().cpu().numpy()
    err = np.abs(got - ref)
    rot = 2 * freqs.numel()
    # half a step: relative to the value, and below the type's smallest normal number relative to that one (steps stay 2^-24
    # below 2^-14 in fp16: 64-bit results rounded to fp16 are off by up to 2^-25 there)
    info = torch.finfo(DT[dtype])
    lim = tol + np.maximum(R.half_step(dtype) * (np.abs(ref) + tol), info.tiny * info.eps / 2)
    lim[..., rot:] = 0   # copied
    assert (err <= lim).all(), f"worst {np.max(err / np.maximum(lim, 1e-300))} of the tolerance"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,Hkv,D,rot", [
    (1, 8, 2, 64, 64), (3, 4, 4, 128, 128), (65, 32, 8, 128, 64), (7, 5, 1, 256, 96), (130, 3, 1, 512, 512), (2, 1, 1, 64, 2),
    (33, 6, 2, 128, 20), (5, 2, 2, 512, 34), (700, 2, 1, 64, 32), (1, 64, 8, 128, 128), (4, 12, 3, 256, 250),
])
def test_layouts_and_sizes(T, H, Hkv, D, rot, dtype, interleaved):
    q, k = data(T, H, Hkv, D, dtype, T + rot)
    pos = np.random.default_rng(rot).integers(0, 40000, T).astype(np.int32)
    freqs = qda.qdecode_rope_freqs(rot, 10000.0)
    qo, ko = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), torch.full(k.shape, 7.0, dtype=k.dtype, device="cuda")
    a, b = qda.qdecode_rope(q.cuda(), k.cuda(), torch.from_numpy(pos).cuda(), freqs.cuda(), qo, ko, interleaved, 1.25)
    assert a is qo and b is ko
    check(qo, q, pos, freqs, dtype, interleaved=interleaved, scale=1.25)
    check(ko, k, pos, freqs, dtype, interleaved=interleaved, scale=1.25)


@pytest.mark.parametrize("factor,context", [(1.0, 0), (8.0, 0), (8.0, 8192)])
def test_far_positions(factor, context):
    """fp32 outputs hold 2^-22 at the far end of the range, where an angle in fp32 would be nothing but noise."""
    pos = np.array([0, 1, 999_983, (1 << 24) + 1, (1 << 31) - 1], dtype=np.int32)
    freqs = qda.qdecode_rope_freqs(128, 500000.0, factor, context, 1.0, 4.0)
    q, k = data(5, 4, 2, 128, "fp32", 5)
    qo, ko = qda.qdecode_rope(q.contiguous().cuda(), k.contiguous().cuda(), torch.from_numpy(pos).cuda(), freqs.cuda())
    check(qo, q, pos, freqs, "fp32")
    check(ko, k, pos, freqs, "fp32")


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (24, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place_in_a_fused_projection(rot, interleaved, dtype):
    """Queries and keys rotated where they lie, as views of one row per token; values and unturned rows are untouched."""
    T, H, Hkv, D = 37, 6, 2, 128
    x = torch.randn(T, H + 2 * Hkv, D, generator=torch.Generator().manual_seed(3), dtype=torch.float64).to(DT[dtype])
    dev = x.cuda()
    pos = np.random.default_rng(1).integers(0, 9000, T).astype(np.int32)
    pos[-3:] = -1
    freqs = qda.qdecode_rope_freqs(rot)
    q, k = dev[:, :H], dev[:, H: H + Hkv]
    a, b = qda.qdecode_rope(q, k, torch.from_numpy(pos).cuda(), freqs.cuda(), interleaved=interleaved)
    assert a is q and b is k
    got = dev.cpu()
    check(got[:, :H], x[:, :H], pos, freqs, dtype, interleaved=interleaved)
    check(got[:, H: H + Hkv], x[:, H: H + Hkv], pos, freqs, dtype, interleaved=interleaved)
    assert torch.equal(got[:, H + Hkv:], x[:, H + Hkv:]) and torch.equal(got[-3:], x[-3:])


def test_one_tensor_other_strides_and_rows_behind_the_last_token():
    T, H, D = 9, 3, 64
    x = torch.randn(H, T, 2 * D, generator=torch.Generator().manual_seed(8))
    q = x.cuda().transpose(0, 1)[..., D:]                       # heads outside, every other row's worth of columns
    out = torch.full((T, 2 * H, D), 7.0, device="cuda")
    pos = np.array([5, 4, 3, 2, 1, 0, 70000, -1, -1], dtype=np.int32)
    freqs = qda.qdecode_rope_freqs(48)
    a, b = qda.qdecode_rope(q, None, torch.from_numpy(pos).cuda(), freqs.cuda(), q_out=out[:, ::2])
    assert b is None
    check(out[:7, ::2], q[:7].cpu(), pos[:7], freqs, "fp32")
    assert (out[7:] == 7).all() and (out[:, 1::2] == 7).all()
    ko = torch.full((T, H, D), 7.0, device="cuda")
    qda.qdecode_rope(None, q, torch.from_numpy(pos).cuda(), freqs.cuda(), k_out=ko)
    assert torch.equal(ko, out[:, ::2])


def test_shift_per_sequence():
    """Rows behind q_start[B] keep their position; the others' grow by their sequence's shift."""
    lens, shift = [3, 0, 5, 1], [100, 7, 0, 9000]
    T = sum(lens) + 2
    pos = np.arange(T, dtype=np.int32)
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    want = pos.copy()
    for b in range(4):
        want[start[b]: start[b + 1]] += shift[b]
    q, k = data(T, 4, 2, 128, "fp32", 2)
    freqs = qda.qdecode_rope_freqs(128)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    a, b = qda.qdecode_rope(q.contiguous().cuda(), k.contiguous().cuda(), i32(pos), freqs.cuda(), q_start=i32(start), shift=i32(shift))
    check(a, q, want, freqs, "fp32")
    check(b, k, want, freqs, "fp32")


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """d loss / d x for loss = sum(g y): turning g back, against differences of the call itself in fp32 (the call is linear, so
    a difference over any step is the derivative; products of 2^-22 relative error, 2 * 64 of them summed)."""
    T, D, rot = 4, 64, 32
    gen = torch.Generator().manual_seed(4)
    x, g, d = (torch.randn(T, 2, D, generator=gen).cuda() for _ in range(3))
    pos, freqs = torch.tensor([3, 77, 12345, 0], dtype=torch.int32).cuda(), qda.qdecode_rope_freqs(rot).cuda()
    kw = dict(interleaved=interleaved, scale=1.5)
    f = lambda v, **k: qda.qdecode_rope(v.contiguous(), None, pos, freqs, q_out=torch.empty_like(v), **kw, **k)[0]  # noqa: E731
    grad = f(g, inverse=True)
    lhs = (g.double() * (f(x + d).double() - f(x).double())).sum()
    rhs = (grad.double() * d.double()).sum()
    assert abs(lhs - rhs) <= T * 2 * D * 64 * 2.0 ** -22
    ref, tol = R.rope(g.double().cpu().numpy(), pos.cpu().numpy(), freqs.cpu().numpy(), inverse=True, **kw)
    assert (np.abs(grad.double().cpu().numpy() - ref) <= tol + 2.0 ** -24 * np.abs(ref)).all()


def test_graph_and_stream():
    T = 50
    q, k = (t.contiguous().cuda() for t in data(T, 8, 2, 128, "bf16", 9))
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), qda.qdecode_rope_freqs(128).cuda()
    want = qda.qdecode_rope(q, k, pos, freqs, torch.empty_like(q), torch.empty_like(k))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q), torch.zeros_like(k)
    qda.qdecode_rope(q, k, pos, freqs, *out, stream=s)
    s.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qda.qdecode_rope(q, k, pos, freqs, *out)
    pos.add_(11)
    g.replay()
    want = qda.qdecode_rope(q, k, pos, freqs, torch.empty_like(q), torch.empty_like(k))
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_outputs_whose_tokens_and_heads_interleave():
    """Rows that lie apart without a token's heads, or a head's tokens, lying together."""
    T, H, D = 4, 3, 64
    q, _ = data(T, H, 1, D, "bf16", 9)
    pos, freqs = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda"), qda.qdecode_rope_freqs(D)
    for ts, hs in ((3 * D, 4 * D), (D, T * D), (H * D, D), (2 * D, 2 * D * T + 3 * D)):
        buf = torch.full((40 * D,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf.as_strided((T, H, D), (ts, hs, 1))
        qda.qdecode_rope(q.cuda(), None, pos, freqs.cuda(), out)
        check(out, q, pos.cpu().numpy(), freqs, "bf16")
        rest = torch.ones(40, dtype=torch.bool)
        rest[[(t * ts + h * hs) // D for t in range(T) for h in range(H)]] = False
        assert (buf.view(40, D)[rest.cuda()] == 7).all()


def test_strides_of_a_single_token_or_head_mean_nothing():
    """In place: one token whose output has another token stride, one head whose output has another head stride."""
    for T, H, other in ((1, 8, (8192, 128, 1)), (5, 1, (1024, 4096, 1))):
        q, _ = data(T, H, 1, 128, "bf16", T)
        x = torch.zeros(T, 8, 128, dtype=torch.bfloat16, device="cuda")
        x[:, :H] = q
        pos, freqs = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda"), qda.qdecode_rope_freqs(128)
        qda.qdecode_rope(x[:, :H], None, pos, freqs.cuda(), x[:, :H].as_strided((T, H, 128), other))
        check(x[:, :H], q, pos.cpu().numpy(), freqs, "bf16")
        assert not x[:, H:].any()
