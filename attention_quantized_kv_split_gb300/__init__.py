"""Quantized-KV single-query decode attention for GB300 (sm_103a).

The work happens in libqdecode_attn.so (hand-written CUDA behind a C ABI, include/qdecode_attn.h). This module
only marshals torch tensors (device memory and streams) into that ABI, under the same names.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import (QDA_BF16, QDA_FP16, QDA_FP32, QdaError, QdaPlan, lib)  # noqa: F401

_DT_CODE = {torch.bfloat16: QDA_BF16, torch.float16: QDA_FP16, torch.float32: QDA_FP32}
_CODE_DT = {v: k for k, v in _DT_CODE.items()}


def dtype_code(in_dtype: torch.dtype, out_dtype: Optional[torch.dtype] = None) -> int:
    """The ABI's dtype argument: input dtype in the low byte, output dtype in the next."""
    return _DT_CODE[in_dtype] | ((_DT_CODE[out_dtype] if out_dtype is not None else 0) << 8)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream, device):
    """Context in which torch allocates (and copies) on ``stream``: memory that a call on another stream than torch's
    current one writes must come from that stream's share of torch's allocator, which may otherwise hand out a block that
    work on the current stream still uses, or give this one away while the call is under way."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):   # a handle; 0 and 1 name the default stream
        stream = torch.cuda.default_stream(device) if int(stream) in (0, 1) else torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def qdecode_attn(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                 v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                 N: Sequence[int], Hkv: int, GS: int, bits: int, stream=None) -> torch.Tensor:
    """out[b, h] = softmax(q[b, h] . K_hat[b, h // (H/Hkv)]^T / sqrt(D)) V_hat[...] from the packed cache.

    q ``[B, H, D]`` bf16/fp16; packed ``[Hkv * sum(N), D*bits/32]`` int32/uint32 (sequences back to back, each
    ``[Hkv, N[b], .]``); scales/biases ``[Hkv * sum(N), D/GS]`` in q's dtype; out ``[B, H, D]`` (bf16, fp16 or
    fp32). Asynchronous on ``stream`` (default: torch's current stream).
    """
    B, H, D = q.shape
    n = _lib.int32_array(N)
    st = lib().qdecode_attn(_ptr(q), _ptr(k_packed), _ptr(k_scales), _ptr(k_biases), _ptr(v_packed),
                            _ptr(v_scales), _ptr(v_biases), _ptr(out), B, H, Hkv, n, D, GS, bits,
                            dtype_code(q.dtype, out.dtype), _stream(stream))
    _lib.check(st, "qdecode_attn")
    return out


def qdecode_attn_noalloc(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                         v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                         N: Sequence[int], Hkv: int, GS: int, bits: int, stream=None) -> torch.Tensor:
    """qdecode_attn for callers that must not allocate device memory: the library's fixed scratch array is used
    instead of a workspace (shapes needing more than QDA_STATIC_SCRATCH_BYTES are rejected). Calls that overlap
    on the GPU share that array and must be serialised by the caller."""
    B, H, D = q.shape
    st = lib().qdecode_attn_noalloc(_ptr(q), _ptr(k_packed), _ptr(k_scales), _ptr(k_biases), _ptr(v_packed),
                                    _ptr(v_scales), _ptr(v_biases), _ptr(out), B, H, Hkv, _lib.int32_array(N), D,
                                    GS, bits, dtype_code(q.dtype, out.dtype), _stream(stream))
    _lib.check(st, "qdecode_attn_noalloc")
    return out


def qdecode_attn_host(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                      v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                      N: Sequence[int], Hkv: int, GS: int, bits: int, stream=None) -> torch.Tensor:
    """qdecode_attn with every tensor in HOST memory (contiguous CPU tensors; pinned ones copy at full speed): the
    library stages the inputs on the current device, decodes and copies out back, asynchronously on `stream`.
    Synchronise the stream before reading out or changing the inputs."""
    ts = (q, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, out)
    if any(t.is_cuda or not t.is_contiguous() for t in ts):
        raise ValueError("qdecode_attn_host takes contiguous host tensors")
    B, H, D = q.shape
    st = lib().qdecode_attn_host(*(_ptr(t) for t in ts), B, H, Hkv, _lib.int32_array(N), D, GS, bits,
                                 dtype_code(q.dtype, out.dtype), _stream(stream))
    _lib.check(st, "qdecode_attn_host")
    return out


def qdecode_attn_compat(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                        v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                        N: Sequence[int], Hkv: int, GS: int, bits: int, stream=None) -> torch.Tensor:
    """qdecode_attn in the two-pass form with compat rounding: scores and normalised probabilities rounded to the
    input dtype, the probability-weighted V rows summed without renormalising."""
    B, H, D = q.shape
    st = lib().qdecode_attn_compat(_ptr(q), _ptr(k_packed), _ptr(k_scales), _ptr(k_biases), _ptr(v_packed),
                                   _ptr(v_scales), _ptr(v_biases), _ptr(out), B, H, Hkv, _lib.int32_array(N), D,
                                   GS, bits, dtype_code(q.dtype, out.dtype), _stream(stream))
    _lib.check(st, "qdecode_attn_compat")
    return out


def qdecode_attn_multi(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                       v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                       N: Sequence[int], Hkv: int, GS: int, bits: int, stream=None) -> torch.Tensor:
    """Small-L multi-query decode: q and out ``[B, L, H, D]``; the L positions are each sequence's last L tokens
    (already the last L rows of its cache, counted in N), and position l attends the first N[b] - L + 1 + l
    rows. Cache arguments as for qdecode_attn."""
    B, L, H, D = q.shape
    st = lib().qdecode_attn_multi(_ptr(q), _ptr(k_packed), _ptr(k_scales), _ptr(k_biases), _ptr(v_packed),
                                  _ptr(v_scales), _ptr(v_biases), _ptr(out), B, L, H, Hkv, _lib.int32_array(N), D,
                                  GS, bits, dtype_code(q.dtype, out.dtype), _stream(stream))
    _lib.check(st, "qdecode_attn_multi")
    return out


def bind_qdecode_attn(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                      v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                      N: Sequence[int], Hkv: int, GS: int, bits: int, stream=None):
    """qdecode_attn with every argument marshalled once: returns a no-argument callable for repeated calls on
    the same buffers (decode loops, timing)."""
    B, H, D = q.shape
    args = (_ptr(q), _ptr(k_packed), _ptr(k_scales), _ptr(k_biases), _ptr(v_packed), _ptr(v_scales),
            _ptr(v_biases), _ptr(out), B, H, Hkv, _lib.int32_array(N), D, GS, bits, dtype_code(q.dtype, out.dtype),
            _stream(stream))
    fn = lib().qdecode_attn

    def call():
        st = fn(*args)
        if st:
            raise _lib.QdaError(st, "qdecode_attn")
    call.keepalive = (q, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, out)
    return call


def qdecode_attn_plan(B: int, H: int, Hkv: int, N: Sequence[int], D: int, GS: int, bits: int, num_sms: int = 0,
                      ctas_per_sm: int = 0) -> dict:
    plan = QdaPlan()
    st = lib().qdecode_attn_plan(B, H, Hkv, _lib.int32_array(N), D, GS, bits, num_sms, ctas_per_sm,
                                 ctypes.byref(plan))
    _lib.check(st, "qdecode_attn_plan")
    return plan.as_dict()


def qdecode_attn_multi_plan(B: int, L: int, H: int, Hkv: int, N: Sequence[int], D: int, GS: int, bits: int,
                            num_sms: int = 0, ctas_per_sm: int = 0) -> dict:
    plan = QdaPlan()
    st = lib().qdecode_attn_multi_plan(B, L, H, Hkv, _lib.int32_array(N), D, GS, bits, num_sms, ctas_per_sm,
                                       ctypes.byref(plan))
    _lib.check(st, "qdecode_attn_multi_plan")
    return plan.as_dict()


def qdecode_attn_workspace_bytes(B: int, H: int, Hkv: int, N: Sequence[int], D: int, GS: int, bits: int) -> int:
    out = ctypes.c_size_t()
    st = lib().qdecode_attn_workspace_bytes(B, H, Hkv, _lib.int32_array(N), D, GS, bits, ctypes.byref(out))
    _lib.check(st, "qdecode_attn_workspace_bytes")
    return out.value


def qdecode_attn_set_workspace(buf: Optional[torch.Tensor]) -> None:
    st = lib().qdecode_attn_set_workspace(_ptr(buf), 0 if buf is None else buf.numel() * buf.element_size())
    _lib.check(st, "qdecode_attn_set_workspace")


def qdecode_attn_debug_force_splits(num_ctas: int) -> None:
    _lib.check(lib().qdecode_attn_debug_force_splits(num_ctas), "qdecode_attn_debug_force_splits")


def qdecode_attn_debug_stall_chunk(chunk: int) -> None:
    """Testing aid: the first CTA's producer stops before its chunk ``chunk`` (-1: off); see the C header."""
    _lib.check(lib().qdecode_attn_debug_stall_chunk(chunk), "qdecode_attn_debug_stall_chunk")


def qdecode_attn_set_split_event(event: Optional[torch.cuda.Event]) -> None:
    handle = None if event is None else event.cuda_event
    _lib.check(lib().qdecode_attn_set_split_event(handle), "qdecode_attn_set_split_event")


def qdecode_quantize(x: torch.Tensor, GS: int, bits: int, dtype: torch.dtype, packed: torch.Tensor,
                     scales: torch.Tensor, biases: torch.Tensor, stream=None) -> None:
    """Quantize fp32 rows ``x [rows, D]`` into ``packed [rows, D*bits/32]``, ``scales``/``biases [rows, D/GS]``
    (dtype bf16 or fp16). Writing into views offset to a cache's next rows appends to that cache."""
    rows, D = x.shape
    st = lib().qdecode_quantize(_ptr(x), rows, D, GS, bits, dtype_code(dtype), _ptr(packed), _ptr(scales),
                                _ptr(biases), _stream(stream))
    _lib.check(st, "qdecode_quantize")


def qdecode_qgemv(x: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor, w_biases: torch.Tensor,
                  y: torch.Tensor, GS: int, bits: int, stream=None) -> torch.Tensor:
    """y[t, n] = sum_k x[t, k] * (scale * code + bias)[n, k]: x ``[T, K]`` bf16/fp16, packed ``[N, K*bits/32]``,
    scales/biases ``[N, K/GS]`` in x's dtype, y ``[T, N]`` (bf16, fp16 or fp32)."""
    T, K = x.shape
    N = w_packed.shape[0]
    st = lib().qdecode_qgemv(_ptr(x), _ptr(w_packed), _ptr(w_scales), _ptr(w_biases), _ptr(y), T, N, K, GS, bits,
                             dtype_code(x.dtype, y.dtype), _stream(stream))
    _lib.check(st, "qdecode_qgemv")
    return y


def _paged_call(op: int, name: str, pack, dev: int, stream, args) -> None:
    """One paged call on device ``dev``: the arguments packed (one foreign-call argument instead of thirty), the stream
    given or the device's current one."""
    if dev < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    if dev == torch.cuda.current_device():
        st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
        st = lib().qdecode_paged_packed(op, pack(*args, st))
    else:
        with torch.cuda.device(dev):
            st = torch.cuda.current_stream().cuda_stream if stream is None else _stream(stream)
            st = lib().qdecode_paged_packed(op, pack(*args, st))
    if st:
        raise _lib.QdaError(st, name)


def _ints(dev: int, names: str, *tensors) -> None:
    """Every tensor given: int32, contiguous, on device ``dev``."""
    for i, t in enumerate(tensors):
        if t is not None and not (t.dtype is torch.int32 and t.is_contiguous() and t.get_device() == dev):
            raise ValueError(f"{names.split()[i]}: expected contiguous int32 on device {dev}, got {t.dtype} on {t.device}, "
                             f"strides {t.stride()}")


def _pool(dev, kp, ks, kb, vp, vs, vb, D, GS, bits):
    """num_pages, Hkv, page and dtype of a pool's six arrays: shapes, dtypes, device and contiguity checked."""
    shape, groups, dt = kp.shape, ks.shape, ks.dtype
    pages, Hkv, page, W = shape
    if GS < 1 or W * 32 != D * bits or vp.shape != shape or kp.element_size() != 4 or vp.element_size() != 4:
        raise ValueError(f"packed arrays {tuple(shape)} {kp.dtype}, {tuple(vp.shape)} {vp.dtype} do not hold {bits}-bit "
                         f"rows of {D} in 32-bit words")
    if not (groups == (pages, Hkv, page, D // GS) == kb.shape == vs.shape == vb.shape and kb.dtype is dt
            and vs.dtype is dt and vb.dtype is dt):
        raise ValueError(f"scales and biases must be [{pages}, {Hkv}, {page}, {D // GS}] of one dtype, got "
                         f"{[(tuple(t.shape), t.dtype) for t in (ks, kb, vs, vb)]}")
    for t in (kp, ks, kb, vp, vs, vb):
        if not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"the pool's arrays must be contiguous and on device {dev}")
    return pages, Hkv, page, dt


_PACK_MAP, _PACK_APPEND, _PACK_ATTN = (struct.Struct(f"={n}q").pack for n in (15, 24, 27))


def qdecode_paged_map(old_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                      page: int, q_start: torch.Tensor, kv_len: torch.Tensor, slots: torch.Tensor,
                      positions: Optional[torch.Tensor], used: torch.Tensor, stream=None) -> None:
    """One step's tables on the GPU (all int32): from ``old_len``, ``new_len [B]`` and ``free_pages [n_free]`` writes
    ``q_start [B + 1]``, ``kv_len [B]``, the new pages' entries of ``block_table [B, max_pages]``, ``slots`` and
    ``positions [max_tokens]`` (-1 behind the last token) and ``used [1]``, the pages that the step takes."""
    dev = old_len.get_device()
    _ints(dev, "old_len new_len block_table free_pages q_start kv_len slots positions used", old_len, new_len, block_table,
          free_pages, q_start, kv_len, slots, positions, used)
    B, max_pages = block_table.shape
    n = slots.numel()
    if not (old_len.numel() == new_len.numel() == kv_len.numel() == B and q_start.numel() == B + 1 and used.numel() >= 1):
        raise ValueError("old_len, new_len and kv_len hold B values, q_start B + 1")
    if positions is not None and positions.numel() < n:
        raise ValueError("positions holds fewer tokens than slots")
    _paged_call(0, "qdecode_paged_map", _PACK_MAP, dev, stream,
                (old_len.data_ptr(), new_len.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), q_start.data_ptr(),
                 kv_len.data_ptr(), slots.data_ptr(), 0 if positions is None else positions.data_ptr(), used.data_ptr(), B,
                 max_pages, free_pages.numel(), page, n))


def qdecode_paged_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_packed: torch.Tensor,
                         k_scales: torch.Tensor, k_biases: torch.Tensor, v_packed: torch.Tensor, v_scales: torch.Tensor,
                         v_biases: torch.Tensor, GS: int, bits: int, k_held: Optional[torch.Tensor] = None,
                         v_held: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantize new rows ``k``, ``v [T, Hkv, D]`` (bf16, fp16 or fp32; last dimension contiguous, other strides free)
    into the pool at ``slots [T]`` (int32; negative: skipped). ``k_held``, ``v_held [T, Hkv, D]`` in the cache dtype
    receive the values the cache now stands for."""
    shape, dev = k.shape, k.get_device()
    T, Hkv, D = shape
    pages, heads, page, dt = _pool(dev, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, D, GS, bits)
    if v.shape != shape or v.dtype is not k.dtype or v.get_device() != dev or heads != Hkv or slots.numel() != T:
        raise ValueError(f"k {tuple(shape)} {k.dtype}, v {tuple(v.shape)} {v.dtype} on {v.device}, {slots.numel()} slots "
                         f"and a pool of {heads} heads do not belong together")
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    if T and (kd != 1 or vd != 1):
        raise ValueError("rows of k and v must be contiguous")
    _ints(dev, "slots", slots)
    for t in (k_held, v_held):
        if t is not None and not (t.shape == shape and t.dtype is dt and t.is_contiguous() and t.get_device() == dev):
            raise ValueError(f"k_held and v_held must be contiguous {tuple(shape)} {dt} on the pool's device")
    _paged_call(1, "qdecode_paged_append", _PACK_APPEND, dev, stream,
                (k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), k_packed.data_ptr(), k_scales.data_ptr(),
                 k_biases.data_ptr(), v_packed.data_ptr(), v_scales.data_ptr(), v_biases.data_ptr(),
                 0 if k_held is None else k_held.data_ptr(), 0 if v_held is None else v_held.data_ptr(), T, Hkv, pages,
                 page, D, GS, bits, _DT_CODE[dt] | _DT_CODE[k.dtype] << 8))


def qdecode_paged_attn(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, k_biases: torch.Tensor,
                       v_packed: torch.Tensor, v_scales: torch.Tensor, v_biases: torch.Tensor, out: torch.Tensor,
                       q_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, max_q: int, GS: int,
                       bits: int, causal: bool = True, stream=None) -> torch.Tensor:
    """Attention of every sequence's new tokens over its pages: q ``[total_q, H, D]`` (rows contiguous), out the same
    shape, contiguous; ``q_start [B + 1]``, ``kv_len [B]``, ``block_table [B, max_pages]`` int32 on the GPU. ``max_q``
    bounds the new tokens of a sequence (it only chooses the kernel). ``causal=False`` is cross attention."""
    shape, dev = q.shape, q.get_device()
    T, H, D = shape
    pages, Hkv, page, dt = _pool(dev, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, D, GS, bits)
    B, max_pages = block_table.shape
    if not (q.dtype is dt and out.dtype is dt and out.shape == shape and out.is_contiguous() and out.get_device() == dev
            and kv_len.numel() == B and q_start.numel() == B + 1):
        raise ValueError(f"q {tuple(shape)} {q.dtype}, out {tuple(out.shape)} {out.dtype} on {out.device} (contiguous), "
                         f"{kv_len.numel()} lengths and {q_start.numel()} starts do not fit a {dt} cache of {B} sequences")
    qt, qh, qd = q.stride()
    if T and qd != 1:
        raise ValueError("rows of q must be contiguous")
    _ints(dev, "q_start kv_len block_table", q_start, kv_len, block_table)
    _paged_call(2, "qdecode_paged_attn", _PACK_ATTN, dev, stream,
                (q.data_ptr(), qt, qh, k_packed.data_ptr(), k_scales.data_ptr(), k_biases.data_ptr(), v_packed.data_ptr(),
                 v_scales.data_ptr(), v_biases.data_ptr(), out.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                 block_table.data_ptr(), T, max_q, B, H, Hkv, pages, page, max_pages, 1 if causal else 0, D, GS, bits,
                 _DT_CODE[dt]))
    return out


def qdecode_paged_attn_workspace_bytes(B: int, H: int, Hkv: int, max_q: int, D: int, GS: int, bits: int) -> int:
    out = ctypes.c_size_t()
    st = lib().qdecode_paged_attn_workspace_bytes(B, H, Hkv, max_q, D, GS, bits, ctypes.byref(out))
    _lib.check(st, "qdecode_paged_attn_workspace_bytes")
    return out.value


def qdecode_attn_device_status() -> int:
    flags = ctypes.c_uint()
    _lib.check(lib().qdecode_attn_device_status(ctypes.byref(flags)), "qdecode_attn_device_status")
    return flags.value


def qdecode_attn_calls() -> int:
    return lib().qdecode_attn_calls()


# ------------------------------------------------------------------------------------------- conveniences


class QuantizedKV:
    """A packed cache in the library's layout: sequences back to back, each ``[Hkv, N[b], .]``."""

    def __init__(self, packed_k, scales_k, biases_k, packed_v, scales_v, biases_v, N, Hkv, D, GS, bits):
        self.kp, self.ks, self.kb = packed_k, scales_k, biases_k
        self.vp, self.vs, self.vb = packed_v, scales_v, biases_v
        self.N, self.Hkv, self.D, self.GS, self.bits = list(N), Hkv, D, GS, bits

    @classmethod
    def empty(cls, N, Hkv, D, GS, bits, dtype, device="cuda"):
        rows = Hkv * sum(N)
        W, NG = D * bits // 32, D // GS
        mk = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        return cls(mk((rows, W), torch.int32), mk((rows, NG), dtype), mk((rows, NG), dtype),
                   mk((rows, W), torch.int32), mk((rows, NG), dtype), mk((rows, NG), dtype), N, Hkv, D, GS, bits)

    @property
    def dtype(self):
        return self.ks.dtype

    def unit_rows(self, b: int, kvh: int):
        r0 = self.Hkv * sum(self.N[:b]) + kvh * self.N[b]
        return r0, r0 + self.N[b]

    def quantize_into(self, b: int, kvh: int, K: torch.Tensor, V: torch.Tensor, row0: int = 0, stream=None):
        """Quantize fp32 K, V rows ``[n, D]`` into rows ``row0 .. row0 + n`` of KV head ``kvh`` of sequence b."""
        r0, r1 = self.unit_rows(b, kvh)
        a = r0 + row0
        e = a + K.shape[0]
        if e > r1:
            raise ValueError("rows past the end of this KV head")
        qdecode_quantize(K, self.GS, self.bits, self.dtype, self.kp[a:e], self.ks[a:e], self.kb[a:e], stream)
        qdecode_quantize(V, self.GS, self.bits, self.dtype, self.vp[a:e], self.vs[a:e], self.vb[a:e], stream)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.kp, self.ks, self.kb, self.vp, self.vs, self.vb))

    def append(self, K_new: torch.Tensor, V_new: torch.Tensor, out: "QuantizedKV" = None, stream=None) -> "QuantizedKV":
        """The cache with T new tokens per sequence (``K_new``, ``V_new`` fp32 ``[B, Hkv, T, D]``): every KV head's
        old rows, then the new rows quantized (qdecode_cache_append). Writes ``out`` (allocated when None)."""
        B, Hkv, T, D = K_new.shape
        with _on(stream, K_new.device):
            kn, vn = K_new.contiguous(), V_new.contiguous()
            if out is None:
                out = QuantizedKV.empty([n + T for n in self.N], self.Hkv, self.D, self.GS, self.bits, self.dtype,
                                        device=K_new.device)
        st = lib().qdecode_cache_append(
            _ptr(self.kp), _ptr(self.ks), _ptr(self.kb), _ptr(self.vp), _ptr(self.vs), _ptr(self.vb),
            _ptr(kn), _ptr(vn), _ptr(out.kp), _ptr(out.ks), _ptr(out.kb),
            _ptr(out.vp), _ptr(out.vs), _ptr(out.vb), B, Hkv, _lib.int32_array(self.N), T, D, self.GS, self.bits,
            dtype_code(self.dtype), _stream(stream))
        _lib.check(st, "qdecode_cache_append")
        return out


def bind_decode_attention(q: torch.Tensor, cache: QuantizedKV, out: torch.Tensor, stream=None):
    """Pre-marshalled decode_attention over a QuantizedKV (see bind_qdecode_attn)."""
    return bind_qdecode_attn(q, cache.kp, cache.ks, cache.kb, cache.vp, cache.vs, cache.vb, out, cache.N, cache.Hkv,
                             cache.GS, cache.bits, stream)


def decode_attention(q: torch.Tensor, cache: QuantizedKV, out_dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Allocating wrapper of qdecode_attn over a QuantizedKV."""
    if out is None:
        with _on(stream, q.device):
            out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    return qdecode_attn(q, cache.kp, cache.ks, cache.kb, cache.vp, cache.vs, cache.vb, out, cache.N, cache.Hkv,
                        cache.GS, cache.bits, stream)


class PagedKV:
    """A pool of pages in the library's layout, and the paged calls on it. Tables, lengths and the free list are the
    caller's (int32 tensors on the GPU); ``step_tables`` allocates one step's and fills them with qdecode_paged_map."""

    def __init__(self, num_pages, Hkv, page, D, GS, bits, dtype, device="cuda"):
        self.num_pages, self.Hkv, self.page, self.D, self.GS, self.bits = num_pages, Hkv, page, D, GS, bits
        mk = lambda last, dt: torch.zeros((num_pages, Hkv, page, last), dtype=dt, device=device)  # noqa: E731
        W, NG = D * bits // 32, D // GS
        self.kp, self.ks, self.kb = mk(W, torch.int32), mk(NG, dtype), mk(NG, dtype)
        self.vp, self.vs, self.vb = mk(W, torch.int32), mk(NG, dtype), mk(NG, dtype)

    @property
    def dtype(self):
        return self.ks.dtype

    def arrays(self):
        return self.kp, self.ks, self.kb, self.vp, self.vs, self.vb

    def step_tables(self, old_len, new_len, block_table, free_pages, max_tokens, stream=None) -> dict:
        """q_start, kv_len, slots, positions and used of a step (qdecode_paged_map; block_table is extended in place)."""
        B = block_table.shape[0]
        mk = lambda n: torch.empty(n, dtype=torch.int32, device=block_table.device)  # noqa: E731
        with _on(stream, block_table.device):
            t = {"q_start": mk(B + 1), "kv_len": mk(B), "slots": mk(max_tokens), "positions": mk(max_tokens), "used": mk(1)}
        qdecode_paged_map(old_len, new_len, block_table, free_pages, self.page, **t, stream=stream)
        return t

    def append(self, k, v, slots, k_held=None, v_held=None, stream=None) -> None:
        qdecode_paged_append(k, v, slots, *self.arrays(), self.GS, self.bits, k_held, v_held, stream)

    def attend(self, q, q_start, kv_len, block_table, max_q, causal=True, out=None, stream=None) -> torch.Tensor:
        """Allocating wrapper of qdecode_paged_attn (rows of q behind q_start[B] leave theirs unwritten)."""
        if out is None:
            with _on(stream, q.device):
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        return qdecode_paged_attn(q, *self.arrays(), out, q_start, kv_len, block_table, max_q, self.GS, self.bits, causal,
                                  stream)
