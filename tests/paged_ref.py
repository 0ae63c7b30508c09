"""Plain 64-bit implementations of the paged calls, and pools of pages for their tests.

Tolerance of the attention (derived, per output element): with weights p_n, values v_n and o = sum p_n v_n,
  * the output is rounded once: half a step, u |o| (u = finfo.eps / 2: bf16 2^-8, fp16 2^-11);
  * a weight is rounded once to the 16-bit type or better and multiplies either a value or its offset from the middle of
    its group, both at most A_n = max(|v_n|, half the group's range): u sum p_n A_n;
  * keys and values may be rounded to 11 significant bits: 2^-11 A_n for a value, and a score s = sum q k / sqrt(D) then
    moves by at most ds = 2^-11 max_n sum |q k| / sqrt(D), a normalised weight by a factor of at most e^(2 ds);
  * sums and exponentials in fp32, over at most 2^14 keys here: 2^-17 of sum p_n A_n covers them.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle as O
import attention_quantized_kv_split_gb300 as qda

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def need(n, page):
    return -(-n // page)


class Case:
    """A batch on a scattered pool: q, the device arrays, and each sequence's dequantised keys and values (64 bits)."""

    def __init__(self, q_lens, kv_lens, H, Hkv, D, bits, GS, dtype, page, seed=0, spare=2, q_scale=1.0, pad_rows=0,
                 unwritten=float("nan"), extra_cols=1):
        rng = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.H, self.Hkv, self.D = list(q_lens), list(kv_lens), H, Hkv, D
        self.bits, self.GS, self.dtype, self.page = bits, GS, dtype, page
        B, dt = len(q_lens), DT[dtype]
        pages = sum(need(n, page) for n in kv_lens)
        pool = pages + spare
        order = rng.permutation(pool)
        cols = max([need(n, page) for n in kv_lens] + [1]) + extra_cols
        table = np.full((B, cols), -1, dtype=np.int32)
        W, NG = D * bits // 32, D // GS
        packed = {x: rng.integers(0, 1 << 32, (pool, Hkv, page, W), dtype=np.uint64).astype(np.uint32) for x in "kv"}
        sc = {x: np.full((pool, Hkv, page, NG), unwritten) for x in ("ks", "kb", "vs", "vb")}
        self.K, self.V, self.A = [], [], []
        at = 0
        for b, n in enumerate(kv_lens):
            m = need(n, page)
            ids = order[at: at + m]
            at += m
            table[b, :m] = ids
            for x, vals in (("k", self.K), ("v", self.V)):
                rows = rng.standard_normal((Hkv * n, D)).astype(np.float32) if n else np.zeros((0, D), np.float32)
                if x == "k" and n:
                    rows[:, rng.integers(D)] *= 6
                codes, s, bi = O.quantize(rows, GS, bits, dtype) if n else (np.zeros((0, D), int),) + (np.zeros((0, NG)),) * 2
                words = O.pack(codes, bits) if n else np.zeros((0, W), np.uint32)
                for h in range(Hkv):
                    for j, pg in enumerate(ids):
                        k = min(page, n - j * page)
                        src = slice(h * n + j * page, h * n + j * page + k)
                        packed[x][pg, h, :k] = words[src]
                        sc[x + "s"][pg, h, :k], sc[x + "b"][pg, h, :k] = s[src], bi[src]
                deq = O.dequantize(codes, s, bi, GS) if n else np.zeros((0, D))
                vals.append(np.asarray(deq, dtype=np.float64).reshape(Hkv, n, D))
                if x == "v":
                    half = np.repeat(np.asarray(s, dtype=np.float64), GS, axis=-1) * (2 ** bits - 1) / 2
                    self.A.append(np.maximum(np.abs(self.V[-1]), half.reshape(Hkv, n, D)))
        self.total = sum(q_lens)
        q = torch.from_numpy(rng.standard_normal((self.total + pad_rows, H, D)) * q_scale).to(dt)
        self.q64 = q.double().numpy()
        self.q = q.cuda()
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        w = lambda a: torch.from_numpy(a.view(np.int32)).cuda()  # noqa: E731
        h = lambda a: torch.from_numpy(a).to(dt).cuda()  # noqa: E731
        self.arrays = [w(packed["k"]), h(sc["ks"]), h(sc["kb"]), w(packed["v"]), h(sc["vs"]), h(sc["vb"])]
        self.table = i32(table)
        self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int64)
        self.q_start, self.kv_len = i32(self.start), i32(kv_lens)

    def run(self, causal=True, max_q=None, out=None, stream=None, q=None):
        q = self.q if q is None else q
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
        return qda.qdecode_paged_attn(q, *self.arrays, out, self.q_start, self.kv_len, self.table,
                                      max_q or max(max(self.q_lens), 1), self.GS, self.bits, causal, stream)

    def reference(self, causal=True, hidden=()):
        """(out, tolerance) [total, H, D] in 64 bits; hidden: (sequence, key) pairs that nobody sees."""
        return attention(self, causal, hidden)

    def check(self, got, causal=True, hidden=()):
        ref, tol = self.reference(causal, hidden)
        g = got[: self.total].double().cpu().numpy()
        assert np.isfinite(g).all()
        err = np.abs(g - ref)
        worst = (err / np.maximum(tol, 1e-300)).max() if err.size else 0.0
        assert (err <= tol).all(), f"worst error is {worst:.2f} of the tolerance"
        return worst


def attention(c, causal, hidden=()):
    u = torch.finfo(DT[c.dtype]).eps / 2
    out = np.zeros((c.total, c.H, c.D))
    tol = np.zeros_like(out)
    nrep = c.H // c.Hkv
    for b, (L, n) in enumerate(zip(c.q_lens, c.kv_lens)):
        if n == 0 or L == 0:
            continue
        key = np.arange(n)
        last = n - L + np.arange(L) if causal else np.full(L, n - 1)
        seen = key[None] <= last[:, None]
        for bb, k in hidden:
            if bb == b:
                seen[:, k] = False
        for h in range(c.H):
            q, K, V, A = c.q64[c.start[b]: c.start[b] + L, h], c.K[b][h // nrep], c.V[b][h // nrep], c.A[b][h // nrep]
            s = np.where(seen, q @ K.T / math.sqrt(c.D), -np.inf)
            any_ = seen.any(1)
            e = np.exp(s - np.where(any_, s.max(1), 0.0)[:, None])
            p = np.where(seen, e, 0.0) / np.where(any_, e.sum(1), 1.0)[:, None]
            o = p @ V
            ds = 2.0 ** -11 * np.where(seen, np.abs(q) @ np.abs(K).T, 0).max(1) / math.sqrt(c.D)
            rows = slice(c.start[b], c.start[b] + L)
            out[rows, h] = o
            tol[rows, h] = u * np.abs(o) + (u + 2.0 ** -11 + np.expm1(2 * ds)[:, None] + 2.0 ** -17) * (p @ A) + 1e-7
    return out, tol


def tables(old, new, table, free, page, max_tokens):
    """qdecode_paged_map on the host: (table, q_start, kv_len, slots, positions, used, whether anything lacked a page)."""
    table = np.array(table)
    B, cols = table.shape
    q_start, kv, taken, bad = [0], [], 0, False
    slots, positions = np.full(max_tokens, -1), np.full(max_tokens, -1)
    for b in range(B):
        bad |= old[b] < 0 or new[b] < 0
        o, n = max(old[b], 0), max(new[b], 0)
        page_of = {c: table[b, c] for c in range(min(need(o, page), cols))}
        for c in range(need(o, page), need(o + n, page)):
            pid = free[taken] if taken < len(free) else -1
            taken += 1
            page_of[c] = pid
            if c < cols:
                table[b, c] = pid
            bad |= pid < 0 or c >= cols
        for i in range(n):
            t, at = q_start[-1] + i, o + i
            pid = page_of.get(at // page, -1) if at // page < cols else -1
            bad |= pid < 0 or t >= max_tokens
            if t < max_tokens:
                positions[t] = at
                slots[t] = pid * page + at % page if pid >= 0 else -1
        q_start.append(q_start[-1] + n)
        kv.append(o + n)
    return table, np.array(q_start), np.array(kv), slots, positions, taken, bad
