"""Plain 64-bit implementations of the calls behind a cache that forgets: rotary positions, accumulated attention weight,
eviction; with the tolerances of the first two, derived beside them."""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_ref import DT


def rope(x, positions, freqs, interleaved=False, scale=1.0, inverse=False):
    """x [T, heads, D] in 64 bits turned by positions [T] * freqs [rot / 2]; rows of negative positions as they are.
    Returns (values, tolerance before the rounding to the output type).

    An angle is kept in turns, rounded to fp32 below half a turn (2^-25 of a turn, pi 2^-24 radians), from a frequency with
    2^-52 of relative error; a sine or cosine is right to 2^-23 beside that, the scale, its product and the two products and
    the sum of the rotation add at most 2^-22 of (|a| + |b|) scale together."""
    x = np.asarray(x, dtype=np.float64)
    r = 2 * len(freqs)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs)[None]
    c, s = np.cos(ang)[:, None], np.sin(-ang if inverse else ang)[:, None]
    out, tol = x.copy(), np.zeros_like(x)
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = scale * (a * c - b * s), scale * (b * c + a * s)
    off = abs(scale) * (np.abs(a) + np.abs(b)) * (math.pi * 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -22 + np.abs(ang)[:, None] * 2.0 ** -52)
    tol[..., ia] = tol[..., ib] = off
    keep = np.asarray(positions) < 0
    out[keep], tol[keep] = x[keep], 0
    return out, tol


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def scores(c, b, h, first=0):
    """Scores [L - first, n] of sequence b's new tokens from `first` on under query head h of a paged_ref.Case, a bound on the
    sum of the products' magnitudes, and which keys are seen."""
    n, L, kv = c.kv_lens[b], c.q_lens[b], h // (c.H // c.Hkv)
    q = c.q64[c.start[b] + first: c.start[b] + L, h]
    K = c.K[b][kv]
    s = q @ K.T / math.sqrt(c.D)
    # |q| (|scale code| + |bias|): a group's codes and bias enter the sum apart
    big = np.abs(K).reshape(n, -1, c.GS).max(-1)
    mag = (np.abs(q).reshape(len(q), -1, c.GS).sum(-1) @ (3 * big).T) / math.sqrt(c.D)
    seen = np.arange(n)[None] <= (n - L + np.arange(first, L))[:, None]
    return s, mag, seen


def log_sums(c):
    """lse [total, H] in 64 bits (-inf where a token sees no key)."""
    out = np.full((c.total, c.H), -np.inf)
    for b, L in enumerate(c.q_lens):
        for h in range(c.H if L and c.kv_lens[b] else 0):
            s, _, seen = scores(c, b, h)
            s = np.where(seen, s, -np.inf)
            top = s.max(1)
            ok = np.isfinite(top)
            e = np.exp(s[ok] - top[ok, None]).sum(1)
            out[c.start[b]: c.start[b] + L, h][ok] = top[ok] + np.log(e)
    return out


def weights(c, lse, mass, token, window=0, decay=1.0, shift=None):
    """(mass, token, tolerance) after qdecode_paged_weights, from mass [pool, Hkv, page] and lse as the call gets them.

    A score is a sum of exact products in fp32: D / 16 steps of the matrix instruction and a few more, each off by at most
    2^-22 of the largest partial sum, which the magnitudes bound; log-sum and its factor are rounded twice; the exponential
    and its argument are off by 2^-21 together; a sum of R terms by R 2^-24, the decayed mass by 2^-23."""
    mass, token = np.array(mass, dtype=np.float64), np.array(token)
    tol = np.zeros_like(mass)
    table = c.table.cpu().numpy()
    rep = c.H // c.Hkv
    for b, (L, n) in enumerate(zip(c.q_lens, c.kv_lens)):
        if L == 0 or n == 0:
            continue
        first = L - (min(window, L) if window else L)
        key = np.arange(n)
        pg, row = table[b][key // c.page], key % c.page
        for kv in range(c.Hkv):
            add, err, terms = np.zeros(n), np.zeros(n), 0
            for h in range(kv * rep, (kv + 1) * rep):
                s, mag, seen = scores(c, b, h, first)
                ls = lse[c.start[b] + first: c.start[b] + L, h].astype(np.float64)[:, None]
                with np.errstate(over="ignore", invalid="ignore"):
                    p = np.where(seen, np.exp(s - ls), 0.0)
                ds = (c.D / 16 + 16) * 2.0 ** -22 * mag + 2.0 ** -22 * np.abs(np.where(np.isfinite(ls), ls, 0)) + 2.0 ** -21
                add += p.sum(0)
                err += (p * np.expm1(ds)).sum(0)
                terms += len(s)
            old = np.where(key < n - L, decay * mass[pg, kv, row], 0.0)
            mass[pg, kv, row] = old + add
            tol[pg, kv, row] = err + (terms + 4) * 2.0 ** -24 * add + 2.0 ** -22 * np.abs(old) + 1e-30
            new = key >= n - L
            token[pg[new], kv, row[new]] = key[new] + (0 if shift is None else shift[b])
    return mass, token, tol


def evict(arrays, mass, token, kv_len, table, freed, page, budget, limit=None, sinks=0, recent=0, shift=None):
    """qdecode_paged_evict on the host: copies of (arrays, mass, token, new_len, table, freed, n_freed, shift), arrays any
    number of [pool, Hkv, page, .]."""
    arrays = [np.array(a) for a in arrays]
    mass, token, table, freed = np.array(mass), np.array(token), np.array(table), np.array(freed)
    new_len, shift = np.array(kv_len), None if shift is None else np.array(shift)
    limit, at = budget if limit is None else limit, 0
    cols = table.shape[1]
    for b, n in enumerate(kv_len):
        if n <= limit or n > cols * page:
            continue
        seen = n + (0 if shift is None else shift[b])
        idx = np.arange(n)
        pg, row = table[b][idx // page], idx % page
        for h in range(mass.shape[1]):
            m, t = mass[pg, h, row].astype(np.float64), token[pg, h, row]
            safe = (t < sinks) | (t >= seen - recent)
            rank = sorted(range(n), key=lambda i: (not safe[i], math.isnan(m[i]), 0.0 if safe[i] or math.isnan(m[i]) else -m[i], i))
            kept = set(rank[:budget])
            holes = [i for i in range(budget) if i not in kept]
            comes = [i for i in range(budget, n) if i in kept]
            assert len(holes) == len(comes)
            for a in (*arrays, mass, token):
                a[pg[holes], h, row[holes]] = a[pg[comes], h, row[comes]]
        for col in range(-(-budget // page), -(-n // page)):
            if at < len(freed):
                freed[at] = table[b, col]
            at += 1
            table[b, col] = -1
        new_len[b] = budget
        if shift is not None:
            shift[b] += n - budget
    return arrays, mass, token, new_len, table, freed, at, shift
