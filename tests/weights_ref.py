"""The accumulated weight in 64 bits with bounds that tell a key of 22 bits from one of 11: queries whose rows have one value
each, so that a score is one product.

A score's error, in units of mag = |q| (|scale| 2^bits + |bias|) / sqrt(D), where one value of a query is not zero: the kernel for
many rows holds a key in two fp16 operands (2^-22 of it, and 2^-39 of the most that the key can hold), which come from an fp32
product and one or two sums (2^-24 each); joining the operands' two products, 2^-23 (sums with zeros are exact); the softmax scale
2^-23, its product with the score 2^-24. In all less than 3 x 2^-22 of mag: 4 x 2^-22 is allowed. Few rows take the codes as they
are: a product of the scale, one of the bias and their sum, less than that. Queries of one value are held exactly by either.
With a second value in a row another 4 x 2^-22 for its products' sums, and what is said of a query's values far below its largest.

Of a weight exp(s - lse) in fp32: lse and its factor 2^-22 of |lse|, the exponential and its argument 2^-21. Of a sum of R weights:
a thread adds at most R / 4 of them one after the other (16 beside that where a chunk is not full), 8 sums join the threads."""
from __future__ import annotations

import numpy as np
import torch

import oracle as O
from paged_ref import DT, need


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).double().numpy()


class Keys:
    """One sequence: codes, scales and biases of n keys under Hkv heads, its new tokens' queries and masses from before."""

    def __init__(self, L, n, H, Hkv, D, bits, GS, dtype, page=16, seed=0):
        rng = np.random.default_rng(seed)
        self.L, self.n, self.H, self.Hkv, self.D, self.bits, self.GS, self.dtype, self.page = L, n, H, Hkv, D, bits, GS, dtype, page
        self.codes = rng.integers(0, 1 << bits, (Hkv, n, D))
        spread = rng.uniform(3, 8, (Hkv, n, D // GS))
        self.s = rounded(spread / ((1 << bits) - 1), dtype)
        self.b = rounded(-spread * rng.uniform(0.02, 0.5, spread.shape), dtype)   # (small ones: low bits beside high ones)
        wide = lambda a: np.repeat(a, GS, axis=-1)  # noqa: E731
        self.K = wide(self.s) * self.codes + wide(self.b)
        self.A = np.abs(wide(self.s)) * (1 << bits) + np.abs(wide(self.b))
        self.mass = rng.random((Hkv, n)).astype(np.float32)
        self.pages = rng.permutation(need(n, page) + 2)[: need(n, page)]
        self.q = np.zeros((L, H, D))
        self.rng = rng

    def one_value_rows(self, first):
        """Row i of a KV head, its queries one token after the other, has one value, at (first + i) modulo D."""
        rep = self.H // self.Hkv
        self.q[:] = 0
        t, h = np.meshgrid(np.arange(self.L), np.arange(self.H), indexing="ij")
        size = self.rng.uniform(1.5, 4.5, t.shape) * self.rng.choice([-1, 1], t.shape) * np.sqrt(self.D) / 2
        self.q[t, h, (first + t * rep + h % rep) % self.D] = rounded(size, self.dtype)
        return self

    def quiet_values(self, below, far):
        """Four rows of five have a value over keys that are 0 there, and one 2^-below of it over keys that bring the score back;
        the fifth has one value alone, 2^far times theirs, over keys that are 0."""
        rep, g = self.H // self.Hkv, self.GS
        t, h = np.meshgrid(np.arange(self.L), np.arange(self.H), indexing="ij")
        row = t * rep + h % rep
        loud = row % 5 == 0
        self.q[:] = 0
        self.q[t, h, (7 * row) % g] = rounded(self.rng.uniform(1, 2, t.shape), self.dtype) * np.where(loud, 2.0 ** far, 1.0)
        self.q[t, h, g + row % (self.D - g)] = rounded(self.rng.uniform(1, 2, t.shape), self.dtype) * np.where(loud, 0, 2.0 ** -below)
        self.codes[..., :g] = 0
        self.b[..., 0] = 0
        f = 2.0 ** below * np.sqrt(self.D) / 4
        self.s[..., 1:], self.b[..., 1:] = rounded(self.s[..., 1:] * f, self.dtype), rounded(self.b[..., 1:] * f, self.dtype)
        wide = lambda a: np.repeat(a, g, axis=-1)  # noqa: E731
        self.K = wide(self.s) * self.codes + wide(self.b)
        self.A = np.abs(wide(self.s)) * (1 << self.bits) + np.abs(wide(self.b))
        self.A[..., :g] = 0   # (their products are exact zeros)
        return self

    def products(self, q, K):
        """[H, L, n] of q [L, H, D] and K [Hkv, n, D]"""
        return np.swapaxes(q, 0, 1) @ np.repeat(np.swapaxes(K, 1, 2), self.H // self.Hkv, axis=0)

    def scores(self, K=None):
        """[H, L, n]"""
        K = self.K if K is None else K
        return self.products(self.q, K) / np.sqrt(self.D)

    def seen(self):
        return np.arange(self.n)[None] <= (self.n - self.L + np.arange(self.L))[:, None]

    def lse(self):
        """[L, H], as a call gets them: fp32."""
        s = np.where(self.seen(), self.scores(), -np.inf)
        top = s.max(-1)
        return (top + np.log(np.exp(s - top[..., None]).sum(-1))).T.astype(np.float32)

    def weights(self, K=None, decay=0.5, steps=4, q_off=0.0):
        """(mass, tolerance) [Hkv, n]; K: other keys than the definition's; steps: 2^-22ths of mag that a score may be off by;
        q_off: how far a query's values may be off, of its row's largest."""
        rep, lse = self.H // self.Hkv, self.lse().T.astype(np.float64)[:, :, None]
        p = np.where(self.seen(), np.exp(self.scores(K) - lse), 0.0)
        mag = self.products(np.abs(self.q), self.A) / np.sqrt(self.D)
        ds = steps * 2.0 ** -22 * mag + 2.0 ** -22 * np.abs(lse) + 2.0 ** -21
        if q_off:
            top = np.abs(self.q).max(-1, keepdims=True) * (self.q != 0)
            ds = ds + q_off * self.products(top, self.A) / np.sqrt(self.D)
        join = lambda x: x.reshape(self.Hkv, rep * self.L, self.n).sum(1)  # noqa: E731
        add = join(p)
        old = np.where(np.arange(self.n) < self.n - self.L, decay * self.mass.astype(np.float64), 0.0)
        R = rep * self.L
        return old + add, join(p * np.expm1(ds)) + (R / 4 + 24) * 2.0 ** -24 * add + 2.0 ** -22 * np.abs(old)

    def device(self):
        """(q, key arrays, lse, mass, q_start, kv_len, table) on the GPU."""
        pool, NG, W = len(self.pages) + 2, self.D // self.GS, self.D * self.bits // 32
        words = O.pack(self.codes.reshape(-1, self.D), self.bits).reshape(self.Hkv, self.n, W)
        arrays = [np.zeros((pool, self.Hkv, self.page, W), np.uint32), *(np.zeros((pool, self.Hkv, self.page, NG)) for _ in "sb")]
        mass = np.zeros((pool, self.Hkv, self.page), np.float32)
        pg, row = self.where()
        for a, x in zip((*arrays, mass), (words, self.s, self.b, self.mass)):
            a[pg, :, row] = np.swapaxes(x, 0, 1)
        dt = DT[self.dtype]
        i32 = lambda a: torch.from_numpy(np.array(a, dtype=np.int32)).cuda()  # noqa: E731
        return (torch.from_numpy(self.q).to(dt).cuda(),
                [torch.from_numpy(arrays[0].view(np.int32)).cuda(), *(torch.from_numpy(a).to(dt).cuda() for a in arrays[1:])],
                torch.from_numpy(np.ascontiguousarray(self.lse())).cuda(), torch.from_numpy(mass).cuda(), i32([0, self.L]),
                i32([self.n]), i32(self.pages[None]))

    def where(self):
        key = np.arange(self.n)
        return self.pages[key // self.page], key % self.page

    def of_pool(self, mass):
        """[Hkv, n] of a pool's masses."""
        pg, row = self.where()
        return np.swapaxes(mass[pg, :, row], 0, 1)


def fewer_bits(K, dims=slice(None)):
    """Keys whose values in `dims` are rounded once to 11 significant bits."""
    m, e = np.frexp(K)
    out = K.copy()
    out[..., dims] = np.ldexp(np.rint(m * 2048) / 2048, e)[..., dims]
    return out
