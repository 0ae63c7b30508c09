"""A serving program over a cache that forgets: map, rotary, append, attention with its row sums, weights, eviction, step after
step, against a cache of 64-bit rows on the host that follows the same rules."""
import math

import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda

import forget_ref as R
from paged_ref import DT

pytestmark = pytest.mark.gpu


class Server:
    """Pool, tables and free list of a batch, as a program holds them."""

    def __init__(self, B, H, Hkv, D, bits, GS, dtype, page, pages, cols):
        self.B, self.H, self.Hkv, self.D, self.dt = B, H, Hkv, D, DT[dtype]
        self.pool = qda.PagedKV(pages, Hkv, page, D, GS, bits, self.dt, track=True)
        i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.i32 = i32
        self.table = i32(np.full((B, cols), -1))
        self.free = i32(np.random.default_rng(0).permutation(pages))
        self.len, self.shift = i32(np.zeros(B)), i32(np.zeros(B))
        self.freqs = qda.qdecode_rope_freqs(D, 10000.0, 2.0).cuda()

    def step(self, q, k, v, new, budget, limit, sinks, recent, decay=0.9, window=0):
        """One step for all layers' worth of one layer: returns what a test wants to see of it."""
        T, max_q = q.shape[0], int(max(new))
        t = self.pool.step_tables(self.len, self.i32(new), self.table, self.free, T)
        qda.qdecode_rope(q, k, t["positions"], self.freqs, q_start=t["q_start"], shift=self.shift)
        held = torch.empty(T, self.Hkv, self.D, dtype=self.dt, device="cuda"), torch.empty(T, self.Hkv, self.D, dtype=self.dt, device="cuda")
        self.pool.append(k, v, t["slots"], *held)
        lse = torch.empty(T, self.H, device="cuda")
        out = self.pool.attend(q, t["q_start"], t["kv_len"], self.table, max_q, lse=lse)
        self.pool.weigh(q, lse, t["q_start"], t["kv_len"], self.table, max_q, window, decay, self.shift)
        seen = {"table": self.table.clone(), "mass": self.pool.mass.clone(), "token": self.pool.token.clone(), "shift": self.shift.clone()}
        e = self.pool.evict(t["kv_len"], self.table, budget, limit, sinks, recent, self.shift)
        # the program's own list: pages taken leave the front, freed ones join behind
        self.free = torch.cat([self.free[int(t["used"]):], e["freed"][: int(e["n_freed"])]])
        self.len = e["new_len"]
        return {"out": out, "lse": lse, "held": held, "kv_len": t["kv_len"], **seen}


@pytest.mark.parametrize("H,Hkv,D,bits,GS,dtype,page", [(8, 2, 64, 8, 32, "fp16", 16), (4, 2, 128, 4, 64, "bf16", 32)])
def test_steps(H, Hkv, D, bits, GS, dtype, page):
    qda.qdecode_attn_device_status()
    B, budget, limit, sinks, recent, decay, window = 3, 96, 120, 2, 16, 0.9, 40
    s = Server(B, H, Hkv, D, bits, GS, dtype, page, 40, 16)
    rng = np.random.default_rng(7)
    u = torch.finfo(DT[dtype]).eps / 2
    # the host's cache: per sequence and KV head lists of (token, key, value, mass), rows in the order of the pool's
    cache = [[[] for _ in range(Hkv)] for _ in range(B)]
    seen = [0] * B
    for step, new in enumerate([[150, 7, 90], [1, 1, 1], [1, 130, 40], [3, 1, 0], [1, 1, 1], [60, 1, 100]]):
        T = sum(new)
        q, k, v = (torch.from_numpy(rng.standard_normal((T, h, D))).to(DT[dtype]).cuda() for h in (H, Hkv, Hkv))
        q0, k0 = q.double().cpu().numpy(), k.double().cpu().numpy()
        pos = np.concatenate([np.arange(seen[b], seen[b] + new[b]) for b in range(B)])
        got = s.step(q, k, v, new, budget, limit, sinks, recent, decay, window)
        for x, x0 in ((q, q0), (k, k0)):   # in place, by the tokens' true positions
            ref, tol = R.rope(x0, pos, s.freqs.cpu().numpy())
            assert (np.abs(x.double().cpu().numpy() - ref) <= tol + u * (np.abs(ref) + tol)).all()
        qr, out, lse = q.double().cpu().numpy(), got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
        kh, vh = (h.double().cpu().numpy() for h in got["held"])
        table, mass, token = (got[n].cpu().numpy() for n in ("table", "mass", "token"))
        at = 0
        for b in range(B):
            L = new[b]
            n = len(cache[b][0]) + L
            assert int(got["kv_len"][b]) == n and int(got["shift"][b]) == seen[b] + L - n
            idx = np.arange(n)
            pg, row = table[b][idx // page], idx % page
            for h in range(Hkv):
                rows = cache[b][h]
                rows += [[seen[b] + i, kh[at + i, h], vh[at + i, h], 0.0] for i in range(L)]
                if n == 0:
                    continue
                if L:
                    K, V = np.array([r[1] for r in rows]), np.array([r[2] for r in rows])
                    vis = idx[None] <= (n - L + np.arange(L))[:, None]
                    drawn, err = np.zeros(n), np.zeros(n)
                    for r in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                        x = qr[at: at + L, r]
                        sc = np.where(vis, x @ K.T / math.sqrt(D), -np.inf)
                        # held values are rounded once where the pool's are not: half a step of every key and value
                        ds = (u + 2.0 ** -11) * (np.abs(x) @ np.abs(K).T).max(1) / math.sqrt(D)
                        top = sc.max(1, keepdims=True)
                        z = np.exp(sc - top).sum(1)
                        assert (np.abs(lse[at: at + L, r] - (top[:, 0] + np.log(z))) <= ds + 2.0 ** -16).all()
                        p = np.exp(sc - top) / z[:, None]
                        lim = (3 * u + 2.0 ** -10 + np.expm1(2 * ds))[:, None] * (p @ np.abs(V) + np.abs(V).max() * u) + 1e-6
                        # (a weight multiplies a value's distance from its group's middle: at most the group's range)
                        span = np.abs(V).reshape(n, -1, GS).max(-1).repeat(GS, -1)
                        lim = np.maximum(lim, (3 * u + 2.0 ** -10 + np.expm1(2 * ds))[:, None] * (p @ span) + 1e-6)
                        assert (np.abs(out[at: at + L, r] - p @ V) <= lim).all()
                        w = slice(max(0, L - window), L)
                        drawn += p[w].sum(0)
                        err += (p[w] * np.expm1(2 * ds[w] + 2.0 ** -16)[:, None]).sum(0)
                    for i in range(n):
                        rows[i][3] = decay * rows[i][3] * (i < n - L) + drawn[i]
                    m = mass[pg, h, row]
                    want = np.array([r[3] for r in rows])
                    assert (np.abs(m - want) <= err + 2.0 ** -18 * want + 1e-9).all()
                    np.testing.assert_array_equal(token[pg, h, row], [r[0] for r in rows])
                # from here on the call's own masses: the rule decides by them, and near ties are its own
                for i in range(n):
                    rows[i][3] = float(mass[pg[i], h, row[i]])
                if n > limit:
                    safe = [r[0] < sinks or r[0] >= seen[b] + L - recent for r in rows]
                    kept = set(sorted(range(n), key=lambda i: (not safe[i], 0 if safe[i] else -rows[i][3], i))[:budget])
                    comes = iter([rows[i] for i in range(budget, n) if i in kept])
                    cache[b][h] = [rows[i] if i in kept else next(comes) for i in range(budget)]
            seen[b] += L
            at += L
        assert qda.qdecode_attn_device_status() == 0
        np.testing.assert_array_equal(s.len.cpu().numpy(), [len(c[0]) for c in cache])
        used = s.table.cpu().numpy()
        ids = np.concatenate([used[used >= 0], s.free.cpu().numpy()])
        assert sorted(ids) == list(range(40))   # every page is in one place


def test_a_decode_step_in_a_graph():
    """Sequences at their budget: a captured step of all calls, replayed, against the same steps made eagerly. The page that a
    step takes for its token is the one that it frees again."""
    B, H, Hkv, D, bits, GS, page, budget = 4, 8, 2, 128, 4, 64, 16, 64

    def start():
        s = Server(B, H, Hkv, D, bits, GS, "bf16", page, 30, 6)
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn(B * budget, H + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
        s.step(x[:, :H], x[:, H: H + Hkv], x[:, H + Hkv:], [budget] * B, budget, budget, 1, 8)
        return s

    def buffers(s):
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"x": torch.zeros(B, H + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda"), "out": torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"),
                "lse": torch.zeros(B, H, device="cuda"), "new": i32(B) + 1, "q_start": i32(B + 1), "kv_len": i32(B), "slots": i32(B),
                "positions": i32(B), "used": i32(1), "freed": i32(24), "n_freed": i32(1), "free": s.free[:B].clone(), "len": s.len.clone()}

    def step(s, f):
        p = s.pool
        qda.qdecode_paged_map(f["len"], f["new"], s.table, f["free"], page, f["q_start"], f["kv_len"], f["slots"], f["positions"], f["used"])
        q, k, v = f["x"][:, :H], f["x"][:, H: H + Hkv], f["x"][:, H + Hkv:]
        qda.qdecode_rope(q, k, f["positions"], s.freqs, q_start=f["q_start"], shift=s.shift)
        p.append(k, v, f["slots"])
        p.attend(q, f["q_start"], f["kv_len"], s.table, 1, out=f["out"], lse=f["lse"])
        p.weigh(q, f["lse"], f["q_start"], f["kv_len"], s.table, 1, 0, 0.9, s.shift)
        qda.qdecode_paged_evict(*p.arrays(), p.mass, p.token, f["kv_len"], f["len"], s.table, f["freed"], f["n_freed"], GS, bits, budget, None,
                                1, 8, s.shift)
        f["free"].copy_(f["freed"][:B])

    xs = torch.randn(6, B, H + 2 * Hkv, D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    qda.qdecode_attn_device_status()
    a = start()
    fa = buffers(a)
    eager = []
    for x in xs:
        fa["x"].copy_(x)
        step(a, fa)
        eager.append((fa["out"].clone(), fa["lse"].clone(), a.pool.mass.clone(), a.pool.token.clone(), a.shift.clone(), a.table.clone()))
    b = start()
    fb = buffers(b)
    fb["x"].copy_(xs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, fb)
    for x, want in zip(xs, eager):
        fb["x"].copy_(x)
        graph.replay()
        for got, w in zip((fb["out"], fb["lse"], b.pool.mass, b.pool.token, b.shift, b.table), want):
            assert torch.equal(got, w)
    assert eager[-1][4].tolist() == [6] * B and qda.qdecode_attn_device_status() == 0
