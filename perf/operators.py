"""The paged quantized KV cache's operators as a serving program uses them, for measurement: the step's block tables and
slot maps, the append of new keys and values, and attention over the pages (single tokens, chunks of a prompt, cross
attention). Every operator is here in its plain form (elementary torch operations in 32 bits) and as the framework's
call; `own` says which one run() takes."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- the cases


def _attn(name, B, H, Hkv, D, bits, GS, dtype, page, q, kv, causal=True, lens=1):
    # q, kv: inclusive ranges of a sequence's new tokens and of its keys (for causal attention the new ones among them)
    return {"name": name, "op": "attn", "B": B, "H": H, "Hkv": Hkv, "D": D, "bits": bits, "GS": GS, "dtype": dtype,
            "page": page, "q_lo": q[0], "q_hi": q[1], "kv_lo": kv[0], "kv_hi": kv[1], "causal": causal, "lens": lens}


def _append(name, B, Hkv, D, bits, GS, dtype, src, page, new, old, lens=1):
    return {"name": name, "op": "append", "B": B, "Hkv": Hkv, "D": D, "bits": bits, "GS": GS, "dtype": dtype, "src": src,
            "page": page, "new_lo": new[0], "new_hi": new[1], "old_lo": old[0], "old_hi": old[1], "lens": lens}


def _map(name, B, page, new, old, lens=1):
    return {"name": name, "op": "map", "B": B, "page": page, "new_lo": new[0], "new_hi": new[1], "old_lo": old[0],
            "old_hi": old[1], "lens": lens}


def listed():
    return [
        # one token of one short conversation: latency
        _attn("token_short", 1, 8, 2, 256, 4, 64, "bf16", 16, (1, 1), (512, 512)),
        # a serving batch, one token each, lengths as a running server holds them
        _attn("token_batch", 64, 32, 8, 128, 4, 64, "bf16", 64, (1, 1), (700, 8200)),
        # one token at the end of a very long document
        _attn("token_128k", 1, 16, 4, 256, 4, 32, "bf16", 64, (1, 1), (131072, 131072)),
        # a chunk of a long prompt: 2048 new tokens behind 30k earlier ones
        _attn("chunk_32k", 1, 32, 8, 128, 4, 64, "bf16", 64, (2048, 2048), (32768, 32768)),
        # chunks and single tokens in one batch, 8-bit codes, odd lengths
        _attn("chunk_mixed", 8, 16, 8, 256, 8, 32, "bf16", 32, (1, 1023), (1024, 9001), lens=4),
        # a chunk at the widest heads
        _attn("chunk_wide", 1, 16, 8, 512, 4, 128, "fp16", 32, (250, 250), (4097, 4097)),
        # decoder tokens attending an encoder's states of another length
        _attn("cross", 16, 16, 16, 64, 8, 32, "fp16", 16, (60, 333), (300, 1500), causal=False, lens=2),
        # one new token per sequence into the cache
        _append("append_tokens", 64, 8, 128, 4, 64, "bf16", "bf16", 64, (1, 1), (700, 8200)),
        # the prompts of a batch into the cache
        _append("append_prompts", 7, 8, 256, 8, 32, "bf16", "bf16", 32, (900, 4097), (0, 0), lens=3),
        # 32-bit rows of wide heads, 4-bit codes
        _append("append_wide", 3, 8, 512, 4, 128, "fp16", "fp32", 16, (333, 2000), (5, 100), lens=2),
        # the tables of one decode step of a batch
        _map("map_tokens", 64, 64, (1, 1), (700, 8200)),
        # the tables of a step that takes prompts and tokens of the largest batch
        _map("map_prompts", 512, 16, (1, 129), (0, 4000), lens=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_one(rng):
    D = rng.choice([64, 128, 256, 512])
    GS = rng.choice([g for g in (32, 64, 128) if g <= D])
    c = {"bits": rng.choice([4, 8]), "GS": GS, "dtype": rng.choice(["bf16", "fp16"]), "page": rng.choice([16, 32, 64, 128]),
         "lens": rng.randrange(1 << 20)}
    op = rng.choice(["attn", "attn", "attn", "append", "map"])
    if op == "map":
        B, new = _log(rng, 1, 512), _log(rng, 1, 2048)
        old = _log(rng, 1, 32768)
        return {"op": op, "B": B, "page": c["page"], "new_lo": 1, "new_hi": new, "old_lo": 0, "old_hi": old, "lens": c["lens"]}
    if op == "append":
        B, new = _log(rng, 1, 128), _log(rng, 1, 4096)
        return {"op": op, "B": B, "Hkv": rng.choice([1, 2, 4, 8]), "D": D, **c, "src": rng.choice([c["dtype"], c["dtype"], "fp32"]),
                "new_lo": 1, "new_hi": new, "old_lo": 0, "old_hi": _log(rng, 1, 4096)}
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "B": _log(rng, 1, 64), "H": Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), "Hkv": Hkv, "D": D, **c, "causal": True}
    kind = rng.choice(["token", "few", "chunk", "cross"])
    kv = _log(rng, 16, 65536)
    if kind == "token":
        q = (1, 1)
    elif kind == "few":
        q = (1, rng.randrange(2, 17))
    else:
        q = (1, _log(rng, 16, 2048))
        c["causal"] = kind != "cross"
    least = q[1] if c["causal"] else 1   # an encoder's states may be fewer than the tokens that attend them
    return {**c, "q_lo": q[0], "q_hi": q[1], "kv_lo": max(least, kv // 8), "kv_hi": max(least, kv)}


def draw(rng):
    """One more case: a serving step of any kind, no larger than the largest listed one of its operator."""
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0, "padded": 0})
        for k, v in (("bytes", w["bytes"]), ("flops", w["flops"]), ("padded", _padded(c))):
            m[k] = max(m[k], v)
    while True:
        c = _draw_one(rng)
        w = work(c)
        m = most[c["op"]]
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and _padded(c) <= m["padded"]:
            return c


def _lens(c, lo, hi, salt):
    r = random.Random(c["lens"] * 7 + salt)
    return [r.randint(lo, hi) for _ in range(c["B"])]


def _attn_lens(c):
    return _lens(c, c["q_lo"], c["q_hi"], 1), _lens(c, c["kv_lo"], c["kv_hi"], 2)


def _step_lens(c):
    return _lens(c, c["old_lo"], c["old_hi"], 3), _lens(c, c["new_lo"], c["new_hi"], 4)


def _padded(c):
    """Scores that a padded batch holds (what the plain form of attention costs in memory)."""
    if c["op"] != "attn":
        return 0
    q, kv = _attn_lens(c)
    return c["B"] * c["H"] * max(q) * max(kv)


def _pairs(q, kv, causal):
    if not causal:
        return q * kv
    first = kv - q + 1   # keys that the first new token sees
    return q * first + q * (q - 1) // 2


def work(case):
    c = case
    if c["op"] == "attn":
        q, kv = _attn_lens(c)
        row = c["D"] * c["bits"] // 8 + c["D"] // c["GS"] * 4   # codes, scales and biases of one key (or value)
        return {"bytes": 2 * 2 * sum(q) * c["H"] * c["D"] + 2 * sum(kv) * c["Hkv"] * row,
                "flops": 4 * c["D"] * c["H"] * sum(_pairs(a, b, c["causal"]) for a, b in zip(q, kv))}
    old, new = _step_lens(c)
    n = sum(new)
    if c["op"] == "append":
        out = c["D"] * c["bits"] // 8 + c["D"] // c["GS"] * 4 + c["D"] * 2   # codes, scales, biases, the values held
        return {"bytes": 2 * n * c["Hkv"] * (c["D"] * (4 if c["src"] == "fp32" else 2) + out) + 4 * n, "flops": 0}
    pages = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(old, new))
    return {"bytes": 4 * (2 * c["B"] + 2 * c["B"] + 1 + 2 * n + 2 * pages), "flops": 0}


# --------------------------------------------------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _tables(c, kv, g):
    """A pool with some pages to spare, the sequences' pages scattered over it, and each sequence's row of the table."""
    P = c["page"]
    need = [-(-n // P) for n in kv]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["B"], max(max(need), 1), dtype=torch.int32, device="cuda")
    n = torch.tensor(need, device="cuda")
    use = torch.arange(table.shape[1], device="cuda")[None] < n[:, None]
    table[use] = order[: sum(need)]
    return pool, order, table, use


def _codec(x, GS, bits, dtype):
    """Codes, scales and biases of rows x [..., D] in 32 bits: scale = (max - min) / (2^bits - 1) and bias = min, kept in
    dtype, code = round((x - bias) / scale)."""
    v = x.float().unflatten(-1, (-1, GS))
    lo, hi = v.amin(-1), v.amax(-1)
    top = torch.full_like(lo, 2 ** bits - 1)   # a tensor: by a number torch multiplies with its reciprocal
    s, b = ((hi - lo) / top).to(dtype), lo.to(dtype)
    code = torch.round((v - b.float()[..., None]) / s.float()[..., None]).clamp(0, 2 ** bits - 1)
    code = torch.where(s[..., None] == 0, torch.zeros_like(code), code)
    return code, s, b


def _pack(code, bits):
    per = 32 // bits
    w = code.flatten(-2).to(torch.int64).unflatten(-1, (-1, per))
    w = (w << (bits * torch.arange(per, device=w.device))).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _pool(c, pool, g):
    """A filled pool's six arrays: keys with a few strong channels, as attention heads have, and plain values."""
    shape = (pool, c["Hkv"], c["page"], c["D"])
    dt = DTYPES[c["dtype"]]
    out = []
    for strong in (True, False):
        x = torch.randn(shape, generator=g, device="cuda")
        if strong:
            x[..., :: max(1, c["D"] // 3)] *= 4
        code, s, b = _codec(x, c["GS"], c["bits"], dt)
        out += [_pack(code, c["bits"]), s, b]
        del x, code
    return out


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dt = DTYPES.get(c.get("dtype"))
    if c["op"] == "attn":
        q, kv = _attn_lens(c)
        pool, _, table, _ = _tables(c, kv, g)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        kp, ks, kb, vp, vs, vb = _pool(c, pool, g)
        qs = torch.randn(sum(q), c["H"], c["D"], generator=g, device="cuda").to(dt)
        start = [sum(q[:i]) for i in range(len(q) + 1)]
        return {"case": c, "q": qs, "kp": kp, "ks": ks, "kb": kb, "vp": vp, "vs": vs, "vb": vb, "table": table,
                "q_start": ints(start), "kv_len": ints(kv), "max_q": max(q), "max_kv": max(kv), "out": torch.empty_like(qs)}
    old, new = _step_lens(c)
    total = [a + b for a, b in zip(old, new)]
    pool, order, table, use = _tables(c, total, g)
    n = sum(new)
    old_t, new_t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (old, new))
    if c["op"] == "map":
        # the rows as the last step left them: pages of the old tokens only; the rest of the pool is free
        had = (old_t + c["page"] - 1) // c["page"]
        held = torch.arange(table.shape[1], device="cuda")[None] < had[:, None]
        free = torch.cat([table[use & ~held], order[int(use.sum()):]])
        free = free[torch.randperm(free.numel(), generator=g, device="cuda")]
        table = torch.where(held, table, torch.full_like(table, -1))
        z = lambda k: torch.full((k,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"case": c, "old": old_t, "new": new_t, "table": table, "free": free, "q_start": z(c["B"] + 1),
                "kv_len": z(c["B"]), "slots": z(n), "positions": z(n), "used": z(1)}
    seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), new_t.long())
    first = torch.cumsum(new_t.long(), 0) - new_t
    pos = torch.arange(n, device="cuda") - first[seq] + old_t[seq]
    slots = (table[seq, pos // c["page"]].long() * c["page"] + pos % c["page"]).to(torch.int32)
    src = DTYPES[c["src"]]
    # keys and values of a fused projection: views of one row per token
    kv = torch.randn(n, 2, c["Hkv"], c["D"], generator=g, device="cuda")
    kv[:, 0, :, :: max(1, c["D"] // 3)] *= 4
    kv = kv.to(src)
    NG, W = c["D"] // c["GS"], c["D"] * c["bits"] // 32
    rows = (pool, c["Hkv"], c["page"])
    st = {"case": c, "k": kv[:, 0], "v": kv[:, 1], "slots": slots}
    for x in "kv":
        st[x + "p"] = torch.zeros(*rows, W, dtype=torch.int32, device="cuda")
        st[x + "s"], st[x + "b"] = (torch.zeros(*rows, NG, dtype=dt, device="cuda") for _ in range(2))
        st[x + "_held"] = torch.empty(n, c["Hkv"], c["D"], dtype=dt, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------------- the plain forms


def _values(packed, s, b, c):
    """The rows that codes, scales and biases stand for, in 32 bits."""
    per = 32 // c["bits"]
    shift = c["bits"] * torch.arange(per, dtype=torch.int32, device=packed.device)
    code = ((packed[..., None] >> shift) & (2 ** c["bits"] - 1)).flatten(-2).float()
    return (code.unflatten(-1, (-1, c["GS"])) * s.float()[..., None] + b.float()[..., None]).flatten(-2)


def _plain_attn(st):
    c = st["case"]
    rows = st["table"].long()
    n = st["max_kv"]

    def gathered(p, s, b):   # [B, Hkv, keys, D]
        return _values(p[rows], s[rows], b[rows], c).transpose(1, 2).flatten(2, 3)[:, :, :n]

    K, V = gathered(st["kp"], st["ks"], st["kb"]), gathered(st["vp"], st["vs"], st["vb"])
    start, kv = st["q_start"].long(), st["kv_len"].long()
    q_len = start[1:] - start[:-1]
    i = torch.arange(st["max_q"], device="cuda")
    real = i[None] < q_len[:, None]                                             # [B, max_q]
    at = (start[:-1, None] + i[None]).clamp(max=max(st["q"].shape[0] - 1, 0))
    q = st["q"].float()[at].unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)  # [B, Hkv, rep, max_q, D]
    B, G, R, L, D = q.shape
    S = (q.reshape(B, G, R * L, D) @ K.transpose(2, 3)).view(B, G, R, L, -1) * (1 / math.sqrt(D))
    key = torch.arange(S.shape[-1], device="cuda")
    last = kv[:, None] - q_len[:, None] + i[None] if c["causal"] else (kv[:, None] - 1).expand(B, L)
    seen = key[None, None] <= torch.minimum(last, kv[:, None] - 1)[..., None]    # [B, L, keys]
    S = S.masked_fill_(~seen[:, None, None], -math.inf)
    top = S.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = S.sub_(top).exp_()
    total = e.sum(-1)
    o = (e.view(B, G, R * L, -1) @ V).view(B, G, R, L, D) / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, L, G * R, D)
    return o[real].to(st["q"].dtype)


def _plain_append(st):
    c = st["case"]
    page, row = (st["slots"].long() // c["page"]), st["slots"].long() % c["page"]
    out = {}
    for x in "kv":
        code, s, b = _codec(st[x], c["GS"], c["bits"], DTYPES[c["dtype"]])
        st[x + "p"][page, :, row], st[x + "s"][page, :, row], st[x + "b"][page, :, row] = _pack(code, c["bits"]), s, b
        out[x] = (code * s.float()[..., None] + b.float()[..., None]).flatten(-2).to(DTYPES[c["dtype"]])
        out[x + "_scales"], out[x + "_biases"] = st[x + "s"], st[x + "b"]
    return out


def _plain_map(st):
    P = st["case"]["page"]
    old, new = st["old"].long(), st["new"].long()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    start = torch.cat([zero, torch.cumsum(new, 0)])
    had, has = (old + P - 1) // P, (old + new + P - 1) // P
    take = torch.cat([zero, torch.cumsum(has - had, 0)])
    # every sequence's new pages, in order, from the head of the free list
    col = torch.arange(st["table"].shape[1], device="cuda")[None]
    fresh = (col >= had[:, None]) & (col < has[:, None])
    nth = (take[:-1, None] + col - had[:, None]).clamp(0, max(st["free"].numel() - 1, 0))
    table = torch.where(fresh, st["free"][nth], st["table"])
    t = torch.arange(st["slots"].numel(), device="cuda")
    seq = (torch.searchsorted(start, t, right=True) - 1).clamp(max=old.numel() - 1)
    pos = t - start[seq] + old[seq]
    slots = table[seq, pos // P].long() * P + pos % P
    ints = lambda v: v.to(torch.int32)  # noqa: E731
    return {"table": table, "q_start": ints(start), "kv_len": ints(old + new), "slots": ints(slots), "positions": ints(pos),
            "used": ints(take[-1:])}


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "append": _plain_append, "map": _plain_map}[op](st)
    import attention_quantized_kv_split_gb300 as qda
    c = st["case"]
    if op == "attn":
        return qda.qdecode_paged_attn(st["q"], st["kp"], st["ks"], st["kb"], st["vp"], st["vs"], st["vb"], st["out"],
                                      st["q_start"], st["kv_len"], st["table"], st["max_q"], c["GS"], c["bits"],
                                      causal=c["causal"])
    if op == "append":
        qda.qdecode_paged_append(st["k"], st["v"], st["slots"], st["kp"], st["ks"], st["kb"], st["vp"], st["vs"], st["vb"],
                                 c["GS"], c["bits"], k_held=st["k_held"], v_held=st["v_held"])
        return {"k": st["k_held"], "k_scales": st["ks"], "k_biases": st["kb"], "v": st["v_held"], "v_scales": st["vs"],
                "v_biases": st["vb"]}
    qda.qdecode_paged_map(st["old"], st["new"], st["table"], st["free"], c["page"], st["q_start"], st["kv_len"], st["slots"],
                          st["positions"], st["used"])
    return {"table": st["table"], "q_start": st["q_start"], "kv_len": st["kv_len"], "slots": st["slots"],
            "positions": st["positions"], "used": st["used"]}


# ------------------------------------------------------------------------------------------------- the definition, 64 bits


def _exact_rows(packed, s, b, bits, GS):
    """[rows, words] -> [rows, D] in 64 bits."""
    w = packed.long() & 0xFFFFFFFF
    cols = [(w >> (bits * j)) & (2 ** bits - 1) for j in range(32 // bits)]
    code = torch.stack(cols, -1).reshape(w.shape[0], -1).double()
    rep = lambda x: x.double().repeat_interleave(GS, dim=1)  # noqa: E731
    return code * rep(s) + rep(b)


def exact(case, seed):
    c = case
    if c["op"] == "map":
        return None
    st = prepare(case, seed)
    if c["op"] == "attn":
        q_len, kv = _attn_lens(c)
        H, G, D, P = c["H"], c["Hkv"], c["D"], c["page"]
        out, t0 = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0
        for b in range(c["B"]):
            n, L = kv[b], q_len[b]
            pages = st["table"][b, : -(-n // P)].long()
            for h in range(G):
                def rows(p, s, bi):
                    part = [x[pages, h].reshape(pages.numel() * P, -1)[:n] for x in (p, s, bi)]
                    return _exact_rows(*part, c["bits"], c["GS"])
                K, V = rows(st["kp"], st["ks"], st["kb"]), rows(st["vp"], st["vs"], st["vb"])
                for r in range(h * (H // G), (h + 1) * (H // G)):
                    x = st["q"][t0: t0 + L, r].double() @ K.T / math.sqrt(D)
                    if c["causal"]:
                        far = torch.arange(n, device="cuda")[None] - torch.arange(L, device="cuda")[:, None] > n - L
                        x[far] = -math.inf
                    out[t0: t0 + L, r] = torch.softmax(x, dim=-1) @ V
            t0 += L
        return out
    res = {}
    for x in "kv":
        v = st[x].double().reshape(-1, c["GS"])
        lo, span = v.min(1).values, v.max(1).values - v.min(1).values
        scale = span / (2 ** c["bits"] - 1)
        s, b = (y.float().to(DTYPES[c["dtype"]]).double() for y in (scale, lo))
        code = torch.clamp(torch.round((v - b[:, None]) / torch.where(s == 0, torch.ones_like(s), s)[:, None]), 0, 2 ** c["bits"] - 1)
        code[s == 0] = 0
        shape = st[x].shape
        res[x] = (code * s[:, None] + b[:, None]).reshape(shape)
        pools = []
        for y, like in ((scale, st[x + "s"]), (lo, st[x + "b"])):
            pool = torch.zeros(like.shape, dtype=torch.float64, device="cuda")
            y = y.reshape(shape[0], shape[1], -1)
            for h in range(shape[1]):
                pool[st["slots"].long() // c["page"], h, st["slots"].long() % c["page"]] = y[:, h]
            pools.append(pool)
        res[x + "_scales"], res[x + "_biases"] = pools
    return res
