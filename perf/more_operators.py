"""A cache that forgets, as a serving program uses it, for measurement: rotary positions for the new tokens' queries and keys,
the attention weight that every cached key has drawn, and the eviction of the keys that drew least. Every operator is here in
its plain form (elementary torch operations) and as the framework's call; `own` says which one run() takes."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- the cases


def _rope(name, B, H, Hkv, D, rot, dtype, new, at, interleaved=False, base=1e4, factor=1.0, ramp=False, inverse=False, lens=1):
    # at: inclusive range of a sequence's first position; factor: how far the context is stretched, `ramp`: slow pairs only
    return {"name": name, "op": "rope", "B": B, "H": H, "Hkv": Hkv, "D": D, "rot": rot, "dtype": dtype, "new_lo": new[0],
            "new_hi": new[1], "at_lo": at[0], "at_hi": at[1], "interleaved": interleaved, "base": base, "factor": factor,
            "ramp": ramp, "inverse": inverse, "lens": lens}


def _weights(name, B, H, Hkv, D, bits, GS, dtype, page, q, kv, window=0, decay=1.0, lens=1):
    # q, kv: inclusive ranges of a sequence's new tokens and of its keys, the new ones among them
    return {"name": name, "op": "weights", "B": B, "H": H, "Hkv": Hkv, "D": D, "bits": bits, "GS": GS, "dtype": dtype,
            "page": page, "q_lo": q[0], "q_hi": q[1], "kv_lo": kv[0], "kv_hi": kv[1], "window": window, "decay": decay,
            "lens": lens}


def _evict(name, B, Hkv, D, bits, GS, dtype, page, kv, budget, limit, sinks, recent, fresh, lens=1):
    # kv: inclusive range of a sequence's rows; fresh: rows stand in the order of their tokens (nothing was evicted before)
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "D": D, "bits": bits, "GS": GS, "dtype": dtype, "page": page,
            "kv_lo": kv[0], "kv_hi": kv[1], "budget": budget, "limit": limit, "sinks": sinks, "recent": recent, "fresh": fresh,
            "lens": lens}


def listed():
    return [
        # one new token of every sequence of a serving batch: latency
        _rope("rope_tokens", 64, 32, 8, 128, 128, "bf16", (1, 1), (700, 8200)),
        # a chunk of a long prompt, the context stretched eightfold over the slow pairs
        _rope("rope_chunk", 1, 32, 8, 128, 128, "bf16", (2048, 2048), (28672, 28672), base=5e5, factor=8.0, ramp=True),
        # the prompts of a batch, interleaved pairs in a quarter of a wide head
        _rope("rope_prompts", 7, 16, 8, 256, 64, "fp16", (900, 4097), (0, 0), interleaved=True, lens=3),
        # gradients in 32 bits through whole wide heads at far positions
        _rope("rope_grad", 3, 16, 8, 512, 512, "fp32", (333, 1100), (900000, 1100000), factor=4.0, inverse=True, lens=2),
        # one token of one short conversation: latency
        _weights("weights_short", 1, 8, 2, 256, 4, 64, "bf16", 16, (1, 1), (512, 512)),
        # a serving batch, one token each, lengths as a running server holds them, old weight fading
        _weights("weights_batch", 64, 32, 8, 128, 4, 64, "bf16", 64, (1, 1), (700, 8200), decay=0.99),
        # one token at the end of a very long document
        _weights("weights_128k", 1, 16, 4, 256, 4, 32, "bf16", 64, (1, 1), (131072, 131072)),
        # the last 64 tokens of a long prompt judge all of its keys
        _weights("weights_window", 1, 32, 8, 128, 4, 64, "bf16", 64, (2048, 2048), (32768, 32768), window=64),
        # every token of a batch's chunks counts, 8-bit codes, odd lengths
        _weights("weights_chunks", 8, 16, 8, 256, 8, 32, "fp16", 32, (1, 1023), (1024, 9001), lens=4),
        # a step of a full batch: each sequence holds one row more than its budget
        _evict("evict_step", 64, 8, 128, 4, 64, "bf16", 64, (2049, 2049), 2048, 2048, 4, 256, False),
        # a long prompt cut to an eighth
        _evict("evict_prompt", 1, 8, 128, 4, 64, "bf16", 64, (32768, 32768), 4096, 4096, 4, 64, True),
        # a batch of which the long sequences are cut, wide rows of 8-bit codes, odd lengths
        _evict("evict_ragged", 16, 8, 256, 8, 32, "fp16", 32, (300, 9001), 1024, 1500, 1, 100, False, lens=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_one(rng):
    op = rng.choice(["rope", "weights", "weights", "evict"])
    D = rng.choice([64, 128, 256, 512])
    GS = rng.choice([g for g in (32, 64, 128) if g <= D])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    lens = rng.randrange(1 << 20)
    if op == "rope":
        new, at = _log(rng, 1, 4096), _log(rng, 1, 1 << 20)
        c = _rope("", _log(rng, 1, 128), H, Hkv, D, D // rng.choice([1, 1, 2, 4]), rng.choice(["bf16", "fp16", "fp32"]), (1, new),
                  (at // 2, at), rng.choice([False, True]), rng.choice([1e4, 5e5]), rng.choice([1.0, 2.5, 8.0]),
                  rng.choice([False, True]), rng.choice([False, False, True]), lens)
    elif op == "weights":
        kv, kind = _log(rng, 16, 65536), rng.choice(["token", "few", "window", "chunk"])
        q = (1, 1) if kind == "token" else (1, rng.randrange(2, 17)) if kind == "few" else (1, _log(rng, 16, 2048))
        c = _weights("", _log(rng, 1, 64), H, Hkv, D, rng.choice([4, 8]), GS, rng.choice(["bf16", "fp16"]),
                     rng.choice([16, 32, 64, 128]), q, (max(q[1], kv // 8), max(q[1], kv)),
                     rng.randrange(1, 100) if kind == "window" else 0, rng.choice([1.0, 0.9]), lens)
    else:
        budget = _log(rng, 16, 8192)
        over = _log(rng, 1, 8 * budget)
        sinks = rng.randrange(0, 9)
        recent = rng.randrange(0, budget - sinks + 1)
        c = _evict("", _log(rng, 1, 64), Hkv, D, rng.choice([4, 8]), GS, rng.choice(["bf16", "fp16"]), rng.choice([16, 32, 64, 128]),
                   (budget // 2 + 1, budget + over), budget, budget + rng.choice([0, over // 4]), sinks, recent,
                   rng.choice([False, True]), lens)
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    """One more case: a serving step of any kind, no larger than the largest listed one of its operator."""
    most = {}
    for c in listed():
        m = most.setdefault(c["op"], {})
        for k, v in _size(c).items():
            m[k] = max(m.get(k, 0), v)
    while True:
        c = _draw_one(rng)
        if all(v <= most[c["op"]][k] for k, v in _size(c).items()):
            return c


def _lens(c, lo, hi, salt):
    r = random.Random(c["lens"] * 7 + salt)
    return [r.randint(lo, hi) for _ in range(c["B"])]


def _new(c):
    return _lens(c, c["new_lo"], c["new_hi"], 1)


def _attn_lens(c):
    return _lens(c, c["q_lo"], c["q_hi"], 1), _lens(c, c["kv_lo"], c["kv_hi"], 2)


def _counted(c, q):
    """New tokens whose weights count."""
    return min(q, c["window"]) if c["window"] else q


def _row(c):
    """Codes, scales and biases of one row of one tensor, in bytes."""
    return c["D"] * c["bits"] // 8 + c["D"] // c["GS"] * 4


def work(case):
    c = case
    if c["op"] == "rope":
        values = sum(_new(c)) * (c["H"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * values * (4 if c["dtype"] == "fp32" else 2) + 4 * sum(_new(c)) + 4 * c["rot"],
                "flops": 3 * values * c["rot"] // c["D"]}
    if c["op"] == "weights":
        q, kv = _attn_lens(c)
        w = [_counted(c, a) for a in q]
        pairs = sum(x * (n - x) + x * (x + 1) // 2 for x, n in zip(w, kv))
        return {"bytes": sum(w) * c["H"] * (2 * c["D"] + 4) + sum(kv) * c["Hkv"] * (_row(c) + 8) + 4 * sum(q) * c["Hkv"],
                "flops": 2 * c["D"] * c["H"] * pairs}
    cut = [n for n in _lens(c, c["kv_lo"], c["kv_hi"], 2) if n > c["limit"]]
    # rows that move: of the budget, the share that comes from behind it when any row is as likely to be kept
    moved = sum(c["budget"] * (n - c["budget"]) / n for n in cut)
    return {"bytes": c["Hkv"] * (8 * sum(cut) + 2 * moved * (2 * _row(c) + 8)) + 12 * c["B"], "flops": 0}


def _size(c):
    """What a drawn case may not have more of than the listed ones."""
    w = work(c)
    if c["op"] == "weights":   # scores of a padded batch too: what the plain form costs in memory
        q, kv = _attn_lens(c)
        w["padded"] = c["B"] * c["H"] * max(_counted(c, a) for a in q) * max(kv)
        w["keys"] = c["B"] * c["Hkv"] * c["D"] * max(kv)
    if c["op"] == "evict":
        w["rows"] = c["B"] * c["Hkv"] * c["kv_hi"]
    return w


# --------------------------------------------------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _freqs(c):
    """Radians per position of every pair, in 64 bits."""
    f = c["base"] ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64) / c["rot"])
    keep = torch.zeros_like(f)
    if c["ramp"]:   # pairs that turn often over 8192 positions stay, those that turn less than once are stretched
        keep = ((f * (8192 / (2 * math.pi)) - 1) / (4 - 1)).clamp(0, 1)
    return (f * (keep + (1 - keep) / c["factor"])).cuda()


def _tables(c, kv, g):
    """A pool with some pages to spare and the sequences' pages scattered over it."""
    need = [-(-n // c["page"]) for n in kv]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    use = torch.arange(table.shape[1], device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[use] = order[: sum(need)]
    return pool, table


def _pool(c, pool, g, names):
    """Filled arrays of a pool. Any words are codes; scales are those of plain rows, with a few strong channels among the
    keys, as attention heads have, and biases put a group's middle near zero."""
    st, dt = {}, DTYPES[c["dtype"]]
    W, NG = c["D"] * c["bits"] // 32, c["D"] // c["GS"]
    for x in names:
        rows = (pool, c["Hkv"], c["page"])
        st[x + "p"] = torch.randint(-(1 << 31), 1 << 31, (*rows, W), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        wide = (0.75 + 0.5 * torch.rand(*rows, NG, generator=g, device="cuda")) * (4 if x == "v" else 3)
        if x == "k":
            wide[..., 0] *= 1.5
        st[x + "s"] = (wide / (2 ** c["bits"] - 1)).to(dt)
        st[x + "b"] = (-wide * (0.4 + 0.2 * torch.rand(*rows, NG, generator=g, device="cuda"))).to(dt)
    return st


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "rope":
        new, at = _new(c), _lens(c, c["at_lo"], c["at_hi"], 2)
        n, H, Hkv, D, dt = sum(new), c["H"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
        first = torch.repeat_interleave(torch.tensor([a - sum(new[:i]) for i, a in enumerate(at)], device="cuda"),
                                        torch.tensor(new, device="cuda"))
        # queries, keys and values of a fused projection: views of one row per token
        x = torch.randn(n, H + 2 * Hkv, D, generator=g, device="cuda").to(dt)
        mk = lambda h: torch.empty(n, h, D, dtype=dt, device="cuda")  # noqa: E731
        return {"case": c, "q": x[:, :H], "k": x[:, H: H + Hkv], "positions": (first + torch.arange(n, device="cuda")).to(torch.int32),
                "freqs": _freqs(c), "q_out": mk(H), "k_out": mk(Hkv), "scale": 1.0 + 0.1 * math.log(c["factor"])}
    if c["op"] == "weights":
        q, kv = _attn_lens(c)
        pool, table = _tables(c, kv, g)
        st = _pool(c, pool, g, "k")
        shape = (pool, c["Hkv"], c["page"])
        start = [sum(q[:i]) for i in range(len(q) + 1)]
        shift = torch.randint(0, 1000, (c["B"],), generator=g, device="cuda").to(torch.int32)
        st.update(case=c, q=torch.randn(sum(q), c["H"], c["D"], generator=g, device="cuda").to(DTYPES[c["dtype"]]), table=table,
                  q_start=_ints(start), kv_len=_ints(kv), max_q=max(q), max_kv=max(kv), shift=shift,
                  # as much weight as a few such steps leave
                  mass=torch.rand(shape, generator=g, device="cuda") * (4 * sum(_counted(c, a) for a in q) * c["H"] / c["Hkv"] / sum(kv)),
                  lse=torch.zeros(sum(q), c["H"], device="cuda"),
                  token=torch.full(shape, -7, dtype=torch.int32, device="cuda"))
        # what the attention call before this one has left: log sum exp of every counted row's scores
        S, _, _, at, counted = _scores(st)
        top = S.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        lse = (S.sub_(top).exp_().sum(-1) + 0.0).log() + top[..., 0]            # [B, Hkv, rep, L]
        st["lse"][at[counted]] = lse.permute(0, 3, 1, 2).flatten(2)[counted]
        return st
    kv = _lens(c, c["kv_lo"], c["kv_hi"], 2)
    pool, table = _tables(c, kv, g)
    st = _pool(c, pool, g, "kv")
    rows, B, N = pool * c["Hkv"] * c["page"], c["B"], table.shape[1] * c["page"]
    # mass, token, table and shift as one step finds them; a pass starts from them
    side = torch.zeros(2 * rows + table.numel() + B, dtype=torch.int32, device="cuda")
    mass, token = (side[i * rows: (i + 1) * rows].view(pool, c["Hkv"], c["page"]) for i in (0, 1))
    mass = mass.view(torch.float32)
    shift = side[2 * rows + table.numel():]
    if not c["fresh"]:
        shift.copy_(torch.randint(1, 5000, (B,), generator=g, device="cuda"))
    # few keys draw most of the weight, and some none at all
    m = torch.exp(1.5 * torch.randn(mass.shape, generator=g, device="cuda"))
    mass.copy_(torch.where(torch.rand(mass.shape, generator=g, device="cuda") < 0.05, torch.zeros_like(m), m))
    n = torch.tensor(kv, device="cuda")[:, None, None]
    at = torch.arange(N, device="cuda").expand(B, c["Hkv"], N)
    if c["fresh"]:
        tok = at
    else:   # rows that took the places of evicted ones stand anywhere
        tok = torch.where(at < n, torch.rand(at.shape, generator=g, device="cuda"), torch.full((), 2.0, device="cuda"))
        tok = tok.argsort(-1).argsort(-1)
        tok = tok + torch.where(tok >= c["sinks"], shift[:, None, None].long(), torch.zeros_like(tok))
    page, h, row = _at(st | {"case": c, "table": table}, at)
    ok = at < n
    token[page[ok], h[ok], row[ok]] = tok[ok].to(torch.int32)
    held = side[2 * rows: 2 * rows + table.numel()].view(table.shape)
    held.copy_(table)
    z = lambda k: torch.full((k,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    st.update(case=c, side=side, before=side.clone(), mass=mass, token=token, table=held, kv_len=_ints(kv), shift=shift,
              new_len=z(B), freed=z(table.numel()), n_freed=z(1))
    return st


# ---------------------------------------------------------------------------------------------------- the plain forms


def _plain_rope(st):
    c = st["case"]
    angle = st["positions"].double()[:, None] * st["freqs"]
    if c["inverse"]:
        angle = -angle
    cos, sin = (st["scale"] * f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    out = []
    for x in (st["q"], st["k"]):
        x = x.float()
        r, rest = x[..., : c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r.chunk(2, -1)
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out.append(torch.cat((y, rest), -1).to(st["q"].dtype))
    return {"q": out[0], "k": out[1]}


def _values(packed, s, b, c):
    """The rows that codes, scales and biases stand for, in 32 bits."""
    shift = c["bits"] * torch.arange(32 // c["bits"], dtype=torch.int32, device=packed.device)
    code = ((packed[..., None] >> shift) & (2 ** c["bits"] - 1)).flatten(-2).float()
    return (code.unflatten(-1, (-1, c["GS"])) * s.float()[..., None] + b.float()[..., None]).flatten(-2)


def _at(st, rows):
    """Page, head and row in the page of each sequence's rows [B, Hkv, .]."""
    c = st["case"]
    col = (rows // c["page"]).clamp(max=st["table"].shape[1] - 1)
    page = st["table"].long()[torch.arange(c["B"], device="cuda")[:, None, None], col].clamp(min=0)
    return page, torch.arange(c["Hkv"], device="cuda")[None, :, None].expand_as(rows), rows % c["page"]


def _scores(st):
    """Scores [B, Hkv, rep, L, keys] of every sequence's counted new tokens, -inf where a token does not see a key; each
    sequence's first new key; rows of q and which are real [B, L]."""
    c, n = st["case"], st["max_kv"]
    rows = st["table"].long().clamp(min=0)
    K = _values(st["kp"][rows], st["ks"][rows], st["kb"][rows], c).transpose(1, 2).flatten(2, 3)[:, :, :n]
    start, kv = st["q_start"].long(), st["kv_len"].long()
    q_len = start[1:] - start[:-1]
    count = q_len.clamp(max=c["window"]) if c["window"] else q_len
    i = torch.arange(_counted(c, st["max_q"]), device="cuda")
    real = i[None] < count[:, None]
    tok = q_len[:, None] - count[:, None] + i[None]                              # place among the new tokens
    at = (start[:-1, None] + tok).clamp(max=max(st["q"].shape[0] - 1, 0))
    q = st["q"].float()[at].unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)   # [B, Hkv, rep, L, D]
    B, G, R, L, D = q.shape
    S = (q.reshape(B, G, R * L, D) @ K.transpose(2, 3)).view(B, G, R, L, -1).mul_(1 / math.sqrt(D))
    key = torch.arange(S.shape[-1], device="cuda")
    old = kv - q_len
    seen = (key[None, None] <= (old[:, None] + tok)[..., None]) & real[..., None] & (key < kv[:, None])[:, None]
    return S.masked_fill_(~seen[:, None, None], -math.inf), old, kv, at, real


def _plain_weights(st):
    c = st["case"]
    S, old, kv, at, real = _scores(st)
    lse = st["lse"][at].unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1)          # [B, Hkv, rep, L]
    drawn = S.sub_(lse[..., None]).exp_().sum((2, 3))                             # [B, Hkv, keys]
    key = torch.arange(drawn.shape[-1], device="cuda").expand(drawn.shape)
    page, h, row = _at(st, key)
    mass, first = st["mass"], old[:, None, None]
    had = torch.where(key < first, mass[page, h, row], torch.zeros_like(drawn))
    ok = (key < kv[:, None, None]) & (kv > old)[:, None, None]
    mass[page[ok], h[ok], row[ok]] = (c["decay"] * had + drawn)[ok]
    fresh = ok & (key >= first)
    st["token"][page[fresh], h[fresh], row[fresh]] = (key + st["shift"][:, None, None])[fresh].to(torch.int32)
    return {"mass": mass, "token": st["token"]}


def _plain_evict(st):
    c = st["case"]
    budget, n = c["budget"], st["kv_len"].long()
    cut = n > c["limit"]
    at = torch.arange(st["table"].shape[1] * c["page"], device="cuda").expand(c["B"], c["Hkv"], -1)
    page, h, row = _at(st, at)
    token, live = st["token"][page, h, row], at < n[:, None, None]
    safe = (token < c["sinks"]) | (token >= (n + st["shift"] - c["recent"])[:, None, None])
    rank = torch.where(live, st["mass"][page, h, row], torch.full((), -math.inf, device="cuda"))
    rank = rank.masked_fill(safe & live, math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.zeros_like(live).scatter_(-1, best, True)
    over = cut[:, None, None]
    hole, come = ~keep & (at < budget) & over, keep & (at >= budget) & live & over
    # the i-th row behind the budget that stays goes to the i-th hole
    nth = torch.zeros_like(at).scatter_(-1, torch.where(come, come.cumsum(-1) - 1, at.shape[-1] - 1), torch.where(come, at, 0))
    src = nth.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0))[hole]
    to = (page[hole], h[hole], row[hole])
    b = torch.arange(c["B"], device="cuda")[:, None, None].expand_as(at)[hole]
    frm = (st["table"].long()[b, src // c["page"]], to[1], src % c["page"])
    for x in ("kp", "ks", "kb", "vp", "vs", "vb", "mass", "token"):
        st[x][to] = st[x][frm]
    st["new_len"].copy_(torch.where(cut, torch.full_like(n, budget), n))
    st["shift"].add_((n - st["new_len"]).to(torch.int32))
    col = torch.arange(st["table"].shape[1], device="cuda")[None]
    gone = cut[:, None] & (col >= -(-budget // c["page"])) & (col < ((n + c["page"] - 1) // c["page"])[:, None])
    ids = st["table"][gone]
    st["freed"][: ids.numel()] = ids
    st["n_freed"].fill_(ids.numel())
    st["table"].masked_fill_(gone, -1)


def run(state):
    st, c = state, state["case"]
    if own:
        import attention_quantized_kv_split_gb300 as qda
    if c["op"] == "rope":
        if not own:
            return _plain_rope(st)
        qda.qdecode_rope(st["q"], st["k"], st["positions"], st["freqs"], st["q_out"], st["k_out"], interleaved=c["interleaved"],
                         scale=st["scale"], inverse=c["inverse"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if c["op"] == "weights":
        if not own:
            return _plain_weights(st)
        qda.qdecode_paged_weights(st["q"], st["kp"], st["ks"], st["kb"], st["lse"], st["mass"], st["token"], st["q_start"],
                                  st["kv_len"], st["table"], st["max_q"], c["GS"], c["bits"], window=c["window"], decay=c["decay"],
                                  shift=st["shift"])
        return {"mass": st["mass"], "token": st["token"]}
    # the step's weights, tokens, table and shifts, of which the last pass has changed some
    st["side"].copy_(st["before"])
    if own:
        qda.qdecode_paged_evict(st["kp"], st["ks"], st["kb"], st["vp"], st["vs"], st["vb"], st["mass"], st["token"], st["kv_len"],
                                st["new_len"], st["table"], st["freed"], st["n_freed"], c["GS"], c["bits"], c["budget"],
                                limit=c["limit"], sinks=c["sinks"], recent=c["recent"], shift=st["shift"])
    else:
        _plain_evict(st)
    return {k: st[k] for k in ("kp", "ks", "kb", "vp", "vs", "vb", "mass", "token", "new_len", "shift", "table", "freed", "n_freed")}


# ------------------------------------------------------------------------------------------------- the definition, 64 bits


def _exact_rope(c, st):
    r, out = c["rot"], {}
    turn = torch.outer(st["positions"].double(), st["freqs"]) * (-1.0 if c["inverse"] else 1.0)
    z = torch.polar(torch.full_like(turn, st["scale"]), turn)[:, None]   # a pair is a complex number that this one turns
    for x in "qk":
        v = st[x].double()
        if c["interleaved"]:
            y = torch.view_as_real(torch.view_as_complex(v[..., :r].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        else:
            w = torch.complex(v[..., : r // 2], v[..., r // 2: r]) * z
            y = torch.cat((w.real, w.imag), -1)
        out[x] = torch.cat((y, v[..., r:]), -1)
    return out


def _exact_weights(c, st):
    q_len, kv = _attn_lens(c)
    mass, P, D, rep, t0 = st["mass"].double(), c["page"], c["D"], c["H"] // c["Hkv"], 0
    lse = st["lse"].double()
    for b in range(c["B"]):
        n, L = kv[b], q_len[b]
        pages = st["table"][b, : -(-n // P)].long()
        for h in range(c["Hkv"]):
            words, s, bias = (st[x][pages, h].reshape(pages.numel() * P, -1)[:n] for x in ("kp", "ks", "kb"))
            w = words.long() & 0xFFFFFFFF
            code = torch.stack([(w >> (c["bits"] * j)) & (2 ** c["bits"] - 1) for j in range(32 // c["bits"])], -1)
            K = code.reshape(n, D).double() * s.double().repeat_interleave(c["GS"], 1) + bias.double().repeat_interleave(c["GS"], 1)
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            first = L - _counted(c, L)
            far = torch.arange(n, device="cuda")[None] - torch.arange(first, L, device="cuda")[:, None] > n - L
            for r in range(h * rep, (h + 1) * rep):
                x = st["q"][t0 + first: t0 + L, r].double() @ K.T / math.sqrt(D) - lse[t0 + first: t0 + L, r, None]
                total += x.exp_().masked_fill_(far, 0).sum(0)
            had = mass[pages, h].reshape(-1)
            had[n - L: n] = 0
            had[:n] = c["decay"] * had[:n] + total
            old = mass[pages, h].reshape(-1)
            old[:n] = had[:n]
            mass[pages, h] = old.view(-1, P)
        t0 += L
    return {"mass": mass, "token": None}


def _exact_evict(c, st):
    names = ("ks", "kb", "vs", "vb", "mass")
    out = {x: st[x].double() for x in names}
    P, budget = c["page"], c["budget"]
    table, token = st["table"].cpu(), st["token"].cpu()
    mass, shift = st["mass"].cpu(), st["shift"].tolist()
    for b, n in enumerate(st["kv_len"].tolist()):
        if n <= c["limit"]:
            continue
        pages = table[b, : -(-n // P)].long()
        for h in range(c["Hkv"]):
            m, t = mass[pages, h].reshape(-1)[:n].double(), token[pages, h].reshape(-1)[:n]
            m[(t < c["sinks"]) | (t >= n + shift[b] - c["recent"])] = math.inf
            kept = torch.sort(-m, stable=True).indices[:budget]
            inside = torch.zeros(budget, dtype=torch.bool)
            inside[kept[kept < budget]] = True
            to, frm = torch.nonzero(~inside)[:, 0], torch.sort(kept[kept >= budget]).values
            for x in names:
                out[x][pages[to // P].cuda(), h, (to % P).cuda()] = st[x][pages[frm // P].cuda(), h, (frm % P).cuda()].double()
    return {x: out.get(x) for x in ("kp", "ks", "kb", "vp", "vs", "vb", "mass", "token", "new_len", "shift", "table", "freed", "n_freed")}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](case, st)
