"""The paged cache on the GPU: step tables, append and attention against plain 64-bit implementations (paged_ref), at the
sizes, layouts and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import oracle as O
import attention_quantized_kv_split_gb300 as qda
from attention_quantized_kv_split_gb300 import build

from paged_ref import DT, Case, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    qda.lib()


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    qda.qdecode_attn_device_status()
    yield


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------------------ tables


def run_map(old, new, cols, page, n_free, max_tokens, seed=0):
    rng = np.random.default_rng(seed)
    B = len(old)
    held = [-(-max(o, 0) // page) for o in old]
    pool = sum(held) + n_free
    order = rng.permutation(pool)
    table = np.full((B, cols), -5, dtype=np.int32)
    at = 0
    for b, m in enumerate(held):
        table[b, : min(m, cols)] = order[at: at + min(m, cols)]
        at += m
    free = order[at:]
    dev = i32(table)
    pad = 3   # canaries behind the outputs
    outs = {k: torch.full((n + pad,), 1234, dtype=torch.int32, device="cuda")
            for k, n in (("q_start", B + 1), ("kv_len", B), ("slots", max_tokens), ("positions", max_tokens), ("used", 1))}
    views = {k: v[:-pad] for k, v in outs.items()}
    qda.qdecode_paged_map(i32(old), i32(new), dev, i32(free), page, **views)
    torch.cuda.synchronize()
    ref = tables(old, new, table, free, page, max_tokens)
    got = (dev, views["q_start"], views["kv_len"], views["slots"], views["positions"])
    for g, r, name in zip(got, ref, ("table", "q_start", "kv_len", "slots", "positions")):
        np.testing.assert_array_equal(g.cpu().numpy(), r, err_msg=name)
    assert int(views["used"]) == ref[5]
    assert all(bool((v[-pad:] == 1234).all()) for v in outs.values())
    assert qda.qdecode_attn_device_status() == (8 if ref[6] else 0)


@pytest.mark.parametrize("old,new,page", [
    ([0], [1], 16), ([15], [1], 16), ([16], [1], 16), ([17], [0], 16), ([0, 0], [0, 0], 32),
    ([0, 31, 32, 100], [33, 1, 1, 200], 32), ([5, 0, 300], [0, 7, 1], 256), ([1000], [3001], 64),
])
def test_map(old, new, page):
    total = sum(new)
    for max_tokens in (total, total + 5):   # exactly full, and padded as a captured step would be
        run_map(old, new, 70 if page < 64 else 64, page, 300, max_tokens)


@pytest.mark.parametrize("B", [2, 31, 33, 512])
def test_map_batches(B):
    rng = np.random.default_rng(B)
    old, new = rng.integers(0, 200, B), rng.integers(0, 70, B)
    run_map(old, new, 20, 16, 6 * B, int(new.sum()) + 9, seed=B)


def test_map_exhausted_pool_narrow_table_and_bad_lengths():
    run_map([10, 20, 3], [40, 40, 5], 10, 16, 3, 85)        # the second sequence gets part of its pages, the third none
    run_map([10, 100], [40, 40], 4, 16, 20, 80)             # tokens past the table's last column
    run_map([-3, 5], [4, -1], 4, 16, 20, 8)                 # negative lengths count as 0
    run_map([0, 0], [20, 20], 4, 16, 20, 30)                # more tokens than the arrays hold


# ------------------------------------------------------------------------------------------------------------ append


def pool_arrays(pages, Hkv, page, D, GS, bits, dt, fill=0):
    W, NG = D * bits // 32, D // GS
    mk = lambda n, d: torch.full((pages, Hkv, page, n), fill, dtype=d, device="cuda")  # noqa: E731
    return [mk(W, torch.int32), mk(NG, dt), mk(NG, dt), mk(W, torch.int32), mk(NG, dt), mk(NG, dt)]


APPEND = [(64, 32, 4, "bf16", "bf16"), (64, 64, 8, "fp16", "fp32"), (128, 128, 4, "fp16", "fp16"),
          (128, 64, 8, "bf16", "fp16"), (256, 32, 8, "bf16", "bf16"), (256, 128, 4, "fp16", "fp32"),
          (512, 128, 4, "bf16", "fp32"), (512, 32, 8, "fp16", "bf16"), (512, 64, 4, "bf16", "bf16")]


@pytest.mark.parametrize("D,GS,bits,cache,src", APPEND)
@pytest.mark.parametrize("T,Hkv,page", [(1, 1, 16), (5, 3, 32), (130, 2, 256)])
def test_append_bit_exact(D, GS, bits, cache, src, T, Hkv, page):
    rng = np.random.default_rng(D + GS + bits + T)
    pages = -(-T // page) + 2
    kv = torch.from_numpy(rng.standard_normal((T, 2, Hkv, D)) * 3).to(DT[src]).cuda()   # a fused projection's rows
    kv[0, 0, 0, :] = 1.5                                                                 # a group of one value
    k, v = kv[:, 0], kv[:, 1]
    slots = rng.permutation(pages * page)[:T]
    slots[T // 2:T // 2 + (T > 1)] = -1                                                  # a skipped token
    arr = pool_arrays(pages, Hkv, page, D, GS, bits, DT[cache], fill=3)
    held = [torch.empty(T, Hkv, D, dtype=DT[cache], device="cuda") for _ in range(2)]
    qda.qdecode_paged_append(k, v, i32(slots), *arr, GS, bits, *held)
    torch.cuda.synchronize()
    for x, (p, s, b), h in ((k, arr[:3], held[0]), (v, arr[3:], held[1])):
        codes, sr, br = O.quantize(x.float().cpu().numpy().reshape(T * Hkv, D), GS, bits, cache)
        words = O.pack(codes, bits).reshape(T, Hkv, -1).view(np.int32)
        ref = [np.full(t.shape, 3.0) for t in (p, s, b)]
        for t, slot in enumerate(slots):
            if slot >= 0:
                ref[0][slot // page, :, slot % page] = words[t]
                ref[1][slot // page, :, slot % page] = sr.reshape(T, Hkv, -1)[t]
                ref[2][slot // page, :, slot % page] = br.reshape(T, Hkv, -1)[t]
        for got, r in zip((p, s, b), ref):
            np.testing.assert_array_equal(got.double().cpu().numpy(), r)
        # the held values: one rounding of scale * code + bias, itself one fp32 rounding off
        deq = np.asarray(O.dequantize(codes, sr, br, GS), dtype=np.float64).reshape(T, Hkv, D)
        u = torch.finfo(DT[cache]).eps / 2
        tiny = 2.0 ** -25 if cache == "fp16" else 0.0   # half of fp16's smallest step
        err = np.abs(h.double().cpu().numpy() - deq)
        assert (err <= u * (1 + 2.0 ** -10) * np.abs(deq) + 2.0 ** -24 * np.abs(sr).max() * 2 ** bits + tiny).all()
    assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("bits,cache", [(4, "bf16"), (8, "bf16"), (4, "fp16"), (8, "fp16")])
def test_append_values_between_two_codes(bits, cache):
    """Rows whose values lie on and next to the middle between two codes, tiny and huge groups, groups of one value, and
    infinities and NaN: the codes are the quantizer's to the bit."""
    D, GS, top = 128, 64, 2 ** bits - 1
    rng = np.random.default_rng(bits)
    rows = []
    for scale in (1.0, 0.375, 2.0 ** -9, 3e-5, 1e-38, 3e4 if cache == "fp16" else 1e35):
        x = (rng.integers(0, 2 * top, (8, D)) * 0.5 - 3) * scale / top     # whole and half codes
        x[:, 0::GS], x[:, 1::GS] = -3 * scale / top, (top - 3) * scale / top
        rows += [x, np.nextafter(x.astype(np.float32), np.float32(np.inf)), np.nextafter(x.astype(np.float32), -np.float32(np.inf))]
    rows.append(rng.standard_normal((300, D)) * np.exp(rng.standard_normal((300, 1)) * 4))
    odd = rng.standard_normal((6, D))
    odd[0, 3], odd[1, 5], odd[2, 7], odd[3, :GS], odd[4, 9], odd[4, 10], odd[5] = np.nan, np.inf, -np.inf, np.nan, np.inf, -np.inf, 0
    x = torch.from_numpy(np.concatenate(rows + [odd]).astype(np.float32)).cuda()
    T = x.shape[0]
    pages = -(-T // 16)
    arr = pool_arrays(pages, 1, 16, D, GS, bits, DT[cache])
    qda.qdecode_paged_append(x[:, None], x[:, None], i32(np.arange(T)), *arr, GS, bits)
    packed = torch.empty(T, D * bits // 32, dtype=torch.int32, device="cuda")
    sc, bi = (torch.empty(T, D // GS, dtype=DT[cache], device="cuda") for _ in range(2))
    qda.qdecode_quantize(x, GS, bits, DT[cache], packed, sc, bi)
    torch.cuda.synchronize()
    for a in (0, 3):
        for got, ref in zip(arr[a: a + 3], (packed, sc, bi)):
            g = got.reshape(pages * 16, -1)[:T]
            view = torch.int32 if g.dtype == torch.int32 else torch.int16
            assert torch.equal(g.view(view), ref.view(view))


def test_append_slots_outside_the_pool_are_skipped():
    T, Hkv, D = 6, 2, 128
    x = torch.randn(T, Hkv, D, device="cuda", dtype=torch.bfloat16)
    arr = pool_arrays(3, Hkv, 16, D, 64, 4, torch.bfloat16, fill=9)
    before = [a.clone() for a in arr]
    qda.qdecode_paged_append(x, x, i32([48, 1 << 30, -1, -7, 2 ** 31 - 1, 49]), *arr, 64, 4)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(arr, before))
    assert qda.qdecode_attn_device_status() == 8


def test_append_nothing():
    arr = pool_arrays(2, 2, 16, 128, 64, 4, torch.bfloat16)
    x = torch.empty(0, 2, 128, device="cuda", dtype=torch.bfloat16)
    qda.qdecode_paged_append(x, x, i32([]), *arr, 64, 4)


# --------------------------------------------------------------------------------------------------------- attention

CODECS = [(64, 32, 4, "bf16"), (64, 64, 8, "fp16"), (128, 32, 8, "bf16"), (128, 64, 4, "bf16"), (128, 128, 4, "fp16"),
          (128, 64, 8, "fp16"), (256, 32, 4, "fp16"), (256, 64, 8, "bf16"), (256, 128, 4, "bf16"), (512, 128, 4, "fp16"),
          (512, 32, 4, "bf16"), (512, 64, 8, "bf16"), (64, 64, 4, "fp16"), (256, 128, 8, "fp16"), (512, 128, 8, "fp16")]


@pytest.mark.parametrize("D,GS,bits,dtype", CODECS)
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(D, GS, bits, dtype, page):
    c = Case([1] * 6, [1, 2, 33, 64, 0, 700], 8, 2, D, bits, GS, dtype, page, seed=D + bits + page)
    c.check(c.run())
    assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("D,GS,bits,dtype", CODECS)
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(D, GS, bits, dtype, causal):
    # a prompt from its start, chunks behind earlier tokens, a lone token, an idle sequence, and one of many tiles
    c = Case([130, 57, 1, 0, 200], [130, 311, 90, 40, 650], 6, 2, D, bits, GS, dtype, 32, seed=D + GS)
    c.check(c.run(causal), causal)
    assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (6, 2), (16, 1), (32, 8), (64, 1), (24, 3)])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [2, 8, 3], [40, 1, 17]])
def test_head_layouts(H, Hkv, q_lens):
    c = Case(q_lens, [50, 300, 129], H, Hkv, 128, 4, 64, "bf16", 16, seed=H + Hkv)
    c.check(c.run())


@pytest.mark.parametrize("page", [16, 32, 128, 256])
@pytest.mark.parametrize("q_len", [1, 5, 70])
def test_lengths_around_tile_and_page_borders(page, q_len):
    kv = [n for n in (q_len, 127, 128, 129, 255, 256, 257, 383, 513) if n >= q_len]
    c = Case([q_len] * len(kv), kv, 4, 2, 128, 4, 32, "fp16", page, seed=page + q_len)
    c.check(c.run())


@pytest.mark.parametrize("q_len,kv,D", [(1, 9000, 128), (1, 16000, 256), (3, 6000, 64), (100, 5000, 128), (64, 4000, 256),
                                        (20, 3000, 512)])
def test_long_sequences_are_split(q_len, kv, D):
    # one sequence over many CTAs; strong scores, so that a key lost or counted twice shows
    c = Case([q_len], [kv], 8, 2, D, 4, 64, "bf16", 64, seed=kv, q_scale=2.0)
    c.check(c.run())


@pytest.mark.parametrize("D,GS,bits", [(64, 32, 8), (128, 64, 4), (256, 32, 8), (256, 128, 4), (512, 64, 8)])
@pytest.mark.parametrize("q_len", [60, 130])
def test_many_tiles_and_blocks_per_cta(D, GS, bits, q_len):
    # more work than CTAs: every CTA walks several tiles of a few dozen key blocks, with and without split ones
    B = {64: 24, 128: 12, 256: 8, 512: 4}[D]
    kv = [2400 + 301 * (i % 5) for i in range(B)]
    c = Case([q_len] * B, kv, 16, 8, D, bits, GS, "bf16", 32, seed=D + q_len)
    ref = None
    for _ in range(3):
        got = c.run()
        ref = got.clone() if ref is None else ref
        assert torch.equal(got, ref)
    assert qda.qdecode_attn_device_status() == 0
    rows = [b for b in range(B) if b % max(1, B // 3) == 0]   # a few sequences in 64 bits
    sub = Case.__new__(Case)
    sub.__dict__.update(c.__dict__)
    sub.q_lens, sub.kv_lens, sub.total = [q_len] * len(rows), [kv[b] for b in rows], q_len * len(rows)
    sub.K, sub.V, sub.A = ([x[b] for b in rows] for x in (c.K, c.V, c.A))
    sub.start = np.arange(len(rows) + 1) * q_len
    pick = np.concatenate([np.arange(b * q_len, (b + 1) * q_len) for b in rows])
    sub.q64 = c.q64[pick]
    sub.check(got[torch.from_numpy(pick).cuda()])


@pytest.mark.parametrize("q_lens", [[1, 1], [90, 140]])
def test_more_queries_than_keys(q_lens):
    # cross attention to fewer states than tokens; with a causal mask the first tokens see nothing and give zeros
    c = Case(q_lens, [0, 33], 8, 2, 128, 8, 32, "bf16", 16, seed=3)
    c.check(c.run(False), False)
    got = c.run(True)
    c.check(got, True)
    assert not got[: q_lens[0]].any()


@pytest.mark.parametrize("max_q", [1, 7, 1000])
def test_max_q_only_chooses_the_kernel(max_q):
    c = Case([1, 130, 9], [400, 500, 77], 8, 2, 128, 4, 64, "bf16", 32, seed=8)
    c.check(c.run(max_q=max_q))


@pytest.mark.parametrize("q_lens", [[1, 1, 2], [70, 3, 150]])
def test_rows_behind_the_last_sequence_stay(q_lens):
    c = Case(q_lens, [200, 31, 400], 8, 2, 128, 4, 64, "bf16", 32, seed=5, pad_rows=9)
    got = c.run()
    c.check(got)
    assert bool((got[c.total:] == 7.0).all())


@pytest.mark.parametrize("q_lens", [[1, 1], [64, 130]])
@pytest.mark.parametrize("D,GS,bits,dtype", [(128, 64, 4, "bf16"), (256, 32, 8, "fp16"), (512, 128, 4, "bf16"), (64, 32, 8, "bf16")])
def test_nothing_behind_a_sequence_reaches_it(q_lens, D, GS, bits, dtype):
    # NaN in every row of the pool that holds no token (Case fills them), and infinities in the last page's rest
    c = Case(q_lens, [77, 145], 4, 2, D, bits, GS, dtype, 64, seed=6, unwritten=float("inf"))
    c.check(c.run())
    c.check(c.run(False), False)


@pytest.mark.parametrize("D,GS,bits,dtype", [(128, 64, 4, "bf16"), (256, 32, 8, "fp16"), (512, 128, 4, "fp16"), (64, 32, 4, "bf16")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_hidden_key_that_is_not_finite(D, GS, bits, dtype, bad):
    # the last token of a chunk is not finite: the tokens before it do not see it
    L, n, page = 150, 200, 32
    c = Case([L], [n], 4, 2, D, bits, GS, dtype, page, seed=7)
    pg = int(c.table[0, (n - 1) // page])
    for a in (c.arrays[1], c.arrays[2], c.arrays[4], c.arrays[5]):
        a[pg, :, (n - 1) % page] = bad
    got = c.run()
    assert not torch.isfinite(got[L - 1]).any()
    got[L - 1] = 0
    ref, tol = c.reference(hidden=[(0, n - 1)])
    err = np.abs(got.double().cpu().numpy() - ref)[: L - 1]
    assert (err <= tol[: L - 1]).all()


@pytest.mark.parametrize("q_lens", [[1, 1], [64, 130]])
def test_pages_outside_the_pool_count_as_absent(q_lens):
    c = Case(q_lens, [100, 200], 4, 2, 128, 4, 64, "bf16", 16, seed=9)
    c.table[0, 1] = c.arrays[0].shape[0]
    c.table[1, 3] = -1
    got = c.run()
    torch.cuda.synchronize()
    assert qda.qdecode_attn_device_status() == 8
    c.check(got, hidden=[(0, n) for n in range(16, 32)] + [(1, n) for n in range(48, 64)])


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [70, 1, 150]])
def test_strided_queries(q_lens):
    c = Case(q_lens, [200, 31, 400], 8, 2, 128, 4, 64, "bf16", 32, seed=11)
    wide = torch.zeros(c.total, 13, 136, dtype=c.q.dtype, device="cuda")
    wide[:, 2:10, 8:] = c.q
    q = wide[:, 2:10, 8:]
    assert torch.equal(c.run(), c.run(q=q, out=torch.empty_like(c.q)))


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [300, 1, 33]])
def test_the_same_bits_every_time_and_on_another_stream(q_lens):
    c = Case(q_lens, [2000, 31, 1400], 8, 2, 128, 4, 64, "bf16", 32, seed=12)
    first = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        out = torch.zeros_like(first)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.run(out=out)
        s.synchronize()
        assert torch.equal(first, out)


def test_repeated_page_in_two_rows():
    # two sequences that share their pages (a common prefix) read the same keys
    c = Case([1, 1], [64, 64], 8, 2, 128, 4, 64, "bf16", 16, seed=13)
    c.table[1] = c.table[0]
    c.K[1], c.V[1], c.A[1] = c.K[0], c.V[0], c.A[0]
    c.check(c.run())


def test_agrees_with_the_contiguous_cache():
    # the same rows through qdecode_attn
    c = Case([1], [777], 8, 2, 256, 4, 64, "bf16", 16, seed=14)
    rows = c.table[0, : 49].long()
    flat = [a[rows].transpose(0, 1).flatten(1, 2)[:, :777].reshape(2 * 777, -1).contiguous() for a in c.arrays]
    out = torch.empty(1, 8, 256, dtype=torch.bfloat16, device="cuda")
    qda.qdecode_attn(c.q, *flat, out, [777], 2, 64, 4)
    ref, tol = c.reference()
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    c.check(c.run())


def test_workspace_of_the_stated_size():
    for q_lens, D in (([1, 1], 128), ([300], 256), ([9], 512)):
        c = Case(q_lens, [4000] * len(q_lens), 8, 2, D, 4, 64, "bf16", 64, seed=15)
        ref = c.run()
        n = qda.qdecode_paged_attn_workspace_bytes(len(q_lens), 8, 2, max(q_lens), D, 64, 4)
        buf = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        try:
            qda.qdecode_attn_set_workspace(buf[:n] if n else None)
            assert torch.equal(ref, c.run())
            torch.cuda.synchronize()
            assert bool((buf[n:] == 0xA5).all())
            if n > 16:
                qda.qdecode_attn_set_workspace(buf[: n - 16])
                with pytest.raises(qda.QdaError):
                    c.run()
        finally:
            qda.qdecode_attn_set_workspace(None)


def test_refusals_in_python():
    c = Case([2], [20], 8, 2, 128, 4, 64, "bf16", 16)
    ok = dict(causal=True)
    call = lambda q=c.q, arr=None, out=None, **kw: qda.qdecode_paged_attn(  # noqa: E731
        q, *(arr or c.arrays), c.q.clone() if out is None else out, kw.get("s", c.q_start), kw.get("n", c.kv_len),
        kw.get("t", c.table), 2, 64, kw.get("bits", 4), **ok)
    for kw in (dict(q=c.q.half()), dict(out=c.q[:1]), dict(s=c.q_start.long()), dict(n=c.kv_len.cpu()), dict(bits=8),
               dict(t=c.table[:, ::2]), dict(out=c.q.transpose(0, 1)), dict(q=c.q.transpose(1, 2)),
               dict(arr=c.arrays[:1] + [c.arrays[1][:, :1]] + c.arrays[2:])):
        with pytest.raises(ValueError):
            call(**kw)
    x = c.q[:, :2]
    with pytest.raises(ValueError):
        qda.qdecode_paged_append(x, x, i32([1]), *c.arrays, 64, 4)
    with pytest.raises(ValueError):
        qda.qdecode_paged_append(x, x.float(), i32([1, 2]), *c.arrays, 64, 4)
    with pytest.raises(ValueError):
        qda.qdecode_paged_append(x.cpu(), x.cpu(), i32([1, 2]), *c.arrays, 64, 4)


# ------------------------------------------------------------------------------------------------- the calls together


def grown(old, new, k, v, lens):
    """Append a step's rows to the host's copy of each sequence."""
    at = 0
    for b, n in enumerate(new):
        for dst, src in ((old[0], k), (old[1], v)):
            dst[b] = np.concatenate([dst[b], src[at: at + n]], axis=0)
        at += n
        lens[b] += n


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_server(captured):
    """Prompts, a chunk, and single tokens through map, append and attend; captured: the three calls are one CUDA graph
    that every step replays with its own lengths, padded to the largest step."""
    H, Hkv, D, GS, bits, page, dtype = 8, 2, 128, 64, 4, 16, "bf16"
    rng = np.random.default_rng(21)
    steps = [[40, 0, 17], [1, 33, 1], [1, 1, 1], [0, 1, 60], [1, 1, 1]]
    B, most = 3, max(sum(s) for s in steps)
    pool = qda.PagedKV(40, Hkv, page, D, GS, bits, DT[dtype])
    free = i32(rng.permutation(40))
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(most, h, D, dtype=DT[dtype], device="cuda") for h in (H, Hkv, Hkv))
    held = [torch.zeros(most, Hkv, D, dtype=DT[dtype], device="cuda") for _ in range(2)]
    out = torch.empty_like(q)
    old, new = i32([0] * B), i32([0] * B)
    free_now = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    state = {}

    def step():
        t = pool.step_tables(old, new, table, free_now, most)
        pool.append(k, v, t["slots"], *held)
        pool.attend(q, t["q_start"], t["kv_len"], table, 64, out=out)
        state.update(t)

    graph = None
    if captured:
        step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    taken, lens = 0, [0] * B
    rows = [[np.zeros((0, Hkv, D)) for _ in range(B)] for _ in range(2)]
    for s in steps:
        n = sum(s)
        for buf, h in ((q, H), (k, Hkv), (v, Hkv)):
            buf.copy_(torch.from_numpy(rng.standard_normal((most, h, D))))
        new.copy_(i32(s))
        left = free[taken:]
        free_now.fill_(-1)
        free_now[: left.numel()] = left
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        taken += int(state["used"])
        deq = []
        for x in (k, v):
            codes, sc, bi = O.quantize(x[:n].float().cpu().numpy().reshape(n * Hkv, D), GS, bits, dtype)
            deq.append(np.asarray(O.dequantize(codes, sc, bi, GS), dtype=np.float64).reshape(n, Hkv, D))
        grown(rows, s, *deq, lens)
        old.copy_(state["kv_len"])
        assert state["kv_len"].tolist() == lens
        ref = Case.__new__(Case)
        ref.q_lens, ref.kv_lens, ref.H, ref.Hkv, ref.D, ref.dtype, ref.total = s, list(lens), H, Hkv, D, dtype, n
        ref.start = np.concatenate([[0], np.cumsum(s)])
        ref.q64 = q.double().cpu().numpy()
        ref.K = [r.transpose(1, 0, 2) for r in rows[0]]
        ref.V = [r.transpose(1, 0, 2) for r in rows[1]]
        ref.A = [np.abs(r) + 3.5 for r in ref.V]   # half of a group's range: the rows are N(0, 1), within 7 of each other
        ref.check(out)
    assert qda.qdecode_attn_device_status() == 0


def test_two_graphs_share_the_workspace():
    # two captured calls of different shapes on the library's workspace, replayed in turn on one stream
    a = Case([1], [5000], 8, 2, 128, 4, 64, "bf16", 64, seed=31)
    b = Case([200], [3000], 8, 2, 256, 4, 64, "bf16", 64, seed=32)
    ref = [a.run(), b.run()]
    outs = [torch.zeros_like(r) for r in ref]
    graphs = []
    for c, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=o)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, ref):
            assert torch.equal(o, r)


@pytest.mark.parametrize("D,GS,bits,dtype", [(64, 32, 8, "bf16"), (128, 64, 4, "fp16"), (256, 32, 8, "bf16"), (512, 128, 4, "bf16")])
def test_pages_outside_the_pool_where_a_tile_has_two_threads_per_row(D, GS, bits, dtype):
    # 60 and 100 query rows per KV head: absent pages in both halves of a block of keys, and a whole absent block
    c = Case([30, 50], [300, 420], 4, 2, D, bits, GS, dtype, 32, seed=21)
    absent = {0: [1, 2], 1: [4, 5, 6, 7, 11]}
    for b, cols in absent.items():
        for i, col in enumerate(cols):
            c.table[b, col] = -1 - i
    got = c.run(False)
    torch.cuda.synchronize()
    assert qda.qdecode_attn_device_status() == 8
    c.check(got, False, hidden=[(b, n) for b, cols in absent.items() for col in cols for n in range(32 * col, 32 * col + 32)])


@pytest.mark.parametrize("D,GS,bits", [(64, 32, 8), (128, 64, 4), (256, 64, 4), (256, 32, 8), (512, 64, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_strong_scores_where_a_tile_has_two_threads_per_row(D, GS, bits, causal):
    # a row's reference rises again and again, from either half of a block of keys
    c = Case([15, 9, 21], [900, 2000, 131], 8, 2, D, bits, GS, "bf16", 16, seed=22, q_scale=4.0)
    c.check(c.run(causal), causal)
