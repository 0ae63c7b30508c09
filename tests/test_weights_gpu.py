"""Accumulated attention weight, and the row sums that it needs, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda

import forget_ref as R
from paged_ref import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    qda.qdecode_attn_device_status()
    yield
    assert qda.qdecode_attn_device_status() == 0


def side(c, seed=0):
    """mass and token as an earlier owner of the pages left them, NaN where no row of these sequences is."""
    rng = np.random.default_rng(seed)
    shape = tuple(c.arrays[1].shape[:3])
    mass = np.full(shape, np.nan, dtype=np.float32)
    table = c.table.cpu().numpy()
    for b, (L, n) in enumerate(zip(c.q_lens, c.kv_lens)):
        key = np.arange(n - L if n > L else 0)
        mass[table[b][key // c.page], :, key % c.page] = rng.random((len(key), c.Hkv))
    return mass, rng.integers(-5, 5, shape).astype(np.int32)


def run(c, lse, mass, token, window=0, decay=1.0, shift=None, max_q=None, q=None, stream=None):
    m, t = torch.from_numpy(mass).cuda(), torch.from_numpy(token).cuda()
    sh = None if shift is None else torch.tensor(shift, dtype=torch.int32, device="cuda")
    qda.qdecode_paged_weights(c.q if q is None else q, *c.arrays[:3], lse, m, t, c.q_start, c.kv_len, c.table,
                              max_q or max(max(c.q_lens), 1), c.GS, c.bits, window, decay, sh, stream)
    torch.cuda.synchronize()
    return m.cpu().numpy(), t.cpu().numpy()


def log_sums(c):
    return torch.from_numpy(R.log_sums(c).astype(np.float32)).cuda()


def check(c, window=0, decay=1.0, shift=None, max_q=None, seed=0):
    lse, (mass, token) = log_sums(c), side(c, seed)
    got, tok = run(c, lse, mass, token, window, decay, shift, max_q)
    ref, want, tol = R.weights(c, lse.cpu().numpy(), mass, token, window, decay, shift)
    np.testing.assert_array_equal(tok, want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))   # rows of nobody are left as they were
    ok = ~np.isnan(ref)
    err = np.abs(got[ok] - ref[ok])
    assert (err <= tol[ok]).all(), f"worst {np.max(err / np.maximum(tol[ok], 1e-300))} of the tolerance"


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1, 1, 1], [33, 1, 300]), ([3], [40]), ([17, 1, 0, 5], [64, 2, 9, 129]),
                                            ([70, 33], [70, 500])])
@pytest.mark.parametrize("D,bits,GS,dtype,page", [
    (64, 4, 32, "bf16", 16), (64, 8, 64, "fp16", 32), (128, 4, 64, "bf16", 64), (128, 8, 128, "fp16", 16), (128, 4, 32, "fp16", 256),
    (256, 8, 32, "bf16", 16), (256, 4, 128, "bf16", 32), (512, 4, 128, "fp16", 32), (512, 8, 32, "bf16", 64),
])
def test_against_the_definition(q_lens, kv_lens, D, bits, GS, dtype, page):
    check(Case(q_lens, kv_lens, 6, 2, D, bits, GS, dtype, page, seed=D + bits), decay=0.75, shift=list(range(len(q_lens))))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (16, 2), (5, 5), (64, 1)])
@pytest.mark.parametrize("L", [1, 2, 9])
def test_heads(H, Hkv, L):
    check(Case([L, 2 * L], [100, 77], H, Hkv, 128, 4, 64, "bf16", 16, seed=H + L))


@pytest.mark.parametrize("window", [1, 3, 64, 1000])
def test_window(window):
    check(Case([100, 2, 1], [333, 2, 50], 4, 2, 64, 8, 32, "fp16", 16, seed=window), window, 0.5)


@pytest.mark.parametrize("max_q", [1, 100])
def test_the_bound_only_chooses_the_kernel(max_q):
    check(Case([1, 13], [90, 200], 4, 2, 128, 4, 32, "bf16", 32, seed=3), max_q=max_q)


def test_long_sequence_among_short_ones():
    check(Case([1, 4, 1, 0, 200], [9000, 5, 1, 40, 5000], 8, 2, 128, 4, 64, "bf16", 64, seed=11), window=9)


@pytest.mark.parametrize("L,n", [(5, 3), (60, 20), (200, 150)])
def test_more_new_tokens_than_keys_sees_nothing(L, n):
    """Lengths that lie (more new tokens than keys): the tokens before the first key see nothing and count nothing."""
    check(Case([L], [n], 2, 1, 64, 4, 32, "bf16", 16, seed=1))


def test_keys_that_are_not_seen_reach_nothing():
    """NaN scales in rows behind the sequence, and in keys that come after a counted token: only such a key's own later
    weights are NaN."""
    c = Case([4], [37], 4, 2, 128, 4, 64, "bf16", 16, seed=6)   # rows behind 37 hold NaN scales
    lse, (mass, token) = log_sums(c), side(c)
    want, _ = run(c, lse, mass, token)
    pg = int(c.table[0, 36 // 16])
    c.arrays[1][pg, :, 36 % 16] = float("nan")                  # the last token's key
    got, _ = run(c, lse, mass, token)
    assert np.isnan(got[pg, :, 36 % 16]).all()
    got[pg, :, 36 % 16] = want[pg, :, 36 % 16]
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("L,D", [(4, 128), (70, 128), (70, 256), (70, 512)])
def test_rows_that_are_no_numbers_reach_only_what_they_see(L, D):
    """A token whose query, or whose lse, is NaN or infinite: keys that it does not see keep their masses bit for bit."""
    c = Case([L], [L + 90], 4, 2, D, 4, 64, "bf16", 16, seed=6)
    lse, (mass, token) = log_sums(c), side(c)
    want, _ = run(c, lse, mass, token)
    key = np.arange(L + 90)
    pg, row = c.table.cpu().numpy()[0][key // 16], key % 16
    first = 90 + L // 2   # the first key that is not seen by token L // 2 - 1, nor by those before it
    for bad in (float("nan"), float("inf"), float("-inf")):
        q, ls = c.q.clone(), lse.clone()
        q[: L // 2, :, 3] = bad
        ls[L // 4: L // 2] = bad
        got, _ = run(c, ls, mass, token, q=q)
        np.testing.assert_array_equal(got[pg, :, row][first:], want[pg, :, row][first:])
        assert np.isfinite(got[pg, :, row][first:]).all()


@pytest.mark.parametrize("L,D,bits", [(3, 128, 4), (70, 64, 8), (70, 128, 4), (70, 256, 8)])
def test_rows_and_keys_of_very_different_size(L, D, bits):
    """Query rows 2^-30 to 2^30 apart and keys 2^-20 to 2^20 apart, side by side: each keeps its own bits. Scores stay small by
    pairing: a key's and a row's factors enter the score together, so rows are taken whose factor undoes their keys'."""
    c = Case([L], [L + 200], 4, 2, D, bits, 32, "bf16", 16, seed=9)
    rng = np.random.default_rng(1)
    power = rng.integers(-20, 21, L + 200)
    table = c.table.cpu().numpy()[0]
    f = torch.from_numpy(2.0 ** power).float().cuda()
    pg = torch.from_numpy(table[np.arange(L + 200) // 16].astype(np.int64)).cuda()
    row = torch.arange(L + 200, device="cuda") % 16
    for a in c.arrays[1:3]:
        a[pg, :, row] = (a[pg, :, row].float() * f[:, None, None]).to(a.dtype)
    c.K = [k * (2.0 ** power)[None, :, None] for k in c.K]
    # every row sees scores of up to 2^20 times its own size: rows from 2^-30 to 2^-20 of a normal one
    scale = 2.0 ** rng.integers(-30, -19, c.total)
    c.q = (c.q.double().cpu() * torch.from_numpy(scale)[:, None, None]).to(torch.bfloat16).cuda()
    c.q64 = c.q.double().cpu().numpy()
    check(c)


def test_query_rows_far_apart_in_a_chunk():
    """One token's queries 2^40 times the others', over keys that are tiny: the others' scores come from their own bits."""
    c = Case([80], [300], 4, 2, 128, 4, 64, "bf16", 16, seed=12)
    c.arrays[1] *= 2.0 ** -40
    c.arrays[2] *= 2.0 ** -40
    c.K = [k * 2.0 ** -40 for k in c.K]
    f = np.full(80, 2.0 ** 40)
    f[::7] = 1.0
    f[::5] = 2.0 ** 20
    c.q = (c.q.double().cpu() * torch.from_numpy(f)[:, None, None]).to(torch.bfloat16).cuda()
    c.q64 = c.q.double().cpu().numpy()
    check(c)


@pytest.mark.parametrize("power", [20, -60, None])
def test_ranges_of_queries(power):
    """Queries beyond fp16's range and far below it, with keys that bring the scores back; and zeros."""
    c = Case([3], [50], 2, 1, 128, 8, 64, "bf16", 16, seed=2)
    f = 0.0 if power is None else 2.0 ** power
    c.q = (c.q.double() * f).to(torch.bfloat16)
    c.q64 = c.q.double().cpu().numpy()
    if power is not None:
        c.arrays[1] /= f
        c.arrays[2] /= f
        c.K = [k / f for k in c.K]
    check(c)


def test_strides_streams_graphs_and_repeats():
    c = Case([2, 1, 7], [130, 65, 300], 8, 2, 128, 4, 64, "bf16", 32, seed=8)
    lse, (mass, token) = log_sums(c), side(c)
    want, tok = run(c, lse, mass, token, 4, 0.5)
    wide = torch.zeros(c.total, 20, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:18:2] = c.q
    again, _ = run(c, lse, mass, token, 4, 0.5, q=wide[:, 2:18:2])
    np.testing.assert_array_equal(again, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, _ = run(c, lse, mass, token, 4, 0.5, stream=s)
    np.testing.assert_array_equal(other, want)
    m, t = torch.from_numpy(mass).cuda(), torch.from_numpy(token).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qda.qdecode_paged_weights(c.q, *c.arrays[:3], lse, m, t, c.q_start, c.kv_len, c.table, 7, 64, 4, 4, 0.5)
    m.copy_(torch.from_numpy(mass))
    g.replay()
    np.testing.assert_array_equal(m.cpu().numpy(), want)
    np.testing.assert_array_equal(t.cpu().numpy(), tok)


@pytest.mark.parametrize("q_lens,kv_lens,window", [([1] * 512, [1 + i % 90 for i in range(512)], 0), ([40, 0] * 60, [60, 9] * 60, 0),
                                                   ([33] * 100, [40 + i for i in range(100)], 17)])
def test_large_batches(q_lens, kv_lens, window):
    check(Case(q_lens, kv_lens, 2, 1, 64, 4, 32, "bf16", 16, seed=len(q_lens)), window, 0.5)


@pytest.mark.parametrize("L,D", [(2, 128), (64, 128), (64, 256), (64, 512)])
def test_own_workspace_is_enough_and_nothing_else_is_touched(L, D):
    """An installed workspace of exactly the bytes asked for, guard bytes around it and around masses and tokens."""
    c = Case([L, 1], [200, 150], 8, 2, D, 4, 64, "fp16", 32, seed=D)
    lse, (mass, token) = log_sums(c), side(c)
    want, tok = run(c, lse, mass, token)
    need = qda.qdecode_paged_weights_workspace_bytes(2, 8, 2, c.total, L, 0, D)
    assert (need > 0) == (L * 4 > 32 and D <= 256)
    buf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    try:
        if need:
            qda.qdecode_attn_set_workspace(buf[4096: 4096 + need])
        got, got_tok = run(c, lse, mass, token)
        if need:
            qda.qdecode_attn_set_workspace(buf[4096: 4096 + need - 256])
            with pytest.raises(qda.QdaError, match="-5"):
                run(c, lse, mass, token)
    finally:
        qda.qdecode_attn_set_workspace(None)
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(got_tok, tok)
    assert bool((buf[:4096] == 0x5A).all()) and bool((buf[4096 + need:] == 0x5A).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [700, 3]), ([4, 1, 0], [300, 1, 5]), ([200, 33], [1300, 33]), ([300], [300])])
@pytest.mark.parametrize("H,Hkv,D,bits,GS,dtype", [(8, 2, 128, 4, 64, "bf16"), (4, 4, 64, 8, 32, "fp16"), (4, 2, 256, 8, 64, "bf16"),
                                                   (16, 2, 512, 4, 128, "fp16")])
def test_log_sums_of_the_attention(H, Hkv, D, bits, GS, dtype, q_lens, kv_lens, causal):
    """lse against 64 bits: a score moves by ds (keys of 11 significant bits, as for the attention itself), queries are exact,
    the sum and its logarithm add 2^-17 and 2^-22 of the logarithm; the outputs are those of the call without lse."""
    c = Case(q_lens, kv_lens, H, Hkv, D, bits, GS, dtype, 16, seed=D, pad_rows=3)
    lse = torch.full((c.total + 3, H), 7.0, device="cuda")
    out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    qda.qdecode_paged_attn(c.q, *c.arrays, out, c.q_start, c.kv_len, c.table, max(q_lens), GS, bits, causal, lse=lse)
    assert torch.equal(out, c.run(causal))
    got = lse.cpu().numpy().astype(np.float64)
    assert (got[c.total:] == 7).all()
    for b, (L, n) in enumerate(zip(q_lens, kv_lens)):
        for h in range(H if L else 0):
            s, _, seen = R.scores(c, b, h)
            if not causal:
                seen = np.ones_like(seen)
            s = np.where(seen, s, -np.inf)
            ref = s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1))
            q, K = c.q64[c.start[b]: c.start[b] + L, h], c.K[b][h // (H // Hkv)]
            ds = 2.0 ** -11 * (np.abs(q) @ np.abs(K).T).max(1) / math.sqrt(D)
            err = np.abs(got[c.start[b]: c.start[b] + L, h] - ref)
            assert (err <= ds + 2.0 ** -17 + 2.0 ** -22 * np.abs(ref)).all(), (b, h, (err / ds).max())


def test_log_sums_where_nothing_is_seen():
    c = Case([4, 2], [2, 0], 2, 1, 64, 4, 32, "bf16", 16, seed=4)
    lse = torch.full((c.total, 2), 7.0, device="cuda")
    out = torch.empty_like(c.q)
    qda.qdecode_paged_attn(c.q, *c.arrays, out, c.q_start, c.kv_len, c.table, 4, 32, 4, lse=lse)
    got = lse.cpu().numpy()
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(R.log_sums(c)))
    assert np.isneginf(got[:2]).all() and np.isneginf(got[4:]).all() and np.isfinite(got[2:4]).all()


def test_log_sums_of_rows_done_anew():
    """A later token's key is far larger than what the others see: their rows are done anew in fp32, sums and all."""
    q_lens, kv_lens = [40], [200]
    c = Case(q_lens, kv_lens, 8, 2, 128, 4, 64, "bf16", 16, seed=5)
    pg = int(c.table[0, 199 // 16])
    c.arrays[1][pg, :, 199 % 16] *= 2.0 ** 20
    c.arrays[2][pg, :, 199 % 16] *= 2.0 ** 20
    c.K[0][:, 199] *= 2.0 ** 20
    lse = torch.zeros(40, 8, device="cuda")
    qda.qdecode_paged_attn(c.q, *c.arrays, torch.empty_like(c.q), c.q_start, c.kv_len, c.table, 40, 64, 4, lse=lse)
    ref = R.log_sums(c)[:39]
    err = np.abs(lse.cpu().numpy()[:39] - ref)
    assert (err <= 2.0 ** -11 * 30 + 2.0 ** -17).all(), err.max()   # (sum |q k| / sqrt(D) stays below 30 here)


def call(c, lse, mass, token, table=None, q_start=None, kv_len=None):
    """The status of a call with other tables; masses and tokens behind it."""
    m, t = torch.from_numpy(mass).cuda(), torch.from_numpy(token).cuda()
    i32 = lambda a, like: like if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    qda.qdecode_paged_weights(c.q, *c.arrays[:3], lse, m, t, i32(q_start, c.q_start), i32(kv_len, c.kv_len), i32(table, c.table),
                              max(c.q_lens), c.GS, c.bits, decay=0.5)
    torch.cuda.synchronize()
    return qda.qdecode_attn_device_status(), m.cpu().numpy(), t.cpu().numpy()


@pytest.mark.parametrize("L,D", [(1, 128), (3, 256), (40, 64), (70, 256), (70, 512)])
@pytest.mark.parametrize("page", [-1, 1 << 30])
def test_absent_pages_are_neither_read_nor_written(L, D, page):
    """A page outside the pool sets bit 8; keys of other pages come out as they would."""
    c = Case([L, 1], [L + 150, 33], 4, 2, D, 4, 64, "bf16", 16, seed=5)
    lse, (mass, token) = log_sums(c), side(c)
    status, want, tok = call(c, lse, mass, token)
    assert status == 0
    table = c.table.cpu().numpy()
    gone = table[0, [3, (L + 149) // 16]]
    table[0, [3, (L + 149) // 16]] = page
    status, got, tk = call(c, lse, mass, token, table=table)
    assert status == 8
    want[gone], tok[gone] = mass[gone], token[gone]
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(tk, tok)


@pytest.mark.parametrize("L", [2, 70])
def test_lengths_and_starts_that_lie(L):
    """A length beyond the table or negative, starts that fall or lie outside q: bit 8; the other sequence comes out right."""
    c = Case([L, L], [L + 60, L + 45], 4, 2, 128, 4, 64, "bf16", 16, seed=4)
    lse, (mass, token) = log_sums(c), side(c)
    _, want, tok = call(c, lse, mass, token)
    second = c.table.cpu().numpy()[1][: -(-(L + 45) // 16)]
    for n in (-3, 1 << 20, (1 << 31) - 1):
        status, got, tk = call(c, lse, mass, token, kv_len=[n, L + 45])
        assert status == 8
        np.testing.assert_array_equal(got[second], want[second])
        np.testing.assert_array_equal(tk[second], tok[second])
    for start in ([0, L, 3 * L], [-5, L, 2 * L], [L, 0, 2 * L], [0, 2 * L, L]):
        assert call(c, lse, mass, token, q_start=start)[0] == 8


def test_starts_that_count_rows_many_times():
    """More chunks than the workspace has room for: nothing is written."""
    B = 40
    c = Case([70] * B, [80] * B, 4, 2, 128, 4, 64, "bf16", 16, seed=4)
    lse, (mass, token) = log_sums(c), side(c)
    status, got, tk = call(c, lse, mass, token, q_start=[0, 70 * B] * (B // 2) + [0])
    assert status == 8
    np.testing.assert_array_equal(got, mass)
    np.testing.assert_array_equal(tk, token)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_captured(D):
    c = Case([70, 0, 33, 200], [170, 5, 33, 500], 4, 2, D, 8, 32, "fp16", 32, seed=8)
    lse, (mass, token) = log_sums(c), side(c)
    want, tok = run(c, lse, mass, token, 64, 0.5)
    m, t = torch.from_numpy(mass).cuda(), torch.from_numpy(token).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qda.qdecode_paged_weights(c.q, *c.arrays[:3], lse, m, t, c.q_start, c.kv_len, c.table, 200, 32, 8, 64, 0.5)
    for _ in range(3):
        m.copy_(torch.from_numpy(mass))
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(m.cpu().numpy(), want)
        np.testing.assert_array_equal(t.cpu().numpy(), tok)
