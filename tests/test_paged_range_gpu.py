"""The paged attention's arithmetic at the ends of its range, against the plain 64-bit implementation (paged_ref): queries
and keys of zero, scales far apart, scores far apart, and what keys that a token does not see may leave in its output."""
import math

import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda
from attention_quantized_kv_split_gb300 import build

from paged_ref import Case

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
    torch.cuda.synchronize()   # absent pages leave their bit to nobody else
    qda.qdecode_attn_device_status()


KP, KS, KB, VP, VS, VB = range(6)


def put(c, array, b, keys, value):
    """Scales or biases of sequence b's keys (every head and group)."""
    keys = torch.as_tensor(list(keys), device="cuda")
    c.arrays[array][c.table[b, keys // c.page].long(), :, keys % c.page] = value


def reload(c):
    """The 64-bit keys and values anew, from what the device's arrays hold."""
    table = c.table.cpu().numpy()
    c.K, c.V, c.A = [], [], []
    for b, n in enumerate(c.kv_lens):
        out = []
        for p, s, z in (c.arrays[:3], c.arrays[3:]):
            pages = torch.as_tensor(table[b, : -(-n // c.page)], device="cuda").long()
            rows = lambda a: a[pages].transpose(1, 2).flatten(0, 1)[:n].transpose(0, 1)  # noqa: E731
            w = rows(p).cpu().numpy().view(np.uint32).astype(np.int64)
            code = np.stack([(w >> (c.bits * j)) & (2 ** c.bits - 1) for j in range(32 // c.bits)], -1).reshape(*w.shape[:2], -1)
            sc, bi = (np.repeat(rows(a).double().cpu().numpy(), c.GS, axis=-1) for a in (s, z))
            out.append((code * sc + bi, sc * (2 ** c.bits - 1) / 2))
        c.K.append(out[0][0])
        c.V.append(out[1][0])
        c.A.append(np.maximum(np.abs(out[1][0]), np.abs(out[1][1])))


def steer(c, scores, b=0):
    """Queries of ones and constant keys: key n of sequence b gets the score scores[n] in log2 units, rounded to the type."""
    c.q.fill_(1.0)
    c.q64[...] = 1.0
    c.arrays[KS].zero_()
    vals = torch.as_tensor(np.asarray(scores), dtype=torch.float64, device="cuda") * (math.log(2) / math.sqrt(c.D))
    keys = torch.arange(len(scores), device="cuda")
    c.arrays[KB][c.table[b, keys // c.page].long(), :, keys % c.page] = vals.to(c.q.dtype)[:, None, None]


KINDS = [(64, 32, 8, "bf16"), (128, 64, 4, "bf16"), (128, 128, 8, "fp16"), (256, 32, 8, "bf16"), (256, 64, 4, "fp16"),
         (512, 128, 4, "bf16")]
FEW, MANY = [1, 3], [64, 130]   # new tokens: the split kernel's calls, the chunk kernel's


@pytest.mark.parametrize("D,GS,bits,dtype", KINDS)
@pytest.mark.parametrize("q_lens", [FEW, MANY])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_size,k_size", [(0.0, 0.0), (0.0, 2.0 ** -22), (2.0 ** -23, 0.0)])
def test_queries_and_keys_of_zero(D, GS, bits, dtype, q_lens, causal, q_size, k_size):
    # a server's warm-up: nothing but zeros (or next to it) in the queries and in the pool's keys; lengths end inside a block
    c = Case(q_lens, [77, 300], 4, 2, D, bits, GS, dtype, 32, seed=41)
    c.q.fill_(q_size)
    c.q64[...] = q_size
    for a in (KS, KB):
        c.arrays[a].fill_(k_size)
    reload(c)
    c.check(c.run(causal), causal)
    assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("D,GS,bits", [(64, 64, 4), (128, 64, 4), (128, 32, 8), (256, 64, 8), (512, 128, 4)])
@pytest.mark.parametrize("small", [2.0 ** -24, 2.0 ** -22, 3 * 2.0 ** -20])
@pytest.mark.parametrize("rise", [3.0, 5.0, 7.5])
@pytest.mark.parametrize("q_lens", [[1], [70]])
def test_value_scales_below_the_normal_ones(D, GS, bits, small, rise, q_lens):
    # fp16: almost constant groups of values first, larger ones behind them with scores a few log2 units higher
    n = 600
    c = Case(q_lens, [n], 2, 1, D, bits, GS, "fp16", 32, seed=42)
    put(c, VS, 0, range(n), 2.0 ** -11)
    put(c, VS, 0, range(300), small)
    put(c, VB, 0, range(n), 0.0)
    steer(c, np.where(np.arange(n) < 300, 0.0, rise))
    reload(c)
    c.check(c.run(False), False)


@pytest.mark.parametrize("D,GS,bits,dtype", KINDS)
@pytest.mark.parametrize("q_lens", [[2], [8], [3, 5]])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40, 2.0 ** 60])
@pytest.mark.parametrize("what", ["v", "vb", "k"])
def test_large_keys_that_some_tokens_do_not_see(D, GS, bits, dtype, q_lens, size, what):
    # the last tokens' own keys or values are large (and finite): the tokens before them do not see those
    c = Case(q_lens, [90 + 111 * b for b in range(len(q_lens))], 4, 2, D, bits, GS, dtype, 32, seed=43)
    size = min(size, 2.0 ** 13) if dtype == "fp16" else size
    for b, n in enumerate(c.kv_lens):
        put(c, {"v": VS, "vb": VB, "k": KS}[what], b, [n - 1], size)
    reload(c)
    ref, tol = c.reference()
    got = c.run().double().cpu().numpy()
    # 2^13 * 255 is beyond fp16: the token that sees it may have a result that its type does not hold
    fits = np.abs(ref) + tol < torch.finfo(c.q.dtype).max
    if what == "k":   # its scores may be off by the rounding of the largest
        fits[c.start[1:] - 1] = False
    assert (np.abs(got - ref) <= tol)[fits].all()
    others = np.delete(np.arange(c.total), c.start[1:] - 1)
    assert fits[others].all() and np.isfinite(got[others]).all()


@pytest.mark.parametrize("D,GS,bits,dtype", KINDS)
@pytest.mark.parametrize("q_lens,kv_lens", [([64, 130], [200, 130]), ([150], [150]), ([129, 40, 300], [700, 513, 300]), ([40, 17], [300, 17])])
@pytest.mark.parametrize("size", [2.0 ** 9, 2.0 ** 20, 2.0 ** 40, 2.0 ** 60])
@pytest.mark.parametrize("what", ["v", "vb", "k", "kb"])
def test_large_keys_that_some_tokens_of_a_chunk_do_not_see(D, GS, bits, dtype, q_lens, kv_lens, size, what):
    # tokens in the middle and at the end of a chunk bring large (and finite) keys or values: the tokens before them do
    # not see those, the tokens behind do
    c = Case(q_lens, kv_lens, 4, 2, D, bits, GS, dtype, 32, seed=44)
    size = min(size, 2.0 ** 13) if dtype == "fp16" else size
    loud = [[n - 1, n - L // 2, n - L // 2 - 7] for L, n in zip(q_lens, kv_lens)]
    for b, keys in enumerate(loud):
        put(c, {"v": VS, "vb": VB, "k": KS, "kb": KB}[what], b, keys, size)
    reload(c)
    ref, tol = c.reference()
    got = c.run().double().cpu().numpy()
    fits = np.abs(ref) + tol < torch.finfo(c.q.dtype).max   # (65499 within 747 may be an infinity in fp16)
    quiet = np.zeros(c.total, bool)
    for b, (L, n) in enumerate(zip(q_lens, kv_lens)):   # tokens that see none of the large ones
        quiet[c.start[b]: c.start[b] + L] = n - L + np.arange(L) < min(loud[b])
    assert np.isfinite(got[quiet]).all()
    assert (np.abs(got - ref) <= tol)[quiet].all()
    # who sees a large value: within the rounding of the largest. Large keys' scores are rounded far beyond the tolerance's
    # bound on a factor: no bound on those tokens
    if what[0] == "v":
        assert (np.abs(got - ref) <= tol)[fits].all()
    assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("D,GS,bits,dtype", [(64, 32, 8, "bf16"), (128, 64, 4, "bf16"), (256, 64, 4, "fp16"), (512, 128, 8, "bf16")])
@pytest.mark.parametrize("zeros", [0, 1, 40])
def test_keys_that_grow_along_a_chunk(D, GS, bits, dtype, zeros):
    # a prompt whose first keys and values are zeros and whose others grow by a factor of four every eight tokens
    L = 140
    c = Case([L, 3], [L, 50], 4, 2, D, bits, GS, dtype, 16, seed=45)
    top = 12 if dtype == "fp16" else 30
    for a in (KS, KB, VS, VB):
        for n in range(L):
            size = 0.0 if n < zeros else 2.0 ** (min(2 * (n // 8), top) - (14 if a in (KS, KB) else 8))
            put(c, a, 0, [n], size if a in (KS, VS) else -size)
    c.q.mul_(2.0 ** -12)
    c.q64 *= 2.0 ** -12
    reload(c)
    ref, tol = c.reference()
    got = c.run().double().cpu().numpy()
    tame = tol < 0.2 * np.maximum(np.abs(ref).max(axis=-1, keepdims=True), 1e-3)   # scores small enough for a bound
    assert tame[: zeros + 24].all()
    assert (np.abs(got - ref) <= tol)[tame].all()


@pytest.mark.parametrize("D,GS,bits,dtype,far", [
    (64, 32, 8, "bf16", 22.3), (128, 64, 4, "bf16", 22.3), (128, 128, 8, "fp16", 20.3), (256, 32, 8, "bf16", 20.3),
    (256, 64, 4, "fp16", 20.3), (512, 128, 4, "bf16", 22.3)])
@pytest.mark.parametrize("q_lens", [FEW, MANY])
def test_weights_far_below_the_largest(D, GS, bits, dtype, far, q_lens):
    # a first key that draws nearly all of the attention and has a value of zeros: the result is what the others leave (some 2^-22
    # of the weight), and it keeps its bits. Weights are taken up by 2^7 (chunks) or 2^8 and more (few tokens), so that 2^-far
    # becomes 2^-13.3 to 2^-16.3 in fp16, off by at most 2^-25 absolute: 2^-8.7 of the weight or less, of which 7 / 15 or less
    # reaches the result (few tokens), or 2^-9.7 (chunks). Values of one sign, so that an error that all weights share shows;
    # the keys' few bits are exact in the operands, so scores are off by fp32's sums alone: D 2^-24 of far log2 units
    far += 2.0 * (q_lens is FEW)
    n = 16 if q_lens is FEW else 1500   # (a warp of the first kind has a reference of its own: all keys are one warp's)
    c = Case(q_lens, [n, n], 4, 2, D, bits, GS, dtype, 32, seed=46)
    c.arrays[VP].fill_(-1)   # the largest codes: as far from the middle of the range as they get
    for b in range(2):
        put(c, VS, b, range(n), 1.0)
        put(c, VB, b, range(n), 0.0)
        put(c, VS, b, [0], 0.0)
        steer(c, np.where(np.arange(n) == 0, far, 0.0), b)
    reload(c)
    got = c.run().double().cpu().numpy()
    u = torch.finfo(c.q.dtype).eps / 2
    for b, L in enumerate(q_lens):
        s = c.K[b][0, 0, 0] * math.sqrt(D) / math.log(2)   # the first key's score as the type holds it
        for i in range(L):
            seen = n - L + i + 1
            p = 2.0 ** -s / (1 + (seen - 1) * 2.0 ** -s)
            ref = np.repeat(p * c.V[b][:, 1:seen].sum(1), 2, axis=0)
            err = np.abs(got[c.start[b] + i] - ref).max() / ref.max()
            assert err <= 2 * u + 2.0 ** -11 + 2.0 ** -17 + math.expm1(D * 2.0 ** -24 * far * math.log(2))


@pytest.mark.parametrize("q_lens", [[1, 2, 1], [40, 70, 9], [200, 130, 1]])
@pytest.mark.parametrize("kv_len", [2 ** 31 - 1, 2 ** 31 - 513, 2 ** 31 - 800, 1 << 30])
@pytest.mark.parametrize("causal", [True, False])
def test_a_length_beyond_the_table(q_lens, kv_len, causal):
    # a length far beyond what the sequence's row of the table reaches: its tokens see all keys that the row has pages for, and
    # the other sequences of the batch are as they were
    c = Case(q_lens, [250, 320, 33], 8, 2, 128, 4, 64, "bf16", 32, seed=47)
    c.kv_len[1] = kv_len
    got = c.run(causal).double().cpu().numpy()
    for rows, (ref, tol) in ((slice(0, c.start[1]), c.reference(causal)), (slice(c.start[1], c.start[2]), c.reference(False)),
                             (slice(c.start[2], c.start[3]), c.reference(causal))):
        assert (np.abs(got - ref) <= tol)[rows].all()


@pytest.mark.parametrize("q_lens", [[1, 2, 1], [40, 70, 9]])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("what", ["negative", "beyond the table", "falling starts", "starts beyond q", "negative start", "idle"])
def test_bad_lengths_show_in_the_status(q_lens, causal, what):
    c = Case(q_lens, [250, 320, 64], 8, 2, 128, 4, 64, "bf16", 32, seed=48, extra_cols=0)
    checked, status = [0, 1, 2], 8
    if what == "negative":
        c.kv_len[2], checked = -5, [0, 1]
    elif what == "beyond the table":
        c.kv_len[1], checked = 321, [0, 2]
    elif what == "falling starts":
        c.q_start[3], checked = c.start[2] - 1, [0, 1]
    elif what == "starts beyond q":
        c.q_start[3] += 7
    elif what == "negative start":   # counts as 0
        c.q_start[0] = -3
    else:   # a sequence without new tokens: its length is not looked at
        c.q_start[3] = c.q_start[2]
        c.kv_len[2], checked, status = 1 << 30, [0, 1], 0
    got = c.run(causal).double().cpu().numpy()
    ref, tol = c.reference(causal)
    for b in checked:
        assert (np.abs(got - ref) <= tol)[c.start[b]: c.start[b + 1]].all()
    if what == "negative":
        assert not got[c.start[2]:].any()
    assert qda.qdecode_attn_device_status() == status


def test_good_lengths_leave_the_status_clean():
    for kv in ([250, 320, 64], [0, 1, 500]):
        for q_lens in ([1, 0, 3], [60, 70, 0]):
            c = Case(q_lens, kv, 8, 2, 128, 4, 64, "bf16", 32, seed=49, extra_cols=0, pad_rows=4)
            c.run(True)
            c.run(False)
            assert qda.qdecode_attn_device_status() == 0


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("where", ["free list", "table"])
def test_map_refuses_pages_whose_slots_pass_32_bits(page, where):
    # a broken free list or table: an id so large that id * page + row would come out as another page's slot
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    last = (2 ** 31 - 1) // page            # the largest page whose slots are int32 numbers
    for pid, good in ((last, True), (last + 1, False), (2 * (last + 1) - 1, False), (2 ** 31 - 1, False), (-9, False)):
        table = i32([[pid if where == "table" else -1, -1], [-1, -1]])
        free = i32([5, 6] if where == "table" else [pid, 6])
        old = [1, 0] if where == "table" else [0, 0]
        new = [2, 1]
        outs = dict(q_start=i32([0] * 3), kv_len=i32([0] * 2), slots=i32([7] * 4), positions=i32([7] * 4), used=i32([7]))
        qda.qdecode_paged_map(i32(old), i32(new), table, free, page, **outs)
        slots = [pid * page + old[0], pid * page + old[0] + 1] if good else [-1, -1]
        assert outs["slots"].tolist() == slots + [(5 if where == "table" else 6) * page, -1]
        if where == "free list":
            assert table[0].tolist() == [pid if good else -1, -1]
        assert outs["positions"].tolist() == [old[0], old[0] + 1, 0, -1]
        assert qda.qdecode_attn_device_status() == (0 if good else 8)


@pytest.mark.parametrize("q_lens", [[1, 1], [40, 50]])
@pytest.mark.parametrize("D", [64, 256])
def test_a_query_that_is_not_a_number(q_lens, D):
    # NaN in one query row: that row's output is NaN wherever the borders between the CTAs fall, and no other's
    for kv0 in range(1000, 1360, 12):
        c = Case(q_lens, [kv0, 700], 2, 2, D, 8, 32, "bf16", 32, seed=50)
        q = c.q.clone()
        q[q_lens[0], 1, 5] = float("nan")
        got = c.run(q=q)
        assert torch.isnan(got[q_lens[0], 1]).all(), kv0
        got[q_lens[0], 1] = c.run()[q_lens[0], 1]
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("q_lens", [[1, 2], [40, 90]])
def test_outputs_next_to_the_queries(q_lens):
    # queries and outputs back to back in one buffer, either way round, and one query row expanded over all tokens and heads
    c = Case(q_lens, [200, 333], 4, 2, 512, 4, 64, "bf16", 32, seed=51)
    ref = c.run()
    both = torch.zeros(2 * c.total, c.H, c.D, dtype=c.q.dtype, device="cuda")
    for q, out in ((both[: c.total], both[c.total:]), (both[c.total:], both[: c.total])):
        q.copy_(c.q)
        assert torch.equal(c.run(q=q, out=out), ref)
    with pytest.raises(qda.QdaError):
        c.run(q=both[: c.total], out=both[1: c.total + 1])
    one = c.q[:1, :1].expand(c.total, c.H, c.D)
    assert torch.equal(c.run(q=one, out=torch.empty_like(ref)), c.run(q=one.contiguous()))


@pytest.mark.parametrize("H,Hkv,D,GS,bits,page", [(5, 1, 128, 64, 4, 16), (12, 4, 64, 32, 8, 256), (64, 1, 64, 64, 4, 32),
                                                  (6, 2, 512, 32, 8, 16), (3, 3, 256, 128, 4, 64)])
def test_rows_done_anew_in_a_ragged_batch(H, Hkv, D, GS, bits, page):
    # forty sequences of any lengths (some idle, some with more tokens than keys), strided queries, absent pages, large keys
    # among the last third of a sequence's new tokens: eager, on another stream and from a captured graph
    rng = np.random.default_rng(D + H)
    q_lens = [int(x) for x in rng.integers(0, 60, 40)]
    q_lens[3], q_lens[7] = 200, 0
    kv_lens = [max(1, L + int(x)) for L, x in zip(q_lens, rng.integers(-10, 200, 40))]
    c = Case(q_lens, kv_lens, H, Hkv, D, bits, GS, "bf16", page, seed=52)
    quiet = np.zeros(c.total, bool)   # tokens that see none of the large keys
    for b, (L, n) in enumerate(zip(q_lens, kv_lens)):
        loud = sorted(int(k) for k in rng.integers(max(n - L // 3 - 1, 0), n, 3))
        for k in loud:
            put(c, int(rng.choice([KB, VS, VB])), b, [k], 2.0 ** int(rng.integers(8, 24)))
        quiet[c.start[b]: c.start[b + 1]] = n - L + np.arange(L) < loud[0]
    assert quiet.sum() > c.total / 3
    hidden = []
    for b in (3, 20, 30):
        col = int(rng.integers(0, -(-kv_lens[b] // page)))
        hidden += [(b, k) for k in range(col * page, min((col + 1) * page, kv_lens[b]))]
        gone = (b, col)
        c.table[gone] = c.arrays[0].shape[0] + b
    table = c.table.clone()
    c.table = torch.where((table >= c.arrays[0].shape[0]) | (table < 0), torch.zeros_like(table), table)
    reload(c)
    c.table = table
    for b, k in hidden:   # (what an absent page would hold is nothing, not page 0's rest)
        c.K[b][:, k] = c.V[b][:, k] = c.A[b][:, k] = 0
    wide = torch.zeros(c.total, H + 3, D + 8, dtype=c.q.dtype, device="cuda")
    wide[:, 2: H + 2, :D] = c.q
    q = wide[:, 2: H + 2, :D]
    ref, tol = c.reference(True, hidden)
    # Beside the tolerance of ordinary inputs: operands are off by 2^-13 of the largest key or value that the token sees (bounds of
    # what a scale and bias allow), that is what "done anew" is measured by
    for b, (L, n) in enumerate(zip(q_lens, kv_lens)):
        keys = torch.arange(n, device="cuda")
        pages = c.table[b, keys // page].long().clamp(0, c.arrays[0].shape[0] - 1)
        there = torch.tensor([(b, k) not in hidden for k in range(n)], device="cuda")[:, None, None]
        sizes = lambda x: torch.where(there, c.arrays[x][pages, :, keys % page].double().abs(), 0)  # noqa: E731
        top = [(sizes(x) * (2 ** bits - 1) + sizes(x + 1)).amax(-1).cummax(0).values.cpu().numpy() for x in (KS, VS)]
        for i in range(L):
            last = n - L + i
            r = int(c.start[b]) + i
            if last < 0 or not quiet[r]:
                continue
            seen = [k for k in range(last + 1) if (b, k) not in hidden]
            for h in range(H):
                g = h // (H // Hkv)
                ds = 2.0 ** -13 * top[0][last, g] * np.abs(c.q64[r, h]).sum() / math.sqrt(D)
                x = c.K[b][g, seen] @ c.q64[r, h] / math.sqrt(D)
                w = np.exp(x - x.max()) if len(seen) else np.zeros(0)
                with np.errstate(over="ignore"):
                    tol[r, h] += 2.0 ** -13 * top[1][last, g] + (np.expm1(2 * ds) * (w @ c.A[b][g, seen]) / w.sum() if len(seen) else 0)
    got = c.run(q=q)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.isfinite(got.double().cpu().numpy()).all()
    assert (err <= tol)[quiet].all(), (err / tol)[quiet].max()
    out, s, graph = torch.zeros_like(got), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    c.run(q=q, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, got)
    with torch.cuda.graph(graph):
        c.run(q=q, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
