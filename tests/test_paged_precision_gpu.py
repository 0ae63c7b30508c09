"""How exact the paged attention is over all of an output (not element by element), and that every key counts once."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda
from attention_quantized_kv_split_gb300 import build

from paged_ref import Case
from test_paged_range_gpu import VB, VS, put, reload, steer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    qda.lib()


# The error of an output over its norm, in units of the error that its one rounding to the type makes. Every rounding to b bits
# adds the variance of one such rounding to b bits: of a sum of products with values of either sign, a relative error of
# one factor is one of the sum. Chunks round keys, values and weights to 11 bits (a key's error enters by the score, times the
# scores' spread of up to 1.3 here): fp16 sqrt(1 + 1 + 1 + 1.3^2) = 2.2 units, operands below the largest of a block
# a little more; bf16 sqrt(1 + 3.7 / 64) = 1.03. Few tokens round the weights alone: sqrt(2) = 1.4 and 1.01.
BOUND = {("few", "bf16"): 1.1, ("few", "fp16"): 1.6, ("many", "bf16"): 1.15, ("many", "fp16"): 2.8}


@pytest.mark.parametrize("D,GS,bits", [(64, 32, 8), (128, 64, 4), (128, 128, 8), (256, 32, 4), (256, 128, 8), (512, 64, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind,q_lens,causal", [("few", [1, 2, 1, 2], True), ("many", [70, 1, 200, 40], True),
                                                ("many", [70, 33, 20, 40], False)])
def test_error_over_the_norm(D, GS, bits, dtype, kind, q_lens, causal):
    c = Case(q_lens, [1500, 900, 700, 2000], 8, 4, D, bits, GS, dtype, 32, seed=61)
    got = c.run(causal).double().cpu().numpy()
    ref, _ = c.reference(causal)
    once = torch.from_numpy(ref).to(c.q.dtype).double().numpy()
    ratio = np.linalg.norm(got - ref) / np.linalg.norm(once - ref)
    assert ratio <= BOUND[kind, dtype], ratio


@pytest.mark.parametrize("q_lens,kv_lens,D,GS,bits", [
    ([1], [2900], 128, 64, 4), ([1, 1], [1111, 1700], 64, 32, 8), ([2], [2500], 256, 64, 4), ([1], [1500], 512, 128, 8),
    ([100], [2700], 128, 64, 4), ([20], [2600], 64, 32, 8), ([70, 9], [1000, 1600], 256, 32, 8), ([90], [2500], 512, 128, 4)])
def test_every_key_counts_once(q_lens, kv_lens, D, GS, bits):
    # queries of zeros give every key the same weight; all values are zeros but those of 16 keys, which are ones: the result is
    # 16 over the number of keys wherever the 16 lie, nothing if they are lost and twice that if they are counted twice
    c = Case(q_lens, kv_lens, 4, 2, D, bits, GS, "bf16", 16, seed=62)
    c.q.zero_()
    c.arrays[VS].zero_()
    for n0 in range(0, max(kv_lens), 16):
        c.arrays[VB].zero_()
        want = torch.zeros(c.total, dtype=torch.float64)
        for b, n in enumerate(kv_lens):
            keys = range(min(n0, n), min(n0 + 16, n))
            if len(keys):
                put(c, VB, b, keys, 1.0)
            want[c.start[b]: c.start[b + 1]] = len(keys) / n
        got = c.run(False).double().cpu()
        assert ((got - want[:, None, None]).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * want[:, None, None]).all(), n0


@pytest.mark.parametrize("D,GS,bits", [(128, 64, 4), (256, 32, 8)])
@pytest.mark.parametrize("q_lens", [[40], [130, 7]])
def test_every_key_counts_once_under_a_causal_mask(D, GS, bits, q_lens):
    kv_lens = [600, 333][: len(q_lens)]
    c = Case(q_lens, kv_lens, 4, 2, D, bits, GS, "bf16", 16, seed=63)
    c.q.zero_()
    c.arrays[VS].zero_()
    for n0 in range(0, 600, 16):
        c.arrays[VB].zero_()
        want = torch.zeros(c.total, dtype=torch.float64)
        for b, (L, n) in enumerate(zip(q_lens, kv_lens)):
            keys = range(min(n0, n), min(n0 + 16, n))
            if len(keys):
                put(c, VB, b, keys, 1.0)
            seen = n - L + 1 + torch.arange(L, dtype=torch.float64)
            want[c.start[b]: c.start[b + 1]] = ((seen - n0).clamp(0, len(keys)) / seen)
        got = c.run().double().cpu()
        assert ((got - want[:, None, None]).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * want[:, None, None]).all(), n0


@pytest.mark.parametrize("D,GS,bits", [(64, 32, 8), (128, 64, 4), (256, 32, 4), (512, 64, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q_lens", [[1, 2], [70, 200]])
def test_small_values_beside_large_ones(D, GS, bits, dtype, q_lens):
    # one value in every hundred is 2^6 (4-bit codes) or 2^9 (8-bit) times larger than the others, and hardly weighs: the
    # others keep their bits beside it as far as the formats say
    kv_lens = [1300, 900]
    c = Case(q_lens, kv_lens, 4, 2, D, bits, GS, dtype, 32, seed=64)
    scores = []
    for b, n in enumerate(kv_lens):
        large = torch.arange(37, n, 100, device="cuda")
        pages = c.table[b, large // c.page].long()
        for a in (VS, VB):
            c.arrays[a][pages, :, large % c.page] *= 2.0 ** (6 if bits == 4 else 9)
        scores.append(np.where(np.arange(n) % 100 == 37, -40.0, 0.0))
        steer(c, scores[-1], b)
    reload(c)
    got = c.run(False).double().cpu().numpy()
    ref, _ = c.reference(False)
    # The largest that the root of the sum of squared errors should be, from the formats: a rounding that is off by at most e is
    # off by e / sqrt(3) in the mean square. The result's rounding: u of it. A weight's: 2^-11 of it, times its value's offset from
    # the middle of the codes (few tokens; next to no more than half the range, A) or its value (chunks). A value's operand in
    # chunks: 2^-11 of it or half of fp16's smallest step, 2^-25, where the block's unit (which never falls) brings the largest
    # value of a block, scale * (2^bits - 1) + |bias|, to [2^-6, 2^-5) with 4-bit codes, [2^-3, 2^-2) with 8-bit ones. The
    # scores are exact (keys of few bits). A quarter more for what is not independent.
    total = (torch.finfo(c.q.dtype).eps / 2) ** 2 / 3 * (ref ** 2).sum()
    for b, (L, n) in enumerate(zip(q_lens, kv_lens)):
        keys = torch.arange(n, device="cuda")
        pages = c.table[b, keys // c.page].long()
        s, z = (c.arrays[a][pages, :, keys % c.page].double().abs().cpu().numpy() for a in (VS, VB))   # [n, Hkv, groups]
        top = (s * (2 ** bits - 1) + z).max(-1)
        p = np.exp2(scores[b]) / np.exp2(scores[b]).sum()
        for h in range(2):
            unit = np.repeat([2.0 ** np.floor(np.log2(top[: j + 128, h].max())) for j in range(0, n, 128)], 128)[:n]
            step = 2.0 ** -25 * unit / 2.0 ** (-6 if bits == 4 else -3)
            off = (2.0 ** -11 * c.A[b][h]) ** 2
            if q_lens[0] > 8:
                off += np.maximum(2.0 ** -11 * np.abs(c.V[b][h]), step[:, None]) ** 2
            total += (p[:, None] ** 2 * off).sum() / 3 * L * (c.H // c.Hkv)
    ratio = np.linalg.norm(got - ref) / np.sqrt(total)
    assert ratio <= 1.25, ratio
