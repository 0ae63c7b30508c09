"""qdecode_paged_weights at the precision that it promises: bounds (weights_ref.py) that keys of 11 bits fail, as
test_weights_bounds.py shows."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_split_gb300 as qda

from weights_ref import Keys

pytestmark = pytest.mark.gpu

SHAPES = [(64, 4, 32), (64, 8, 64), (128, 4, 64), (128, 8, 32), (256, 4, 128), (256, 8, 32), (512, 4, 64), (512, 8, 128)]


@pytest.fixture(autouse=True)
def clean_status():
    qda.qdecode_attn_device_status()
    yield
    assert qda.qdecode_attn_device_status() == 0


def check(k, **kw):
    q, arrays, lse, mass, start, kv_len, table = k.device()
    token = torch.zeros(mass.shape, dtype=torch.int32, device="cuda")
    qda.qdecode_paged_weights(q, *arrays, lse, mass, token, start, kv_len, table, k.L, k.GS, k.bits, decay=0.5)
    ref, tol = k.weights(**kw)
    err = np.abs(k.of_pool(mass.cpu().numpy()) - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max()} of the tolerance"


@pytest.mark.parametrize("D,bits,GS", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_product_a_score(D, bits, GS, dtype):
    """D rows under a KV head, one for each of its dimensions (at D = 512 in the kernel for few rows)."""
    check(Keys(D // 4, D // 4 + 200, 8, 2, D, bits, GS, dtype, seed=D + bits).one_value_rows(0))


@pytest.mark.parametrize("D,bits,GS", SHAPES)
@pytest.mark.parametrize("rows", [8, 16, 32])
def test_one_product_a_score_in_few_rows(D, bits, GS, rows):
    k = Keys(rows // 4, 200, 8, 2, D, bits, GS, "bf16", seed=D + bits)
    for first in range(0, D, rows):
        check(k.one_value_rows(first))


@pytest.mark.parametrize("D,bits,GS", [(64, 8, 32), (128, 4, 64), (256, 8, 32)])
@pytest.mark.parametrize("below,far", [(12, 0), (20, 0), (20, 12), (24, 12), (24, 30)])
def test_queries_far_below_their_rows_largest(D, bits, GS, below, far):
    """Beside rows 2^far times as large: a row's values are held to 2^-27 of its largest."""
    check(Keys(64, 264, 8, 2, D, bits, GS, "bf16", seed=D + below).quiet_values(below, far), steps=8, q_off=2.0 ** -27)


@pytest.mark.parametrize("D,bits,GS", [(64, 8, 32), (128, 4, 64), (256, 8, 32), (512, 4, 64)])
@pytest.mark.parametrize("below,far", [(20, 0), (30, 0), (30, 12), (30, 30)])
@pytest.mark.parametrize("L", [2, 8])
def test_queries_far_below_their_rows_largest_in_few_rows(D, bits, GS, below, far, L):
    """To 2^-35 of its largest."""
    check(Keys(L, 200, 8, 2, D, bits, GS, "bf16", seed=D + below).quiet_values(below, far), steps=8, q_off=2.0 ** -35)
