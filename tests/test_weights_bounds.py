"""The bounds of test_weights_precision_gpu.py, shown on the CPU to tell keys of 11 bits from keys of 22."""
import numpy as np
import pytest

from weights_ref import Keys, fewer_bits

SHAPES = [(64, 4, 32), (64, 8, 64), (128, 4, 64), (128, 8, 32), (256, 4, 128), (256, 8, 32), (512, 4, 64), (512, 8, 128)]


def worst(k, K, **kw):
    ref, tol = k.weights(**kw)
    return (np.abs(k.weights(K, **kw)[0] - ref) / tol).max()


@pytest.mark.parametrize("D,bits,GS", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_keys_of_eleven_bits_are_seen(D, bits, GS, dtype):
    """All values of the keys, and those of one slice of 64 dimensions alone, wherever it lies."""
    k = Keys(D // 4, D // 4 + 200, 8, 2, D, bits, GS, dtype, seed=D + bits).one_value_rows(0)
    assert worst(k, fewer_bits(k.K)) > 4
    for d in range(0, D, 64):
        assert worst(k, fewer_bits(k.K, slice(d, d + 64))) > 4, d


@pytest.mark.parametrize("D,bits,GS", SHAPES)
@pytest.mark.parametrize("rows", [8, 16, 32])
def test_keys_of_eleven_bits_are_seen_by_few_rows(D, bits, GS, rows):
    k = Keys(rows // 4, 200, 8, 2, D, bits, GS, "bf16", seed=D + bits)
    for first in range(0, D, rows):
        k.one_value_rows(first)
        assert worst(k, fewer_bits(k.K)) > 4, first


@pytest.mark.parametrize("D,bits,GS", SHAPES)
def test_keys_in_two_operands_stay_inside(D, bits, GS):
    """Each value to 11 bits and what those leave to 11 bits: within half of the bound."""
    k = Keys(D // 4, D // 4 + 200, 8, 2, D, bits, GS, "bf16", seed=D + bits).one_value_rows(0)
    high = fewer_bits(k.K)
    assert worst(k, high + fewer_bits(k.K - high)) < 0.5


def test_queries_held_to_their_bounds_stay_inside():
    """A row of 2^-far of its neighbours' largest, in steps of 2^-24 under a scale that brings those to 2^14, stays inside the
    bound for 2^-27 of its own largest and not inside that for 2^-39; so do odd values in steps of 2^-20, with 2^-35."""
    for L, below, far, step, bound in ((64, 20, 12, 2.0 ** -26, 2.0 ** -27), (64, 24, 12, 2.0 ** -26, 2.0 ** -27),
                                       (2, 30, 0, 2.0 ** -34, 2.0 ** -35)):
        k = Keys(L, 264, 8, 2, 256, 8, 32, "bf16", seed=3).quiet_values(below, far)
        exact, lse = k.q.copy(), k.lse()
        k.lse = lambda: lse   # noqa: B023
        ref, tol = k.weights(steps=8, q_off=bound)
        _, tight = k.weights(steps=8, q_off=2.0 ** -39)
        k.q = np.rint(exact / step) * step
        got, _ = k.weights()
        assert (np.abs(got - ref) <= tol).all()
        assert (np.abs(got - ref) > tight).any()
