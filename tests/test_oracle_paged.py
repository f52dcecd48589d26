"""The scale that the oracle gives for rounding errors of attention (no GPU): tight enough that a kernel which drops small
weights is seen, wide enough for the one that is there. The mistake is planted here, in numpy."""
import numpy as np
import pytest

import oracle.paged as op

U, FP32 = 2.0 ** -11, 2.0 ** -12     # f16's half step, and what fp32 costs


def sink_row(keys, below, seed=0):
    """One query, one head, d = 2 twice over (scores; values): a key with V = 0 and `keys` weights of 2^-below behind it."""
    rng = np.random.default_rng(seed)
    k, v = np.zeros((keys + 1, 1, 2)), np.zeros((keys + 1, 1, 2))
    k[0, 0, 0] = below * op.LN2
    k[1:, 0, 1] = rng.uniform(-0.1, 0.1, keys)
    v[1:, 0] = 1 + rng.standard_normal((keys, 2))
    return np.ones((1, 1, 2)), k, v, np.ones((1, keys + 1), bool)


def through_f16(q, k, v, shift):
    s = q[0, 0] @ k[:, 0].T
    p = np.exp(s - s.max())
    held = (p * 2.0 ** shift).astype(np.float16).astype(np.float64) * 2.0 ** -shift
    return (held @ v[:, 0]) / p.sum()


@pytest.mark.parametrize("keys,below", [(32768, 26), (16384, 25.3), (4096, 27)])
def test_the_scale_sees_weights_that_f16_drops(keys, below):
    q, k, v, seen = sink_row(keys, below)
    O, _, A = op.attend(q, k, v, seen, 1.0)
    dropped = np.abs(through_f16(q, k, v, 0) - O[0, 0])
    kept = np.abs(through_f16(q, k, v, 7) - O[0, 0])
    assert np.all(dropped > 0.5 * np.abs(O[0, 0]))
    assert np.all(dropped > (U + FP32) * A[0, 0]), "a bound that lets a dropped tail pass"
    assert np.all(kept <= U * A[0, 0])


def test_the_scale_without_a_floor_is_that_of_the_terms():
    q, k, v, seen = sink_row(1000, 22)
    O, L, A = op.attend(q, k, v, seen, 1.0, floor=0.0)
    p = np.exp((q[0, 0] @ k[:, 0].T) - 22 * op.LN2)
    assert np.allclose(A[0, 0], (p @ np.abs(v[:, 0])) / p.sum(), rtol=1e-12)
    cu = np.array([0, 1]), np.array([0, 1001])
    assert np.array_equal(op.prompt_attention(q, k, v, *cu, 1.0, floor=0.0)[2], A)
    pages = np.concatenate([k, np.zeros((7, 1, 2))]).reshape(63, 16, 1, 2), np.concatenate([v, np.zeros((7, 1, 2))]).reshape(63, 16, 1, 2)
    got = op.paged_attention(q, *pages, np.arange(63)[None], np.array([1001]), cu[0], 1.0, floor=0.0)
    assert np.array_equal(got[2], A) and np.array_equal(got[0], O) and np.array_equal(got[1], L)
    assert np.all(op.attend(q, k, v, seen, 1.0)[2] > A)
