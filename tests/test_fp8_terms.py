"""The checks of tests/fp8_cases.py tell: a model of the decode's 8-bit terms
passes them, and one with a mistake planted does not."""
import numpy as np
import pytest
import torch

from tests import fp8_cases as c


def bf16(x):
    return torch.from_numpy(x).bfloat16().double().numpy()


def scores_through(q, k, s, gain):
    x = (c.query_model(q, gain) @ k.T) * (s * c.SCALE)
    p = np.exp(x - x.max(1, keepdims=True))
    return bf16(p / p.sum(1, keepdims=True) @ k[:, :512] * s)


@pytest.mark.parametrize("ratio", [2.0 ** 8, 2.0 ** 13])
def test_queries_are_exact_to_a_ratio_of_2_to_the_13(ratio):
    q, _ = c.wide_query(20, ratio)
    q = q.double().numpy()
    assert np.array_equal(c.query_model(q), q)
    assert not c.query_floor(q).any()


@pytest.mark.parametrize("spread", [14, 20])
def test_queries_are_within_their_floor(spread):
    rng = np.random.default_rng(spread)
    q = torch.from_numpy(rng.standard_normal((50, 576)) * np.exp2(rng.integers(-spread, 1, (50, 576)))).bfloat16()
    q = q.double().numpy()
    assert np.all(np.abs(c.query_model(q) - q) <= c.query_floor(q))


@pytest.mark.parametrize("ratio", [2.0 ** 13, 2.0 ** 14])  # (further up the floor's worst case hides it)
def test_a_second_term_without_its_factor_is_told(ratio):
    q, k = c.wide_query(40, ratio)
    q = q[0].double().numpy()
    c.check_scores(scores_through(q, k, 2.0 ** -6, 16), q, k, 2.0 ** -6, 40, "two terms")
    with pytest.raises(AssertionError, match="times the tolerance"):
        c.check_scores(scores_through(q, k, 2.0 ** -6, 1), q, k, 2.0 ** -6, 40, "no factor")


@pytest.mark.parametrize("heads", [16, 40])
@pytest.mark.parametrize("n,gap", [(2000, 9.0), (2000, 16.5), (8192, 30.0), (8192, 60.0)])
def test_offsets_leave_weights_of_zero_alone(n, gap, heads):
    q, k, s = c.alternating_tail(heads, n, gap)
    q = q[0].double().numpy()
    c.check_alternating(c.decode_model(q, k, s, heads), q, k, s, "two terms")
    if heads > 32 and gap > 16:
        with pytest.raises(AssertionError, match="times the tolerance"):
            c.check_alternating(c.decode_model(q, k, s, heads, steps=False), q, k, s, "e5m2's own steps")


@pytest.mark.parametrize("heads", [16, 40])
@pytest.mark.parametrize("n,gap", [(3000, 6.0), (3000, 9.0), (20000, 12.0)])
def test_a_tail_dropped_halved_or_raised_is_told(n, gap, heads):
    q, k, s = c.peak_over_tail(heads, n, gap)
    q = q[0].double().numpy()
    c.check_tail(c.decode_model(q, k, s, heads), q, k, s, "two terms")
    for factor in (0, 0.5, 1.5):
        with pytest.raises(AssertionError, match="times the tolerance"):
            c.check_tail(c.decode_model(q, k, s, heads, tail=factor), q, k, s, f"tail times {factor}")


def test_a_tail_rounded_to_nearest_is_told():
    q, k, s = c.peak_over_tail(16, 20000, 12.0)
    q = q[0].double().numpy()
    with pytest.raises(AssertionError, match="times the tolerance"):
        c.check_tail(c.decode_model(q, k, s, 16, offsets=False), q, k, s, "no offsets")
