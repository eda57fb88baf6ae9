"""Queries that are not finite, for every kind of work split: their own rows become NaN, every other row keeps
every bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_scene import Held, rounded  # noqa: E402

pytestmark = pytest.mark.gpu

# kind, d, group, bf16, T, gamma, L: one and two row tiles, four and eight waves, both joins
CASES = [("int8", 128, 128, True, 2, 4, 100), ("int8", 128, 128, True, 1, 4, 500), ("fp8", 128, 64, True, 12, 4, 300),
         ("int4", 64, 32, True, 12, 4, 200), ("int8", 64, 64, False, 40, 4, 200), ("fp8", 256, 64, False, 3, 4, 150),
         ("int8", 128, 32, False, 2, 4, 3000), ("int4", 128, 64, True, 2, 4, 9000)]


@pytest.mark.parametrize("kind,d,g,bf16,T,gamma,L", CASES)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_query_that_is_not_finite_stays_in_its_row(kind, d, g, bf16, T, gamma, L, bad):
    rng = np.random.default_rng(d + L)
    k, v = rng.standard_normal((2, 1, L, 1, d))
    held = Held(k, v, kind, g, bf16, gamma)
    q = rounded(rng.standard_normal((1, T, gamma, d)), bf16)
    clean, lse = held.attend(q, T)
    assert np.all(np.isfinite(clean)) and np.all(np.isfinite(lse))
    q[0, T - 1, 1, 7] = bad
    o, l2 = held.attend(q, T)
    keep = np.ones((T, gamma), dtype=bool)
    keep[T - 1, 1] = False
    assert np.array_equal(o[0][keep], clean[0][keep]) and np.array_equal(l2[0][keep], lse[0][keep])
    assert np.all(np.isnan(o[0, T - 1, 1])) and np.isnan(l2[0, T - 1, 1])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T", [1, 40])
def test_an_infinite_query_whose_scores_are_all_minus_infinity(bf16, T):
    """It sees tokens, so it is NaN and not a row that sees nothing."""
    k, v = np.full((1, 45, 1, 64), -1.0), np.ones((1, 45, 1, 64))
    held = Held(k, v, "int8", 64, bf16)
    for sign in (1, -1):
        q = np.ones((1, T, 1, 64), dtype=np.float32)
        q[0, 0, 0, 3] = sign * np.inf
        o, lse = held.attend(q, T)
        assert np.all(np.isnan(o[0, 0])) and np.isnan(lse[0, 0, 0])
        assert np.all(np.isfinite(o[0, 1:])) and np.all(np.isfinite(lse[0, 1:]))
