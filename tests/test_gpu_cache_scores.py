"""Attention where scores, keys or queries are far from 1, against the fp64 oracle.

In these cases one token leads its row by far more than a score's error, so the softmax is
that token's one-hot whatever the scores' last bits, which the tests check on the oracle's side first.
What is left of the error is the leader's own weight: 2^-11 of the output (bf16: a weight is rounded to
fp16) or 2^-21 (fp32: two fp16 pieces), half a bf16 step (2^-8) for bf16 outputs, and for lse
(d + 16) 2^-24 + 2^-21 of sum |q k| scale (the fp32 product, two-piece queries, the base-2 units and back)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_scene import Held, rounded  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = [("int8", 128, 128), ("int4", 128, 32), ("fp8", 64, 64)]


def one_hot(held, q, T=1, tokens=None, max_len=None, sequences=None):
    """Checks rows that one token leads (of these sequences; the others only have to be finite)."""
    s = held.d ** -0.5
    wo, wl, w = held.wanted(q, T)
    dz = np.zeros(q.shape[:-1])
    sequences = list(range(held.B)) if sequences is None else sequences
    for b in sequences:
        for hq in range(held.cfg.Hq):
            k = held.k[b, :, hq // held.gamma]
            z_abs = (np.abs(q[b, :, hq].astype(np.float64)) @ np.abs(k).T * abs(s)).max(-1)
            dz[b, :, hq] = ((held.d + 16) * 2.0 ** -24 + 2.0 ** -21) * z_abs
            assert np.all(z_abs * 1.45 < 2.0 ** 128), "the case has to fit fp32"
            z = np.where(held.visible(T), q[b, :, hq].astype(np.float64) @ k.T * s, -np.inf)
            z = np.sort(z, axis=-1)
            if z.shape[-1] > 1:
                assert np.all(z[:, -1] - z[:, -2] > 4 * dz[b, :, hq] + 60), "the case has to be one-hot"
    if tokens is not None:
        assert np.all(w[sequences].argmax(-1) == tokens)
    o, lse = held.attend(q, T, max_len=max_len)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    E = 2.0 ** -8 * (1 + 2.0 ** -11) + 2.0 ** -11 if held.bf16 else 2.0 ** -21
    for b in sequences:
        assert np.all(np.abs(o[b] - wo[b]) <= E * np.abs(wo[b]) + 1e-30)
        assert np.all(np.abs(lse[b] - wl[b]) <= dz[b] + 2.0 ** -21 * np.abs(wl[b]))


@pytest.mark.parametrize("kind,d,g", KINDS)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("size", [1e6, 1e9, 1e12, 1e20, 1e30])
def test_scores_of_every_size(kind, d, g, bf16, size):
    """Queries so long that scores reach 1e31: the leader's weight is exp(0) exactly, however coarse
    fp32 is at its score."""
    rng = np.random.default_rng(int(np.log10(size)) + d)
    k, v = rng.standard_normal((2, 1, 300, 1, d))
    held = Held(k, v, kind, g, bf16, gamma=3)
    q = rounded(rng.standard_normal((1, 2, 3, d)) * size, bf16)
    one_hot(held, q, T=2)
    one_hot(held, q, T=2, max_len=4000)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("size", [1e28, 1e31, 1e34])
def test_rows_whose_every_score_is_far_below_zero(bf16, size):
    """A softmax does not depend on a common offset: rows whose scores are all near -1e30 or -1e35 are not
    rows that see nothing."""
    rng = np.random.default_rng(3)
    d = 128
    k, v = rng.standard_normal((2, 1, 40, 1, d))
    k = np.abs(k) + 0.5
    held = Held(k, v, "int8", 128, bf16)
    q = rounded(-(np.abs(rng.standard_normal((1, 1, 1, d))) + 0.5) * size, bf16)
    one_hot(held, q)
    alone = Held(k[:, :1], v[:, :1], "int8", 128, bf16)
    one_hot(alone, q)


@pytest.mark.parametrize("kind,d,g", KINDS)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("size", [1e30, 1e34, 1e36, np.inf])
@pytest.mark.parametrize("channels", [1, 7])
def test_keys_up_to_the_largest_that_a_cache_holds(kind, d, g, bf16, size, channels):
    """A cache holds magnitudes up to 2^127 (infinities are stored so).  Scores over them are
    finite for queries of ordinary size and smaller, so rows have to be as well."""
    rng = np.random.default_rng(channels + d)
    k, v = rng.standard_normal((2, 2, 77, 1, d))
    for b, t, sign in ((0, 5, 1), (0, 40, -1), (1, 76, 1)):
        k[b, t, 0, rng.permutation(d)[:channels]] = sign * size
    held = Held(k, v, kind, g, bf16, gamma=2)
    for scale in (1.0, 0.1, 1e-5):
        q = rounded(np.abs(rng.standard_normal((2, 1, 2, d))) * scale, bf16)
        one_hot(held, q, tokens=np.array([5, 76]).reshape(2, 1, 1))
    # the other way round: one token far above, one or two far below the ordinary ones
    q = rounded(-np.abs(rng.standard_normal((2, 1, 2, d))) * 0.3, bf16)
    one_hot(held, q, sequences=[0], tokens=np.array([40]).reshape(1, 1, 1))


@pytest.mark.parametrize("bf16", [True, False])
def test_tiny_queries_over_large_keys_and_the_reverse(bf16):
    """Scores of ordinary size from factors that are not: queries of 1e-30 over keys of 1e30, and queries
    of 1e25 over keys of 1e-25.  Tolerance as for ordinary scores (tests/test_gpu_cache.py)."""
    rng = np.random.default_rng(9)
    d, L = 128, 200
    for size in (1e30, 1e36, 1e-25):
        k, v = rng.standard_normal((2, 1, L, 1, d))
        held = Held(k * size, v, "int8", 64, bf16)
        q = rounded(rng.standard_normal((1, 1, 1, d)) / size, bf16)
        o, lse = held.attend(q, 1)
        wo, wl, w = held.wanted(q, 1)
        z_abs = (np.abs(q[0, 0].astype(np.float64)) @ np.abs(held.k[0, :, 0]).T).max() * d ** -0.5
        dz = ((d + 16) * 2.0 ** -24 + (0 if bf16 else 2.0 ** -22)) * z_abs + 4 * 2.0 ** -24 * (z_abs + 16)
        sums = (L / 8 + 64) * 2.0 ** -24
        E = (2.0 ** -11 if bf16 else 2.0 ** -21) + 2 * dz + sums
        v = np.abs(held.v[0, :, 0])
        tol = E * (w[0, 0] @ v) + L * 2.0 ** -28 * v.max()
        if bf16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(wo[0, 0])
        assert np.all(np.abs(o[0, 0] - wo[0, 0]) <= tol)
        assert np.all(np.abs(lse - wl) <= dz + sums + 2.0 ** -22 * np.abs(wl))
