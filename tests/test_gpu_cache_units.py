"""Attention over values of very different size, against the fp64 oracle: what a row may not see does
not touch it, and what it sees costs it no more than the rounding of its own weights.

Tolerance of a row's output in a channel of group G, over L tokens with exact weights w:
    E sum_t w_t |v_t| + L 2^-28 max_t (w_t max_G |v_t|)  (+ 2^-8 |o*| for bf16 outputs)
  E    2^-11 (bf16: weights times value scales in fp16) or 2^-21 (fp32: two fp16 pieces), 2 dz for the scores'
       own error dz ((d + 16) 2^-24, for fp32 + 2^-22, of sum |q k| scale, and 4 2^-24 (|z| + 16) for the
       exponential), (L / 8 + 64) 2^-24 for the fp32 sums;
  the second term: a weight so small that fp16 holds it with fewer bits, or not at all, is off by at most 2^-25
       of the row's unit, which the row's largest (weight x group's largest |value|) exceeds 2^3 times at
       least.
Only weights and values that the row sees, in the channel's own group, enter it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_scene import Held, rounded  # noqa: E402

pytestmark = pytest.mark.gpu

SHAPES = [("int8", 128, 128), ("int8", 64, 32), ("int4", 128, 32), ("int4", 64, 64), ("fp8", 128, 64), ("fp8", 256, 64)]


def tokens(rng, L, d, T, gamma):
    """Keys, values and queries; channel 0 sets a token's weight for all rows alike (see weigh)."""
    k, v = rng.standard_normal((2, 1, L, 1, d))
    q = rng.standard_normal((1, T, gamma, d))
    k[..., 0], q[..., 0] = 0.0, d ** 0.5 / 2
    return k, v, q


def weigh(k, t, nats):
    """Token t's scores go up by this much."""
    k[:, t, :, 0] = 2 * nats


def check(held, q, T, parents=None, max_len=None, rows=None):
    q = rounded(q, held.bf16)
    o, lse = held.attend(q, T, parents, max_len)
    wo, wl, w = held.wanted(q, T, parents)
    L, d, g = held.L, held.d, held.group
    vis = held.visible(T, parents)
    for hq in range(held.cfg.Hq):
        k, v = held.k[0, :, hq // held.gamma], np.abs(held.v[0, :, hq // held.gamma])
        top = v.reshape(L, d // g, g).max(-1).repeat(g, axis=-1)
        for i in range(T) if rows is None else rows:
            z_abs = (np.abs(k[vis[i]]) @ np.abs(q[0, i, hq].astype(np.float64))).max() * d ** -0.5
            dz = ((d + 16) * 2.0 ** -24 + (0 if held.bf16 else 2.0 ** -22)) * z_abs + 4 * 2.0 ** -24 * (z_abs + 16)
            sums = (L / 8 + 64) * 2.0 ** -24
            E = (2.0 ** -11 if held.bf16 else 2.0 ** -21) + 2 * dz + sums
            wt = w[0, i, hq][:, None]
            tol = E * (wt * v).sum(0) + L * 2.0 ** -28 * (wt * top).max(0)
            if held.bf16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(wo[0, i, hq])
            off = np.abs(o[0, i, hq] - wo[0, i, hq])
            assert np.all(off <= tol), (hq, i, off.max(), float((off / np.maximum(tol, 1e-300)).max()))
            assert abs(lse[0, i, hq] - wl[0, i, hq]) <= dz + sums + 2.0 ** -22 * abs(wl[0, i, hq])
    return o


@pytest.mark.parametrize("kind,d,g", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40, np.inf])
def test_a_large_value_in_a_later_draft_or_another_branch(kind, d, g, bf16, size):
    """Rows that may not see it are as exact as without it, and what they give does not change by a bit."""
    rng = np.random.default_rng(d + g)
    L, T, gamma = 70, 5, 4
    k, v, q = tokens(rng, L, d, T, gamma)
    plain = Held(k, v, kind, g, bf16, gamma)
    v = v.copy()
    v[0, L - 2, 0, 3::7] = size                            # token 3 of 5
    held = Held(k, v, kind, g, bf16, gamma)
    o = check(held, q, T, rows=None if np.isfinite(size) else [0, 1, 2])
    assert np.array_equal(o[:, :3], check(plain, q, T)[:, :3])
    parents = [-1, 0, 1, 0, 2]                             # node 3 is nobody's ancestor
    o = check(held, q, T, parents, rows=[0, 1, 2, 4])
    assert np.array_equal(o[:, [0, 1, 2, 4]], check(plain, q, T, parents)[:, [0, 1, 2, 4]])


@pytest.mark.parametrize("kind,d,g", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("L", [150, 1100])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40])
def test_a_large_value_of_small_weight(kind, d, g, bf16, size, L):
    """At the front, where it is met first, and at the end."""
    rng = np.random.default_rng(d + g + L)
    for at in (2, L - 9):
        for nats in (-16.0, -40.0):
            k, v, q = tokens(rng, L, d, 2, 4)
            weigh(k, at, nats)
            v[0, at] *= size
            check(Held(k, v, kind, g, bf16, 4), q, 2)


@pytest.mark.parametrize("kind,d,g", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("size", [2.0 ** -8, 2.0 ** -20, 2.0 ** -60])
def test_a_small_value_of_large_weight(kind, d, g, bf16, size):
    """A token that takes nearly all of the weight and gives nearly nothing, first or last."""
    rng = np.random.default_rng(d + g + 1)
    L = 150
    for at in (0, L - 9):
        for nats in (8.0, 30.0):
            k, v, q = tokens(rng, L, d, 2, 4)
            weigh(k, at, nats)
            v[0, at] *= size
            check(Held(k, v, kind, g, bf16, 4), q, 2)


@pytest.mark.parametrize("kind,d,g", [s for s in SHAPES if s[1] > s[2]])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -20, 2.0 ** -60, 0.0])
def test_groups_of_different_size(kind, d, g, bf16, size):
    """Every group of channels keeps its own precision; the first is zero until the last tokens."""
    rng = np.random.default_rng(d + g + 2)
    for T, gamma in ((2, 4), (9, 4)):
        k, v, q = tokens(rng, 140, d, T, gamma)
        v[..., g:2 * g] *= size or 2.0 ** -30
        if size == 0.0:
            v[:, :-20, :, :g] = 0.0
        check(Held(k, v, kind, g, bf16, gamma), q, T)


@pytest.mark.parametrize("kind,d,g", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
def test_values_that_grow_and_shrink_along_the_context(kind, d, g, bf16):
    """By 2^60 over 300 tokens, with scores that follow them down or up: rows of two tiles."""
    rng = np.random.default_rng(d + g + 3)
    L, T, gamma = 300, 12, 4
    ramp = np.linspace(-30, 30, L)
    for sign, follow in ((1, 0.0), (-1, 0.0), (1, -0.7), (-1, -0.7), (1, 0.4)):
        k, v, q = tokens(rng, L, d, T, gamma)
        v *= 2.0 ** (sign * ramp)[None, :, None, None]
        k[0, :, 0, 0] = 2 * follow * sign * ramp
        check(Held(k, v, kind, g, bf16, gamma), q, T)


@pytest.mark.parametrize("kind,d,g", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("L,max_len", [(150, None), (900, None), (5000, 5000)])
def test_mean_of_the_largest_values_is_finite(kind, d, g, bf16, L, max_len):
    """Infinities are held as 2^127: the mean of many is one, not infinite, however the context is cut."""
    rng = np.random.default_rng(L)
    v = rng.standard_normal((1, L, 1, d))
    v[..., 5], v[..., 17] = np.inf, -np.inf
    held = Held(rng.standard_normal((1, L, 1, d)), v, kind, g, bf16)
    o, _ = held.attend(np.zeros((1, 1, 1, d), dtype=np.float32), 1, max_len=max_len)
    want = held.v[0, 0, 0]
    assert np.all(np.isfinite(o))
    E = (2.0 ** -8 if bf16 else 0.0) + 2.0 ** -10 + (L / 8 + 64) * 2.0 ** -24
    for c in (5, 17):
        assert abs(o[0, 0, 0, c] - want[c]) <= E * abs(want[c])
