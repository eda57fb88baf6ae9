"""Verification of many refused siblings: what is left of a row shrinks with every one of them, and the following token and
the next sibling's chance are taken from it however little it is."""
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import draft_oracle as do  # noqa: E402
from test_gpu_draft import IO, run_verify, same  # noqa: E402


def siblings(seed, B, T, V, bf16, keep):
    """A root with T - 1 children whose tokens are not the one of which most is left (but, with `keep`, the last one's), and rows
    of which a third to a fiftieth is left by every refusal."""
    rng = np.random.default_rng(seed)
    target, draft = np.zeros((B, T, V), dtype=np.float32), np.zeros((B, T, V), dtype=np.float32)
    tokens, best = np.zeros((B, T), dtype=np.int64), rng.integers(0, V, size=B)
    for b in range(B):
        for x, most in ((target, 0.985), (draft, rng.uniform(0.7, 0.97))):
            z = rng.random((T, V)) ** 4
            z[:, best[b]] = 0.0
            x[b] = (1.0 - most) * z / z.sum(-1, keepdims=True)
            x[b, :, best[b]] = most
        others = np.setdiff1d(np.arange(V), best[b])
        tokens[b] = rng.choice(others, T)
        if keep:
            tokens[b, -1] = best[b]
    target, draft = (torch.from_numpy(x).to(IO[bf16]).float().numpy() for x in (target, draft))
    u = rng.random((B, T)).astype(np.float32)
    u[::2, 0] = 0.0                            # (the first token of which anything is left)
    u[:, 1:] = 1.0
    if keep:
        u[:, -1] = rng.random(B)
    return target, draft, tokens, np.array([[-1] + [0] * (T - 1)] * B), u


def literally(target, draft, tokens, u):
    """The accepted child (0: none) and the following token of one star, in rational numbers."""
    number = lambda row: [Fraction(float(x)) for x in row]  # noqa: E731
    w, W, q, x = number(target[0]), Fraction(1), number(draft[0]), 0
    for c in range(1, len(tokens)):
        t = int(tokens[c])
        if Fraction(float(u[c])) * W * q[t] < w[t]:
            x, w = c, number(target[c])
            break
        w = [max(a - W * b, Fraction(0)) for a, b in zip(w, q)]
        W = sum(w)
    at, passed = Fraction(0), Fraction(float(u[0])) * sum(w)
    for t, a in enumerate(w):
        at += a
        if at > passed:
            return x, t
    raise AssertionError


@pytest.mark.parametrize("T", [5, 20, 40])
def test_the_oracle_goes_by_what_is_left(T):
    """64 bits, refusal by refusal, against rational numbers."""
    for keep in (False, True):
        target, draft, tokens, par, u = siblings(T, 12, T, 5, False, keep)
        nodes, counts, following = do.draft_verify(target, draft, tokens, par, u, [T] * 12)
        for b in range(12):
            x, t = literally(target[b], draft[b], tokens[b], u[b])
            assert (nodes[b, 1] if counts[b] > 1 else 0, following[b]) == (x, t)


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("keep", [False, True])
# (one kernel; two kernels, which go on with the walk; more nodes than a wave looks at once)
@pytest.mark.parametrize("B,T,V", [(200, 5, 5), (200, 20, 5), (60, 33, 600), (16, 9, 40000), (16, 20, 40000), (8, 100, 7), (140, 24, 3000)])
def test_what_is_left_after_many_refusals(B, T, V, keep, bf16):
    target, draft, tokens, par, u = siblings(B * T + V, B, T, V, bf16, keep)
    same(run_verify(target, draft, tokens, par, u, bf16=bf16), do.draft_verify(target, draft, tokens, par, u, [T] * B))
