"""The token that follows the accepted path, drawn with uniforms at the upper end of their range over vocabularies
whose last tokens have no weight: sums of many chunks, formed in more than one order, next to a border."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import draft_oracle as do  # noqa: E402
from test_gpu_draft import run_verify, same  # noqa: E402

pytestmark = pytest.mark.gpu


def masked(rng, shape, first, last):
    """Probabilities of which only tokens [first, last) have any, spread over so many powers of two that sums of them in 64 bits
    depend on their order."""
    p = np.zeros(shape, dtype=np.float32)
    z = np.exp(5.0 * rng.standard_normal((*shape[:-1], last - first)))
    p[..., first:last] = z / z.sum(-1, keepdims=True)
    return p


# V: one kernel; two kernels (few sequences); one kernel of many chunks (many sequences); more chunks than LDS holds sums of
@pytest.mark.parametrize("B,V,first,last", [(60, 32768, 0, 20000), (40, 131072, 0, 50000), (40, 131072, 9000, 131072), (130, 70000, 4096, 40000),
                                            (140, 270000, 0, 150000)])
@pytest.mark.parametrize("drawn", [False, True])
def test_uniforms_at_the_end_take_the_last_token_of_any_weight(B, V, first, last, drawn):
    rng, T = np.random.default_rng(V + B), 2 if drawn and B < 100 else 1
    target = masked(rng, (B, T, V), first, last)
    draft = (0.5 * target + 0.5 * masked(rng, (B, T, V), first, last)).astype(np.float32) if drawn else None
    tokens = rng.integers(first, last, size=(B, T))
    par = np.array([[-1, 0][:T]] * B)
    for u0 in (1.0, np.nextafter(np.float32(1), np.float32(0)), 7.0):
        u = np.full((B, T), u0, dtype=np.float32)           # (the child is refused)
        want = do.draft_verify(target, draft, tokens, par, u, [T] * B)
        got = run_verify(target, draft, tokens, par, u)
        assert (got[2] >= 0).all()
        same(got, want)
