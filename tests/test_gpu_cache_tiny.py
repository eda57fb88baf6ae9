"""Codes of groups whose scales are the smallest that a cache holds."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as co  # noqa: E402
from cache_scene import dev, host  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int8", "int4", "fp8"])
def test_values_next_to_ties_at_every_small_scale(kind):
    """From 2^-108 on the bytes are the oracle's; under that a value is still within half a step (int) or half an
    e4m3 step (fp8), and 2^-22 of it."""
    import bit_recurrent_state_amd as pace
    rng = np.random.default_rng(6)
    exps, T, d, g, P = list(range(-126, -99)), 48, 64, 64, 16
    L = co.LEVELS[kind]
    s = np.ldexp(1 + rng.integers(0, 128, (len(exps), T, 1, 1)) / 128.0, np.array(exps)[:, None, None, None])
    mid = (rng.integers(-(L - 1), L - 1, (len(exps), T, 1, d)) + 0.5) if kind != "fp8" else \
        0.5 * (co.E4M3[(j := rng.integers(1, 125, (len(exps), T, 1, d)))] + co.E4M3[j + 1]) * rng.choice([-1, 1], j.shape)
    x = (mid * s).astype(np.float32)
    x = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, 0, 2 * x).astype(np.float32))
    x[..., 0] = (L * s[..., 0]).astype(np.float32)            # fixes the scale
    B = len(exps)
    cfg = pace.CacheConfig(B=B, Hq=1, Hkv=1, d=d, num_pages=B * 3, max_pages=3, kind=kind, group=g, page=P, bf16_io=False)
    oc = co.Cache(B=B, Hkv=1, d=d, kind=kind, group=g, page=P, num_pages=B * 3, max_pages=3)
    table = np.arange(B * 3, dtype=np.int32).reshape(B, 3)
    pos = np.broadcast_to(np.arange(T, dtype=np.int32), (B, T))
    want = np.zeros(oc.nbytes, dtype=np.uint8)
    co.write(oc, want, table, pos, x, x)
    cache = torch.zeros(oc.nbytes, dtype=torch.uint8, device="cuda")
    pace.cache_write(cfg, cache, dev(table), dev(pos), dev(x), dev(x))
    k, v = (torch.empty((B, T, 1, d), device="cuda") for _ in range(2))
    pace.cache_read(cfg, cache, dev(table), dev(pos), k, v)
    got = cache.cpu().numpy().reshape(B, -1)
    for b, e in enumerate(exps):
        if e >= -108:
            assert np.array_equal(got[b], want.reshape(B, -1)[b]), e
    q = np.abs(x.astype(np.float64) / s)
    step = 1.0
    if kind == "fp8":                                        # 2^-3 of the power of two under it, down to 2^-9
        step = np.ldexp(1.0, np.floor(np.log2(q * (1 + 2.0 ** -22) + 2.0 ** -20)).astype(int).clip(-6) - 3)
    for y in (k, v):
        off = np.abs(host(y) - x) / s
        assert np.all(off <= step * (0.5 + 2.0 ** -22) + np.abs(q) * 2.0 ** -22)
