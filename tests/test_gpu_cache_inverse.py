"""What `inverse` of rotary is: with the same magnitude the transpose, with one over it the inverse."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_scene import dev, host  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_are_taken_back_with_one_over_the_magnitude(interleaved):
    """Two turns of at most 8 half steps of 2^-24 of m (|x_i| + |x_j|) each (tests/test_gpu_cache.py), the
    second of a pair whose sum is at most sqrt(2) m times the first's."""
    import bit_recurrent_state_amd as pace
    n, H, d, rd = 50, 2, 64, 48
    rng = np.random.default_rng(2)
    x = rng.standard_normal((n, H, d)).astype(np.float32)
    pos = dev(rng.integers(0, 100000, n).astype(np.int32))
    f, m = pace.rotary_freqs(rd, scaling="blend", factor=16.0, original_len=4096.0)
    assert m > 1.25
    f = dev(f)
    cfg = pace.RotaryConfig(Hq=0, Hk=H, d=d, rd=rd, interleaved=interleaved, bf16_io=False)
    y = dev(x)
    pace.rotary(cfg, pos, f, None, y, None, y, magnitude=m)
    pace.rotary(cfg, pos, f, None, y, None, y, magnitude=1.0 / m, inverse=True)
    part = np.arange(d)
    for i in range(rd // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
        part[a], part[b] = b, a
    both = np.abs(x) + np.abs(x[..., part])
    # the fp64 angles: 4 half steps of 2^-53 of the position in each turn, far below
    tol = 16 * 2.0 ** -24 * (1 + 2 ** 0.5) * both
    tol[..., rd:] = 0
    assert np.all(np.abs(host(y) - x) <= tol)
