"""Attention at the end of the largest context that positions in 32 bits allow."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as co  # noqa: E402
from cache_scene import dev, host, rounded  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_last_positions_of_the_largest_table():
    """2^31 - 16 positions, of which the first and the last 48 are on pages that are there.  Tolerance as for
    ordinary scores over the tokens that are there (tests/test_gpu_cache.py)."""
    import bit_recurrent_state_amd as pace
    P, MP, d, g = 16, (1 << 27) - 1, 64, 64
    cfg = pace.CacheConfig(B=1, Hq=4, Hkv=1, d=d, num_pages=7, max_pages=MP, kind="int4", group=g, page=P)
    rng = np.random.default_rng(3)
    table = torch.full((1, MP), -1, dtype=torch.int32, device="cuda")
    table[0, :3] = dev(np.array([2, 0, 4], dtype=np.int32))
    table[0, -3:] = dev(np.array([6, 1, 3], dtype=np.int32))
    at = np.concatenate([np.arange(48), np.arange(MP * P - 48, MP * P)]).astype(np.int32)
    k, v = (rounded(x, True) for x in rng.standard_normal((2, at.size, 1, d)))
    cache = torch.full((pace.cache_layout(cfg)["cache_bytes"],), 0xFF, dtype=torch.uint8, device="cuda")
    pace.cache_write(cfg, cache, table, dev(at[None]), dev(k[None], torch.bfloat16), dev(v[None], torch.bfloat16))
    q = rounded(rng.standard_normal((1, 2, 4, d)), True)
    o = torch.full((1, 2, 4, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 2, 4), float("nan"), device="cuda")
    ws = torch.empty(pace.cache_attention_workspace_bytes(cfg, 2, MP * P), dtype=torch.uint8, device="cuda")
    print("[cache] attention over 2^31 - 16 positions", flush=True)
    pace.cache_attention(cfg, cache, table, dev(q, torch.bfloat16), dev(np.array([MP * P - 2], dtype=np.int32)), o,
                         lse=lse, workspace=ws)
    kq, vq = (co.quantise(x[:, 0], "int4", g)[2] for x in (k, v))
    L = at.size
    for i in range(2):
        seen = np.broadcast_to(at <= MP * P - 2 + i, (4, L))
        wo, wl, w = co.attention(q[0, i].astype(np.float64), kq, vq, d ** -0.5, seen)
        z_abs = (np.abs(q[0, i].astype(np.float64)) @ np.abs(kq).T * d ** -0.5).max(-1)
        dz = (d + 16) * 2.0 ** -24 * z_abs + 4 * 2.0 ** -24 * (z_abs + 16)
        sums = (L / 8 + 64) * 2.0 ** -24
        tol = (2.0 ** -11 + 2 * dz + sums)[:, None] * (w @ np.abs(vq)) + L * 2.0 ** -28 * np.abs(vq).max()
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(wo)
        assert np.all(np.abs(host(o)[0, i] - wo) <= tol)
        assert np.all(np.abs(host(lse)[0, i] - wl) <= dz + sums + 2.0 ** -22 * np.abs(wl))


@pytest.mark.parametrize("n,d,wide", [((1 << 24) + 3, 2, False), ((1 << 26) + 5, 16, True)])
def test_rotary_of_more_tokens_than_a_launch_holds(n, d, wide):
    """Cut into launches: the tokens around the cuts and at the ends, against calls of their own."""
    import bit_recurrent_state_amd as pace
    print(f"[cache] rotary of {n} tokens", flush=True)
    cfg = pace.RotaryConfig(Hq=0, Hk=1, d=d, rd=d)
    gen = torch.Generator(device="cuda").manual_seed(4)
    pos = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda", dtype=torch.int32)
    x = torch.randn((n, 1, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    f = dev(pace.rotary_freqs(d)[0])
    cuts = [0] + list(range(1 << 23, n, 1 << 23)) + [n]
    parts = []
    for c in cuts:
        lo, hi = max(0, c - 300), min(n, c + 300)
        part = x[lo:hi].clone()
        pace.rotary(cfg, pos[lo:hi].clone(), f, None, part, None, part)
        parts.append((lo, hi, part))
    pace.rotary(cfg, pos, f, None, x, None, x)
    for lo, hi, part in parts:
        assert torch.equal(x[lo:hi], part)
