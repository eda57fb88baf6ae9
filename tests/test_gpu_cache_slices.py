"""The last token of long prompts, as a slice of their projections: token strides of millions of elements."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_scene import dev  # noqa: E402

pytestmark = pytest.mark.gpu


def test_last_tokens_of_long_prompts_as_slices():
    import bit_recurrent_state_amd as pace
    B, T, H, d = 3, 4096, 32, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((B, T, H, d), generator=gen, device="cuda").to(torch.bfloat16)[:, -1:] for _ in range(3))
    assert q.stride(0) == 1 << 24
    cfg = pace.CacheConfig(B=B, Hq=H, Hkv=H, d=d, num_pages=B, max_pages=1, kind="int8", group=128, page=16)
    table = dev(np.arange(B, dtype=np.int32)[:, None])
    pos, ctx = dev(np.zeros((B, 1), dtype=np.int32)), dev(np.zeros(B, dtype=np.int32))
    rot = pace.RotaryConfig(Hq=H, Hk=H, d=d, rd=d)
    f = dev(pace.rotary_freqs(d)[0])
    n = pace.cache_attention_workspace_bytes(cfg, 1, 16)
    assert n == 0
    out = []
    for x, y, z in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
        cache = torch.zeros(pace.cache_layout(cfg)["cache_bytes"], dtype=torch.uint8, device="cuda")
        xr, yr = torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda")
        pace.rotary(rot, dev(np.arange(5, 5 + B, dtype=np.int32)), f, x[:, 0], y[:, 0], xr, yr)
        pace.cache_write(cfg, cache, table, pos, y, z)
        o = torch.empty((B, 1, H, d), dtype=torch.bfloat16, device="cuda")
        pace.cache_attention(cfg, cache, table, x, ctx, o, max_len=16)
        out.append((cache, xr, yr, o))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    wide = torch.zeros((B, T, H, d), dtype=torch.bfloat16, device="cuda")
    k2, v2 = wide[:, -1:], torch.empty((B, 1, H, d), dtype=torch.bfloat16, device="cuda")
    k1, v1 = torch.empty_like(v2), torch.empty_like(v2)
    pace.cache_read(cfg, out[0][0], table, pos, k1, v1)
    pace.cache_read(cfg, out[0][0], table, pos, k2, v2)
    assert torch.equal(k1, k2) and torch.equal(v1, v2) and not wide[:, :-1].any()
