"""A cache with given keys and values, for the GPU tests of attention over it: written by
pace_cache_write into pages of old bytes, with the oracle's dequantised fp64 values beside it."""
import numpy as np
import torch

from oracle import cache_oracle as co

IO = {True: torch.bfloat16, False: torch.float32}


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(dtype) if dtype is not None else t).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rounded(x, bf16):
    """What a tensor of the io type holds of x, as fp32."""
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(IO[bf16]).float().numpy()


class Held:
    """k, v fp32 [B, L, Hkv, d], all of them in the cache."""

    def __init__(self, k, v, kind, g, bf16, gamma=1, page=16, seed=0):
        import bit_recurrent_state_amd as pace
        self.pace, self.bf16, self.gamma, self.group = pace, bf16, gamma, g
        self.B, self.L, self.H, self.d = k.shape
        k, v = rounded(k, bf16), rounded(v, bf16)
        self.k, self.v = (co.quantise(x, kind, g)[2] for x in (k, v))
        MP = -(-self.L // page)
        table = np.random.default_rng(seed).permutation(self.B * MP + 2)[: self.B * MP].reshape(self.B, MP).astype(np.int32)
        self.cfg = pace.CacheConfig(B=self.B, Hq=self.H * gamma, Hkv=self.H, d=self.d, num_pages=self.B * MP + 2,
                                    max_pages=MP, kind=kind, group=g, page=page, bf16_io=bf16)
        self.cache = torch.full((pace.cache_layout(self.cfg)["cache_bytes"],), 0xFF, dtype=torch.uint8, device="cuda")
        self.table = dev(table)
        pos = np.broadcast_to(np.arange(self.L, dtype=np.int32), (self.B, self.L))
        pace.cache_write(self.cfg, self.cache, self.table, dev(pos), dev(k, IO[bf16]), dev(v, IO[bf16]))

    def attend(self, q, T, parents=None, max_len=None, scale=None):
        """The last T tokens ask: (o, lse) fp64 [B, T, Hq, d], [B, T, Hq] for q fp32 [B, T, Hq, d]."""
        pace, cfg = self.pace, self.cfg
        tree = None if parents is None else dev(pace.tree_bits(parents)[None])
        o = torch.full((self.B, T, cfg.Hq, self.d), float("nan"), dtype=IO[self.bf16], device="cuda")
        lse = torch.full((self.B, T, cfg.Hq), float("nan"), device="cuda")
        max_len = max_len or self.L
        n = pace.cache_attention_workspace_bytes(cfg, T, max_len)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
        ctx = dev(np.full(self.B, self.L - T, dtype=np.int32))
        pace.cache_attention(cfg, self.cache, self.table, dev(q, IO[self.bf16]), ctx, o, lse=lse, tree=tree, scale=scale,
                             max_len=max_len, workspace=ws)
        return host(o), host(lse)

    def visible(self, T, parents=None):
        near = np.tril(np.ones((T, T), dtype=bool)) if parents is None else co.tree_mask(parents)
        return np.concatenate([np.ones((T, self.L - T), dtype=bool), near], axis=1)

    def wanted(self, q, T, parents=None, scale=None):
        """(o, lse, weights [B, T, Hq, L]) of the oracle."""
        scale = self.d ** -0.5 if scale is None else scale
        vis = self.visible(T, parents)
        o, lse, w = np.zeros(q.shape), np.zeros(q.shape[:-1]), np.zeros((*q.shape[:-1], self.L))
        for b in range(self.B):
            for hq in range(self.cfg.Hq):
                o[b, :, hq], lse[b, :, hq], w[b, :, hq] = co.attention(
                    q[b, :, hq].astype(np.float64), self.k[b, :, hq // self.gamma], self.v[b, :, hq // self.gamma], scale, vis)
        return o, lse, w
