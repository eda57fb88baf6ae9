"""GPU parity of the attention-layer operators (include/pace_cache.h) against the fp64 oracle:
rotary positions, the cache's bytes as written and its values as read, and attention over it.

Tolerances, derived from what the kernels round:
  rotary: cosine, sine, their magnitude product, two products and a sum in fp32, at most 8 half
    steps of 2^-24 of m (|x_i| + |x_j|), and the fp64 angle, four half steps of 2^-53 of |pos|
    (frequencies are at most 1); bf16 outputs add half a bf16 step, 2^-8 |y|.
  cache bytes: equal (scale and code decisions are exact); values read: equal to the oracle's
    rounded once to the io type.
  attention, per output |o - o*| <= E sum_t w_t |v_t| + F max|v| + 2^-8 |o*| (bf16 only), with
    w the exact weights and
      E = 2^-11 (bf16; weights in fp16) or 2^-21 (fp32; two fp16 pieces), plus
          2 dz (numerator and denominator), dz the error of a score in e-units:
          ((d + 16) 2^-24 + 2^-22 for the two-piece queries) max_t scale sum_c |q_c k_tc|
          + 4 2^-24 (|z| + 16) for the exponent's argument and the exponential, plus
          (L / 8 + 64) 2^-24 for the fp32 sums over L tokens (32 at a time) and their joins;
      F = L 2^-28: weights under 2^-14 lose bits in fp16 (2^-25 absolute, weights lifted by 2^7,
          values within 2^3 of their unit; the second piece of fp32 halves it again).
  lse: dz + (L / 8 + 64) 2^-24, plus 2^-22 |lse| for the logarithm and its scaling.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as co  # noqa: E402

pytestmark = pytest.mark.gpu

IO = {True: torch.bfloat16, False: torch.float32}


def _pace():
    import bit_recurrent_state_amd as pace
    return pace


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(dtype) if dtype is not None else t).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rounded(x, bf16):
    """fp64 values of what a tensor of the io type holds of x."""
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(IO[bf16]).float().numpy()


# ----------------------------------------------------------------------------- rotary

ROTARY = [
    # n, Hq, Hk, d, rd, interleaved, bf16, inverse, far
    (1, 4, 2, 64, 64, False, True, False, 10),
    (7, 3, 1, 128, 64, False, True, False, 131072),
    (5, 2, 2, 128, 32, True, False, True, 2 ** 30),
    (3, 1, 1, 256, 16, False, False, False, 4096),
    (4, 2, 1, 80, 24, True, True, False, 4096),       # units of 8
    (4, 2, 1, 70, 22, False, True, True, 4096),       # pair by pair
    (2, 1, 3, 10, 10, True, False, False, 100),
    (8200, 1, 1, 64, 16, False, True, False, 1 << 20),  # several tokens a workgroup, ragged end
]


def _rotary_tol(x, pos, pairs_of, magnitude, y, bf16):
    a = np.abs(x)
    both = a + a[..., pairs_of]
    angle = 8 * 2.0 ** -24 + 4 * 2.0 ** -53 * np.abs(pos.astype(np.float64))[:, None, None]
    return angle * magnitude * both + (2.0 ** -8 * np.abs(y) if bf16 else 0) + 1e-30


def _partner(d, rd, il):
    p = np.arange(d)
    for i in range(rd // 2):
        u, w = (2 * i, 2 * i + 1) if il else (i, i + rd // 2)
        p[u], p[w] = w, u
    return p


@pytest.mark.parametrize("case", ROTARY)
def test_rotary(case):
    n, Hq, Hk, d, rd, il, bf16, inv, far = case
    pace = _pace()
    print(f"[cache] rotary {case}", flush=True)
    rng = np.random.default_rng(n + d)
    pos = rng.integers(0, far, n).astype(np.int32)
    pos[0] = -3 if n > 3 else pos[0]
    q, k = (rounded(rng.standard_normal((n, H, d)), bf16) for H in (Hq, Hk))
    f, m = pace.rotary_freqs(rd, 10000.0, "blend", 4.0, 1024.0)
    cfg = pace.RotaryConfig(Hq=Hq, Hk=Hk, d=d, rd=rd, interleaved=il, bf16_io=bf16)
    qd, kd = dev(q, IO[bf16]), dev(k, IO[bf16])
    qo, ko = torch.full_like(qd, float("nan")), torch.full_like(kd, float("nan"))
    pace.rotary(cfg, dev(pos), dev(f), qd, kd, qo, ko, magnitude=m, inverse=inv)
    part = _partner(d, rd, il)
    rows = np.arange(n) if n < 100 else np.concatenate([np.arange(3), np.arange(n - 5, n)])
    for x, y in ((q, qo), (k, ko)):
        want = co.rotary(x[rows], pos[rows], f, rd, il, m, inv)
        got = host(y)
        assert np.all(np.isfinite(got))
        tol = _rotary_tol(x[rows].astype(np.float64), pos[rows], part, m, want, bf16)
        tol[..., rd:] = 0                               # copied
        assert np.all(np.abs(got[rows] - want) <= tol)
    # in place, the same bits
    pace.rotary(cfg, dev(pos), dev(f), qd, kd, qd, kd, magnitude=m, inverse=inv)
    assert torch.equal(qd, qo) and torch.equal(kd, ko)


def test_rotary_on_slices_of_a_projection_and_one_side_only():
    pace = _pace()
    n, Hq, Hk, d, rd = 9, 4, 2, 64, 32
    rng = np.random.default_rng(0)
    wide = dev(rng.standard_normal((n, (Hq + 2 * Hk) * d)), torch.bfloat16)
    q, k = wide[:, : Hq * d].view(n, Hq, d), wide[:, Hq * d: (Hq + Hk) * d].view(n, Hk, d)
    pos, (f, _) = dev(np.arange(n, dtype=np.int32)), pace.rotary_freqs(rd)
    f = dev(f)
    cfg = pace.RotaryConfig(Hq=Hq, Hk=Hk, d=d, rd=rd)
    qo, ko = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k))
    pace.rotary(cfg, pos, f, q, k, qo, ko)
    q1, k1 = torch.empty_like(qo), torch.empty_like(ko)
    pace.rotary(cfg, pos, f, q.contiguous(), k.contiguous(), q1, k1)
    assert torch.equal(qo, q1) and torch.equal(ko, k1)
    keep = wide.clone()
    pace.rotary(cfg, pos, f, q, k, q, k)                 # in place in the projection
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(wide[:, (Hq + Hk) * d:], keep[:, (Hq + Hk) * d:])
    k2 = torch.empty_like(ko)
    pace.rotary(pace.RotaryConfig(Hq=0, Hk=Hk, d=d, rd=rd), pos, f, None, keep[:, Hq * d: (Hq + Hk) * d].view(n, Hk, d),
                None, k2)
    assert torch.equal(k2, ko)
    with pytest.raises(ValueError):
        pace.rotary(cfg, pos, f, q.transpose(1, 2).contiguous().transpose(1, 2), k, qo, ko)
    # an odd element offset takes the pair-by-pair form: the same bits
    shifted = torch.zeros(n * Hq * d + 1, dtype=torch.bfloat16, device="cuda")[1:].view(n, Hq, d)
    shifted.copy_(keep[:, : Hq * d].view(n, Hq, d))
    q3 = torch.empty_like(qo)
    pace.rotary(cfg, pos, f, shifted, k1, q3, k2)
    assert torch.equal(q3, qo)


def test_rotary_inverse_is_the_gradient():
    """sum(g . rotary(x)) has the gradient inverse-rotary(g) in x: against the formula (the
    transpose) and against differences of the fp64 oracle along random directions."""
    pace = _pace()
    n, H, d, rd = 3, 2, 64, 48
    rng = np.random.default_rng(5)
    x, g = rng.standard_normal((2, n, H, d))
    g = g.astype(np.float32)
    pos = np.array([0, 77, 5000], dtype=np.int32)
    f, m = pace.rotary_freqs(rd, scaling="blend", factor=2.0, original_len=256.0)
    cfg = pace.RotaryConfig(Hq=H, Hk=0, d=d, rd=rd, bf16_io=False)
    out = torch.empty((n, H, d), device="cuda")
    pace.rotary(cfg, dev(pos), dev(f), dev(g), None, out, None, magnitude=m, inverse=True)
    grad = host(out)
    for _ in range(4):
        u = rng.standard_normal((n, H, d))
        up = (g * co.rotary(x + u, pos, f, rd, False, m)).sum()
        dn = (g * co.rotary(x - u, pos, f, rd, False, m)).sum()
        # linear: the central difference is exact; the error is the gradient's own rounding
        tol = 8 * 2.0 ** -24 * m * 2 * np.abs(u).sum() * np.abs(g).max()
        assert abs((up - dn) / 2 - (grad * u).sum()) <= tol


# ------------------------------------------------------------------- writing and reading

STORE = [(kind, d, g) for kind in ("int8", "int4", "fp8") for d, g in
         ((64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128))]


def _vectors(rng, shape, bf16):
    x = rng.standard_normal(shape)
    x[..., 5::16] *= 8
    x[..., :32] *= rng.choice([0.0, 1.0, 1e-3], size=(*shape[:-1], 1))
    # exact ties: small multiples of a power of two
    x[..., 32:64] = rng.integers(-14, 15, size=(*shape[:-1], 32)) / 4.0
    return rounded(x, bf16)


def _table(rng, B, MP, spare=2):
    return rng.permutation(B * MP + spare)[: B * MP].reshape(B, MP).astype(np.int32), B * MP + spare


@pytest.mark.parametrize("kind,d,g", STORE)
@pytest.mark.parametrize("bf16", [True, False])
def test_written_bytes_and_read_values(kind, d, g, bf16):
    pace = _pace()
    print(f"[cache] store {kind} d={d} g={g} bf16={bf16}", flush=True)
    rng = np.random.default_rng(d + g)
    B, T, H, P, MP = 2, 11, 2, 16, 2
    table, N = _table(rng, B, MP)
    oc = co.Cache(B=B, Hkv=H, d=d, kind=kind, group=g, page=P, num_pages=N, max_pages=MP)
    cfg = pace.CacheConfig(B=B, Hq=H, Hkv=H, d=d, num_pages=N, max_pages=MP, kind=kind, group=g, page=P, bf16_io=bf16)
    k, v = _vectors(rng, (B, T, H, d), bf16), _vectors(rng, (B, T, H, d), bf16)
    # a run from 6 over the page's end with a hole; scattered positions
    pos = np.stack([np.arange(6, 6 + T), rng.permutation(MP * P)[:T]]).astype(np.int32)
    pos[0, 4] = -1
    pos[1, 2] = MP * P + 5                              # past the table
    old = rng.integers(0, 256, oc.nbytes).astype(np.uint8)
    want = old.copy()
    co.write(oc, want, table, pos, k, v)
    cache = dev(old)
    pace.cache_write(cfg, cache, dev(table), dev(pos), dev(k, IO[bf16]), dev(v, IO[bf16]))
    got = cache.cpu().numpy()
    assert np.array_equal(got, want)
    ko = torch.full((B, T, H, d), float("nan"), dtype=IO[bf16], device="cuda")
    vo = torch.full_like(ko, float("nan"))
    pace.cache_read(cfg, cache, dev(table), dev(pos), ko, vo)
    for y, w in zip((ko, vo), co.read(oc, want, table, pos)):
        assert np.array_equal(host(y), rounded(w, bf16).astype(np.float64))
    # whole quads (aligned runs) read and write the same bytes as single tokens
    pos = np.stack([np.arange(1, 1 + T), np.arange(20, 20 + T)]).astype(np.int32)
    one, two = dev(old), dev(old)
    kd, vd = dev(k, IO[bf16]), dev(v, IO[bf16])
    pace.cache_write(cfg, one, dev(table), dev(pos), kd, vd)
    for t in range(T):
        pace.cache_write(cfg, two, dev(table), dev(pos[:, t: t + 1]), kd[:, t: t + 1].contiguous(), vd[:, t: t + 1])
    assert torch.equal(one, two)
    pace.cache_read(cfg, one, dev(table), dev(pos), ko, vo)
    for t in range(T):
        k1, v1 = torch.empty_like(ko[:, :1]).contiguous(), torch.empty_like(vo[:, :1]).contiguous()
        pace.cache_read(cfg, one, dev(table), dev(pos[:, t: t + 1]), k1, v1)
        assert torch.equal(k1, ko[:, t: t + 1]) and torch.equal(v1, vo[:, t: t + 1])


@pytest.mark.parametrize("kind", ["int8", "int4", "fp8"])
def test_non_finite_inputs_and_absent_pages(kind):
    """NaN is stored as 0, infinities at 2^127, tiny groups as zeros; positions whose page is not
    there are dropped and read as zeros."""
    pace = _pace()
    rng = np.random.default_rng(2)
    B, T, H, d, g, P, MP = 1, 6, 1, 64, 32, 16, 3
    table = np.array([[1, -1, 7]], dtype=np.int32)      # 7: not a page of the pool
    N = 3
    oc = co.Cache(B=B, Hkv=H, d=d, kind=kind, group=g, page=P, num_pages=N, max_pages=MP)
    cfg = pace.CacheConfig(B=B, Hq=H, Hkv=H, d=d, num_pages=N, max_pages=MP, kind=kind, group=g, page=P, bf16_io=False)
    k = rng.standard_normal((B, T, H, d)).astype(np.float32)
    k[0, 0, 0, 3], k[0, 1, 0, 3], k[0, 1, 0, 40], k[0, 2, 0, 1] = np.nan, np.inf, -np.inf, 3e38
    k[0, 3] = np.nan
    k[0, 4] *= 1e-38
    v = k[:, ::-1].copy()
    pos = np.array([[0, 5, 16, 33, 15, 1]], dtype=np.int32)
    old = np.zeros(oc.nbytes, dtype=np.uint8)
    want = old.copy()
    co.write(oc, want, table, pos, k, v)
    cache = dev(old)
    pace.cache_write(cfg, cache, dev(table), dev(pos), dev(k), dev(v))
    assert np.array_equal(cache.cpu().numpy(), want)
    ko, vo = (torch.full((B, T, H, d), float("nan"), device="cuda") for _ in range(2))
    pace.cache_read(cfg, cache, dev(table), dev(pos), ko, vo)
    for y, w in zip((ko, vo), co.read(oc, want, table, pos)):
        got = host(y)
        assert np.all(np.isfinite(got)) and np.array_equal(got, w.astype(np.float32).astype(np.float64))
        assert np.all(got[0, 2:4] == 0)


# ------------------------------------------------------------------------- attention

class Scene:
    """A cache with known contents: codes drawn through the oracle's quantiser, written by
    pace_cache_write into a pool of old bytes (fp8 NaN patterns and NaN scales among them)."""

    def __init__(self, seed, B, Hkv, gamma, d, kind, g, page, lens, bf16, spare=2, max_pages=None):
        self.pace = _pace()
        rng = np.random.default_rng(seed)
        self.rng, self.B, self.H, self.gamma, self.d, self.bf16, self.kind, self.g = rng, B, Hkv, gamma, d, bf16, kind, g
        MP = max_pages or max(1, -(-max(lens) // page))
        self.table_h, N = _table(rng, B, MP, spare)
        self.cfg = self.pace.CacheConfig(B=B, Hq=Hkv * gamma, Hkv=Hkv, d=d, num_pages=N, max_pages=MP, kind=kind,
                                         group=g, page=page, bf16_io=bf16)
        self.cache = torch.full((self.cfg._bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        self.table = dev(self.table_h)
        self.lens = lens
        L = max(max(lens), 1)
        x = rng.standard_normal((2, B, L, Hkv, d)).astype(np.float32)
        x[0, ..., 5::16] *= 4
        x[1] *= np.exp(rng.standard_normal((B, L, Hkv, 1)))    # value scales differ by token
        x = rounded(x, bf16)
        pos = np.where(np.arange(L) < np.array(lens)[:, None], np.arange(L), -1).astype(np.int32)
        self.pace.cache_write(self.cfg, self.cache, self.table, dev(pos), dev(x[0], IO[bf16]), dev(x[1], IO[bf16]))
        self.k, self.v = (co.quantise(y, kind, g)[2] for y in x)     # [B, L, H, d]

    def run(self, T, ctx, parents=None, drafts=None, scale=None, max_len=None, q=None, stream=None):
        """(o, lse) on the host and the q used (fp64)."""
        pace, cfg = self.pace, self.cfg
        if q is None:
            q = rounded(self.rng.standard_normal((self.B, T, cfg.Hq, self.d)), self.bf16)
        tree = None
        if parents is not None:
            tree = dev(np.stack([pace.tree_bits(p) for p in parents]))
        o = torch.full((self.B, T, cfg.Hq, self.d), float("nan"), dtype=IO[self.bf16], device="cuda")
        lse = torch.full((self.B, T, cfg.Hq), float("nan"), device="cuda")
        n = pace.cache_attention_workspace_bytes(cfg, T, max_len or cfg.max_pages * cfg.page)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
        pace.cache_attention(cfg, self.cache, self.table, dev(q, IO[self.bf16]), dev(np.array(ctx, dtype=np.int32)), o,
                             lse=lse, tree=tree, draft_lens=None if drafts is None else
                             dev(np.array(drafts, dtype=np.int32)), scale=scale, max_len=max_len, workspace=ws,
                             stream=stream)
        return host(o), host(lse), q.astype(np.float64)

    def check(self, T, ctx, parents=None, drafts=None, scale=None, max_len=None, q=None, hidden=None, rows=None):
        """Runs and compares with the oracle; hidden[b]: positions that are not there."""
        o, lse, q = self.run(T, ctx, parents, drafts, scale, max_len, q)
        scale = self.d ** -0.5 if scale is None else scale
        for b in range(self.B):
            n = T if drafts is None else drafts[b]
            L = ctx[b] + n
            near = np.tril(np.ones((T, T), dtype=bool)) if parents is None else \
                co.tree_mask(parents[b] if len(parents) > 1 else parents[0])
            vis = np.zeros((T, L), dtype=bool)
            vis[:n, : ctx[b]] = True
            vis[:n, ctx[b]:] = near[:n, :n]
            if hidden is not None:
                vis[:, [p for p in hidden[b] if p < L]] = False
            pick = range(T) if rows is None else rows
            for hq in range(self.cfg.Hq):
                h = hq // self.gamma
                k, v = self.k[b, :L, h], self.v[b, :L, h]
                qr, vi = q[b, pick, hq] if rows is not None else q[b, :, hq], vis[list(pick)]
                wo, wl, w = co.attention(qr, k, v, scale, vi)
                z_abs = (np.abs(qr) @ np.abs(k).T * abs(scale)).max(-1, initial=0.0)
                dz = ((self.d + 16) * 2.0 ** -24 + (0 if self.bf16 else 2.0 ** -22)) * z_abs + \
                    4 * 2.0 ** -24 * (z_abs + 16)
                sums = (L / 8 + 64) * 2.0 ** -24
                E = (2.0 ** -11 if self.bf16 else 2.0 ** -21) + 2 * dz + sums
                tol = E[:, None] * (w @ np.abs(v)) + L * 2.0 ** -28 * np.abs(v).max(initial=0.0)
                if self.bf16:
                    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(wo)
                go, gl = o[b, pick, hq] if rows is not None else o[b, :, hq], lse[b, list(pick), hq]
                empty = ~vi.any(-1)
                assert np.all(go[empty] == 0) and np.all(gl[empty] == -np.inf), (b, hq, "empty rows")
                assert np.all(np.isfinite(go)) and np.all(np.isfinite(gl[~empty])), (b, hq)
                bad = np.abs(go - wo) > tol
                assert not bad.any(), (b, hq, np.argwhere(bad)[:4], np.abs(go - wo).max(), tol.max())
                lt = dz + sums + 2.0 ** -22 * np.abs(np.where(empty, 0, wl))
                assert np.all(np.abs(np.where(empty, 0, gl) - np.where(empty, 0, wl)) <= lt), (b, hq, "lse")
        return o, lse


@pytest.mark.parametrize("kind,d,g", STORE)
@pytest.mark.parametrize("bf16", [True, False])
def test_attention_every_layout(kind, d, g, bf16):
    """Single tokens and a chain over ragged contexts, short and past several 32-token steps."""
    print(f"[cache] attention {kind} d={d} g={g} bf16={bf16}", flush=True)
    s = Scene(d + g, 3, 2, 4, d, kind, g, 16, [1, 200, 77], bf16)
    s.check(1, [0, 199, 76])
    s.check(3, [0, 197, 30], drafts=[1, 3, 2])


@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 17, 30, 31, 32, 33, 63, 64, 65, 127, 129])
def test_attention_context_ends_at_every_place(ctx):
    s = Scene(ctx, 1, 1, 3, 128, "int8", 128, 32, [ctx + 5], True)
    s.check(5, [ctx])


@pytest.mark.parametrize("gamma,T", [(1, 1), (1, 16), (1, 17), (2, 9), (3, 11), (5, 7), (7, 5), (16, 1), (16, 3), (32, 2),
                                     (8, 33)])
@pytest.mark.parametrize("kind", ["int4", "fp8"])
def test_attention_head_layouts(gamma, T, kind):
    s = Scene(gamma + T, 2, 2, gamma, 64, kind, 32, 32, [90 + T, 40 + T], True)
    s.check(T, [90, 40])


@pytest.mark.parametrize("kind", ["int8", "int4", "fp8"])
@pytest.mark.parametrize("T", [2, 31, 32, 33, 70])
def test_attention_trees(kind, T):
    rng = np.random.default_rng(T)
    parents = [[int(rng.integers(max(-1, i - 5), i)) if i else -1 for i in range(T)] for _ in range(3)]
    s = Scene(T, 3, 1, 2, 64, kind, 64, 16, [T, 45 + T, 100 + T], True)
    s.check(T, [0, 45, 100], parents=parents)
    s.check(T, [0, 45, 100], parents=parents, drafts=[T, 0, T // 2])
    s.check(T, [0, 45, 100], parents=parents[:1])       # one tree for all


def test_attention_rows_that_see_nothing():
    """Sequences without drafts or context, and a mask row of zeros."""
    pace = _pace()
    s = Scene(1, 3, 1, 2, 128, "fp8", 64, 16, [4, 40, 4], True)
    s.check(4, [0, 36, 0], drafts=[0, 0, 4])
    tree = np.zeros((1, 4, 1), dtype=np.int32)
    tree[0, 2] = 0b0101
    q = rounded(np.random.default_rng(0).standard_normal((3, 4, 2, 128)), True)
    o = torch.full((3, 4, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 4, 2), float("nan"), device="cuda")
    n = pace.cache_attention_workspace_bytes(s.cfg, 4, 48)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    pace.cache_attention(s.cfg, s.cache, s.table, dev(q, torch.bfloat16), dev(np.zeros(3, np.int32)), o, lse=lse,
                         tree=dev(tree), max_len=48, workspace=ws)
    o, lse = host(o), host(lse)
    for i in (0, 1, 3):
        assert np.all(o[:, i] == 0) and np.all(lse[:, i] == -np.inf)
    assert np.all(np.isfinite(o[:, 2])) and np.all(np.isfinite(lse[:, 2]))


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_attention_pages_that_are_not_there(kind):
    """Entries outside the pool hide their positions, wherever a 32-token step meets them."""
    s = Scene(4, 1, 1, 2, 64, kind, 32, 16, [150], True)
    table = s.table_h.copy()
    table[0, 2], table[0, 5], table[0, 9] = -1, s.cfg.num_pages, 2 ** 30
    s.table = dev(table)
    hidden = [[p for e in (2, 5, 9) for p in range(16 * e, 16 * e + 16)]]
    s.check(3, [147], hidden=hidden)
    table[:] = -7
    s.table = dev(table)
    s.check(3, [147], hidden=[list(range(160))])


@pytest.mark.parametrize("kind,d,g,bf16", [("int8", 128, 128, True), ("int4", 128, 32, True), ("fp8", 256, 64, False),
                                           ("int8", 64, 64, False)])
def test_attention_long_contexts_cut_over_workgroups(kind, d, g, bf16):
    """Pieces joined by the second kernel; a max_len under the true length (the last piece takes
    the rest) and far over it (empty pieces) give the same result within tolerance."""
    s = Scene(11, 2, 1, 4, d, kind, g, 64, [5003, 1200], bf16)
    for max_len in (None, 700, 5003, 1 << 20):
        s.check(2, [5001, 1198], max_len=max_len)
    s.check(1, [5002, 0], max_len=5003)


def test_attention_prompt_chunk_rows():
    """A chunk of 150 tokens over a cached context: many row tiles, sampled rows."""
    s = Scene(12, 1, 2, 4, 128, "int8", 64, 64, [650], True)
    s.check(150, [500], rows=[0, 1, 3, 31, 32, 63, 64, 100, 148, 149])


@pytest.mark.parametrize("bf16", [True, False])
def test_attention_sharp_and_tiny_scores(bf16):
    """Softmax over scores far apart (the maximum moves late), tiny and huge queries, scale 0."""
    s = Scene(13, 1, 1, 2, 64, "int8", 64, 16, [300], bf16)
    q = rounded(s.rng.standard_normal((1, 1, 2, 64)) * 30, bf16)
    s.check(1, [299], q=q)
    s.check(1, [299], q=rounded(q * 1e-30, bf16))
    s.check(1, [299], q=rounded(q * 0, bf16))
    s.check(1, [299], scale=0.0)
    s.check(1, [299], scale=-0.3)
    # one token towers over the others at the very end
    s.check(1, [299], q=rounded(s.k[:, 299:, :, :].repeat(2, axis=2) * 3, bf16))


def test_attention_nan_query_stays_in_its_row():
    s = Scene(14, 1, 1, 4, 128, "fp8", 128, 16, [100], True)
    q = rounded(s.rng.standard_normal((1, 2, 4, 128)), True)
    clean, lse, _ = s.run(2, [98], q=q)
    q[0, 1, 2, 7] = np.nan
    o, l2, _ = s.run(2, [98], q=q)
    keep = np.ones((2, 4), dtype=bool)
    keep[1, 2] = False
    assert np.array_equal(o[0][keep], clean[0][keep]) and np.array_equal(l2[0][keep], lse[0][keep])
    assert np.all(np.isnan(o[0, 1, 2])) and np.isnan(l2[0, 1, 2])


def test_attention_repeats_bit_for_bit_and_ignores_other_sequences():
    s = Scene(15, 3, 2, 4, 128, "int4", 64, 32, [2100, 900, 33], True)
    q = rounded(s.rng.standard_normal((3, 2, 8, 128)), True)
    a = s.run(2, [2098, 898, 31], q=q, max_len=2112)
    b = s.run(2, [2098, 898, 31], q=q, max_len=2112)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    c = s.run(2, [2098, 5, 0], q=q, max_len=2112)
    assert np.array_equal(a[0][0], c[0][0]) and np.array_equal(a[1][0], c[1][0])


def test_attention_on_slices_of_a_projection():
    s = Scene(16, 2, 2, 2, 64, "int8", 64, 16, [50, 20], True)
    pace, cfg = s.pace, s.cfg
    wide = torch.randn((2, 3, (4 + 4) * 64), device="cuda").to(torch.bfloat16)
    q = wide[..., :256].view(2, 3, 4, 64)
    ctx = dev(np.array([47, 17], dtype=np.int32))
    n = pace.cache_attention_workspace_bytes(cfg, 3, 64)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    o1, o2 = (torch.empty((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pace.cache_attention(cfg, s.cache, s.table, q, ctx, o1, max_len=64, workspace=ws)
    pace.cache_attention(cfg, s.cache, s.table, q.contiguous(), ctx, o2, max_len=64, workspace=ws)
    assert torch.equal(o1, o2)
    with pytest.raises(ValueError):
        pace.cache_attention(cfg, s.cache, s.table, q.transpose(1, 2), ctx, o1, max_len=64, workspace=ws)
    with pytest.raises(ValueError):
        pace.cache_attention(cfg, s.cache[:-1], s.table, q, ctx, o1, max_len=64, workspace=ws)


def test_offsets_past_32_bits():
    """A pool of over 4 GiB whose last pages are used."""
    pace = _pace()
    B, H, d, P, MP = 1, 8, 128, 64, 4
    rec = co.Cache(B=B, Hkv=H, d=d, kind="int8", group=128, page=P, num_pages=1, max_pages=MP).nbytes
    N = (1 << 32) // rec + 40
    cfg = pace.CacheConfig(B=B, Hq=16, Hkv=H, d=d, num_pages=N, max_pages=MP, kind="int8", group=128, page=P)
    assert cfg._bytes > 1 << 32
    rng = np.random.default_rng(8)
    cache = torch.empty(cfg._bytes, dtype=torch.uint8, device="cuda")
    x = dev(rounded(rng.standard_normal((2, B, 200, H, d)), True), torch.bfloat16)
    pos = dev(np.arange(200, dtype=np.int32)[None])
    q = dev(rounded(rng.standard_normal((B, 1, 16, d)), True), torch.bfloat16)
    ctx = dev(np.array([199], dtype=np.int32))
    n = pace.cache_attention_workspace_bytes(cfg, 1, 256)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    got = []
    for first in (0, N - MP):                           # the same tokens in the first and the last pages
        table = dev(np.arange(first, first + MP, dtype=np.int32)[None])
        pace.cache_write(cfg, cache, table, pos, x[0], x[1])
        k, v, o = (torch.empty_like(y) for y in (x[0], x[1], q))
        pace.cache_read(cfg, cache, table, pos, k, v)
        pace.cache_attention(cfg, cache, table, q, ctx, o, max_len=256, workspace=ws)
        got.append((k, v, o))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(cache[: 4 * rec], cache[-4 * rec:])


def test_a_step_captured_in_a_graph_replays_as_eager():
    """rotary, write and attention of a decode step on their own stream, captured and replayed
    with other inputs and eager work between the replays."""
    pace = _pace()
    B, Hq, H, d, P, MP = 3, 8, 2, 128, 16, 200
    rng = np.random.default_rng(6)
    table, N = _table(rng, B, MP)
    cfg = pace.CacheConfig(B=B, Hq=Hq, Hkv=H, d=d, num_pages=N, max_pages=MP, kind="int4", group=32, page=P)
    rot = pace.RotaryConfig(Hq=Hq, Hk=H, d=d, rd=64)
    table, (f, _) = dev(table), pace.rotary_freqs(64)
    f = dev(f)
    lens = np.array([3000, 17, 800], dtype=np.int32)
    hist = dev(rounded(rng.standard_normal((2, B, 3000, H, d)), True), torch.bfloat16)
    hpos = dev(np.where(np.arange(3000) < lens[:, None], np.arange(3000), -1).astype(np.int32))
    steps = [dev(rounded(rng.standard_normal((B, 1, (Hq + 2 * H) * d)), True), torch.bfloat16) for _ in range(4)]
    stream = torch.cuda.Stream()
    n = pace.cache_attention_workspace_bytes(cfg, 1, MP * P)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def buffers():
        cache = torch.zeros(cfg._bytes, dtype=torch.uint8, device="cuda")
        pace.cache_write(cfg, cache, table, hpos, hist[0], hist[1])
        return dict(cache=cache, x=torch.empty_like(steps[0]), pos=dev(lens[:, None]), ctx=dev(lens),
                    qr=torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda"),
                    kr=torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda"),
                    o=torch.empty((B, 1, Hq, d), dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty((B, 1, Hq), device="cuda"))

    def step(u):
        x = u["x"].view(B, -1)
        q, k = x[:, : Hq * d].view(B, Hq, d), x[:, Hq * d: (Hq + H) * d].view(B, H, d)
        v = u["x"][..., (Hq + H) * d:].view(B, 1, H, d)
        pace.rotary(rot, u["ctx"], f, q, k, u["qr"], u["kr"], stream=stream)
        pace.cache_write(cfg, u["cache"], table, u["pos"], u["kr"].view(B, 1, H, d), v, stream=stream)
        pace.cache_attention(cfg, u["cache"], table, u["qr"].view(B, 1, Hq, d), u["ctx"], u["o"], lse=u["lse"],
                             workspace=ws, stream=stream)

    def load(u, i):
        u["x"].copy_(steps[i])
        u["ctx"].copy_(dev(lens + i))
        u["pos"].copy_(dev((lens + i)[:, None]))
        torch.cuda.synchronize()

    eager, want = buffers(), []
    for i in range(4):
        load(eager, i)
        step(eager)
        torch.cuda.synchronize()
        want.append((eager["o"].clone(), eager["lse"].clone(), eager["cache"].clone()))
    u = buffers()
    load(u, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(u)
    for i in range(4):
        load(u, i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((u["o"], u["lse"], u["cache"]), want[i]):
            assert torch.equal(a, b), f"replay {i}"
        torch.randn(1 << 20, device="cuda").mul_(2.0).sum().item()      # the program's own work between
    del graph


def test_accepted_drafts_written_again_equal_a_plain_decode():
    """A tree is verified, its accepted path's keys and values are written at their final
    positions, and the next token's attention equals that of a cache that never held a tree."""
    pace = _pace()
    s = Scene(21, 1, 2, 2, 64, "int8", 64, 16, [40], True, max_pages=5)
    parents = [-1, 0, 0, 1, 2, 4]
    path = [0, 2, 4]
    new = dev(rounded(s.rng.standard_normal((2, 1, 6, 2, 64)), True), torch.bfloat16)
    plain = s.cache.clone()
    at = lambda p: dev(np.array([p], dtype=np.int32))  # noqa: E731
    pace.cache_write(s.cfg, s.cache, s.table, at(np.arange(40, 46)), new[0], new[1])
    s.run(6, [40], parents=[parents])
    final = [40 + path.index(i) if i in path else -1 for i in range(6)]
    pace.cache_write(s.cfg, s.cache, s.table, at(final), new[0], new[1])
    pace.cache_write(s.cfg, plain, s.table, at([40, 41, 42]), new[0][:, path].contiguous(), new[1][:, path].contiguous())
    q = rounded(s.rng.standard_normal((1, 1, 4, 64)), True)
    a = s.run(1, [42], q=q)
    s.cache = plain
    b = s.run(1, [42], q=q)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_attention_fp32_weights_keep_both_pieces_at_ties():
    """Many rows over few tokens in fp32: one weight in some ten thousand lies next to a tie of
    its fp16 piece, and its second piece has to match the first as the matrix unit got it."""
    s = Scene(31, 24, 4, 4, 64, "fp8", 32, 16, [9] * 24, False)
    s.check(6, [3] * 24)


def test_prepared_calls_equal_plain_ones():
    pace = _pace()
    s = Scene(41, 2, 2, 2, 64, "int8", 64, 16, [60, 33], True, max_pages=6)
    n = pace.cache_attention_workspace_bytes(s.cfg, 2, 96)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    x = dev(rounded(s.rng.standard_normal((3, 2, 2, 4, 64)), True), torch.bfloat16)
    q, k, v = x[0], x[1, :, :, :2].contiguous(), x[2, :, :, :2].contiguous()
    ctx, pos = dev(np.array([60, 33], np.int32)), dev(np.array([[60, 61], [33, 34]], np.int32))
    f = dev(pace.rotary_freqs(32)[0])
    rot = pace.RotaryConfig(Hq=4, Hk=2, d=64, rd=32)
    out = []
    for prepared in (False, True):
        cache, qr, kr, o = s.cache.clone(), torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
        flat = lambda t: t.view(4, -1, 64)  # noqa: E731
        a = (rot, pos.view(-1), f, flat(q), flat(k), flat(qr), flat(kr))
        b = (s.cfg, cache, s.table, pos, kr, v)
        c = (s.cfg, cache, s.table, qr, ctx, o)
        if prepared:
            calls = [pace.prepare_rotary(*a), pace.prepare_cache_write(*b),
                     pace.prepare_cache_attention(*c, max_len=96, workspace=ws)]
            for call in calls + calls:
                call()
        else:
            pace.rotary(*a)
            pace.cache_write(*b)
            pace.cache_attention(*c, max_len=96, workspace=ws)
        torch.cuda.synchronize()
        out.append((cache, qr, kr, o))
    for x, y in zip(*out):
        assert torch.equal(x, y)


@pytest.mark.parametrize("longest", [256, 257, 768, 769])
@pytest.mark.parametrize("T,gamma,bf16", [(1, 4, True), (8, 4, True), (11, 3, True), (32, 4, False), (43, 3, False)])
def test_attention_at_the_edges_of_the_split(T, gamma, bf16, longest):
    """One row tile or two, four waves or eight, one piece or more: rows on both sides of each
    bound, with several row blocks, a ragged context and a sequence without one."""
    s = Scene(43, 3, 1, gamma, 128, "int8", 128, 16, [longest, 200, T], bf16)
    s.check(T, [longest - T, 200 - T, 0], max_len=longest)
