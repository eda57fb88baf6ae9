"""GPU parity of the operators that serve drafted tokens (include/pace_draft.h) against their fp64
oracle, through the C ABI: outputs of drafts, commits, verification, moves."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as co  # noqa: E402
from oracle import draft_oracle as do  # noqa: E402
from oracle import packing as pk  # noqa: E402
from pace_synth import make_tokens, random_bf16_state, random_buffer_parts, random_packed_state_parts  # noqa: E402

pytestmark = pytest.mark.gpu
IO = {True: torch.bfloat16, False: torch.float32}


def _lib():
    import bit_recurrent_state_amd as pace
    return pace


def dev(x, dtype=None):
    t = torch.from_numpy(np.array(x, order="C"))
    return (t.to(dtype) if dtype is not None else t).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------- layers

LAYERS = {
    # name: (B, Hv, Hk, d, group, state, buf, bf16_io, dP, head_bits)
    "pace4": (3, 32, 16, 128, 64, "sym", "int8", True, 8, None),
    "pace48_mixed": (2, 16, 8, 128, 32, "asym", "mixed", True, 8, "quarter"),
    "pace48_int8_f32": (2, 8, 4, 128, 32, "asym", "int8", False, 8, "quarter"),
    "tiny_f32": (2, 4, 4, 64, 32, "sym", "int8", False, 8, None),
    "d64_asym_mixed": (3, 8, 4, 64, 32, "asym", "mixed", True, 5, [8, 4, 4, 8, 4, 4, 4, 8]),
    "asym_g64_dP32": (2, 6, 2, 128, 64, "asym", "int8", True, 32, [4, 8, 4, 4, 8, 4]),
    "sym8_dP16": (2, 4, 2, 128, 64, "sym", "int8", True, 16, [8, 8, 4, 8]),
    "d64_g64_dP1": (2, 3, 1, 64, 64, "sym", "int8", True, 1, None),
    "asym4_g64": (2, 8, 4, 128, 64, "asym", "int8", True, 8, None),
    "f32_g32_mixed_dP32": (2, 2, 1, 128, 32, "sym", "mixed", False, 32, None),
    "bf16_state": (2, 8, 4, 128, 32, "bf16", "int8", True, 8, None),
    "bf16_state_f32_d64": (2, 4, 2, 64, 32, "bf16", "int8", False, 12, None),
}


def layer(name, seed, counts=None, B=None):
    """(oracle config, library config, state bytes, buffer bytes)."""
    nB, Hv, Hk, d, g, kind, buf, bf16, dP, hb = LAYERS[name]
    B = B or nB
    if hb == "quarter":
        hb = [8 if h % 4 == 1 else 4 for h in range(Hv)]
    ocfg = pk.LayerCfg(B=B, Hv=Hv, Hk=Hk, dk=d, dv=d, group=g, asym=kind == "asym", buf=buf, dP=dP, bf16_io=bf16,
                       head_bits=hb, bf16_state=kind == "bf16")
    gcfg = _lib().LayerConfig(B=B, Hv=Hv, Hk=Hk, dk=d, dv=d, group=g, asym=kind == "asym", buf=buf, bf16_io=bf16, dP=dP,
                              head_bits=hb, bf16_state=kind == "bf16")
    if kind == "bf16":
        S = random_bf16_state(seed, B, Hv, d, d)
        parts = [[S[b, h] for h in range(Hv)] for b in range(B)]
    else:
        parts = pk.state_from_parts(ocfg, random_packed_state_parts(seed, B, Hv, d, d, g, [ocfg.bits(h) for h in range(Hv)],
                                                                    kind == "asym"))
    return ocfg, gcfg, pk.pack_state(ocfg, parts), \
        pk.pack_buffer(ocfg, random_buffer_parts(seed + 1, B, Hv, Hk, d, d, dP, buf == "mixed", counts=counts))


def trees(rng, B, T, kind):
    """parents [B][T]: a chain, trees with one root, or forests (several nodes hang on the sequence itself)."""
    low = {"tree": 0, "forest": -1}
    return [[-1] + [i - 1 if kind == "chain" else int(rng.integers(low[kind], i)) for i in range(1, T)] for _ in range(B)]


def paths(parents):
    out = []
    for p in parents:
        rows = []
        for i in range(len(p)):
            rows.append(rows[p[i]] + [p[i]] if p[i] >= 0 else [])
        out.append(rows)
    return out


def bits(parents):
    return dev(np.stack([_lib().tree_bits(p) for p in parents]))


def step(gcfg, state, buf, toks, T, tree=None, lens=None, fill=float("nan")):
    pace = _lib()
    io = IO[gcfg.bf16_io]
    st, bu = dev(state), dev(buf)
    q, k, v = (dev(x, io) for x in (toks.q, toks.k, toks.v))
    o = torch.full((gcfg.B, T, gcfg.Hv, gcfg.dv), fill, dtype=io, device="cuda")
    pace.draft_step(gcfg, st, bu, q, k, v, dev(toks.a), dev(toks.beta), o, tree=tree,
                    draft_lens=None if lens is None else dev(np.asarray(lens, dtype=np.int32)))
    torch.cuda.synchronize()
    assert np.array_equal(st.cpu().numpy(), state) and np.array_equal(bu.cpu().numpy(), buf)
    return o


def check_step(ocfg, o, state, buf, toks, rows, lens, tiles):
    args = (ocfg, state, buf, toks.q, toks.k, toks.v, toks.a, toks.beta, rows, lens, tiles)
    want = do.draft_step(*args)
    # products of a projection (queries in three pieces in fp32), their offsets, the scale and decay factors
    off = do.draft_step_bound(*args, roundings=2 * ocfg.dk * (1 if ocfg.bf16_io else 3) + ocfg.dP + o.shape[1] + 32)
    got = host(o)
    for b, h in tiles:
        room = off[b, :, h] + (np.abs(want[b, :, h]) + off[b, :, h]) * (2.0 ** -8 if ocfg.bf16_io else 2.0 ** -24)
        d = np.abs(got[b, :, h] - want[b, :, h])
        assert np.all(d <= room), (b, h, float((d / np.maximum(room, 1e-300)).max()))
        n = int(lens[b])
        assert np.all(got[b, n:, h] == 0.0)


@pytest.mark.parametrize("kind", ["chain", "tree", "forest"])
@pytest.mark.parametrize("T", [1, 5, 17, 33])
@pytest.mark.parametrize("name", list(LAYERS))
def test_outputs_of_drafts(name, T, kind):
    rng = np.random.default_rng(T * 7 + len(kind))
    ocfg, gcfg, state, buf = layer(name, 3 * T)
    toks = make_tokens(11 + T, ocfg.B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    par = trees(rng, ocfg.B, T, kind)
    lens = rng.integers(0, T + 1, size=ocfg.B)
    lens[0] = T
    o = step(gcfg, state, buf, toks, T, None if kind == "chain" else bits(par), lens)
    tiles = [(b, h) for b in range(ocfg.B) for h in sorted({0, 1, ocfg.Hv // 2, ocfg.Hv - 1})]
    check_step(ocfg, o, state, buf, toks, paths(par), lens, tiles)


@pytest.mark.parametrize("name,T,count", [("pace4", 64, 7), ("asym_g64_dP32", 64, 31), ("f32_g32_mixed_dP32", 64, 31), ("pace4", 9, 0),
                                          ("pace4", 9, 7), ("asym_g64_dP32", 32, 16), ("bf16_state", 64, 3), ("tiny_f32", 50, 6),
                                          ("pace4", 8, 40), ("pace4", 8, -3)])
def test_outputs_of_the_largest_drafts_and_at_every_count(name, T, count):
    ocfg, gcfg, state, buf = layer(name, 5, counts=[count] * LAYERS[name][0])
    toks = make_tokens(6, ocfg.B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    par = trees(np.random.default_rng(T), 1, T, "tree") * ocfg.B
    o = step(gcfg, state, buf, toks, T, bits(par[:1]))                       # one tree for all sequences
    check_step(ocfg, o, state, buf, toks, paths(par), [T] * ocfg.B, [(0, 0), (ocfg.B - 1, ocfg.Hv - 1)])


def test_a_chain_is_a_tree_and_rows_do_not_depend_on_other_sequences_or_what_lies_behind():
    ocfg, gcfg, state, buf = layer("pace4", 8)
    T = 11
    toks = make_tokens(9, ocfg.B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=True)
    lens = [T, 4, 9]
    a = step(gcfg, state, buf, toks, T, None, lens)
    b = step(gcfg, state, buf, toks, T, bits(trees(None, 1, T, "chain")), lens)
    assert torch.equal(a, b)
    for x in (toks.q, toks.k, toks.v, toks.a, toks.beta):                    # rows behind the last token may hold anything
        x[1, 4:] = np.nan
        x[2, 9:] = np.inf
    c = step(gcfg, state, buf, toks, T, None, lens)
    assert torch.equal(a, c)
    toks.v[1] *= 3
    d = step(gcfg, state, buf, toks, T, None, lens)
    assert torch.equal(a[[0, 2]], d[[0, 2]]) and not torch.equal(a[1], d[1])
    toks2 = type(toks)(*(x[:, :4] if isinstance(x, np.ndarray) else x for x in (toks.q, toks.k, toks.v, toks.a, toks.beta)), None)
    e = step(gcfg, state, buf, toks2, 4)
    assert torch.equal(d[:, :4][1], e[1])


@pytest.mark.parametrize("name", list(LAYERS))
def test_a_single_draft_is_the_decoded_token(name):
    """T = 1 gives what pace_decode_step gives (another order of sums)."""
    pace = _lib()
    ocfg, gcfg, state, buf = layer(name, 21)
    toks = make_tokens(22, ocfg.B, 1, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    o = step(gcfg, state, buf, toks, 1)
    io = IO[gcfg.bf16_io]
    w = torch.empty((gcfg.B, gcfg.Hv, gcfg.dv), dtype=io, device="cuda")
    pace.decode_step(gcfg, dev(state), dev(buf), *(dev(x[:, 0], io) for x in (toks.q, toks.k, toks.v)), dev(toks.a[:, 0]),
                     dev(toks.beta[:, 0]), w)
    x, y = host(o[:, 0]), host(w)
    assert np.abs(x - y).max() <= np.abs(y).max() * (2.0 ** -7 if gcfg.bf16_io else 1e-5)


# ------------------------------------------------------------------- commit

def run_commit(gcfg, state, buf, toks, nodes, counts, most=None):
    pace = _lib()
    io = IO[gcfg.bf16_io]
    st, bu = dev(state), dev(buf)
    n = pace.draft_commit_workspace_bytes(gcfg, most or nodes.shape[1])
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    pace.draft_commit(gcfg, st, bu, dev(toks.k, io), dev(toks.v, io), dev(toks.a), dev(toks.beta), dev(nodes), dev(counts), ws,
                      most=most)
    return st, bu


def by_steps(gcfg, state, buf, toks, nodes, counts):
    pace = _lib()
    io = IO[gcfg.bf16_io]
    st, bu = dev(state), dev(buf)
    o = torch.empty((gcfg.B, gcfg.Hv, gcfg.dv), dtype=io, device="cuda")
    each = np.arange(gcfg.B)
    for i in range(int(max(counts.max(), 0))):
        at = nodes[:, i].clip(0, nodes.shape[1] - 1)
        active = (i < counts).astype(np.uint8)
        pace.decode_step(gcfg, st, bu, *(dev(x[each, at], io) for x in (toks.q, toks.k, toks.v)), dev(toks.a[each, at]),
                         dev(toks.beta[each, at]), o, active=dev(active))
    return st, bu


def same_layer(ocfg, got, want):
    """The states' bytes, the counts, and the slots below them (what lies in the others is no token: the decode
    hands the period's last one to the fold without storing it, a commit stores it first)."""
    assert torch.equal(got[0], want[0])
    x, y = (pk.unpack_buffer(ocfg, t.cpu().numpy()) for t in (got[1], want[1]))
    assert np.array_equal(x["count"], y["count"])
    for name in x:
        if name == "count":
            continue
        n = y["count"] if y[name].shape[1] == ocfg.Hv else y["count"][:, :: ocfg.gamma]
        live = np.arange(ocfg.dP) < n[..., None]
        assert np.array_equal(x[name][live].view(np.uint8), y[name][live].view(np.uint8)), name


@pytest.mark.parametrize("T", [1, 7, 30])
@pytest.mark.parametrize("name", list(LAYERS))
def test_commit_is_decoding_the_path_bit_for_bit(name, T):
    rng = np.random.default_rng(T)
    B = 6
    ocfg, gcfg, state, buf = layer(name, 31 + T, B=B)
    toks = make_tokens(32, B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    counts = rng.integers(0, T + 1, size=B).astype(np.int32)
    counts[0], counts[1] = T, 0
    nodes = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        nodes[b, : counts[b]] = np.sort(rng.choice(T, counts[b], replace=False))
    nodes[2] = nodes[2][::-1].copy() if counts[2] == T else nodes[2]
    same_layer(ocfg, run_commit(gcfg, state, buf, toks, nodes, counts), by_steps(gcfg, state, buf, toks, nodes, counts))


def test_commit_ends_at_a_bad_node_and_keeps_to_its_bounds():
    ocfg, gcfg, state, buf = layer("pace4", 41, B=6, counts=[0, 3, 7, 2, 5, 6])
    T = 9
    toks = make_tokens(42, 6, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=True)
    nodes = np.tile(np.arange(T, dtype=np.int32), (6, 1))
    nodes[1, 3], nodes[2, 0], nodes[3, 5] = T, -7, 2 ** 31 - 1
    nodes[4] = 4                                                              # the same node again and again
    counts = np.array([-5, 9, 9, 9, 9, 2 ** 31 - 1], dtype=np.int32)
    got = run_commit(gcfg, state, buf, toks, nodes, counts, most=6)
    want = by_steps(gcfg, state, buf, toks, nodes, np.array([0, 3, 0, 5, 6, 6], dtype=np.int32))
    same_layer(ocfg, got, want)


# ------------------------------------------------------------- verification

def run_verify(target, draft, tokens, parents, u, lens=None, pad=0, bf16=False, offset=0):
    pace = _lib()
    B, T, V = target.shape
    cfg = pace.VerifyConfig(B=B, T=T, V=V, bf16_probs=bf16)

    def rows(x):
        if x is None:
            return None
        wide = torch.full((B * T * (V + pad) + offset,), 7.0, dtype=IO[bf16], device="cuda")[offset:].view(B, T, V + pad)
        wide[..., :V] = dev(np.asarray(x, dtype=np.float32), IO[bf16])
        return wide[..., :V]

    nodes = torch.full((B, T), 99, dtype=torch.int32, device="cuda")
    counts, following = (torch.full((B,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    n = pace.draft_verify_workspace_bytes(cfg)
    pace.draft_verify(cfg, rows(target), dev(np.asarray(tokens, dtype=np.int32)),
                      None if parents is None else dev(np.asarray(parents, dtype=np.int32)), dev(np.asarray(u, dtype=np.float32)),
                      nodes, counts, following, draft=rows(draft),
                      draft_lens=None if lens is None else dev(np.asarray(lens, dtype=np.int32)),
                      workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None)
    return nodes.cpu().numpy(), counts.cpu().numpy(), following.cpu().numpy()


def probabilities(rng, shape, sharp, bf16):
    z = rng.standard_normal(shape) * sharp
    p = np.exp(z - z.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True)).astype(np.float32)
    return torch.from_numpy(p).to(IO[bf16]).float().numpy()


def same(got, want):
    for x, y, name in zip(got, want, ("nodes", "counts", "next")):
        assert np.array_equal(x, y), (name, x, y)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("T,V,kind,pad", [(1, 1, "chain", 0), (1, 5000, "chain", 3), (4, 2, "chain", 0), (8, 2047, "chain", 1),
                                          (8, 2048, "tree", 0), (25, 2049, "tree", 5), (25, 6151, "forest", 0), (63, 40, "tree", 0),
                                          (64, 600, "chain", 8), (65, 600, "chain", 0), (200, 97, "tree", 0), (1024, 9, "forest", 0)])
def test_verification(T, V, kind, pad, drawn, bf16):
    rng = np.random.default_rng(T * V + drawn)
    B = 7
    target, q = probabilities(rng, (B, T, V), 2.0, bf16), probabilities(rng, (B, T, V), 2.0, bf16)
    q = torch.from_numpy(0.7 * target + 0.3 * q).to(IO[bf16]).float().numpy()
    par = np.array(trees(rng, B, T, kind))
    tokens = np.zeros((B, T), dtype=np.int64)
    for b in range(B):
        for i in range(1, T):
            p = q[b, max(par[b, i], 0)].astype(np.float64)
            tokens[b, i] = rng.choice(V, p=p / p.sum()) if drawn else np.argsort(-p)[min(V - 1, int(rng.integers(0, 3)))]
    u = rng.random((B, T)).astype(np.float32)
    u[1] *= 0.3
    lens = np.full(B, T)
    lens[2], lens[3] = T // 2, 0
    chain = None if kind == "chain" and drawn else par
    want = do.draft_verify(target, q if drawn else None, tokens, par, u, lens)
    same(run_verify(target, q if drawn else None, tokens, chain, u, lens, pad, bf16, offset=pad % 3), want)


def test_verification_of_rows_that_are_no_probabilities():
    """Zero rows, NaN, infinities and negative entries, all weight on refused tokens, uniforms at and past the ends."""
    rng = np.random.default_rng(4)
    B, T, V = 16, 6, 37
    target, q = probabilities(rng, (B, T, V), 1.0, False), probabilities(rng, (B, T, V), 1.0, False)
    tokens = rng.integers(0, V, size=(B, T))
    par = np.array([[-1, 0, 0, 0, 1, 2]] * B)
    u = rng.random((B, T)).astype(np.float32)
    target[0] = 0.0
    target[1, :, ::2] = np.nan
    target[2, :, 5:] = -1.0
    target[3, :, 3] = np.inf
    q[3, :, 4] = np.nan
    target[4], q[4] = 0.0, 0.0
    target[4, :, 9], q[4, :, 9] = 1.0, 1.0
    tokens[4] = 3
    u[5] = 0.0
    u[6] = 1.0
    u[7] = np.nan
    u[8] = 5.0
    u[9] = -1.0
    tokens[10, 1:3] = [-1, V]
    tokens[11] = 8                                                             # the same token for every node
    target[12, :, :] = 0.25
    target[13], q[13] = 0.0, 1.0 / V                                             # nothing is left of a row that the draft covers
    target[13, :, 2] = 1e-3
    target[14] = 1e-40                                                           # subnormal
    par[15] = [-1, 7, -3, 2 ** 31 - 1, -2 ** 31, 5]                              # nobody's children
    for draft in (q, None):
        want = do.draft_verify(target, draft, tokens, par, u, [T] * B)
        same(run_verify(target, draft, tokens, par, u), want)


def test_verification_at_ties():
    """Dyadic probabilities: every sum is exact, and u on a border takes the token behind it."""
    V = 8
    p = np.array([0.25, 0.125, 0.0, 0.125, 0.25, 0.0, 0.125, 0.125], dtype=np.float32)
    us = np.arange(0, 17) / 16.0
    B = len(us)
    target = np.broadcast_to(p, (B, 1, V))
    u = us[:, None].astype(np.float32)
    want = do.draft_verify(target, None, np.zeros((B, 1), int), np.full((B, 1), -1), u, [1] * B)
    got = run_verify(target, None, np.zeros((B, 1), int), None, u)
    same(got, want)
    assert got[2][4] == 1 and got[2][16] == 7 and got[2][0] == 0
    # accepted below p / q, refused at it
    target = np.broadcast_to(p, (2, 2, V)).copy()
    draft = np.full((2, 2, V), 0.125, dtype=np.float32)
    draft[:, :, 4] = 0.5
    u = np.array([[0.0, 0.5], [0.0, np.nextafter(np.float32(0.5), np.float32(0))]], dtype=np.float32)
    tokens = np.full((2, 2), 4)
    got = run_verify(target, draft, tokens, None, u)
    assert list(got[1]) == [1, 2]
    same(got, do.draft_verify(target, draft, tokens, np.array([[-1, 0]] * 2), u, [2, 2]))


# -------------------------------------------------------------------- moves

class Cached:
    def __init__(self, seed, B, Hkv, d, kind, group, page, MP, spare=5):
        pace, rng = _lib(), np.random.default_rng(seed)
        N = 2 * B * MP + spare
        self.c = co.Cache(B=B, Hkv=Hkv, d=d, kind=kind, group=group, page=page, num_pages=N, max_pages=MP)
        self.cfg = pace.CacheConfig(B=B, Hq=Hkv, Hkv=Hkv, d=d, num_pages=N, max_pages=MP, kind=kind, group=group, page=page)
        self.bytes = rng.integers(0, 256, self.c.nbytes, dtype=np.uint8)
        order = rng.permutation(N)[: 2 * B * MP].astype(np.int32).reshape(2, B, MP)
        self.src, self.other = order

    def check(self, start, nodes, counts, src=None, dst=None, most=None):
        src, dst = self.src if src is None else src, self.src if dst is None else dst
        cache = dev(self.bytes)
        start, counts = np.asarray(start, dtype=np.int32), np.asarray(counts, dtype=np.int32)
        _lib().cache_move(self.cfg, cache, dev(src), dev(dst), dev(start), dev(counts),
                          nodes=None if nodes is None else dev(np.asarray(nodes, dtype=np.int32)), most=most)
        top = most if nodes is None or most is not None else nodes.shape[1]
        want = do.cache_move(self.c, self.bytes, src, dst, start, nodes, np.clip(counts, 0, top))
        got = cache.cpu().numpy()
        assert np.array_equal(got, want), np.nonzero(got != want)[0][:10]


KINDS = [("int8", 128, 64, 64), ("int4", 128, 32, 16), ("fp8", 64, 64, 32), ("int4", 64, 32, 64), ("int8", 256, 128, 16), ("int4", 256, 64, 128)]


@pytest.mark.parametrize("kind,d,group,page", KINDS)
@pytest.mark.parametrize("T", [1, 4, 25, 70, 300])
def test_accepted_paths_and_kept_entries_move_in_place(kind, d, group, page, T):
    rng = np.random.default_rng(T)
    B = 4
    s = Cached(T, B, 2, d, kind, group, page, MP=-(-(T + 100) // page))
    nodes, counts = np.full((B, T), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        n = [T, max(1, T // 2), 0, max(1, T // 3)][b]
        nodes[b, :n], counts[b] = np.sort(rng.choice(T, n, replace=False)), n
    s.check([0, 3, 7, 61], nodes, counts)


@pytest.mark.parametrize("kind,d,group,page", KINDS)
@pytest.mark.parametrize("T", [65, 200])
def test_kept_entries_of_many_sequences_move_in_place(kind, d, group, page, T):
    """As many (sequence, head) pairs as the kernel of small steps takes, several steps each."""
    rng, B = np.random.default_rng(T + 7), 34
    s = Cached(T + 7, B, 4, d, kind, group, page, MP=-(-(T + 40) // page))
    nodes, counts = np.full((B, T), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        counts[b] = rng.integers(0, T + 1)
        nodes[b, : counts[b]] = np.sort(rng.choice(T, counts[b], replace=False))
    s.check(rng.integers(0, 40, B), nodes, counts)


@pytest.mark.parametrize("kind,d,group,page", KINDS)
@pytest.mark.parametrize("T", [1, 63, 257])
def test_forks_copy_into_other_pages(kind, d, group, page, T):
    B = 3
    s = Cached(T + 1, B, 2, d, kind, group, page, MP=-(-(T + 30) // page))
    src = np.repeat(s.src[:1], B, axis=0)
    s.check([0, 0, 17], None, [T, T // 2, T], src=src, dst=s.other, most=T)
    nodes = np.random.default_rng(T).integers(0, T, size=(B, T))                # any order, repeats too, between tables without a common page
    s.check([5, 0, 1], nodes, [T, T, T - 1], src=src, dst=s.other)


@pytest.mark.parametrize("kind,d,group,page", KINDS)
def test_forks_that_keep_a_prefix(kind, d, group, page):
    """Tables that hold the same pages at their first entries: what lies there stays, or moves in place."""
    T = 2 * page + 21
    s = Cached(23, 1, 2, d, kind, group, page, MP=4)
    dst = s.other.copy()
    dst[:, :2] = s.src[:, :2]
    s.check([0], None, [T], dst=dst, most=T)
    s.check([3], None, [T - 9], dst=dst, most=T)
    nodes = np.sort(np.random.default_rng(page).choice(T, T // 2, replace=False))[None]
    s.check([2], nodes, [T // 2], dst=dst)


def test_moves_leave_out_what_is_not_there():
    s = Cached(3, 3, 2, 64, "int8", 32, 16, MP=6)
    T = 50
    nodes = np.tile(np.arange(T) + 20, (3, 1))
    nodes[0, ::5] = -1
    src, dst = s.src.copy(), s.other.copy()
    src[1, 2], dst[1, 1] = -1, s.c.num_pages
    src[2, :], dst[2, 3:] = 2 ** 31 - 1, -2 ** 31
    s.check([0, 40, 5], nodes, [T, T + 30, T], src=src, dst=dst)               # past the table, more than there are
    s.check([-30, 2 ** 31 - 1, -2 ** 31], nodes, [T, T, T], src=src, dst=dst)
    s.check([0, 0, 0], nodes, [-1, 0, -2 ** 31], src=src, dst=dst)
    nodes[0] = 2 ** 31 - 1
    s.check([2 ** 31 - 1, 0, 0], nodes, [T, T, T], src=src, dst=dst)
