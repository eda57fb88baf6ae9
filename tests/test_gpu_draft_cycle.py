"""A step of drafted tokens as a serving program makes it: outputs of the drafts in every layer, verification,
commits and moves, from one call's device results to the next; eager, on other streams, and captured in a graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import draft_oracle as do  # noqa: E402
from test_gpu_draft import IO, _lib, bits, dev, host, probabilities, run_verify, same, trees  # noqa: E402

pytestmark = pytest.mark.gpu
B, T, V, HEADS, D, PAGE, MAX_PAGES = 5, 7, 48, 8, 128, 16, 8


class Stack:
    """A gated-delta layer and an attention layer in mid-service, and the inputs of one step of drafts."""

    def __init__(self, seed=0, dP=8):
        pace, self.rng = _lib(), np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.delta = pace.pace4(B=B, Hv=HEADS, Hk=HEADS // 2, d=D, dP=dP)
        sizes = pace.layout(self.delta)
        self.state = torch.zeros(sizes["state_bytes"], dtype=torch.uint8, device="cuda")
        self.buffer = torch.zeros(sizes["buffer_bytes"], dtype=torch.uint8, device="cuda")
        self.att = pace.CacheConfig(B=B, Hq=HEADS, Hkv=2, d=D, num_pages=B * MAX_PAGES, max_pages=MAX_PAGES, kind="int8",
                                    group=64, page=PAGE)
        self.cache = torch.randint(0, 256, (pace.cache_layout(self.att)["cache_bytes"],), generator=self.gen, device="cuda").to(torch.uint8)
        self.table = dev(self.rng.permutation(B * MAX_PAGES).astype(np.int32).reshape(B, MAX_PAGES))
        self.lens = dev(np.array([40, 0, 17, 63, 5], dtype=np.int32))
        prompt = 64
        q, k, v, a, b = self.tokens(prompt)
        pace.prefill_chunk(self.delta, self.state, q, k, v, a, b, torch.empty_like(v))
        for _ in range(5):                                   # some buffered tokens
            q, k, v, a, b = self.tokens(1)
            pace.decode_step(self.delta, self.state, self.buffer, q[:, 0], k[:, 0], v[:, 0], a[:, 0].contiguous(), b[:, 0].contiguous(),
                             torch.empty_like(v[:, 0]))
        ck, cv = self.normal(B, 64, 2, D), self.normal(B, 64, 2, D)
        at = torch.arange(64, device="cuda", dtype=torch.int32).expand(B, 64)
        pace.cache_write(self.att, self.cache, self.table, torch.where(at < self.lens[:, None], at, -1).contiguous(), ck, cv)
        # one step's inputs
        self.parents = trees(self.rng, B, T, "tree")
        self.bits = bits(self.parents)
        self.parents_dev = dev(np.array(self.parents, dtype=np.int32))
        self.drafts = self.tokens(T)
        self.q, self.k, self.v = self.normal(B, T, HEADS, D), self.normal(B, T, 2, D), self.normal(B, T, 2, D)
        self.target, self.draft = probabilities(self.rng, (B, T, V), 1.5, False), probabilities(self.rng, (B, T, V), 1.5, False)
        self.draft = 0.8 * self.target + 0.2 * self.draft
        self.ids = np.zeros((B, T), dtype=np.int32)
        for x in range(B):
            for i in range(1, T):
                p = self.draft[x, self.parents[x][i]].astype(np.float64)
                self.ids[x, i] = self.rng.choice(V, p=p / p.sum())
        self.u = self.rng.random((B, T)).astype(np.float32)
        self.vcfg = pace.VerifyConfig(B=B, T=T, V=V)
        self.inputs = (dev(self.target), dev(self.draft), dev(self.ids), dev(self.u))
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.nodes, self.counts, self.next = i32(B, T), i32(B), i32(B)
        self.o_delta = torch.empty((B, T, HEADS, D), dtype=torch.bfloat16, device="cuda")
        self.o_att = torch.empty_like(self.o_delta)
        scratch = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws_v, self.ws_c = scratch(pace.draft_verify_workspace_bytes(self.vcfg)), scratch(pace.draft_commit_workspace_bytes(self.delta, T))
        n = pace.cache_attention_workspace_bytes(self.att, T, MAX_PAGES * PAGE)
        self.ws_a = scratch(n) if n else None
        self.at = (self.lens[:, None] + torch.arange(T, device="cuda")).to(torch.int32)
        torch.cuda.synchronize()

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def tokens(self, n):
        unit = lambda: torch.nn.functional.normalize(torch.randn((B, n, HEADS // 2, D), generator=self.gen, device="cuda"), dim=-1).to(torch.bfloat16)  # noqa: E731
        a = torch.exp(-torch.nn.functional.softplus(torch.randn((B, n, HEADS), generator=self.gen, device="cuda") - 3))
        return unit(), unit(), self.normal(B, n, HEADS, D), a, torch.sigmoid(torch.randn((B, n, HEADS), generator=self.gen, device="cuda"))

    def step(self):
        pace = _lib()
        q, k, v, a, b = self.drafts
        pace.draft_step(self.delta, self.state, self.buffer, q, k, v, a, b, self.o_delta, tree=self.bits)
        pace.cache_write(self.att, self.cache, self.table, self.at, self.k, self.v)
        pace.cache_attention(self.att, self.cache, self.table, self.q, self.lens, self.o_att, tree=self.bits, workspace=self.ws_a)
        target, draft, ids, u = self.inputs
        pace.draft_verify(self.vcfg, target, ids, self.parents_dev, u, self.nodes, self.counts, self.next, draft=draft, workspace=self.ws_v)
        pace.draft_commit(self.delta, self.state, self.buffer, k, v, a, b, self.nodes, self.counts, self.ws_c)
        pace.cache_move(self.att, self.cache, self.table, self.table, self.lens, self.counts, nodes=self.nodes)
        self.lens.add_(self.counts)

    def held(self):
        return [self.state, self.buffer, self.cache, self.lens, self.nodes, self.counts, self.next, self.o_delta, self.o_att]


def by_hand(s):
    """The accepted path of a Stack that has not stepped yet, token by token: (outputs of the delta layer per node, state,
    buffer, cache, path)."""
    pace = _lib()
    nodes, counts, _ = do.draft_verify(s.target, s.draft, s.ids, np.array(s.parents), s.u, [T] * B)
    state, buffer, cache = s.state.clone(), s.buffer.clone(), s.cache.clone()
    q, k, v, a, b = s.drafts
    each = torch.arange(B, device="cuda")
    outs = []
    for i in range(int(counts.max())):
        at = dev(nodes[:, i].clip(0).astype(np.int64))
        o = torch.empty((B, HEADS, D), dtype=torch.bfloat16, device="cuda")
        pace.decode_step(s.delta, state, buffer, q[each, at], k[each, at], v[each, at], a[each, at], b[each, at], o,
                         active=dev((i < counts).astype(np.uint8)))
        outs.append(o)
        pos = torch.where(dev(i < counts), s.lens + i, torch.full_like(s.lens, -1)).view(B, 1)
        pace.cache_write(s.att, cache, s.table, pos, s.k[each, at][:, None].contiguous(), s.v[each, at][:, None].contiguous())
    return outs, state, buffer, cache, nodes, counts


def read(s, cache, n):
    pace = _lib()
    k, v = (torch.empty((B, n, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = torch.arange(n, device="cuda", dtype=torch.int32).expand(B, n).contiguous()
    pace.cache_read(s.att, cache, s.table, at, k, v)
    return k, v


@pytest.mark.parametrize("dP", [8, 16])
def test_a_step_ends_as_decoding_the_accepted_path(dP):
    from oracle import packing as pk
    from test_gpu_draft import same_layer
    s = Stack(3, dP)
    outs, state, buffer, cache, nodes, counts = by_hand(s)
    before = s.lens.clone()
    s.step()
    assert np.array_equal(s.nodes.cpu().numpy(), nodes) and np.array_equal(s.counts.cpu().numpy(), counts)
    ocfg = pk.LayerCfg(B=B, Hv=HEADS, Hk=HEADS // 2, dk=D, dv=D, group=64, asym=False, buf="int8", dP=dP, bf16_io=True)
    same_layer(ocfg, (s.state, s.buffer), (state, buffer))
    # the cache: codes and scales of the accepted entries at their places, those of the context where they were
    assert torch.equal(s.lens, before + dev(counts))
    n = int(s.lens.max())
    live = (torch.arange(n, device="cuda") < s.lens[:, None])[:, :, None, None]
    for x, y in zip(read(s, s.cache, n), read(s, cache, n)):
        assert torch.equal(torch.where(live, x, torch.zeros_like(x)), torch.where(live, y, torch.zeros_like(y)))
    # outputs of accepted nodes against decoding them, where no rounding of the state lay between (count 5 of dP)
    for i, o in enumerate(outs):
        if 5 + i >= dP:
            break
        for b in range(B):
            if i < counts[b]:
                x, y = host(s.o_delta[b, nodes[b, i]]), host(o[b])
                # both round fp32 values that differ by sums' orders: a step of bf16 at most next to a tie
                assert np.abs(x - y).max() <= 2.0 ** -7 * np.abs(y).max()


def test_a_captured_step_replays_as_the_eager_one():
    s, e = Stack(5), Stack(5)
    start = [t.clone() for t in s.held()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.step()                                              # (warms up)
        for t, x in zip(s.held(), start):
            t.copy_(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.step()
    torch.cuda.synchronize()
    wanted = []
    for _ in range(3):                                        # steps that go on from one another (the drafts' places move with lens)
        e.at.copy_(e.lens[:, None] + torch.arange(T, device="cuda"))
        e.step()
        wanted.append([t.clone() for t in e.held()])
    for t, x in zip(s.held(), start):
        t.copy_(x)
    for want in wanted:
        s.at.copy_(s.lens[:, None] + torch.arange(T, device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 20, device="cuda").sum().item()  # noqa: F841  (eager work between)
        for i, (x, y) in enumerate(zip(s.held(), want)):
            assert torch.equal(x, y), i


def test_two_stacks_on_streams_of_their_own():
    a, b, ea, eb = Stack(7), Stack(8), Stack(7), Stack(8)
    ea.step()
    eb.step()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(sa):
        a.step()
    with torch.cuda.stream(sb):
        b.step()
    torch.cuda.synchronize()
    for x, y in zip(a.held() + b.held(), ea.held() + eb.held()):
        assert torch.equal(x, y)


def test_prepared_calls_are_the_calls():
    pace = _lib()
    s, e = Stack(9), Stack(9)
    q, k, v, a, b = s.drafts
    target, draft, ids, u = s.inputs
    calls = [pace.prepare_draft_step(s.delta, s.state, s.buffer, q, k, v, a, b, s.o_delta, tree=s.bits),
             pace.prepare_cache_write(s.att, s.cache, s.table, s.at, s.k, s.v),
             pace.prepare_cache_attention(s.att, s.cache, s.table, s.q, s.lens, s.o_att, tree=s.bits, workspace=s.ws_a),
             pace.prepare_draft_verify(s.vcfg, target, ids, s.parents_dev, u, s.nodes, s.counts, s.next, draft=draft, workspace=s.ws_v),
             pace.prepare_draft_commit(s.delta, s.state, s.buffer, k, v, a, b, s.nodes, s.counts, s.ws_c),
             pace.prepare_cache_move(s.att, s.cache, s.table, s.table, s.lens, s.counts, nodes=s.nodes)]
    for c in calls:
        c()
    s.lens.add_(s.counts)
    e.step()
    for x, y in zip(s.held(), e.held()):
        assert torch.equal(x, y)


# ----------------------------------------------------- verification in two kernels

@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("Bn,Tn,Vn,kind,pad", [(1, 3, 32769, "chain", 0), (2, 12, 40001, "tree", 0), (3, 9, 65536, "star", 8), (2, 70, 34817, "tree", 3),
                                              (1, 6, 300007, "star", 1), (260, 2, 36000, "chain", 0)])
def test_verification_over_large_vocabularies(Bn, Tn, Vn, kind, pad, drawn, bf16):
    rng = np.random.default_rng(Vn)
    par = np.array([[-1] + [0] * (Tn - 1)] * Bn if kind == "star" else trees(rng, Bn, Tn, kind))
    target = probabilities(rng, (Bn, Tn, Vn), 3.0, bf16)
    q = torch.from_numpy(np.float32(0.6) * target + np.float32(0.4) * np.roll(target, 7, axis=-1)).to(IO[bf16]).float().numpy()
    tokens = np.zeros((Bn, Tn), dtype=np.int64)
    for b in range(Bn):
        for i in range(1, Tn):
            p = q[b, max(par[b, i], 0)].astype(np.float64)
            tokens[b, i] = np.searchsorted(np.cumsum(p), rng.random() * p.sum()) if drawn else np.argpartition(-p, 3)[i % 3]
    tokens = tokens.clip(0, Vn - 1)
    u = rng.random((Bn, Tn)).astype(np.float32)
    u[0, 1:] = 0.999                                           # most children refused: several rows summed
    lens = np.full(Bn, Tn)
    if Bn > 1:
        lens[1] = 0
    want = do.draft_verify(target, q if drawn else None, tokens, par, u, lens)
    same(run_verify(target, q if drawn else None, tokens, par, u, lens, pad, bf16, offset=pad % 3), want)


def test_verification_of_rows_behind_2_to_32_bytes():
    """Probabilities of 6.4 GB: rows past 2^31 elements."""
    pace = _lib()
    Bn, Tn, Vn = 3, 1024, 1 << 20
    target = torch.zeros((Bn, Tn, Vn), dtype=torch.bfloat16, device="cuda")
    # a chain that is accepted to its end; the following token is the last of the vocabulary but one
    ids = torch.randint(0, Vn, (Bn, Tn), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    each = torch.arange(Bn, device="cuda")[:, None]
    target[each, torch.arange(Tn - 1, device="cuda")[None], ids[:, 1:]] = 1.0
    target[:, Tn - 1, Vn - 2] = 1.0
    cfg = pace.VerifyConfig(B=Bn, T=Tn, V=Vn, bf16_probs=True)
    nodes, counts, following = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((Bn, Tn), (Bn,), (Bn,)))
    ws = torch.empty(pace.draft_verify_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    pace.draft_verify(cfg, target, ids.to(torch.int32), None, torch.full((Bn, Tn), 0.5, device="cuda"), nodes, counts, following, workspace=ws)
    assert counts.tolist() == [Tn] * Bn and following.tolist() == [Vn - 2] * Bn
    assert torch.equal(nodes, torch.arange(Tn, device="cuda", dtype=torch.int32).expand(Bn, Tn))


# --------------------------------------------------------------------- large caches

def test_moves_in_a_cache_of_more_than_2_to_32_bytes():
    pace = _lib()
    H, page, N = 8, 64, 40000
    cfg = pace.CacheConfig(B=2, Hq=H, Hkv=H, d=128, num_pages=N, max_pages=4, kind="int8", group=64, page=page)
    bytes_ = pace.cache_layout(cfg)["cache_bytes"]
    assert bytes_ > 2 ** 32
    cache = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    src = dev(np.array([[N - 1, N - 2, 3, 4], [5, N - 3, 6, N - 4]], dtype=np.int32))
    dst = dev(np.array([[N - 5, 7, N - 6, 8], [9, 10, N - 7, N - 8]], dtype=np.int32))
    n = 4 * page
    k, v = (torch.randn((2, n, H, 128), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    at = torch.arange(n, device="cuda", dtype=torch.int32).expand(2, n).contiguous()
    pace.cache_write(cfg, cache, src, at, k, v)
    out = [torch.empty_like(k) for _ in range(4)]
    pace.cache_read(cfg, cache, src, at, out[0], out[1])
    zero, full = dev(np.zeros(2, dtype=np.int32)), dev(np.array([n, n - 37], dtype=np.int32))
    pace.cache_move(cfg, cache, src, dst, zero, full, most=n)
    pace.cache_read(cfg, cache, dst, at, out[2], out[3])
    for x, y in ((out[0], out[2]), (out[1], out[3])):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1, : n - 37], y[1, : n - 37]) and not y[1, n - 37:].any()
    kept = torch.arange(0, n, 2, device="cuda", dtype=torch.int32).expand(2, n // 2).contiguous()
    pace.cache_move(cfg, cache, dst, dst, zero, dev(np.array([n // 2, n // 2 - 19], dtype=np.int32)), nodes=kept)
    pace.cache_read(cfg, cache, dst, at, out[2], out[3])
    for x, y in ((out[0], out[2]), (out[1], out[3])):
        assert torch.equal(x[0, ::2], y[0, : n // 2]) and torch.equal(x[1, : n - 38: 2], y[1, : n // 2 - 19])


@pytest.mark.parametrize("with_nodes", [True, False])
def test_moves_of_the_most_sequences(with_nodes):
    """65535 sequences at once, against the same moves in two calls."""
    pace = _lib()
    Bn, H, T_, page = 65535, 32, 50, 16
    halves = (slice(0, 30000), slice(30000, Bn))
    cfg = lambda n: pace.CacheConfig(B=n, Hq=H, Hkv=H, d=64, num_pages=2 * Bn, max_pages=1, kind="int4", group=32, page=page)  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = torch.randint(0, 256, (pace.cache_layout(cfg(Bn))["cache_bytes"],), generator=gen, device="cuda", dtype=torch.uint8)
    tables = torch.randperm(2 * Bn, generator=gen, device="cuda").to(torch.int32).view(2, Bn, 1)
    src, dst = tables[0], tables[0] if with_nodes else tables[1]
    start = torch.randint(0, 6, (Bn,), generator=gen, device="cuda").to(torch.int32)
    counts = torch.randint(0, T_, (Bn,), generator=gen, device="cuda").to(torch.int32)
    nodes = (2 * torch.arange(T_, device="cuda", dtype=torch.int32)).expand(Bn, T_).contiguous() if with_nodes else None
    want = cache.clone()
    pace.cache_move(cfg(Bn), cache, src, dst, start, counts, nodes=nodes, most=T_)
    assert not torch.equal(cache, want)
    for h in halves:
        n = h.stop - h.start
        pace.cache_move(cfg(n), want, src[h], dst[h], start[h].clone(), counts[h].clone(), nodes=nodes[h] if with_nodes else None, most=T_)
    assert torch.equal(cache, want)


def test_moves_of_nothing_read_no_nodes():
    """Sequences without entries to move, whose start lies inside a tile: rows of nodes next to what they may not be taken
    for, and caches as they were."""
    pace = _lib()
    for start in (0, 5, 15, 16, 37):
        cfg = pace.CacheConfig(B=2, Hq=2, Hkv=2, d=64, num_pages=8, max_pages=4, kind="int8", group=64, page=16)
        cache = torch.randint(0, 256, (pace.cache_layout(cfg)["cache_bytes"],), device="cuda", dtype=torch.uint8)
        want, table = cache.clone(), dev(np.array([[7, 1, 3, 0], [2, 6, 4, 5]], dtype=np.int32))
        nodes = torch.arange(3, 23, device="cuda", dtype=torch.int32).view(2, 10)
        for counts in ([0, 0], [-3, 0], [0, -2 ** 31]):
            pace.cache_move(cfg, cache, table, table, dev(np.array([start, start], dtype=np.int32)), dev(np.array(counts, dtype=np.int32)), nodes=nodes)
            assert torch.equal(cache, want)
