"""Measured cases of the attention-layer operators that run beside the gated-delta layers of a
hybrid stack: rotary positions, the quantised paged key/value cache (written and read back), and
attention for drafted tokens over that cache.

`listed()` gives the cases, `draw(rng)` more of the same ranges, `prepare(case, seed)` what a
serving program has in hand, `run(state)` one pass: in plain torch operations, or through the
library where `own` is true.  `work(case)` is what a pass cannot do without and `exact(case, seed)`
the result in 64 bits.

Cache format (one record per page and key/value head, P tokens of d channels, b bits, groups of g):
    key codes | key scales bf16 [P/4][d/g][4] | value codes | value scales bf16 [P/4][d/g][4]
Codes are laid out in the order in which the matrix instructions take them.  With G = c div 32 and
LB = d b / 32 bytes, cut in pieces of W = min(16, LB):
    keys   in tiles of 16 tokens; lane g4 = (c mod 32) div 8 of token r holds the LB bytes of its
           8-channel units G = 0, 1, ..; byte x sits at (x div W) 64 W + (16 g4 + r) W + x mod W.
           int4: a unit is 4 bytes, channel e in nibble (e div 2) + 4 (e mod 2).
    values in quads of 4 tokens; lane m = (c mod 32) div 2 holds channels 32 G + 2 m + {0, 1} of the
           four tokens t: 8 bits: byte x = 4 (2 G + c mod 2) + t; 4 bits: byte x = 4 G + t, the even
           channel in the low nibble; byte x sits at (x div W) 16 W + m W + x mod W.
int8 codes are stored plus 128, int4 codes plus 8, fp8 codes as e4m3 bit patterns.
"""
import json
import math
import random

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = {"int8": 127.0, "int4": 7.0, "fp8": 448.0}
BITS = {"int8": 8, "int4": 4, "fp8": 8}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # The step of 64 sequences that each decode one token, half of every head rotated: the
        # latency of a call in a decode step.
        {"name": "rotary-step", "op": "rotary", "tokens": 64, "Hq": 32, "Hk": 8, "d": 128, "rd": 64,
         "interleaved": False, "scaling": "none", "far": 4096, "inverse": False, "io": "bf16"},
        # A long prompt at once, whole heads, neighbouring pairs, frequencies scaled for a context
        # far past the original one.
        {"name": "rotary-prompt", "op": "rotary", "tokens": 32768, "Hq": 32, "Hk": 8, "d": 128, "rd": 128,
         "interleaved": True, "scaling": "blend", "far": 1000000, "inverse": False, "io": "bf16"},
        # Rotating back (keys taken out of a cache to be placed elsewhere; the gradient), odd count, fp32.
        {"name": "rotary-back", "op": "rotary", "tokens": 1021, "Hq": 16, "Hk": 4, "d": 256, "rd": 64,
         "interleaved": False, "scaling": "linear", "far": 131072, "inverse": True, "io": "f32"},
        # One token of 64 sequences goes into the cache in a decode step (and is read back: what
        # the cache then holds of it).
        {"name": "store-step", "op": "store", "B": 64, "T": 1, "H": 8, "d": 128, "kind": "int8", "group": 128,
         "page": 64, "start": 511, "skip": False, "io": "bf16"},
        # Four prompts of odd length in a chunked prefill, 4-bit cache with short groups.
        {"name": "store-prompt", "op": "store", "B": 4, "T": 4093, "H": 8, "d": 128, "kind": "int4", "group": 32,
         "page": 64, "start": 3, "skip": False, "io": "bf16"},
        # A short shared prefix read back for a new request.
        {"name": "read-short", "op": "read", "B": 1, "T": 257, "H": 4, "d": 64, "kind": "fp8", "group": 64,
         "page": 16, "start": 0, "skip": True, "io": "f32"},
        # Long prefixes read back.
        {"name": "read-long", "op": "read", "B": 4, "T": 16384, "H": 8, "d": 128, "kind": "int8", "group": 64,
         "page": 64, "start": 0, "skip": False, "io": "bf16"},
        # One sequence, one token, a 512-token context: the smallest decode call.
        {"name": "attend-one", "op": "attend", "B": 1, "T": 1, "Hq": 32, "H": 8, "d": 128, "kind": "int8",
         "group": 128, "page": 64, "ctx": 512, "spread": False, "tree": "none", "io": "bf16"},
        # The decode step of 64 sequences of all ages, 4-bit cache.
        {"name": "attend-step", "op": "attend", "B": 64, "T": 1, "Hq": 32, "H": 8, "d": 128, "kind": "int4",
         "group": 64, "page": 64, "ctx": 8192, "spread": True, "tree": "none", "io": "bf16"},
        # Trees of up to 25 drafted tokens checked for 16 sequences, 8-bit floating-point cache.
        {"name": "attend-tree", "op": "attend", "B": 16, "T": 25, "Hq": 32, "H": 8, "d": 128, "kind": "fp8",
         "group": 128, "page": 64, "ctx": 4096, "spread": True, "tree": "tree", "io": "bf16"},
        # Few sequences with very long contexts.
        {"name": "attend-long", "op": "attend", "B": 3, "T": 1, "Hq": 32, "H": 8, "d": 128, "kind": "int8",
         "group": 128, "page": 64, "ctx": 131072, "spread": False, "tree": "none", "io": "bf16"},
        # A chunk of two prompts over what is cached already: the matrix products bound it.
        {"name": "attend-chunk", "op": "attend", "B": 2, "T": 512, "Hq": 32, "H": 8, "d": 128, "kind": "int8",
         "group": 128, "page": 64, "ctx": 7680, "spread": False, "tree": "none", "io": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "store", "store", "read", "attend", "attend", "attend", "attend"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        d = rng.choice([64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4])
        tokens = _log(rng, 1, 32768)
        while tokens * (Hq + Hk) * d * (2 if io == "f32" else 1) > 32768 * 40 * 128:
            tokens = _log(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "Hq": Hq, "Hk": Hk, "d": d, "rd": rng.choice([d, d // 2, d // 4]),
                "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "ntk", "blend"]),
                "far": _log(rng, 64, 1000000), "inverse": rng.random() < 0.3, "io": io}
    kind = rng.choice(["int8", "int4", "fp8"])
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    page = rng.choice([16, 32, 64, 128])
    if op in ("store", "read"):
        most = 4 * 16384 * 8 * 128 if op == "read" else 4 * 4093 * 8 * 128
        while True:
            B, T, H = _log(rng, 1, 64), _log(rng, 1, 16384), rng.choice([1, 2, 4, 8])
            if B * T * H * d * (2 if io == "f32" else 1) <= most:
                break
        return {"op": op, "B": B, "T": T, "H": H, "d": d, "kind": kind, "group": group, "page": page,
                "start": rng.randrange(0, 600) if op == "store" else 0, "skip": rng.random() < 0.3, "io": io}
    tree = rng.choice(["none", "tree", "chain"])
    H = rng.choice([1, 2, 4, 8])
    Hq = H * rng.choice([1, 2, 3, 4, 8])
    while True:
        B, ctx = _log(rng, 1, 64), rng.choice([0, _log(rng, 1, 131072), _log(rng, 1, 131072), _log(rng, 1, 131072)])
        T = 1 if tree == "none" else _log(rng, 2, 64) if tree == "tree" else _log(rng, 2, 512)
        held, rows = B * H * d * (ctx + T), B * Hq * T * (ctx + T)
        if held <= 3 * 8 * 128 * 131072 and rows * d <= 2 * 32 * 512 * 8192 * 128:
            break
    return {"op": op, "B": B, "T": T, "Hq": Hq, "H": H, "d": d, "kind": kind, "group": group, "page": page,
            "ctx": ctx, "spread": rng.random() < 0.5, "tree": "tree" if tree == "tree" else "none", "io": io}


def _plan(case):
    """A case's lengths and trees (host values that work() needs too): by the case alone."""
    r = random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))
    B, T = case["B"], case["T"]
    if case["op"] != "attend":
        start = [case["start"]] * B
        if case["op"] == "store" and case["skip"]:
            start = [r.randrange(case["start"] + 1) for _ in range(B)]
        drop = [[case["skip"] and r.random() < 0.25 for _ in range(T)] for _ in range(B)]
        return {"start": start, "drop": drop}
    ctx = [r.randrange(case["ctx"] // 16, case["ctx"] + 1) if case["spread"] else case["ctx"] for _ in range(B)]
    parents, drafts = None, [T] * B
    if case["tree"] == "tree":
        # every node hangs on one of the few before it; -1: on the context itself
        parents = [[r.randrange(max(-1, i - 6), i) for i in range(T)] for _ in range(B)]
        drafts = [r.randrange(T // 2, T + 1) if case["spread"] else T for _ in range(B)]
    return {"ctx": ctx, "parents": parents, "drafts": drafts}


def _tree_mask(parents):
    """[B][T][T] truth values: node j is node i or one of its ancestors."""
    B, T = len(parents), len(parents[0])
    m = torch.zeros((B, T, T), dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            if parents[b][i] >= 0:
                m[b, i] = m[b, parents[b][i]]
            m[b, i, i] = True
    return m


# ------------------------------------------------------------- inputs and the cache's bytes

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _vectors(gen, shape, io, outliers):
    """Keys or values: normal, four channels of every 64 eight times as large in keys."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if outliers:
        x[..., 5::16] *= 8.0
    return x.to(IO[io])


def _scale_up(m, levels):
    """The smallest bf16 value that is not under m / levels, zero where that is under 2^-126."""
    q = m.float() / torch.full_like(m, levels, dtype=torch.float32)   # a tensor: a number's reciprocal would be multiplied by
    over = q.double() * levels < m.double()          # the division rounded down
    q = torch.where(over, (q.view(torch.int32) + 1).view(torch.float32), q)
    u = (q.view(torch.int32) + 0xFFFF) & -65536
    s = u.view(torch.float32)
    return torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)


def _quantise(x, kind, group):
    """(codes as the values they are, scales) of vectors [..., d]; scales [..., d/group]."""
    f = x.float().unflatten(-1, (-1, group))
    f = torch.where(f.isnan(), torch.zeros_like(f), f.clamp(-2.0 ** 127, 2.0 ** 127))
    s = _scale_up(f.abs().amax(-1), LEVELS[kind])
    c = f / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)
    c = torch.where(s.unsqueeze(-1) > 0, c, torch.zeros_like(c))
    c = c.clamp(-LEVELS[kind], LEVELS[kind])
    c = c.to(torch.float8_e4m3fn) if kind == "fp8" else c.round().to(torch.int8)
    return c.flatten(-2), s


def _stored(c, kind):
    """Codes as stored fields, uint8 (int4: one field a byte still)."""
    if kind == "fp8":
        return c.view(torch.uint8)
    return (c.to(torch.int16) + (128 if kind == "int8" else 8)).to(torch.uint8)


def _valued(u, kind):
    """Stored fields as the values of their codes, fp32."""
    if kind == "fp8":
        return u.view(torch.float8_e4m3fn).float()
    return u.float() - (128.0 if kind == "int8" else 8.0)


def _dims(case):
    d, P, b = case["d"], case["page"], BITS[case["kind"]]
    LB = d * b // 32
    W = min(16, LB)
    codes, scales = P * d * b // 8, P * (d // case["group"]) * 2
    return {"LB": LB, "W": W, "NI": LB // W, "codes": codes, "scales": scales, "rec": 2 * (codes + scales)}


def _key_bytes(u, kind):
    """Fields [..., d] of keys -> bytes [..., 4 lanes, LB]."""
    u = u.unflatten(-1, (-1, 4, 8)).transpose(-3, -2)                   # [..., g4, G, 8]
    if kind == "int4":
        u = u.unflatten(-1, (2, 2, 2))                                  # e = 4 a + 2 h + odd
        lo, hi = u[..., 0, :], u[..., 1, :]                             # nibbles 2 n, 2 n + 1
        u = (lo | (hi << 4)).transpose(-1, -2).flatten(-2)              # bytes: even channels, odd ones
    return u.flatten(-2)


def _key_fields(y, kind):
    """The reverse of _key_bytes."""
    if kind == "int4":
        y = y.unflatten(-1, (-1, 2, 2))                                 # [.., G, odd, a]
        y = torch.stack([y & 15, y >> 4], dim=-1)                       # [.., G, odd, a, h]
        y = y.movedim(-3, -1).flatten(-3)                               # e = 4 a + 2 h + odd
    else:
        y = y.unflatten(-1, (-1, 8))
    return y.transpose(-3, -2).flatten(-3)


def _value_bytes(u, kind):
    """Fields [..., d] of values -> one token's bytes [..., 16 lanes, LB / 4]."""
    u = u.unflatten(-1, (-1, 16, 2)).transpose(-3, -2)                  # [..., m, G, e]
    return u[..., 0] | (u[..., 1] << 4) if kind == "int4" else u.flatten(-2)


def _value_fields(y, kind):
    """The reverse of _value_bytes."""
    y = torch.stack([y & 15, y >> 4], dim=-1) if kind == "int4" else y.unflatten(-1, (-1, 2))
    return y.transpose(-3, -2).flatten(-3)


def _pack(case, kf, ks, vf, vs):
    """Pages [N, H, rec] of whole pages' fields and scales [N, P, H, d], [N, P, H, d/g]."""
    D, kind, P = _dims(case), case["kind"], case["page"]
    N, H = kf.shape[0], kf.shape[2]
    k = _key_bytes(kf, kind).view(N, P // 16, 16, H, 4, D["NI"], D["W"]).permute(0, 3, 1, 5, 4, 2, 6)
    v = _value_bytes(vf, kind).view(N, P // 4, 4, H, 16, D["LB"] // 4).permute(0, 3, 1, 4, 5, 2)
    v = v.reshape(N, H, P // 4, 16, D["NI"], D["W"]).transpose(3, 4)
    bits = lambda s: s.unflatten(1, (-1, 4)).permute(0, 3, 1, 4, 2).contiguous().view(torch.uint8)  # noqa: E731
    return torch.cat([k.reshape(N, H, -1), bits(ks).reshape(N, H, -1), v.reshape(N, H, -1),
                      bits(vs).reshape(N, H, -1)], dim=-1)


def _unpack(case, pages):
    """Pages [..., H, rec] -> dequantised keys and values fp32 [..., P, H, d]."""
    D, kind, P, g = _dims(case), case["kind"], case["page"], case["group"]
    lead, H = pages.shape[:-2], pages.shape[-2]
    k, ks, v, vs = pages.reshape(-1, H, D["rec"]).split([D["codes"], D["scales"]] * 2, dim=-1)
    N = k.shape[0]
    k = k.reshape(N, H, P // 16, D["NI"], 4, 16, D["W"]).permute(0, 2, 5, 1, 4, 3, 6).reshape(N, P, H, 4, D["LB"])
    v = v.reshape(N, H, P // 4, D["NI"], 16, D["W"]).transpose(3, 4).reshape(N, H, P // 4, 16, D["LB"] // 4, 4)
    v = v.permute(0, 2, 5, 1, 3, 4).reshape(N, P, H, 16, D["LB"] // 4)
    full = lambda s: s.contiguous().view(torch.bfloat16).view(N, H, P // 4, -1, 4).permute(0, 2, 4, 1, 3).reshape(  # noqa: E731
        N, P, H, -1).float()
    spread = lambda f, s: (_valued(f, kind).unflatten(-1, (-1, g)) * full(s).unsqueeze(-1)).flatten(-2)  # noqa: E731
    return (spread(_key_fields(k, kind), ks).view(*lead, P, H, -1),
            spread(_value_fields(v, kind), vs).view(*lead, P, H, -1))


def _logical(case, seed, length):
    """What the sequences hold: codes and scales of keys and values for `length` tokens of each."""
    gen = _gen(seed)
    shape = (case["B"], length, case["H"], case["d"])
    k = _quantise(_vectors(gen, shape, case["io"], True), case["kind"], case["group"])
    return k, _quantise(_vectors(gen, shape, case["io"], False), case["kind"], case["group"])


def _cache(case, seed, lens, MP):
    """A pool of recycled pages (old bytes in them) with `lens[b]` tokens of each sequence written."""
    gen, (P, H, B) = _gen(seed + 7919), (case["page"], case["H"], case["B"])
    rec, N = _dims(case)["rec"], B * MP + 3
    table = torch.randperm(N, generator=gen, device="cuda")[: B * MP].to(torch.int32).view(B, MP)
    pool = torch.randint(-2 ** 62, 2 ** 62, (N * H * rec // 8,), generator=gen, device="cuda", dtype=torch.int64)
    pool = pool.view(torch.uint8).view(N, H, rec)
    L = -(-max(lens) // P) * P
    if L:
        (kc, ks), (vc, vs) = _logical(case, seed, L)
        live = torch.arange(L, device="cuda") < torch.tensor(lens, device="cuda").view(B, 1)
        most = 16 if case["kind"] == "int4" else 256

        def codes(x, b):                                 # old bytes stay where the last page ends
            junk = torch.randint(0, most, x[b].shape, generator=gen, device="cuda", dtype=torch.uint8)
            return torch.where(live[b].view(L, 1, 1), _stored(x[b], case["kind"]), junk).view(L // P, P, H, -1)

        def scales(x, b):
            junk = torch.randint(-32768, 32768, x[b].shape, generator=gen, device="cuda", dtype=torch.int16)
            x = torch.where(live[b].view(L, 1, 1), x[b].to(torch.bfloat16).view(torch.int16), junk)
            return x.view(torch.bfloat16).view(L // P, P, H, -1)

        for b in range(B):                               # sequence by sequence, for memory's sake
            pages = _pack(case, codes(kc, b), scales(ks, b), codes(vc, b), scales(vs, b))
            n = -(-lens[b] // P)
            pool[table[b, :n].long()] = pages[:n]
    return pool.view(-1), table


# ------------------------------------------------------------------------------- prepare

def _freqs(rd, scaling, far):
    """Frequencies (radians a position) in 64 bits and the factor on the rotated values."""
    i = torch.arange(0, rd, 2, dtype=torch.float64)
    base, factor, original = 1.0e6, 8.0, max(64, far // 8)
    if scaling == "ntk":
        return (base * factor ** (rd / max(1, rd - 2))) ** (-i / rd), 1.0
    f = base ** (-i / rd)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "blend":
        turns = lambda n: rd * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(turns(32.0))), min(rd - 1, math.ceil(turns(1.0)))
        ramp = ((torch.arange(rd // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotary_inputs(case, seed):
    gen, n, d = _gen(seed), case["tokens"], case["d"]
    q = torch.randn((n, case["Hq"], d), generator=gen, device="cuda").to(IO[case["io"]])
    k = torch.randn((n, case["Hk"], d), generator=gen, device="cuda").to(IO[case["io"]])
    pos = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
    return q, k, pos


def prepare(case, seed):
    s = dict(case)
    io = IO[case["io"]]
    if case["op"] == "rotary":
        s["q"], s["k"], s["pos"] = _rotary_inputs(case, seed)
        f, s["magnitude"] = _freqs(case["rd"], case["scaling"], case["far"])
        s["freqs"] = f.cuda()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["kept"] = {}
        return s
    plan, B, T, P = _plan(case), case["B"], case["T"], case["page"]
    if case["op"] == "attend":
        lens = [c + n for c, n in zip(plan["ctx"], plan["drafts"])]
        MP = -(-(case["ctx"] + T) // P)
        s["cache"], s["table"] = _cache(case, seed, lens, MP)
        s["q"] = torch.randn((B, T, case["Hq"], case["d"]), generator=_gen(seed + 1), device="cuda").to(io)
        s["ctx_lens"] = torch.tensor(plan["ctx"], dtype=torch.int32, device="cuda")
        s["mask"] = s["bits"] = s["drafts"] = None
        if plan["parents"] is not None:
            m = _tree_mask(plan["parents"])
            s["mask"] = m.cuda()
            w = torch.zeros((B, T, -(-T // 32) * 32), dtype=torch.int64)
            w[..., :T] = m
            w = (w.view(B, T, -1, 32) << torch.arange(32)).sum(-1)
            s["bits"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).cuda()
            s["drafts"] = torch.tensor(plan["drafts"], dtype=torch.int32, device="cuda")
        s["o"] = torch.empty((B, T, case["Hq"], case["d"]), dtype=io, device="cuda")
        s["lse"] = torch.empty((B, T, case["Hq"]), dtype=torch.float32, device="cuda")
        s["longest"] = case["ctx"] + T
        s["kept"] = {}
        return s
    start = torch.tensor(plan["start"], dtype=torch.int32).view(B, 1)
    pos = start + torch.arange(T, dtype=torch.int32)
    if case["skip"]:
        pos = torch.where(torch.tensor(plan["drop"]), torch.full_like(pos, -1), pos)
    s["pos"] = pos.cuda()
    MP = -(-(case["start"] + T) // P)
    s["cache"], s["table"] = _cache(case, seed, [0 if case["op"] == "store" else T] * B, MP)
    if case["op"] == "store":
        s["k"], s["v"] = _store_inputs(case, seed)
    s["k_out"] = torch.empty((B, T, case["H"], case["d"]), dtype=io, device="cuda")
    s["v_out"] = torch.empty_like(s["k_out"])
    s["kept"] = {}
    return s


def _store_inputs(case, seed):
    gen, shape = _gen(seed), (case["B"], case["T"], case["H"], case["d"])
    return _vectors(gen, shape, case["io"], True), _vectors(gen, shape, case["io"], False)


# ----------------------------------------------------------------------------- plain forms

def _plain_rotary(s):
    rd, half = s["rd"], s["rd"] // 2
    a = s["pos"].double().unsqueeze(-1) * s["freqs"]
    c, n = (a.cos() * s["magnitude"]).float().unsqueeze(1), (a.sin() * s["magnitude"]).float().unsqueeze(1)
    n = -n if s["inverse"] else n

    def turn(x):
        y, rest = x[..., :rd].float(), x[..., rd:]
        u, w = (y[..., 0::2], y[..., 1::2]) if s["interleaved"] else (y[..., :half], y[..., half:])
        u, w = u * c - w * n, u * n + w * c
        y = torch.stack([u, w], dim=-1).flatten(-2) if s["interleaved"] else torch.cat([u, w], dim=-1)
        return torch.cat([y.to(x.dtype), rest], dim=-1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _places(s):
    """Page and place in the page of every position (0 where it is skipped), and which are not."""
    live = s["pos"] >= 0
    at = s["pos"].clamp(min=0).long()
    page = torch.gather(s["table"].long(), 1, at // s["page"])
    return page, at % s["page"], live


def _plain_write(s):
    D, kind, H = _dims(s), s["kind"], s["H"]
    page, r, live = _places(s)
    page, r = page[live], r[live]
    pool = s["cache"].view(-1, H, D["rec"])
    dev = pool.device
    head = torch.arange(H, device=dev)
    (kc, ks), (vc, vs) = (_quantise(s[n][live], kind, s["group"]) for n in ("k", "v"))
    x = torch.arange(D["LB"], device=dev)
    lane = torch.arange(4, device=dev).view(4, 1)
    r_ = r.view(-1, 1, 1)
    at = (r_ // 16) * (64 * D["LB"]) + (x // D["W"]) * (64 * D["W"]) + (16 * lane + r_ % 16) * D["W"] + x % D["W"]
    page_, head_ = page.view(-1, 1, 1, 1), head.view(1, -1, 1, 1)
    pool[page_, head_, at.unsqueeze(1)] = _key_bytes(_stored(kc, kind), kind)
    x = 4 * torch.arange(D["LB"] // 4, device=dev) + r_ % 4
    lane = torch.arange(16, device=dev).view(16, 1)
    at = (r_ // 4) * (16 * D["LB"]) + (x // D["W"]) * (16 * D["W"]) + lane * D["W"] + x % D["W"]
    pool[page_, head_, at.unsqueeze(1) + D["codes"] + D["scales"]] = _value_bytes(_stored(vc, kind), kind)
    ng = s["d"] // s["group"]
    at = 2 * ((r_ // 4 * ng + torch.arange(ng, device=dev).view(-1, 1)) * 4 + r_ % 4) + torch.arange(2, device=dev)
    for shift, v in ((D["codes"], ks), (2 * D["codes"] + D["scales"], vs)):
        pool[page_, head_, at.unsqueeze(1) + shift] = v.to(torch.bfloat16).unsqueeze(-1).view(torch.uint8)


def _plain_read(s):
    page, r, live = _places(s)
    pages = s["cache"].view(-1, s["H"], _dims(s)["rec"])[s["table"].long()]
    at = s["pos"].clamp(min=0).long()
    out = {}
    for name, x in zip(("k", "v"), _unpack(s, pages)):
        x = torch.gather(x.flatten(1, 2), 1, at.view(*at.shape, 1, 1).expand(*at.shape, s["H"], s["d"]))
        out[name] = torch.where(live.view(*at.shape, 1, 1), x, torch.zeros_like(x)).to(IO[s["io"]])
    return out


def _plain_attend(s):
    B, T, H, d = s["B"], s["T"], s["H"], s["d"]
    pages = s["cache"].view(-1, H, _dims(s)["rec"])[s["table"].long()]
    k, v = (x.flatten(1, 2) for x in _unpack(s, pages))                      # [B, L, H, d]
    at = torch.arange(k.shape[1], device=k.device)
    ctx = s["ctx_lens"].view(B, 1, 1)
    j, i = at - ctx, torch.arange(T, device=k.device).view(1, T, 1)           # [B, 1, L], [1, T, 1]
    if s["mask"] is None:
        seen = j <= i
    else:
        drafts = s["drafts"].view(B, 1, 1)
        near = torch.gather(s["mask"], 2, j.clamp(0, T - 1).expand(B, T, at.numel()))
        seen = (i < drafts) & ((j < 0) | (near & (j >= 0) & (j < drafts)))
    held = seen.any(1).view(B, -1, 1, 1)
    k, v = (torch.where(held, x, torch.zeros_like(x)).permute(0, 2, 1, 3) for x in (k, v))  # [B, H, L, d]
    q = s["q"].float().view(B, T, H, -1, d).permute(0, 2, 1, 3, 4).flatten(2, 3)            # [B, H, T G, d]
    z = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(d)
    seen = seen.expand(B, T, at.numel()).repeat_interleave(q.shape[2] // T, dim=1).unsqueeze(1)
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (z - top).exp()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.contiguous()) / torch.where(total > 0, total, torch.ones_like(total))
    back = lambda x: x.view(B, H, T, -1, x.shape[-1]).permute(0, 2, 1, 3, 4).flatten(2, 3)  # noqa: E731
    return {"o": back(o).to(IO[s["io"]]), "lse": back(total.log() + top).squeeze(-1)}


# ------------------------------------------------------------------------------------- run

def _kept(s):
    """The layer's configuration and scratch, made once, as a serving program keeps them."""
    import bit_recurrent_state_amd as pace
    if not s["kept"]:
        bf16 = s["io"] == "bf16"
        if s["op"] == "rotary":
            s["kept"]["cfg"] = pace.RotaryConfig(Hq=s["Hq"], Hk=s["Hk"], d=s["d"], rd=s["rd"],
                                                 interleaved=s["interleaved"], bf16_io=bf16)
        else:
            cfg = pace.CacheConfig(B=s["B"], Hq=s.get("Hq", s["H"]), Hkv=s["H"], d=s["d"], kind=s["kind"],
                                   group=s["group"], page=s["page"], max_pages=s["table"].shape[1],
                                   num_pages=s["cache"].numel() // (s["H"] * _dims(s)["rec"]), bf16_io=bf16)
            s["kept"]["cfg"] = cfg
            n = pace.cache_attention_workspace_bytes(cfg, s["T"], s["longest"]) if s["op"] == "attend" else 0
            s["kept"]["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    return pace, s["kept"]["cfg"]


def run(state):
    s = state
    if not own:
        if s["op"] == "rotary":
            return _plain_rotary(s)
        if s["op"] == "attend":
            return _plain_attend(s)
        if s["op"] == "store":
            _plain_write(s)
        return _plain_read(s)
    pace, cfg = _kept(s)
    if s["op"] == "rotary":
        pace.rotary(cfg, s["pos"], s["freqs"], s["q"], s["k"], s["q_out"], s["k_out"],
                    magnitude=s["magnitude"], inverse=s["inverse"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "attend":
        pace.cache_attention(cfg, s["cache"], s["table"], s["q"], s["ctx_lens"], s["o"], lse=s["lse"],
                             tree=s["bits"], draft_lens=s["drafts"], max_len=s["longest"],
                             workspace=s["kept"]["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "store":
        pace.cache_write(cfg, s["cache"], s["table"], s["pos"], s["k"], s["v"])
    pace.cache_read(cfg, s["cache"], s["table"], s["pos"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


# ------------------------------------------------------------------------ work and 64 bits

def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "rotary":
        values = case["tokens"] * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": 2 * e * values + 4 * case["tokens"] + 4 * case["rd"],
                "flops": 3 * case["tokens"] * (case["Hq"] + case["Hk"]) * case["rd"]}
    plan = _plan(case)
    token = 2 * case["H"] * (case["d"] * BITS[case["kind"]] // 8 + 2 * (case["d"] // case["group"]))
    if case["op"] != "attend":
        live = sum(not x for row in plan["drop"] for x in row)
        wide, n = 2 * case["H"] * case["d"] * e, case["B"] * case["T"]
        moved = live * (wide + token) if case["op"] == "store" else 0
        return {"bytes": moved + live * token + n * wide + 4 * n, "flops": 4 * live * case["H"] * case["d"]}
    T, rows = case["T"], case["Hq"] // case["H"]
    held = sum(plan["ctx"]) + sum(plan["drafts"])
    if plan["parents"] is None:
        seen = sum(T * c + T * (T + 1) // 2 for c in plan["ctx"])
    else:
        m = _tree_mask(plan["parents"])
        seen = sum(n * c + int(m[b, :n, :n].sum()) for b, (c, n) in enumerate(zip(plan["ctx"], plan["drafts"])))
    outer = case["B"] * T * case["Hq"] * (2 * case["d"] * e + 4)
    return {"bytes": held * token + outer + 4 * case["B"], "flops": 4 * case["d"] * seen * rows * case["H"]}


def _meant(x, kind, group):
    """What a cache of this kind holds of vectors x [..., d]: from the definition, in 64 bits."""
    f = x.double().reshape(*x.shape[:-1], -1, group)
    f = torch.nan_to_num(f, nan=0.0, posinf=2.0 ** 127, neginf=-2.0 ** 127).clamp(-2.0 ** 127, 2.0 ** 127)
    top = f.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / torch.full_like(top, LEVELS[kind]))
    s = torch.ldexp(torch.ceil(m * 256.0) / 256.0, e)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    y = torch.where(s > 0, f / s, torch.zeros_like(f))
    y = torch.where(s > 0, y, torch.zeros_like(y)).clamp(-LEVELS[kind], LEVELS[kind])
    if kind == "fp8":                                    # 3 bits after the leading one, down to 2^-9
        step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 4).clamp(min=-9))
        y = torch.round(y / step) * step
    else:
        y = torch.round(y)
    return (y * s).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "rotary":
        q, k, pos = _rotary_inputs(case, seed)
        f, magnitude = _freqs(case["rd"], case["scaling"], case["far"])
        angle = pos.double()[:, None] * f.cuda()[None, :] * (-1.0 if case["inverse"] else 1.0)
        spin = torch.polar(torch.full_like(angle, magnitude), angle)[:, None, :]
        out = {}
        for name, x in (("q", q), ("k", k)):
            y = x.double()
            part = y[..., : case["rd"]]
            pairs = part.reshape(*part.shape[:-1], -1, 2) if case["interleaved"] else \
                part.reshape(*part.shape[:-1], 2, -1).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * spin)
            z = z.reshape(part.shape) if case["interleaved"] else z.transpose(-1, -2).reshape(part.shape)
            out[name] = torch.cat([z, y[..., case["rd"]:]], dim=-1)
        return out
    plan, B, T = _plan(case), case["B"], case["T"]
    if case["op"] == "attend":
        P, lens = case["page"], [c + n for c, n in zip(plan["ctx"], plan["drafts"])]
        L = -(-max(lens) // P) * P if max(lens) else 0
        (kc, ks), (vc, vs) = _logical(case, seed, L)
        q = torch.randn((B, T, case["Hq"], case["d"]), generator=_gen(seed + 1), device="cuda").to(IO[case["io"]])
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
        wide = lambda c, s: c.double() * s.double().repeat_interleave(case["group"], dim=-1)  # noqa: E731
        per = case["Hq"] // case["H"]
        tree = _tree_mask(plan["parents"]).cuda() if plan["parents"] is not None else \
            torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(B, T, T)
        for b in range(B):
            c, n = plan["ctx"][b], plan["drafts"][b]
            if not n:
                continue
            seen = torch.cat([torch.ones((n, c), dtype=torch.bool, device="cuda"), tree[b, :n, :n]], dim=1)
            for h in range(case["H"]):
                k, v = (wide(x[b, : c + n, h], y[b, : c + n, h]) for x, y in ((kc, ks), (vc, vs)))
                z = q[b, :n, h * per: (h + 1) * per].double() @ k.t() * case["d"] ** -0.5     # [n, per, c + n]
                z = z.masked_fill(~seen[:, None, :], -math.inf)
                lse[b, :n, h * per: (h + 1) * per] = torch.logsumexp(z, -1)
                o[b, :n, h * per: (h + 1) * per] = torch.softmax(z, -1) @ v
        return {"o": o, "lse": lse}
    if case["op"] == "store":
        k, v = (_meant(x, case["kind"], case["group"]) for x in _store_inputs(case, seed))
    else:
        P = case["page"]
        gen, shape = _gen(seed), (B, -(-T // P) * P, case["H"], case["d"])
        k, v = (_meant(_vectors(gen, shape, case["io"], o)[:, :T], case["kind"], case["group"]) for o in (True, False))
    live = ~torch.tensor(plan["drop"], device="cuda")[:, :, None, None]
    return {"k": torch.where(live, k, torch.zeros_like(k)), "v": torch.where(live, v, torch.zeros_like(v))}
