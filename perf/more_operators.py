"""Measured cases of the operators that serve drafted tokens through a hybrid stack: the gated-delta
layers' outputs for a tree of drafts, the verification of drafts against the target's
probabilities, the accepted path's way into the decode buffers, and cached entries moved to other places.

`listed()` gives the cases, `draw(rng)` more of the same ranges, `prepare(case, seed)` what a
serving program has in hand, `run(state)` one pass: in plain torch operations, or through the
library where `own` is true.  `work(case)` is what a pass cannot do without and `exact(case, seed)`
the result in 64 bits.

Packed state: records of (sequence, value head), [codes | bf16 scales | zero points], parts padded
to 16 bytes and records to 256.  A value column's codes lie in units of 8 keys; key 32 m + 8 a + e is
in unit a (d / 32) + m; 4 bits: byte w of a unit holds e = w (low) and e = 4 + w (high).
Decode buffer: regions count | key codes | key scales | values | value scales | a | beta, padded to 256 bytes.
Cache: see `_token_bytes`.
"""
import json
import math
import random

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # One sequence, a chain of five drafts through one layer: the smallest call, latency counts.
        {"name": "step-one", "op": "step", "B": 1, "T": 5, "Hv": 32, "Hk": 16, "d": 128, "state": "sym", "group": 64,
         "buf": "int8", "dP": 8, "tree": False, "ragged": False, "io": "bf16"},
        # The serving batch of the benchmark, chains of up to eight drafts.
        {"name": "step-batch", "op": "step", "B": 64, "T": 8, "Hv": 32, "Hk": 16, "d": 128, "state": "sym",
         "group": 64, "buf": "int8", "dP": 8, "tree": False, "ragged": True, "io": "bf16"},
        # Trees of up to 25 drafts, asymmetric state with a quarter of the heads in 8 bits, mixed buffer.
        {"name": "step-tree", "op": "step", "B": 16, "T": 25, "Hv": 32, "Hk": 16, "d": 128, "state": "asym",
         "group": 32, "buf": "mixed", "dP": 8, "tree": True, "ragged": True, "io": "bf16"},
        # The small fp32 configuration, an odd tree, a longer period.
        {"name": "step-f32", "op": "step", "B": 3, "T": 13, "Hv": 4, "Hk": 4, "d": 64, "state": "sym", "group": 32,
         "buf": "int8", "dP": 16, "tree": True, "ragged": False, "io": "f32"},
        # One sequence's chain against sampled drafts, a small vocabulary.
        {"name": "verify-one", "op": "verify", "B": 1, "T": 5, "V": 32768, "pad": 0, "sampled": True, "tree": False,
         "ragged": False, "probs": "f32"},
        # The serving batch, chains of sampled drafts, a large vocabulary.
        {"name": "verify-batch", "op": "verify", "B": 64, "T": 8, "V": 131072, "pad": 0, "sampled": True,
         "tree": False, "ragged": True, "probs": "f32"},
        # Trees of the draft's likeliest tokens, an odd vocabulary, probabilities in bf16.
        {"name": "verify-tree", "op": "verify", "B": 16, "T": 25, "V": 100003, "pad": 0, "sampled": False,
         "tree": True, "ragged": True, "probs": "bf16"},
        # The accepted tokens of the serving batch into one layer's buffers.
        {"name": "commit-batch", "op": "commit", "B": 64, "T": 8, "Hv": 32, "Hk": 16, "d": 128, "state": "sym",
         "group": 64, "buf": "int8", "dP": 8, "tree": False, "io": "bf16"},
        # The accepted paths of trees, mixed buffer, fp32 inputs.
        {"name": "commit-tree", "op": "commit", "B": 5, "T": 25, "Hv": 8, "Hk": 4, "d": 128, "state": "asym",
         "group": 32, "buf": "mixed", "dP": 16, "tree": True, "io": "f32"},
        # The accepted paths' keys and values to their places behind the contexts of one layer.
        {"name": "move-path", "op": "move", "B": 64, "T": 25, "H": 8, "d": 128, "kind": "int8", "group": 64, "page": 64,
         "far": 1000, "how": "path"},
        # Half of four long contexts kept, moved together in place.
        {"name": "move-kept", "op": "move", "B": 4, "T": 16384, "H": 8, "d": 128, "kind": "int8", "group": 64,
         "page": 64, "far": 0, "how": "keep"},
        # A prompt of odd length copied into the pages of eight forks, 4-bit cache with short groups.
        {"name": "move-fork", "op": "move", "B": 8, "T": 4093, "H": 8, "d": 128, "kind": "int4", "group": 32,
         "page": 64, "far": 0, "how": "fork"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "step", "step", "verify", "verify", "commit", "move", "move"])
    if op in ("step", "commit"):
        d = rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        state = rng.choice(["sym", "asym", "bf16"])
        c = {"op": op, "Hv": Hk * rng.choice([1, 2] if Hk > 4 else [1, 2, 3, 4]), "Hk": Hk, "d": d, "state": state,
             "group": 32 if state == "asym" and d == 64 else rng.choice([32, 64]),
             "buf": "int8" if state == "bf16" else rng.choice(["int8", "mixed"]), "dP": rng.choice([4, 8, 8, 16, 32]),
             "tree": rng.random() < 0.5, "io": rng.choice(["bf16", "bf16", "f32"])}
        while True:
            c["B"], c["T"] = _log(rng, 1, 64), _log(rng, 1, 48)
            if c["B"] * c["T"] * c["Hv"] * d * (2 if c["io"] == "f32" else 1) <= 64 * 8 * 32 * 128:
                break
        return dict(c, ragged=rng.random() < 0.5) if op == "step" else c
    if op == "verify":
        while True:
            B, T, V = _log(rng, 1, 64), _log(rng, 1, 32), _log(rng, 300, 131072)
            if B * T * V <= 64 * 8 * 131072:
                break
        return {"op": op, "B": B, "T": T, "V": V, "pad": rng.choice([0, 0, 8, 61]), "sampled": rng.random() < 0.6,
                "tree": rng.random() < 0.5, "ragged": rng.random() < 0.5, "probs": rng.choice(["f32", "f32", "bf16"])}
    how = rng.choice(["path", "keep", "fork"])
    d, kind = rng.choice([64, 128, 128, 256]), rng.choice(["int8", "int4", "fp8"])
    c = {"op": op, "H": rng.choice([1, 2, 4, 8]), "d": d, "kind": kind,
         "group": rng.choice([g for g in (32, 64, 128) if g <= d]), "page": rng.choice([16, 32, 64, 128]),
         "far": _log(rng, 1, 2000) if how == "path" else 0, "how": how}
    while True:
        c["B"], c["T"] = _log(rng, 1, 64), _log(rng, 1, 48 if how == "path" else 16384)
        if c["B"] * (c["T"] + c["far"]) * c["H"] * d <= 4 * 16384 * 8 * 128 // (2 if kind != "int4" else 1):
            return c


def _parents(r, B, T, tree):
    """Every node but the first hangs on one of the few before it, in a tree; on the last one, in a chain."""
    return [[-1] + [r.randrange(max(0, i - 6), i) if tree else i - 1 for i in range(1, T)] for _ in range(B)]


def _some_path(r, parents, most):
    """The nodes of one path from the root, `most` at most (none where that is 0)."""
    path = [0] if most else []
    for i in range(1, len(parents)):
        if path and len(path) < most and parents[i] == path[-1] and r.random() < 0.8:
            path.append(i)
    return path


def _plan(case):
    """A case's lengths, trees and paths (host values that work() needs too): by the case alone."""
    r = random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))
    B, T, op = case["B"], case["T"], case["op"]
    if op == "step":
        return {"parents": _parents(r, B, T, case["tree"]), "count": [r.randrange(case["dP"]) for _ in range(B)],
                "drafts": [r.randrange((T + 1) // 2, T + 1) if case["ragged"] else T for _ in range(B)]}
    if op == "verify":
        return {"parents": _parents(r, B, T, case["tree"]),
                "drafts": [r.randrange((T + 1) // 2, T + 1) if case["ragged"] else T for _ in range(B)]}
    if op == "commit":
        # What a step accepts stays within the period here.  A path that ends it is rounded by the layer's existing flush, and
        # which way a code next to a tie goes is then no value that two computations share.
        count = [r.randrange(case["dP"] // 2) for _ in range(B)]
        paths = [_some_path(r, p, case["dP"] - 1 - n) for p, n in zip(_parents(r, B, T, case["tree"]), count)]
        return {"count": count, "nodes": paths, "most": min(T, case["dP"] - 1)}
    start = [r.randrange(case["far"] // 2, case["far"] + 1) for _ in range(B)]
    if case["how"] == "path":
        nodes = [_some_path(r, p, T) for p in _parents(r, B, T, True)]
    elif case["how"] == "keep":
        nodes = [sorted(r.sample(range(T), max(1, T // 2 - r.randrange(1 + T // 8)))) for _ in range(B)]
    else:
        nodes = [list(range(T)) for _ in range(B)]
    return {"start": start, "nodes": nodes}


def _rows(lists, T, fill=-1):
    return torch.tensor([x + [fill] * (T - len(x)) for x in lists], dtype=torch.int32).view(len(lists), T)


def _seen(parents):
    """[B][T][T] truth values: node j is node i or one of its ancestors."""
    B, T = len(parents), len(parents[0])
    m = torch.zeros((B, T, T), dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            if parents[b][i] >= 0:
                m[b, i] = m[b, parents[b][i]]
            m[b, i, i] = True
    return m


def _bits(m):
    """Truth values [B][T][T] as int32 words [B][T][ceil(T / 32)]."""
    B, T = m.shape[:2]
    w = torch.zeros((B, T, -(-T // 32) * 32), dtype=torch.int64)
    w[..., :T] = m
    w = (w.view(B, T, -1, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


# ------------------------------------------------------- the gated-delta layer's bytes

def _up(n, a):
    return -(-n // a) * a


def _wide(case, h):
    """Whether head h keeps 8 bits: a quarter of the heads of an asymmetric state."""
    return case["state"] == "asym" and h % 4 == 1


def _record(case, h):
    """(bits, byte offsets of scales and zero points, size) of a head's record."""
    d = case["d"]
    if case["state"] == "bf16":
        return 16, 0, 0, 2 * d * d
    b, n = 8 if _wide(case, h) else 4, d * (d // case["group"])
    scales = _up(d * d * b // 8, 16)
    zeros = scales + _up(2 * n, 16)
    return b, scales, zeros, _up(zeros + (_up(n * b // 8, 16) if case["state"] == "asym" else 0), 256)


def _regions(case):
    """Name, type and shape of the decode buffer's regions."""
    B, Hv, Hk, dP, d = (case[k] for k in ("B", "Hv", "Hk", "dP", "d"))
    if case["buf"] == "int8":
        keys, values = ("kc", torch.int8, (B, Hk, dP, d)), [("v", torch.int8, (B, Hv, dP, d)), ("vs", torch.float32, (B, Hv, dP))]
    else:
        keys, values = ("kc", torch.uint8, (B, Hk, dP, d // 2)), [("v", torch.bfloat16, (B, Hv, dP, d))]
    return [("count", torch.int32, (B, Hv)), keys, ("ks", torch.float32, (B, Hk, dP)), *values,
            ("a", torch.float32, (B, Hv, dP)), ("beta", torch.float32, (B, Hv, dP))]


def _views(case, buffer):
    """The decode buffer's regions as tensors over its bytes."""
    at, out = 0, {}
    for name, dtype, shape in _regions(case):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        out[name] = buffer[at: at + n].view(dtype).view(shape)
        at += _up(n, 256)
    return out


def _buffer_bytes(case):
    return sum(_up(math.prod(shape) * torch.empty((), dtype=t).element_size(), 256) for _, t, shape in _regions(case))


def _buffered(x, levels):
    """(codes as fp32 whole numbers, scale) of vectors [..., d]: one symmetric scale each."""
    x = x.float()
    s = x.abs().amax(-1) / torch.full((), levels, device=x.device)    # a tensor: a number's reciprocal would be multiplied by
    c = (x / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)).round().clamp(-levels, levels)
    return c, s


def _nibbles(c):
    """4-bit codes [..., d] as bytes: unit of 8, byte w holds e = w and e = 4 + w, plus 8."""
    u = (c + 8).to(torch.uint8).unflatten(-1, (-1, 2, 4))
    return (u[..., 0, :] | (u[..., 1, :] << 4)).flatten(-2)


def _of_nibbles(y):
    y = y.unflatten(-1, (-1, 4))
    return torch.stack([y & 15, y >> 4], dim=-2).flatten(-3).float() - 8.0


def _slots(case, k, v):
    """What the buffer holds of keys [..., Hk, d] and values [..., Hv, d]."""
    kc, ks = _buffered(k, 127.0 if case["buf"] == "int8" else 7.0)
    if case["buf"] == "int8":
        vc, vs = _buffered(v, 127.0)
        return {"kc": kc.to(torch.int8), "ks": ks, "v": vc.to(torch.int8), "vs": vs}
    return {"kc": _nibbles(kc), "ks": ks, "v": v.to(torch.bfloat16)}


def _meant(case, w):
    """Keys and values that buffered slots stand for, fp32."""
    kc = w["kc"].float() if case["buf"] == "int8" else _of_nibbles(w["kc"])
    v = w["v"].float()
    return kc * w["ks"].unsqueeze(-1), v * w["vs"].unsqueeze(-1) if case["buf"] == "int8" else v


def _units(c):
    """Fields [..., d] of a column in the order of its units [..., d / 8, 8]."""
    return c.unflatten(-1, (-1, 4, 8)).transpose(-3, -2).flatten(-3, -2)


def _unpack_state(case, state):
    """The dequantised state, fp32 [B, Hv, value column, key]."""
    B, Hv, d = case["B"], case["Hv"], case["d"]
    raw = state.view(B, -1)
    if case["state"] == "bf16":
        return raw.view(torch.bfloat16).view(B, Hv, d, d).float()
    out, at, ng = torch.empty((B, Hv, d, d), device=state.device), 0, d // case["group"]
    groups = {}
    for h in range(Hv):
        groups.setdefault(_record(case, h), []).append((h, at))
        at += _record(case, h)[3]
    for (b, scales, zeros, size), heads in groups.items():
        at = torch.tensor([o for _, o in heads]).view(-1, 1) + torch.arange(size)
        rec = raw[:, at.to(raw.device)]                                           # [B, heads, size]
        y = rec[..., : d * d * b // 8].unflatten(-1, (d, 4, d // 32, b))
        if b == 4:
            y = torch.stack([y & 15, y >> 4], dim=-2).flatten(-2)
        y = y.transpose(-3, -2).flatten(-3).float()                               # [B, heads, column, key]
        s = rec[..., scales: scales + 2 * d * ng].contiguous().view(torch.bfloat16).float().unflatten(-1, (d, ng))
        z = torch.full_like(s, 1 << (b - 1))
        if case["state"] == "asym":
            z = rec[..., zeros: zeros + d * ng * b // 8]
            z = (torch.stack([z & 15, z >> 4], dim=-1).flatten(-2) if b == 4 else z).float().unflatten(-1, (d, ng))
        full = ((y.unflatten(-1, (ng, -1)) - z.unsqueeze(-1)) * s.unsqueeze(-1)).flatten(-2)
        out[:, torch.tensor([h for h, _ in heads], device=out.device)] = full
    return out


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _layer_inputs(case, seed):
    """A layer's state and buffer in mid-service and the drafts' q, k, v and gates."""
    gen, plan = _gen(seed), _plan(case)
    B, Hv, Hk, d, T, dP = (case[k] for k in ("B", "Hv", "Hk", "d", "T", "dP"))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    s = {}
    parts = []
    for h in range(Hv):
        b, scales, zeros, size = _record(case, h)
        if b == 16:
            parts.append((0.1 * normal(B, d, d)).to(torch.bfloat16).view(B, -1).view(torch.uint8))
            continue
        rec, ng, top = torch.zeros((B, size), dtype=torch.uint8, device="cuda"), d // case["group"], (1 << b) - 1
        mid = (top / 2 + top / 10 * normal(B, d, ng)).round().clamp(0, top) if case["state"] == "asym" else \
            torch.full((B, d, ng), (top + 1) / 2, device="cuda")
        c = (mid.unsqueeze(-1) + top / 5 * normal(B, d, ng, case["group"])).round()
        c = c.clamp(0 if case["state"] == "asym" else 1, top).to(torch.uint8).flatten(-2)
        c = _units(c)
        if b == 4:
            c = c.unflatten(-1, (2, 4))
            c = c[..., 0, :] | (c[..., 1, :] << 4)
        rec[:, : d * d * b // 8] = c.reshape(B, -1)
        sc = (0.32 / top * (0.5 * normal(B, d * ng)).exp()).to(torch.bfloat16)
        rec[:, scales: scales + 2 * d * ng] = sc.view(torch.uint8)
        if case["state"] == "asym":
            z = mid.to(torch.uint8).flatten(1)
            z = z[:, 0::2] | (z[:, 1::2] << 4) if b == 4 else z
            rec[:, zeros: zeros + z.shape[1]] = z
        parts.append(rec)
    s["packed"] = torch.cat(parts, dim=1).reshape(-1)

    def tokens(n):
        k, q = (torch.nn.functional.normalize(normal(B, n, Hk, d), dim=-1).to(IO[case["io"]]) for _ in range(2))
        a = torch.exp(-torch.nn.functional.softplus(normal(B, n, Hv) - 4.0))
        return q, k, normal(B, n, Hv, d).to(IO[case["io"]]), a, torch.sigmoid(normal(B, n, Hv))

    s["buffer"] = torch.zeros(_buffer_bytes(case), dtype=torch.uint8, device="cuda")
    held = _views(case, s["buffer"])
    _, k, v, a, beta = tokens(dP)
    for name, x in dict(_slots(case, k, v), a=a, beta=beta).items():
        held[name].copy_(x.transpose(1, 2))
    held["count"].copy_(torch.tensor(plan["count"], dtype=torch.int32).view(B, 1).expand(B, Hv))
    s["q"], s["k"], s["v"], s["a"], s["beta"] = tokens(T)
    return s


# ---------------------------------------------------------------------- verification's inputs

def _verify_inputs(case, seed):
    """The target's probabilities, the draft's (None where its likeliest tokens were taken), tokens and uniforms."""
    gen, plan = _gen(seed), _plan(case)
    B, T, V, pad = (case[k] for k in ("B", "T", "V", "pad"))
    dtype = IO[case["probs"]]
    z = 3.0 * torch.randn((B, T, V), generator=gen, device="cuda")
    y = z + torch.randn((B, T, V), generator=gen, device="cuda")

    def probabilities(x):
        p = torch.full((B, T, V + pad), 1.0, dtype=dtype, device="cuda")      # what lies between rows is nobody's
        p[..., :V] = torch.softmax(x, dim=-1).to(dtype)
        return p[..., :V]

    target = probabilities(z)
    del z
    parents = torch.tensor(plan["parents"], device="cuda")
    tokens = torch.randint(0, V, (B, T), generator=gen, device="cuda")
    each = torch.arange(B, device="cuda")
    older = torch.zeros((B,), dtype=torch.long, device="cuda")
    for c in range(1, T):
        row = y[each, parents[:, c]]
        if case["sampled"]:
            noise = -torch.log(-torch.log(torch.rand((B, V), generator=gen, device="cuda").clamp(1e-30, 1 - 1e-7)))
            tokens[:, c] = (row + noise).argmax(-1)
        else:
            older = (parents[:, 1:c] == parents[:, c: c + 1]).sum(-1)
            tokens[:, c] = row.topk(min(V, 8), dim=-1).indices.gather(1, older.clamp(max=min(V, 8) - 1).view(B, 1)).view(B)
    return {"target": target, "draft": probabilities(y) if case["sampled"] else None, "tokens": tokens.to(torch.int32),
            "uniforms": torch.rand((B, T), generator=gen, device="cuda"),
            "parents": parents.to(torch.int32), "drafts": torch.tensor(plan["drafts"], dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------------------------- prepare

def _cache_sizes(case):
    b = 4 if case["kind"] == "int4" else 8
    LB = case["d"] * b // 32
    codes, scales = case["page"] * case["d"] * b // 8, case["page"] * (case["d"] // case["group"]) * 2
    return {"LB": LB, "W": min(16, LB), "codes": codes, "scales": scales, "rec": 2 * (codes + scales),
            "max_pages": -(-(case["far"] + case["T"]) // case["page"])}


def prepare(case, seed):
    s = dict(case, kept={})
    plan, B, T = _plan(case), case["B"], case["T"]
    if case["op"] in ("step", "commit"):
        s.update(_layer_inputs(case, seed))
        s["held"] = _views(case, s["buffer"])
    if case["op"] == "step":
        m = _seen(plan["parents"])
        s["seen"], s["bits"] = m.cuda(), _bits(m).cuda() if case["tree"] else None
        s["drafts"] = torch.tensor(plan["drafts"], dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["o"] = torch.empty_like(s["v"])
    elif case["op"] == "commit":
        s["nodes"] = _rows(plan["nodes"], T).cuda()
        s["counts"] = torch.tensor([len(x) for x in plan["nodes"]], dtype=torch.int32, device="cuda")
        s["most"] = plan["most"]
        s["count"] = s["held"]["count"].clone()
    elif case["op"] == "verify":
        s.update(_verify_inputs(case, seed))
        s["nodes"] = torch.empty((B, T), dtype=torch.int32, device="cuda")
        s["counts"], s["next"] = (torch.empty((B,), dtype=torch.int32, device="cuda") for _ in range(2))
    else:
        gen, z = _gen(seed), _cache_sizes(case)
        N = 2 * B * z["max_pages"] + 3
        order = torch.randperm(N, generator=gen, device="cuda")[: 2 * B * z["max_pages"]].to(torch.int32)
        tables = order.view(2, B, z["max_pages"])
        words = torch.randint(-2 ** 62, 2 ** 62, (N * case["H"] * z["rec"] // 8,), generator=gen, device="cuda", dtype=torch.int64)
        s["cache"], s["pages"] = words.view(torch.uint8), N
        s["table"] = tables[0].contiguous()
        s["to"] = s["table"]
        if case["how"] == "fork":                 # all read the first sequence's pages
            s["table"], s["to"] = tables[0, :1].expand(B, -1).contiguous(), tables[1].contiguous()
        s["start"] = torch.tensor(plan["start"], dtype=torch.int32, device="cuda")
        s["nodes"] = None if case["how"] == "fork" else _rows(plan["nodes"], T).cuda()
        s["counts"] = torch.tensor([len(x) for x in plan["nodes"]], dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms

def _plain_step(s):
    B, T, Hv, d, dP = (s[k] for k in ("B", "T", "Hv", "d", "dP"))
    per, n0 = Hv // s["Hk"], dP - 1
    N, dev = n0 + T, s["q"].device
    S = _unpack_state(s, s["packed"])                                             # [B, Hv, column, key]
    held = s["held"]
    new = {k: x.transpose(1, 2) for k, x in dict(_slots(s, s["k"], s["v"]), a=s["a"], beta=s["beta"]).items()}
    both = {k: torch.cat([held[k][:, :, :n0], new[k]], dim=2) for k in new}
    k, v = _meant(s, both)
    k = k.repeat_interleave(per, dim=1)                                           # [B, Hv, N, d]
    q = s["q"].float().transpose(1, 2).repeat_interleave(per, dim=1)              # [B, Hv, T, d]
    # slots past the count neither decay nor write
    live = torch.arange(n0, device=dev) < held["count"].clamp(0, n0).unsqueeze(-1)
    live = torch.cat([live, torch.ones((B, Hv, T), dtype=torch.bool, device=dev)], dim=-1)
    a, beta = torch.where(live, both["a"], torch.ones(())), torch.where(live, both["beta"], torch.zeros(()))
    k, v = (torch.where(live.unsqueeze(-1), x, torch.zeros(())) for x in (k, v))
    # path[i, j]: token j is token i or comes before it on its path
    path = torch.ones((N, N), dtype=torch.bool, device=dev).tril().expand(B, N, N).clone()
    path[:, n0:, n0:] = s["seen"]
    w = torch.where(path.unsqueeze(1), a.unsqueeze(-2), torch.ones(()))           # [B, Hv, i, m]
    after = w.flip(-1).cumprod(-1).flip(-1)                                       # prod over m >= j
    D = torch.cat([after[..., 1:], torch.ones((B, Hv, N, 1), device=dev)], dim=-1)
    D = torch.where(path.unsqueeze(1), D, torch.zeros(()))
    gamma = after[..., 0]
    St, kt = S.transpose(-1, -2).contiguous(), k.transpose(-1, -2).contiguous()
    A = torch.matmul(k, kt) * D
    U = beta.unsqueeze(-1) * (v - gamma.unsqueeze(-1) * torch.matmul(k, St))
    for i in range(1, N):
        U[:, :, i] -= beta[:, :, i, None] * torch.matmul(A[:, :, i: i + 1, :i], U[:, :, :i].contiguous()).squeeze(-2)
    o = gamma[:, :, n0:, None] * torch.matmul(q, St) + torch.matmul(torch.matmul(q, kt) * D[:, :, n0:], U)
    o = o.transpose(1, 2).to(s["v"].dtype)
    if s["drafts"] is not None:
        there = torch.arange(T, device=dev) < s["drafts"].unsqueeze(-1)
        o = torch.where(there[:, :, None, None], o, torch.zeros((), dtype=o.dtype))
    return {"o": o}


def _plain_verify(s):
    B, T, V = s["B"], s["T"], s["V"]
    dev = s["target"].device
    each = torch.arange(B, device=dev)
    parents, tokens, u = s["parents"].long(), s["tokens"].long(), s["uniforms"].double()
    row = torch.zeros((B,), dtype=torch.long, device=dev)
    taken, left = torch.zeros((B,), dtype=torch.float64, device=dev), torch.ones((B,), dtype=torch.float64, device=dev)
    nodes = torch.full((B, T), -1, dtype=torch.int32, device=dev)
    nodes[:, 0] = 0
    counts = torch.ones((B,), dtype=torch.long, device=dev)
    refused = torch.zeros((B, T), dtype=torch.bool, device=dev)              # children of the present node
    for c in range(1, T):
        child, t = (parents[:, c] == row) & (c < s["drafts"]), tokens[:, c]
        w = s["target"][each, row, t].double()
        if s["sampled"]:
            q = s["draft"][each, row, t].double()
            w = (w - taken * q).clamp(min=0.0)
            accept = child & (u[:, c] * left * q < w)
            taken = torch.where(child & ~accept, taken + left, taken)
            rest = (s["target"][each, row].double() - taken.unsqueeze(-1) * s["draft"][each, row].double()).clamp(min=0.0).sum(-1)
        else:
            again = (refused[:, :c] & (tokens[:, :c] == t.unsqueeze(-1))).any(-1)
            w = torch.where(again, torch.zeros_like(w), w)
            accept = child & (u[:, c] * left < w)
            rest = (left - w).clamp(min=0.0)
        refused[:, c] = child & ~accept
        left = torch.where(refused[:, c], rest, left)
        nodes.scatter_(1, counts.clamp(max=T - 1).unsqueeze(-1),
                       torch.where(accept, torch.full_like(counts, c), torch.full_like(counts, -1)).to(torch.int32).unsqueeze(-1))
        counts = counts + accept
        row = torch.where(accept, torch.full_like(row, c), row)
        taken, left = torch.where(accept, torch.zeros_like(taken), taken), torch.where(accept, torch.ones_like(left), left)
        refused = refused & ~accept.unsqueeze(-1)
    p = s["target"][each, row].double()
    if s["sampled"]:
        w = (p - taken.unsqueeze(-1) * s["draft"][each, row].double()).clamp(min=0.0)
    else:
        gone = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, tokens, refused.to(torch.int32))
        w = torch.where(gone > 0, torch.zeros_like(p), p)
    sums = w.cumsum(-1)
    sums = torch.where(sums[:, -1:] > 0, sums, p.cumsum(-1))
    at = (sums <= u[:, :1] * sums[:, -1:]).sum(-1)
    last = (sums < sums[:, -1:]).sum(-1)                                      # the last token of any weight
    at = torch.where(at < V, at, last)
    return {"nodes": nodes, "counts": counts.to(torch.int32), "next": torch.where(sums[:, -1] > 0, at, -1).to(torch.int32)}


def _plain_commit(s):
    B, dP = s["B"], s["dP"]
    held, dev = s["held"], s["k"].device
    n = held["count"][:, 0].long()
    at = torch.arange(dP, device=dev) - n.view(B, 1)                           # the slot's place in the path
    take = (at >= 0) & (at < s["counts"].view(B, 1))
    node = torch.gather(s["nodes"].long(), 1, at.clamp(0, s["T"] - 1)).clamp(min=0)
    pick = lambda x: x[torch.arange(B, device=dev).view(B, 1), node]  # noqa: E731
    new = dict(_slots(s, pick(s["k"]), pick(s["v"])), a=pick(s["a"]), beta=pick(s["beta"]))
    for name, x in new.items():
        x = x.transpose(1, 2)
        held[name].copy_(torch.where(take.view(B, 1, dP, *[1] * (x.dim() - 3)), x, held[name]))
    held["count"].add_(s["counts"].view(B, 1))
    return {k: x for k, x in held.items()}


def _token_bytes(case, r, dev):
    """Where a page's record keeps the bytes of its tokens r [...]: [..., bytes of a token].
    Keys, in tiles of 16: lane a of 4 holds LB bytes of token r in pieces of W: byte x at (x div W) 64 W + (16 a + r mod 16) W
    + x mod W.  Values, in quads: lane m of 16 holds LB bytes of the four tokens, byte x (x mod 4 = r mod 4) at (x div W) 16 W
    + m W + x mod W.  Scales bf16 [P/4][d/g][4]."""
    z, r = _cache_sizes(case), r.unsqueeze(-1)
    LB, W, ng = z["LB"], z["W"], case["d"] // case["group"]
    i = torch.arange(4 * LB, device=dev)
    a, x = i // LB, i % LB
    keys = (r // 16) * (64 * LB) + (x // W) * (64 * W) + (16 * a + r % 16) * W + x % W
    m, x = i // (LB // 4), 4 * (i % (LB // 4)) + r % 4
    values = (r // 4) * (16 * LB) + (x // W) * (16 * W) + m * W + x % W
    g = torch.arange(2 * ng, device=dev)
    scales = 2 * (((r // 4) * ng + g // 2) * 4 + r % 4) + g % 2
    half = z["codes"] + z["scales"]
    return torch.cat([keys, z["codes"] + scales, half + values, half + z["codes"] + scales], dim=-1)


def _plain_move(s):
    z, B, T, P = _cache_sizes(s), s["B"], s["T"], s["page"]
    dev = s["cache"].device
    i = torch.arange(T, device=dev).expand(B, T)
    live = i < s["counts"].view(B, 1)
    src = s["start"].long().view(B, 1) + (i if s["nodes"] is None else s["nodes"].long())
    dst = s["start"].long().view(B, 1) + i
    pool = s["cache"].view(-1, s["H"], z["rec"])
    places = []
    for table, at in ((s["table"], src), (s["to"], dst)):
        page = torch.gather(table.long(), 1, at.clamp(min=0) // P)[live]
        places.append((page.view(-1, 1, 1), torch.arange(s["H"], device=dev).view(1, -1, 1),
                       _token_bytes(s, at[live] % P, dev).unsqueeze(1)))
    pool[places[1]] = pool[places[0]]
    return {"cache": s["cache"]}


# ------------------------------------------------------------------------------------- run

def _kept(s):
    """The layer's configuration and scratch, made once, as a serving program keeps them."""
    import bit_recurrent_state_amd as pace
    if s["kept"]:
        return pace, s["kept"]["cfg"]
    n = 0
    if s["op"] in ("step", "commit"):
        bits = [8 if _wide(s, h) else 4 for h in range(s["Hv"])] if s["state"] == "asym" else None
        cfg = pace.LayerConfig(B=s["B"], Hv=s["Hv"], Hk=s["Hk"], dk=s["d"], dv=s["d"], group=s["group"],
                               asym=s["state"] == "asym", buf=s["buf"], bf16_io=s["io"] == "bf16", dP=s["dP"], head_bits=bits,
                               bf16_state=s["state"] == "bf16")
        n = pace.draft_commit_workspace_bytes(cfg, s["most"]) if s["op"] == "commit" else 0
    elif s["op"] == "verify":
        cfg = pace.VerifyConfig(B=s["B"], T=s["T"], V=s["V"], bf16_probs=s["probs"] == "bf16")
        n = pace.draft_verify_workspace_bytes(cfg)
    else:
        cfg = pace.CacheConfig(B=s["B"], Hq=s["H"], Hkv=s["H"], d=s["d"], kind=s["kind"], group=s["group"], page=s["page"],
                               max_pages=s["table"].shape[1], num_pages=s["pages"])
    s["kept"] = {"cfg": cfg, "workspace": torch.empty(n, dtype=torch.uint8, device="cuda") if n else None}
    return pace, cfg


def run(state):
    s = state
    if s["op"] == "commit":
        s["held"]["count"].copy_(s["count"])           # the same step again: the buffers as they were before it
    if not own:
        return {"step": _plain_step, "verify": _plain_verify, "commit": _plain_commit, "move": _plain_move}[s["op"]](s)
    pace, cfg = _kept(s)
    if s["op"] == "step":
        pace.draft_step(cfg, s["packed"], s["buffer"], s["q"], s["k"], s["v"], s["a"], s["beta"], s["o"], tree=s["bits"],
                        draft_lens=s["drafts"])
        return {"o": s["o"]}
    if s["op"] == "verify":
        pace.draft_verify(cfg, s["target"], s["tokens"], s["parents"], s["uniforms"], s["nodes"], s["counts"], s["next"],
                          draft=s["draft"], draft_lens=s["drafts"], workspace=s["kept"]["workspace"])
        return {"nodes": s["nodes"], "counts": s["counts"], "next": s["next"]}
    if s["op"] == "commit":
        pace.draft_commit(cfg, s["packed"], s["buffer"], s["k"], s["v"], s["a"], s["beta"], s["nodes"], s["counts"],
                          most=s["most"], workspace=s["kept"]["workspace"])
        return {k: x for k, x in s["held"].items()}
    pace.cache_move(cfg, s["cache"], s["table"], s["to"], s["start"], s["counts"], nodes=s["nodes"], most=s["T"])
    return {"cache": s["cache"]}


# ------------------------------------------------------------------------ work and 64 bits

def work(case):
    plan, B, T = _plan(case), case["B"], case["T"]
    if case["op"] in ("step", "commit"):
        Hv, Hk, d, e = case["Hv"], case["Hk"], case["d"], 2 if case["io"] == "bf16" else 4
        slot = (Hk * d + Hv * d + 4 * (Hk + Hv) if case["buf"] == "int8" else Hk * d // 2 + 2 * Hv * d + 4 * Hk) + 8 * Hv
        if case["op"] == "commit":
            m = sum(len(x) for x in plan["nodes"])
            return {"bytes": m * ((Hk + Hv) * d * e + 8 * Hv + slot + 4) + 12 * B * Hv, "flops": 4 * m * (Hk + Hv) * d}
        seq = sum(_record(case, h)[3] for h in range(Hv))
        total, flops = 0, 0
        for n, m, p in zip(plan["count"], plan["drafts"], plan["parents"]):
            total += seq + n * slot + m * ((2 * Hk + Hv) * d * e + 8 * Hv) + T * Hv * d * e
            pairs = n * (n + 1) // 2 + m * n + int(_seen([p])[0, :m, :m].sum())
            flops += Hv * (2 * d * d * (n + 2 * m) + 8 * d * pairs)
        return {"bytes": total + 4 * B * Hv, "flops": flops}
    if case["op"] == "verify":
        e, rows = 2 if case["probs"] == "bf16" else 4, 2 if case["sampled"] else 1
        return {"bytes": rows * B * (case["V"] + T) * e + B * (16 * T + 16), "flops": 4 * B * case["V"]}
    b = 4 if case["kind"] == "int4" else 8
    token = 2 * case["H"] * (case["d"] * b // 8 + 2 * (case["d"] // case["group"]))
    moved = [sum(i != j for i, j in enumerate(x)) for x in plan["nodes"]]
    if case["how"] == "fork":
        return {"bytes": token * (T + B * T) + 8 * B, "flops": 0}
    return {"bytes": 2 * token * sum(moved) + 4 * sum(len(x) for x in plan["nodes"]) + 8 * B, "flops": 0}


def _exact_step(case, seed):
    s, plan = _layer_inputs(case, seed), _plan(case)
    B, T, Hv, Hk, d, dP = (case[k] for k in ("B", "T", "Hv", "Hk", "d", "dP"))
    per, held = Hv // Hk, _views(case, s["buffer"])
    start = _unpack_state(case, s["packed"]).double().transpose(-1, -2).contiguous()     # [B, Hv, key, column]
    out = torch.zeros((B, T, Hv, d), dtype=torch.float64, device="cuda")

    def through(x, levels):                     # the buffer's codes are decided on the fp32 quotient
        top = x.float().abs().amax(-1, keepdim=True)
        scale = top / torch.full_like(top, levels)
        code = torch.round(x.float() / scale).clamp(-levels, levels)
        return torch.where(top > 0, code.double() * scale.double(), torch.zeros((), dtype=torch.float64))

    def step(S, k, v, a, beta):                 # S [Hv, key, column], k [Hk, d], v [Hv, d]
        k = k.repeat_interleave(per, 0)
        S = a[:, None, None] * S
        u = beta[:, None] * (v - torch.bmm(k[:, None, :], S)[:, 0])
        return S + k[:, :, None] * u[:, None, :]

    mixed = case["buf"] == "mixed"
    for b in range(B):
        S = start[b]
        for i in range(plan["count"][b]):
            kc = _of_nibbles(held["kc"][b, :, i]) if mixed else held["kc"][b, :, i]
            k = kc.double() * held["ks"][b, :, i, None].double()
            v = held["v"][b, :, i].double() * (1.0 if mixed else held["vs"][b, :, i, None].double())
            S = step(S, k, v, held["a"][b, :, i].double(), held["beta"][b, :, i].double())
        after = {-1: S}
        for i in range(plan["drafts"][b]):
            k = through(s["k"][b, i], 7.0 if mixed else 127.0)
            v = s["v"][b, i].to(torch.bfloat16).double() if mixed else through(s["v"][b, i], 127.0)
            S = step(after[plan["parents"][b][i]], k, v, s["a"][b, i].double(), s["beta"][b, i].double())
            after[i] = S
            out[b, i] = torch.bmm(s["q"][b, i].double().repeat_interleave(per, 0)[:, None, :], S)[:, 0]
    return {"o": out}


def _exact_verify(case, seed):
    s, plan = _verify_inputs(case, seed), _plan(case)
    B, T = case["B"], case["T"]
    tokens, u = s["tokens"].tolist(), s["uniforms"].double().tolist()
    nodes, following = [], []
    for b in range(B):
        x, path, c = 0, [0], 1
        w, total = s["target"][b, 0].double(), 1.0
        while c < plan["drafts"][b]:
            if plan["parents"][b][c] == x:
                t = tokens[b][c]
                q = float(s["draft"][b, x, t]) if case["sampled"] else 1.0
                if u[b][c] * total * q < float(w[t]):
                    x, w, total = c, s["target"][b, c].double(), 1.0
                    path.append(c)
                elif case["sampled"]:
                    w = (w - total * s["draft"][b, x].double()).clamp(min=0.0)
                    total = float(w.sum())
                else:
                    total = max(0.0, total - float(w[t]))
                    w[t] = 0.0
            c += 1
        if not float(w.sum()) > 0.0:
            w = s["target"][b, x].double()
        sums = torch.cumsum(w, 0)
        at = int(torch.searchsorted(sums, u[b][0] * float(sums[-1]), right=True))
        following.append(min(at, int(torch.nonzero(w)[-1])))
        nodes.append(path)
    return {"nodes": _rows(nodes, T), "counts": torch.tensor([len(x) for x in nodes], dtype=torch.int32),
            "next": torch.tensor(following, dtype=torch.int32)}


def _exact_commit(case, seed):
    """What the buffers hold afterwards: the scales from 64-bit quotients, the codes from the header's fp32 ones."""
    s, plan = _layer_inputs(case, seed), _plan(case)
    held = {k: x.clone() for k, x in _views(case, s["buffer"]).items()}
    for name in ("ks", "vs", "a", "beta"):
        if name in held:
            held[name] = held[name].double()
    for b, path in enumerate(plan["nodes"]):
        for i, node in enumerate(path):
            at = plan["count"][b] + i
            for h, x in (("k", s["k"][b, node]), ("v", s["v"][b, node])):
                if h == "v" and case["buf"] == "mixed":
                    held["v"][b, :, at] = x.to(torch.bfloat16)
                    continue
                levels = 7 if case["buf"] == "mixed" else 127
                top = x.float().abs().amax(-1, keepdim=True)
                scale = top / torch.full_like(top, levels)
                code = torch.round(x.float() / torch.where(top > 0, scale, torch.ones(()))).clamp(-levels, levels)
                held[h + "s"][b, :, at] = (top.double() / levels)[:, 0]
                held["kc" if h == "k" else "v"][b, :, at] = _nibbles(code) if case["buf"] == "mixed" else code.to(torch.int8)
            held["a"][b, :, at], held["beta"][b, :, at] = s["a"][b, node].double(), s["beta"][b, node].double()
        held["count"][b] += len(path)
    return held


def exact(case, seed):
    if case["op"] == "step":
        return _exact_step(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    if case["op"] == "commit":
        return _exact_commit(case, seed)
    return None                                  # bytes are moved: nothing is computed
