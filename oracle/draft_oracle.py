"""fp64 NumPy oracle of the operators that serve drafted tokens (include/pace_draft.h).

Everything follows the header's definitions literally: the state of every node for the outputs of
drafts, child by child for the verification, entry by entry for moves.  Nothing is shared with the HIP path.
"""
from __future__ import annotations

import numpy as np

from . import packing as pk
from . import pace_oracle as po


# -------------------------------------------------------- outputs of drafts

def draft_step(cfg: pk.LayerCfg, state, buf, q, k, v, a, beta, rows, lens, tiles):
    """o [B, T, Hv, dv] fp64 (NaN outside `tiles`).  rows[b][i]: the tokens before i on its path, ascending."""
    qstates, d = pk.unpack_state(cfg, state, tiles), pk.unpack_buffer(cfg, buf)
    T = a.shape[1]
    o = np.full((cfg.B, T, cfg.Hv, cfg.dv), np.nan)
    for b, h in tiles:
        kh, n = h // cfg.gamma, min(max(int(d["count"][b, h]), 0), cfg.dP - 1)
        S0 = po._replay(qstates[b][h], [pk._entry(cfg, d, b, h, i) for i in range(n)])
        o[b, :, h] = 0.0
        states = {}
        for i in range(int(lens[b])):
            path = rows[b][i]
            S = states[path[-1]] if path else S0
            e = po.buffer_entry(k[b, i, kh], v[b, i, h], a[b, i, h], beta[b, i, h], cfg.buf)
            states[i], _ = po.exact_step(S, e.k, e.v, e.a, e.beta)
            o[b, i, h] = po.readout(states[i], np.asarray(q[b, i, kh], dtype=np.float64))
    return o


def draft_step_bound(cfg: pk.LayerCfg, state, buf, q, k, v, a, beta, rows, lens, tiles, roundings):
    """What fp32 arithmetic in the projections' form may be off, per output: every output and every u is a sum of
    products; with at most `roundings` roundings of 2^-24 on the way of any term, a sum is off by roundings 2^-24 of
    the sum of its terms' magnitudes, and by what its u's are off."""
    qstates, d = pk.unpack_state(cfg, state, tiles), pk.unpack_buffer(cfg, buf)
    T, eps = a.shape[1], roundings * 2.0 ** -24
    out = np.zeros((cfg.B, T, cfg.Hv, cfg.dv))
    for b, h in tiles:
        kh, n = h // cfg.gamma, min(max(int(d["count"][b, h]), 0), cfg.dP - 1)
        es = [pk._entry(cfg, d, b, h, i) for i in range(n)]
        es += [po.buffer_entry(k[b, i, kh], v[b, i, h], a[b, i, h], beta[b, i, h], cfg.buf) for i in range(int(lens[b]))]
        S = po._deq(qstates[b][h])
        mag = np.abs(S)
        if not cfg.bf16_state:
            # codes enter as 16 + c (8-bit heads: c) and their offsets are taken off again
            s = np.repeat(np.asarray(qstates[b][h].scales), cfg.group, axis=0)
            mag = s * (2.0 * (2 ** cfg.bits(h)) + 32.0)
        m, e = [], []
        for i, x in enumerate(es):
            before = list(range(min(i, n))) + ([n + j for j in rows[b][i - n]] if i >= n else [])
            g = x.a
            mu, er = np.zeros(cfg.dv), np.zeros(cfg.dv)
            for j in reversed(before):
                wm = x.beta * g * (np.abs(es[j].k) @ np.abs(x.k))
                mu += wm * m[j]
                er += wm * e[j]
                g *= es[j].a
            mu += x.beta * (np.abs(x.v) + g * (np.abs(x.k) @ mag))
            m.append(mu)
            e.append(eps * mu + er)
            if i >= n:
                qa = np.abs(np.asarray(q[b, i - n, kh], dtype=np.float64))
                g, tot, er = 1.0, np.zeros(cfg.dv), np.zeros(cfg.dv)
                for j in reversed(before + [i]):
                    w = g * (np.abs(es[j].k) @ qa)
                    tot += w * m[j]
                    er += w * e[j]
                    g *= es[j].a
                out[b, i - n, h] = eps * (tot + g * (qa @ mag)) + er
    return out


# ------------------------------------------------------------- verification

def weights(p):
    p = np.asarray(p, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(p) & (p > 0), p, 0.0)


def draft_verify(target, draft, tokens, parents, uniforms, lens):
    """(nodes [B, T], counts, next) from target [B, T, V], draft [B, T, V] or None."""
    B, T, V = target.shape
    nodes = np.full((B, T), -1, dtype=np.int32)
    counts, following = np.zeros(B, dtype=np.int32), np.full(B, -1, dtype=np.int32)
    u = np.nan_to_num(np.asarray(uniforms, dtype=np.float64), nan=0.0).clip(0.0, 1.0)
    for b in range(B):
        n = min(max(int(lens[b]), 0), T)
        if n == 0:
            continue
        x, path = 0, [0]
        w, W = weights(target[b, 0]), 1.0
        for c in range(1, n):
            t = int(tokens[b, c])
            if int(parents[b, c]) != x or not 0 <= t < V:
                continue
            q = weights(draft[b, x]) if draft is not None else None
            if u[b, c] * W * (q[t] if q is not None else 1.0) < w[t]:
                x = c
                path.append(c)
                w, W = weights(target[b, c]), 1.0
            elif q is not None:
                w = np.maximum(w - W * q, 0.0)
                W = float(w.sum())
            else:
                W = max(W - w[t], 0.0)
                w[t] = 0.0
        if not w.sum() > 0:
            w = weights(target[b, x])
        nodes[b, : len(path)], counts[b] = path, len(path)
        if w.sum() > 0:
            sums = np.cumsum(w)
            over = np.nonzero(sums > u[b, 0] * sums[-1])[0]
            following[b] = over[0] if len(over) else np.nonzero(w)[0][-1]
    return nodes, counts, following


# ------------------------------------------------------------- moved entries

def entry_bytes(c):
    """Byte offsets in a record of everything that belongs to token r of a page: [page][n]."""
    out = []
    for r in range(c.page):
        at = set()
        for ch in range(c.d):
            at.add(c.key_byte(r, ch)[0])
            at.add(c.value_byte(r, ch)[0])
        for G in range(c.d // c.group):
            for v in (False, True):
                at.update((c.scale_at(r, G, v), c.scale_at(r, G, v) + 1))
        out.append(sorted(at))
    return np.array(out)


def cache_move(c, cache, src_table, dst_table, start, nodes, counts):
    """The cache's bytes afterwards: every entry read before any is written."""
    cache = np.array(cache, dtype=np.uint8)
    old, place = cache.copy(), entry_bytes(c)
    for b in range(c.B):
        for i in range(max(0, int(counts[b]))):
            node = i if nodes is None else int(nodes[b, i])
            if node < 0:
                continue
            src, dst = int(start[b]) + node, int(start[b]) + i
            for h in range(c.Hkv):
                x, y = c.record_of(src_table, b, h, src), c.record_of(dst_table, b, h, dst)
                if x is not None and y is not None:
                    cache[y + place[dst % c.page]] = old[x + place[src % c.page]]
    return cache
