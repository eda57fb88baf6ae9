"""CPU tests of the host side of the operators that serve drafted tokens (include/pace_draft.h): exports,
sizes and every refusal, and pins of their oracle.  Nothing is launched: the pointers of the refusal
tests are aligned stand-ins that nothing dereferences, and each call is refused."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import cache_oracle as co
from oracle import draft_oracle as do
from oracle import packing as pk
from pace_synth import make_tokens, random_buffer_parts, random_packed_state_parts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)
EINVAL, EUNSUPPORTED = -1, -2


def _pace():
    import bit_recurrent_state_amd as pace
    return pace


def test_library_exports_every_declared_symbol():
    pace = _pace()
    text = open(os.path.join(ROOT, "include", "pace_draft.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(pace_[a-z0-9_]+)\s*\(", text))
    assert names == set(pace.DRAFT_EXPORTS)
    lib = ctypes.CDLL(pace.LIB_PATH)
    for n in names:
        assert hasattr(lib, n)


# ------------------------------------------------------------------- refusals

def refuse(fn, args, changes):
    """Every change (index -> value) of otherwise good arguments is refused with its status."""
    for change, status in changes:
        bad = list(args)
        for i, x in change.items():
            bad[i] = x
        assert fn(*bad) == status, change


def test_step_refuses():
    pace = _pace()
    c = pace.pace4(B=2)._c()
    good = [ctypes.byref(c)] + [FAKE] * 7 + [8, FAKE, FAKE, 0, FAKE, None]
    nulls = [({i: None}, EINVAL) for i in (0, 1, 2, 3, 4, 5, 6, 7, 12)]
    odd = [({i: ODD}, EINVAL) for i in (1, 2, 3, 4, 5, 6, 7, 9, 10, 12)]
    odd[5] = ({6: ctypes.c_void_p(0x10001)}, EINVAL)
    refuse(pace.LIB.pace_draft_step, good, nulls + odd + [
        ({8: 0}, EINVAL), ({8: -1}, EINVAL), ({8: 65}, EUNSUPPORTED), ({11: -1}, EINVAL), ({11: 1 << 62}, EINVAL)])
    for kw, status in ((dict(dk=96, dv=96, group=32), EUNSUPPORTED), (dict(Hk=3), EINVAL), (dict(dP=33), EUNSUPPORTED), (dict(group=48), EINVAL)):
        base = dict(B=2, Hv=32, Hk=16, dk=128, dv=128, group=64)
        base.update(kw)
        bad = pace.LayerConfig(**base)._c()
        refuse(pace.LIB.pace_draft_step, good, [({0: ctypes.byref(bad)}, status)])


def test_commit_refuses():
    pace = _pace()
    cfg = pace.pace4(B=2)
    c = cfg._c()
    need = pace.draft_commit_workspace_bytes(cfg, 8)
    good = [ctypes.byref(c)] + [FAKE] * 6 + [9, FAKE, FAKE, 8, FAKE, need, None]
    refuse(pace.LIB.pace_draft_commit, good,
           [({i: None}, EINVAL) for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 11)] + [({i: ODD}, EINVAL) for i in (1, 2, 3, 4, 5, 8, 9, 11)] + [
               ({7: 0}, EINVAL), ({7: 65}, EUNSUPPORTED), ({7: 7}, EINVAL), ({10: 0}, EINVAL), ({10: 10}, EINVAL), ({12: need - 1}, EINVAL)])
    with pytest.raises(pace.PaceError):
        pace.draft_commit_workspace_bytes(cfg, 0)
    with pytest.raises(pace.PaceError):
        pace.draft_commit_workspace_bytes(cfg, 65)
    # one list of taken tokens a launch that appends: 1 + ceil(most / dP)
    for most in (1, 8, 9, 16, 64):
        assert pace.draft_commit_workspace_bytes(cfg, most) == (1 + -(-most // 8)) * 2 * 32 * 4


def test_verify_refuses():
    pace = _pace()
    cfg = pace.VerifyConfig(B=2, T=4, V=1000)
    need = pace.draft_verify_workspace_bytes(cfg)
    good = [ctypes.byref(cfg._c), FAKE, 1000, FAKE, 1000, FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, need, None]
    required, optional = (1, 5, 8, 10, 11, 12), (3, 6, 9)
    refuse(pace.LIB.pace_draft_verify, good,
           [({i: None}, EINVAL) for i in (0, *required)] + [({i: ODD}, EINVAL) for i in (*required, *optional)] + [
               ({2: 999}, EINVAL), ({4: 999}, EINVAL), ({7: -1}, EINVAL), ({2: 1 << 46}, EUNSUPPORTED), ({4: 1 << 46}, EUNSUPPORTED),
               ({7: 1 << 60}, EUNSUPPORTED)]
           + ([({13: None}, EINVAL), ({13: ODD}, EINVAL), ({14: need - 1}, EINVAL)] if need else []))
    for kw, status in ((dict(B=0), EINVAL), (dict(T=0), EINVAL), (dict(V=0), EINVAL), (dict(B=65536), EUNSUPPORTED), (dict(T=1025), EUNSUPPORTED),
                       (dict(V=(1 << 24) + 1), EUNSUPPORTED)):
        base = dict(B=2, T=4, V=1000)
        base.update(kw)
        bad = pace.VerifyConfig(**base)
        refuse(pace.LIB.pace_draft_verify, good, [({0: ctypes.byref(bad._c)}, status)])
        with pytest.raises(pace.PaceError) as e:
            pace.draft_verify_workspace_bytes(bad)
        assert e.value.status == status


def test_move_refuses():
    pace = _pace()
    cfg = pace.CacheConfig(B=2, Hq=8, Hkv=2, d=128, num_pages=9, max_pages=4)
    good = [ctypes.byref(cfg._c), FAKE, FAKE, FAKE, FAKE, FAKE, 16, FAKE, 16, None]
    refuse(pace.LIB.pace_cache_move, good, [({i: None}, EINVAL) for i in (0, 1, 2, 3, 4, 7)] + [({i: ODD}, EINVAL) for i in (1, 2, 3, 4, 5, 7)] + [
        ({6: 15}, EINVAL), ({6: 1 << 60}, EINVAL), ({8: -1}, EINVAL), ({8: (1 << 30) + 1}, EUNSUPPORTED)])
    assert pace.LIB.pace_cache_move(ctypes.byref(cfg._c), None, None, None, None, None, 0, None, 0, None) == 0
    bad = pace.CacheConfig(B=2, Hq=8, Hkv=2, d=96, num_pages=9, max_pages=4, group=32)
    refuse(pace.LIB.pace_cache_move, good, [({0: ctypes.byref(bad._c)}, EUNSUPPORTED)])


# ------------------------------------------------------------- pins of the oracle

def test_a_node_sees_what_decoding_its_path_sees():
    """Every output of a tree equals that of the decode oracle on the path alone."""
    cfg = pk.LayerCfg(B=1, Hv=2, Hk=1, dk=64, dv=64, group=32, asym=False, buf="int8", dP=16)
    state = pk.pack_state(cfg, pk.state_from_parts(cfg, random_packed_state_parts(1, 1, 2, 64, 64, 32, [4, 4], False)))
    buf = pk.pack_buffer(cfg, random_buffer_parts(2, 1, 2, 1, 64, 64, 16, False, counts=[5]))
    parents = [-1, 0, 0, 1, 3, 2, -1, 6]
    t = make_tokens(3, 1, len(parents), 2, 1, 64, 64)
    rows = [[]]
    for p in parents[1:]:
        rows.append(rows[p] + [p] if p >= 0 else [])
    tiles = [(0, 0), (0, 1)]
    o = do.draft_step(cfg, state, buf, t.q, t.k, t.v, t.a, t.beta, [rows], [len(parents)], tiles)
    for i, row in enumerate(rows):
        s, b = state, buf
        for j in row + [i]:
            w, s, b, _ = pk.decode_step_layer(cfg, s, b, *(x[:, j] for x in (t.q, t.k, t.v, t.a, t.beta)))
        assert np.abs(w[0] - o[0, i]).max() <= 1e-12 * np.abs(w[0]).max()


@pytest.mark.parametrize("children", [1, 2, 3])
def test_verification_keeps_the_targets_distribution(children):
    """The token that follows the root is distributed as the target's, whatever the draft's distribution."""
    rng, V, N = np.random.default_rng(children), 5, 30000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    T = 1 + children
    tokens = rng.choice(V, size=(N, T), p=q)
    target = np.broadcast_to(np.stack([p] + [rng.dirichlet(np.ones(V)) for _ in range(children)]), (N, T, V))
    par = np.array([[-1] + [0] * children] * N)
    for draft in (np.broadcast_to(q, (N, T, V)), None):
        tok = tokens if draft is not None else np.broadcast_to(np.arange(T) - 1, (N, T))
        nodes, counts, following = do.draft_verify(target, draft, tok, par, rng.random((N, T)), [T] * N)
        first = np.where(counts > 1, tok[np.arange(N), nodes[:, 1 % T].clip(0)], following)
        seen = np.bincount(first, minlength=V) / N
        # five standard deviations of a frequency over N draws
        assert np.all(np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / N) + 1e-9), (seen, p)


def test_an_entrys_bytes_are_its_own():
    for kind, d, g, page in (("int8", 128, 64, 32), ("int4", 64, 32, 16), ("fp8", 256, 128, 16)):
        c = co.Cache(B=1, Hkv=1, d=d, kind=kind, group=g, page=page, num_pages=1, max_pages=1)
        at = do.entry_bytes(c)
        assert sorted(at.reshape(-1)) == list(range(c.record))
