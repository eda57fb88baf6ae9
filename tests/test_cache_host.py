"""CPU tests of the attention-layer operators' host side (include/pace_cache.h): exports,
sizes, rotary frequencies, tree bits and every refusal.  Nothing is launched: the pointers of
the refusal tests are aligned stand-ins that nothing dereferences, and each call is refused."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import cache_oracle as co

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def _pace():
    import bit_recurrent_state_amd as pace
    return pace


def _cfg(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, num_pages=9, max_pages=4, kind="int8", group=64, page=64)
    base.update(kw)
    return _pace().CacheConfig(**base)


def test_library_exports_every_declared_symbol():
    pace = _pace()
    text = open(os.path.join(ROOT, "include", "pace_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(pace_[a-z0-9_]+)\s*\(", text))
    assert names == set(pace.CACHE_EXPORTS)
    lib = ctypes.CDLL(pace.LIB_PATH)
    for n in names:
        assert hasattr(lib, n)


@pytest.mark.parametrize("kind", ["int8", "int4", "fp8"])
@pytest.mark.parametrize("d,group,page", [(64, 32, 16), (64, 64, 1024), (128, 128, 64), (256, 32, 32)])
def test_layout_agrees_with_the_oracle(kind, d, group, page):
    pace = _pace()
    c = co.Cache(B=2, Hkv=2, d=d, kind=kind, group=group, page=page, num_pages=9, max_pages=4)
    L = pace.cache_layout(_cfg(d=d, group=group, page=page, kind=kind))
    assert L["record_bytes"] == c.record and L["page_bytes"] == 2 * c.record and L["cache_bytes"] == c.nbytes
    assert L["bits_per_value"] == co.BITS[kind] + 16 / group
    assert c.record * 8 == 2 * page * d * L["bits_per_value"]


@pytest.mark.parametrize("kind", ["int8", "int4", "fp8"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_oracle_layout_places_every_code_once(kind, d):
    """The header's formulas put the codes of a page one to one on the record's bytes."""
    c = co.Cache(B=1, Hkv=1, d=d, kind=kind, group=32, page=32, num_pages=1, max_pages=1)
    seen = set()
    for r in range(c.page):
        for ch in range(d):
            for at, shift in (c.key_byte(r, ch), c.value_byte(r, ch)):
                for bit in range(co.BITS[kind]):
                    seen.add(8 * at + shift + bit)
        for G in range(d // 32):
            for vals in (False, True):
                for bit in range(16):
                    seen.add(8 * c.scale_at(r, G, vals) + bit)
    assert len(seen) == 8 * c.record and min(seen) == 0 and max(seen) == 8 * c.record - 1


@pytest.mark.parametrize("rd,scaling,factor,original", [
    (64, "none", 1.0, 0.0), (128, "linear", 4.0, 0.0), (64, "ntk", 8.0, 0.0), (2, "ntk", 8.0, 0.0),
    (128, "blend", 16.0, 4096.0), (32, "blend", 1.0, 128.0)])
def test_rotary_frequencies(rd, scaling, factor, original):
    pace = _pace()
    f, m = pace.rotary_freqs(rd, 10000.0, scaling, factor, original)
    g, n = co.rotary_freqs(rd, 10000.0, scaling, factor, original)
    assert f.shape == (rd // 2,)
    assert np.allclose(f, g, rtol=1e-13, atol=0) and m == pytest.approx(n, rel=1e-14)


def test_blended_frequencies_keep_the_fast_pairs_and_stretch_the_slow_ones():
    f, _ = _pace().rotary_freqs(128, 10000.0, "blend", 8.0, 4096.0)
    plain, _ = _pace().rotary_freqs(128, 10000.0)
    assert f[0] == plain[0] and f[-1] == plain[-1] / 8.0
    assert np.all(np.diff(f) < 0)


@pytest.mark.parametrize("kw", [dict(rd=3), dict(rd=0), dict(base=1.0), dict(scaling="linear", factor=0.0),
                                dict(scaling="blend", factor=0.5, original_len=10.0),
                                dict(scaling="blend", factor=2.0, original_len=0.0),
                                dict(scaling="blend", factor=2.0, original_len=9.0, fast_turns=1.0),
                                dict(base=float("nan")), dict(scaling="ntk", factor=float("inf"))])
def test_rotary_frequency_refusals(kw):
    pace = _pace()
    with pytest.raises(pace.PaceError) as e:
        pace.rotary_freqs(**{"rd": 64, **kw})
    assert e.value.status == pace.PACE_EINVAL
    with pytest.raises(ValueError):
        pace.rotary_freqs(64, scaling="what")


def test_tree_bits():
    pace = _pace()
    rng = np.random.default_rng(3)
    for T in (1, 2, 31, 32, 33, 100):
        parents = [int(rng.integers(-1, i)) if i else -1 for i in range(T)]
        bits = pace.tree_bits(parents).view(np.uint32)
        m = co.tree_mask(parents)
        got = (bits[:, np.arange(T) // 32] >> (np.arange(T) % 32).astype(np.uint32)) & 1
        assert bits.shape == (T, (T + 31) // 32) and np.array_equal(got.astype(bool), m)
        assert int(np.sum([bin(int(w)).count("1") for w in bits.ravel()])) == int(m.sum())   # no bit past T
    for bad in ([0], [-2], [-1, 1], [-1, 0, 5]):
        with pytest.raises(pace.PaceError) as e:
            pace.tree_bits(bad)
        assert e.value.status == pace.PACE_EINVAL
    with pytest.raises(pace.PaceError):
        pace.tree_bits([])


INVALID = [dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(group=48), dict(d=64, group=128), dict(page=0),
           dict(num_pages=0), dict(max_pages=0), dict(group=0)]
UNSUPPORTED = [dict(d=96, group=32), dict(d=512), dict(group=16), dict(page=8), dict(page=48), dict(page=2048),
               dict(B=65536), dict(Hq=2048), dict(max_pages=1 << 26)]


@pytest.mark.parametrize("kw", INVALID + UNSUPPORTED)
def test_configuration_refusals_hold_for_every_call(kw):
    pace = _pace()
    want = pace.PACE_EINVAL if kw in INVALID else pace.PACE_EUNSUPPORTED
    cfg = _cfg(**kw)
    with pytest.raises(pace.PaceError) as e:
        pace.cache_layout(cfg)
    assert e.value.status == want
    with pytest.raises(pace.PaceError) as e:
        pace.cache_attention_workspace_bytes(cfg, 1, 64)
    assert e.value.status == want
    c, lib = ctypes.byref(cfg._c), pace.LIB
    assert lib.pace_cache_write(c, FAKE, FAKE, FAKE, 1, FAKE, 1 << 16, FAKE, 1 << 16, None) == want
    assert lib.pace_cache_read(c, FAKE, FAKE, FAKE, 1, FAKE, 1 << 16, FAKE, 1 << 16, None) == want
    assert lib.pace_cache_attention(c, FAKE, FAKE, FAKE, 1 << 20, 1, FAKE, None, None, 0, 1.0, 64, FAKE, None,
                                    None, 0, None) == want


def test_cache_io_refusals():
    pace = _pace()
    c = _cfg()._c
    names = ["cfg", "cache", "table", "positions", "T", "k", "ks", "v", "vs", "stream"]
    good = [ctypes.byref(c), FAKE, FAKE, FAKE, 1, FAKE, 256, FAKE, 256, None]
    bad = [dict(cfg=None), dict(cache=None), dict(cache=ODD), dict(table=None), dict(positions=None),
           dict(positions=ctypes.c_void_p(0x10002)), dict(T=-1), dict(k=None), dict(k=ODD), dict(ks=255), dict(ks=260),
           dict(v=None), dict(vs=128), dict(vs=-256), dict(ks=1 << 60)]
    for fn in (pace.LIB.pace_cache_write, pace.LIB.pace_cache_read):
        for kw in bad:
            args = [kw.get(n, g) for n, g in zip(names, good)]
            assert fn(*args) == pace.PACE_EINVAL, kw
        args = list(good)
        args[4] = 0                                   # nothing to do
        assert fn(*args) == pace.PACE_OK
    for kind in (-1, 3):
        cc = _cfg()._c
        old, cc.kind = cc.kind, kind
        assert pace.LIB.pace_cache_write(ctypes.byref(cc), FAKE, FAKE, FAKE, 1, FAKE, 256, FAKE, 256, None) == \
            pace.PACE_EINVAL
    with pytest.raises(ValueError):
        pace.cache_layout(_cfg(kind="int3"))


def test_attention_refusals():
    pace = _pace()
    cfg = _cfg(max_pages=1024, num_pages=4096)
    names = ["cfg", "cache", "table", "q", "qs", "T", "ctx", "drafts", "tree", "ts", "scale", "max_len", "o", "lse",
             "ws", "wsb", "stream"]
    need = pace.cache_attention_workspace_bytes(cfg, 1, 65536)
    assert need > 0
    good = [ctypes.byref(cfg._c), FAKE, FAKE, FAKE, 1024, 1, FAKE, None, None, 0, 0.1, 65536, FAKE, None, FAKE, need,
            None]
    bad = [dict(cfg=None), dict(cache=None), dict(cache=ODD), dict(table=None), dict(q=None), dict(q=ODD),
           dict(qs=1023), dict(qs=1028), dict(T=0), dict(T=-3), dict(ctx=None), dict(ts=-1), dict(scale=float("nan")),
           dict(scale=float("inf")), dict(max_len=0), dict(o=None), dict(o=ODD), dict(lse=ctypes.c_void_p(0x10001)),
           dict(ws=None), dict(wsb=need - 1), dict(ws=ODD), dict(drafts=ctypes.c_void_p(0x10001)),
           dict(tree=ctypes.c_void_p(0x10002))]
    for kw in bad:
        args = [kw.get(n, g) for n, g in zip(names, good)]
        assert pace.LIB.pace_cache_attention(*args) == pace.PACE_EINVAL, kw
    args = [dict(T=1 << 23).get(n, g) for n, g in zip(names, good)]
    assert pace.LIB.pace_cache_attention(*args) == pace.PACE_EUNSUPPORTED
    out = ctypes.c_size_t(77)
    assert pace.LIB.pace_cache_attention_workspace_bytes(ctypes.byref(cfg._c), 1, 64, None) == pace.PACE_EINVAL
    assert pace.LIB.pace_cache_attention_workspace_bytes(ctypes.byref(cfg._c), 0, 64, ctypes.byref(out)) == \
        pace.PACE_EINVAL
    assert out.value == 77


def test_rotary_refusals():
    pace = _pace()
    names = ["cfg", "n", "pos", "freqs", "mag", "inv", "q", "qs", "k", "ks", "qo", "qos", "ko", "kos", "stream"]

    def call(c=None, **kw):
        base = dict(Hq=4, Hk=2, d=64, rd=32)
        base.update(c or {})
        cfg = pace.RotaryConfig(**base)._c
        k_out = ctypes.c_void_p(0x20000)
        good = [ctypes.byref(cfg), 5, FAKE, FAKE, 1.0, 0, FAKE, 256, FAKE, 128, k_out, 256, k_out, 128, None]
        return pace.LIB.pace_rotary(*[kw.get(n, g) for n, g in zip(names, good)])

    for kw in (dict(cfg=None), dict(n=-1), dict(pos=None), dict(freqs=None), dict(freqs=ctypes.c_void_p(0x10004)),
               dict(mag=float("nan")), dict(q=None), dict(k=None), dict(qo=None), dict(qs=255), dict(kos=64),
               dict(q=ctypes.c_void_p(0x10001)), dict(qo=FAKE, qos=512)):
        assert call(**kw) == pace.PACE_EINVAL, kw
    for c in (dict(Hq=-1), dict(Hq=0, Hk=0), dict(d=63), dict(rd=31), dict(rd=66), dict(rd=0), dict(d=0)):
        assert call(c) == pace.PACE_EINVAL, c
    for c in (dict(d=2048), dict(d=1024, rd=514), dict(Hq=2000)):
        assert call(c, qs=1 << 22, qos=1 << 22, ks=1 << 22, kos=1 << 22) == pace.PACE_EUNSUPPORTED, c
    assert call(n=0, pos=None) == pace.PACE_OK


def test_workspace_is_needed_only_where_the_context_is_cut():
    """One short sequence and one token: cut over workgroups; many rows: not."""
    pace = _pace()
    few = _cfg(B=1, max_pages=64)
    many = _cfg(B=512, Hq=8, Hkv=8, max_pages=64, num_pages=32768)
    assert pace.cache_attention_workspace_bytes(few, 1, 4096) > 0
    assert pace.cache_attention_workspace_bytes(many, 1, 4096) == 0
    assert pace.cache_attention_workspace_bytes(few, 1, 16) == 0


def test_oracle_quantiser_rules():
    """Half-step errors, scale rounding, the stand-ins of non-finite values, zero groups."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 128)).astype(np.float32)
    x[0, :32] = 0
    x[1, 3], x[1, 40], x[2, 5] = np.nan, np.inf, -np.inf
    x[3, 64:96] *= 1e-39
    for kind in co.LEVELS:
        st, s, y = co.quantise(x, kind, 32)
        assert np.all(np.isfinite(y)) and np.all(y[0, :32] == 0) and s[0, 0] == 0 and s[3, 2] == 0
        fin = np.isfinite(x)
        S = np.repeat(s, 32, -1)
        err = np.abs(y - np.where(fin, x, y))
        # half a step of the integer grids; for e4m3 half a step is at most 2^-4 of the value or
        # 2^-10 of the scale; the quotient's own fp32 rounding moves a tie by 2^-24 of it
        half = S / 2 if kind != "fp8" else np.maximum(np.abs(np.where(fin, x, 0)) * 2.0 ** -4, S * 2.0 ** -10)
        plain = np.ones_like(fin)
        plain[3, 64:96] = False                       # stored as zeros
        ok = err <= half * (1 + 1e-6)
        assert np.all(ok[plain & fin])
        assert y[1, 3] == 0 and y[1, 40] >= 2.0 ** 126 and y[2, 5] <= -2.0 ** 126


def test_e4m3_encoding_is_nearest_even():
    v = co.E4M3[:127]
    assert v[126] == 448 and v[1] == 2.0 ** -9 and np.all(np.diff(v) > 0)
    assert np.array_equal(co.e4m3_encode(v), np.arange(127))
    mid = (v[:-1] + v[1:]) / 2
    even = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(co.e4m3_encode(mid), even)
    assert np.array_equal(co.e4m3_encode(-mid), even + 128)
