"""fp64 NumPy oracle of the attention-layer operators (include/pace_cache.h): rotary positions,
the cache's quantiser and byte layout, and attention over what a cache holds.

Everything follows the header's definitions literally, byte by byte and row by row; nothing is
shared with the HIP path.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

LEVELS = {"int8": 127, "int4": 7, "fp8": 448}
BITS = {"int8": 8, "int4": 4, "fp8": 8}


# ----------------------------------------------------------------------------- rotary

def rotary_freqs(rd, base, scaling="none", factor=1.0, original_len=0.0, fast=32.0, slow=1.0):
    f = np.array([base ** (-2.0 * i / rd) for i in range(rd // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        b = base * factor ** (rd / max(1, rd - 2))
        return np.array([b ** (-2.0 * i / rd) for i in range(rd // 2)]), 1.0
    if scaling == "blend":
        # pair i turns original_len f_i / (2 pi) times over the original length
        def pair(turns):
            return rd * np.log(original_len / (2 * np.pi * turns)) / (2 * np.log(base))
        lo, hi = max(0.0, np.floor(pair(fast))), min(rd - 1.0, np.ceil(pair(slow)))
        r = np.clip((np.arange(rd // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - r) + f / factor * r, 0.1 * np.log(factor) + 1.0
    return f, 1.0


def rotary(x, positions, freqs, rd, interleaved, magnitude=1.0, inverse=False):
    """x [n, H, d] -> rotated, fp64."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    for t, pos in enumerate(positions):
        for i in range(rd // 2):
            a = float(pos) * float(freqs[i])
            c, s = np.cos(a) * magnitude, np.sin(a) * magnitude * (-1 if inverse else 1)
            u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
            y[t, :, u] = x[t, :, u] * c - x[t, :, w] * s
            y[t, :, w] = x[t, :, w] * c + x[t, :, u] * s
    return y


# ------------------------------------------------------------------------- quantiser

def bf16_up(x):
    """Smallest bf16 value >= x >= 0 (fp64 in, fp64 out)."""
    m, e = np.frexp(x)
    return np.ldexp(np.ceil(m * 256.0) / 256.0, e)


def e4m3_values():
    """Value of every e4m3 byte (NaN at 0x7F, 0xFF)."""
    b = np.arange(256)
    e, m, s = (b >> 3) & 15, b & 7, np.where(b & 128, -1.0, 1.0)
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e.astype(float) - 7))
    v = s * v
    v[(b & 127) == 127] = np.nan
    return v


E4M3 = e4m3_values()


def e4m3_encode(y):
    """Nearest e4m3 byte of |y| <= 448, ties to the even significand; keeps the sign of zero."""
    pos = E4M3[:127]
    a = np.abs(y)
    hi = np.searchsorted(pos, a)                       # first value >= a
    hi = np.minimum(hi, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - pos[lo], pos[hi] - a
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    code = np.where(pos[hi] == a, hi, code)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x, kind, g):
    """Vectors x [..., d] (fp32 values) -> (stored fields uint8 [..., d], scales fp64
    [..., d / g], dequantised fp64 [..., d])."""
    x = np.asarray(x, dtype=np.float64)
    f = np.where(np.isnan(x), 0.0, np.clip(x, -2.0 ** 127, 2.0 ** 127)).reshape(*x.shape[:-1], -1, g)
    L = LEVELS[kind]
    s = bf16_up(np.abs(f).max(-1) / L)
    s = np.where(s < 2.0 ** -126, 0.0, s)
    S = s[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(S > 0, f / np.where(S > 0, S, 1.0), 0.0).astype(np.float32).astype(np.float64)
    y = np.clip(y, -L, L)
    if kind == "fp8":
        st = e4m3_encode(y)
        val = E4M3[st]
    else:
        c = np.rint(y)
        st = (c + (128 if kind == "int8" else 8)).astype(np.uint8)
        val = c
    return st.reshape(x.shape), s, (val * S).reshape(x.shape)


# ---------------------------------------------------------------------------- layout

@dataclass
class Cache:
    B: int
    Hkv: int
    d: int
    kind: str
    group: int
    page: int
    num_pages: int
    max_pages: int

    @property
    def codes(self):
        return self.page * self.d * BITS[self.kind] // 8

    @property
    def scales(self):
        return self.page * (self.d // self.group) * 2

    @property
    def record(self):
        return 2 * (self.codes + self.scales)

    @property
    def nbytes(self):
        return self.num_pages * self.Hkv * self.record

    def key_byte(self, r, c):
        """(byte offset in the record, shift) of key channel c of token r of a page."""
        b = BITS[self.kind]
        LB, G, a, e = self.d * b // 32, c // 32, (c % 32) // 8, c % 8
        W = min(16, LB)
        if b == 8:
            x, shift = 8 * G + e, 0
        else:
            nib = e // 2 + 4 * (e % 2)
            x, shift = 4 * G + nib // 2, 4 * (nib % 2)
        tile = (r // 16) * (16 * self.d * b // 8)
        return tile + (x // W) * 64 * W + (16 * a + r % 16) * W + x % W, shift

    def value_byte(self, r, c):
        b = BITS[self.kind]
        LB, G, m, e = self.d * b // 32, c // 32, (c % 32) // 2, c % 2
        W = min(16, LB)
        x, shift = (4 * (2 * G + e) + r % 4, 0) if b == 8 else (4 * G + r % 4, 4 * e)
        quad = (r // 4) * (4 * self.d * b // 8)
        return self.codes + self.scales + quad + (x // W) * 16 * W + m * W + x % W, shift

    def scale_at(self, r, G, values):
        at = self.codes + (self.codes + self.scales if values else 0)
        return at + 2 * (((r // 4) * (self.d // self.group) + G) * 4 + r % 4)

    def record_of(self, table, b, h, pos):
        """Byte offset of the record that holds position pos, or None."""
        if pos < 0 or pos // self.page >= self.max_pages:
            return None
        p = int(table[b, pos // self.page])
        return None if not 0 <= p < self.num_pages else (p * self.Hkv + h) * self.record


def _bf16_bits(s):
    return (np.float32(s).view(np.uint32) >> 16).astype(np.uint16)


def _bf16_value(lo, hi):
    return np.array([(int(lo) | int(hi) << 8) << 16], dtype=np.uint32).view(np.float32)[0]


def write(c: Cache, cache, table, positions, k, v):
    """k, v [B, T, Hkv, d] (fp32 values) into the byte array `cache`, in place."""
    B, T, H, d = k.shape
    mask = 255 if BITS[c.kind] == 8 else 15
    parts = [(quantise(x, c.kind, c.group), place, vals) for x, place, vals in
             ((k, c.key_byte, False), (v, c.value_byte, True))]
    for b in range(B):
        for t in range(T):
            pos = int(positions[b, t])
            for h in range(H):
                rec = c.record_of(table, b, h, pos)
                if rec is None:
                    continue
                r = pos % c.page
                for (st, s, _), place, vals in parts:
                    for ch in range(d):
                        at, shift = place(r, ch)
                        cache[rec + at] = (int(cache[rec + at]) & ~(mask << shift) & 255) | (int(st[b, t, h, ch]) << shift)
                    for G in range(d // c.group):
                        at = rec + c.scale_at(r, G, vals)
                        bits = int(_bf16_bits(s[b, t, h, G]))
                        cache[at], cache[at + 1] = bits & 255, bits >> 8


def read(c: Cache, cache, table, positions):
    """(k, v) fp64 [B, T, Hkv, d]; zeros where a position is skipped."""
    B, T = positions.shape
    mask = 255 if BITS[c.kind] == 8 else 15
    out = np.zeros((2, B, T, c.Hkv, c.d))
    for b in range(B):
        for t in range(T):
            pos = int(positions[b, t])
            for h in range(c.Hkv):
                rec = c.record_of(table, b, h, pos)
                if rec is None:
                    continue
                r = pos % c.page
                for i, place in enumerate((c.key_byte, c.value_byte)):
                    for ch in range(c.d):
                        at, shift = place(r, ch)
                        f = (int(cache[rec + at]) >> shift) & mask
                        val = E4M3[f] if c.kind == "fp8" else f - (128 if c.kind == "int8" else 8)
                        sa = rec + c.scale_at(r, ch // c.group, i == 1)
                        out[i, b, t, h, ch] = val * float(_bf16_value(cache[sa], cache[sa + 1]))
    return out[0], out[1]


# ------------------------------------------------------------------------- attention

def tree_mask(parents):
    T = len(parents)
    m = np.zeros((T, T), dtype=bool)
    for i in range(T):
        j = i
        while j >= 0:
            m[i, j] = True
            j = parents[j]
    return m


def attention(q, k, v, scale, visible):
    """Rows q [n, d] over tokens k, v [L, d] with visible [n, L] -> (o, lse, weights), fp64.
    A row that sees nothing: o = 0, lse = -inf."""
    z = np.where(visible, (q @ k.T) * scale, -np.inf)
    top = z.max(-1, initial=-np.inf)
    base = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(z - base[:, None])
    total = e.sum(-1)
    w = e / np.where(total > 0, total, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, np.log(np.where(total > 0, total, 1.0)) + base, -np.inf)
    return w @ v, lse, w
