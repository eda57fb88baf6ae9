"""ctypes binding of the attention-layer operators (the C ABI declared in
include/pace_cache.h): rotary positions, the quantised paged key/value cache, and attention for
drafted tokens over it.

Argument marshalling only, as in `_lib`: the work is done by the HIP kernels of libpace.so.
Tensors may be slices of a wider projection output as long as their heads and channels are
contiguous and their tokens evenly spaced.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from functools import cached_property

import numpy as np
import torch

from ._lib import IO_BF16, IO_F32, LIB, PACE_OK, PaceError, _check

CACHE_KINDS = {"int8": 0, "int4": 1, "fp8": 2}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "blend": 3}

CACHE_EXPORTS = ["pace_rotary_freqs", "pace_rotary", "pace_cache_layout", "pace_cache_write",
                 "pace_cache_read", "pace_tree_bits", "pace_cache_attention",
                 "pace_cache_attention_workspace_bytes"]


class _RotaryCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("Hq", "Hk", "d", "rd", "interleaved", "io_dtype")]


class _CacheCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "d", "kind", "group", "page", "num_pages",
                                              "max_pages", "io_dtype")]


class _CacheInfo(ctypes.Structure):
    _fields_ = [("cache_bytes", ctypes.c_size_t), ("page_bytes", ctypes.c_size_t),
                ("record_bytes", ctypes.c_size_t), ("bits_per_value", ctypes.c_double)]


def _declare():
    P, i32, i64, f64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    C, D = ctypes.POINTER(_CacheCfg), ctypes.POINTER(ctypes.c_double)
    LIB.pace_rotary_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, D, D]
    LIB.pace_rotary.argtypes = [ctypes.POINTER(_RotaryCfg), i32, P, P, f64, i32, P, i64, P, i64, P, i64, P, i64, P]
    LIB.pace_cache_layout.argtypes = [C, ctypes.POINTER(_CacheInfo)]
    LIB.pace_cache_write.argtypes = [C, P, P, P, i32, P, i64, P, i64, P]
    LIB.pace_cache_read.argtypes = [C, P, P, P, i32, P, i64, P, i64, P]
    LIB.pace_tree_bits.argtypes = [ctypes.POINTER(i32), i32, ctypes.POINTER(ctypes.c_uint32)]
    LIB.pace_cache_attention.argtypes = [C, P, P, P, i64, i32, P, P, P, i64, f64, i32, P, P, P, sz, P]
    LIB.pace_cache_attention_workspace_bytes.argtypes = [C, i32, i32, ctypes.POINTER(sz)]
    for name in CACHE_EXPORTS:
        getattr(LIB, name).restype = ctypes.c_int


_declare()


@dataclass(frozen=True)
class RotaryConfig:
    """Python mirror of pace_rotary_cfg."""
    Hq: int
    Hk: int
    d: int
    rd: int
    interleaved: bool = False
    bf16_io: bool = True

    @cached_property
    def _c(self):
        return _RotaryCfg(self.Hq, self.Hk, self.d, self.rd, int(self.interleaved),
                          IO_BF16 if self.bf16_io else IO_F32)


@dataclass(frozen=True)
class CacheConfig:
    """Python mirror of pace_cache_cfg."""
    B: int
    Hq: int
    Hkv: int
    d: int
    num_pages: int
    max_pages: int
    kind: str = "int8"           # 'int8' | 'int4' | 'fp8'
    group: int = 64
    page: int = 64
    bf16_io: bool = True

    @cached_property
    def _c(self):
        if self.kind not in CACHE_KINDS:
            raise ValueError(f"kind must be one of {sorted(CACHE_KINDS)}, got {self.kind!r}")
        return _CacheCfg(self.B, self.Hq, self.Hkv, self.d, CACHE_KINDS[self.kind], self.group, self.page,
                         self.num_pages, self.max_pages, IO_BF16 if self.bf16_io else IO_F32)

    @cached_property
    def _bytes(self):
        return cache_layout(self)["cache_bytes"]


def _io(cfg):
    return torch.bfloat16 if cfg.bf16_io else torch.float32


def _ptr(t, name, dtype, numel=None, optional=False):
    """Address of a contiguous GPU tensor (None where an optional one is left out)."""
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _stream(stream):
    """The stream's handle; the current stream without building a Stream object for it (2.8 of
    the 11 us that a call's host side took)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _call(fn, name, args):
    st = fn(*args)
    if st != PACE_OK:
        raise PaceError(st, name)


def _prepared(fn, name, args, keep):
    """The same call again with no Python-side checks (graph capture, timing loops); the tensors
    stay alive with the callable."""
    def call():
        st = fn(*args)
        if st != PACE_OK:
            raise PaceError(st, name)
    call._keep = (keep, args)
    return call


def _rows(t, name, dtype, lead, H, d):
    """(address, token stride) of a tensor [*lead, H, d] whose tokens are evenly spaced."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (*lead, H, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(*lead, H, d)}")
    if t.is_contiguous():
        return t.data_ptr(), H * d
    st = t.stride()
    n = len(lead)
    if (d > 1 and st[-1] != 1) or (H > 1 and st[-2] != d):
        raise ValueError(f"{name}: heads and channels must be contiguous")
    step = st[n - 1]
    if lead[-1] == 1:                      # one token a sequence: the sequences' spacing counts
        step = st[0] if n > 1 and lead[0] > 1 else H * d
    elif n > 1 and lead[0] > 1 and st[0] != lead[1] * step:
        raise ValueError(f"{name}: tokens must be evenly spaced over the sequences")
    return t.data_ptr(), step


# ----------------------------------------------------------------------------- rotary

def rotary_freqs(rd: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_len: float = 0.0, fast_turns: float = 32.0, slow_turns: float = 1.0):
    """pace_rotary_freqs: (fp64 frequencies [rd / 2], magnitude) on the host."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    f = np.zeros(max(1, rd // 2), dtype=np.float64)
    m = ctypes.c_double(0.0)
    _check(LIB.pace_rotary_freqs(rd, base, ROPE_SCALINGS[scaling], factor, original_len, fast_turns, slow_turns,
                                 f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(m)),
           "pace_rotary_freqs")
    return f, m.value


def _rotary_args(cfg, positions, freqs, q, k, q_out, k_out, magnitude, inverse, stream):
    n = positions.numel()
    io, lead, d = _io(cfg), (n,), cfg.d
    qp = qo = kp = ko = None
    qs = qos = ks = kos = 0
    if cfg.Hq:
        (qp, qs), (qo, qos) = _rows(q, "q", io, lead, cfg.Hq, d), _rows(q_out, "q_out", io, lead, cfg.Hq, d)
    if cfg.Hk:
        (kp, ks), (ko, kos) = _rows(k, "k", io, lead, cfg.Hk, d), _rows(k_out, "k_out", io, lead, cfg.Hk, d)
    return (ctypes.byref(cfg._c), n, _ptr(positions, "positions", torch.int32),
            _ptr(freqs, "freqs", torch.float64, cfg.rd // 2), magnitude, int(inverse),
            qp, qs, kp, ks, qo, qos, ko, kos, _stream(stream))


def rotary(cfg: RotaryConfig, positions, freqs, q, k, q_out, k_out, magnitude: float = 1.0,
           inverse: bool = False, stream=None):
    """pace_rotary.  q, q_out [n, Hq, d] and k, k_out [n, Hk, d] (None where the config has no
    heads of it; the output may be the input); positions int32 [n]; freqs fp64 [rd / 2]."""
    _call(LIB.pace_rotary, "pace_rotary",
          _rotary_args(cfg, positions, freqs, q, k, q_out, k_out, magnitude, inverse, stream))


def prepare_rotary(cfg: RotaryConfig, positions, freqs, q, k, q_out, k_out, magnitude: float = 1.0,
                   inverse: bool = False, stream=None):
    """Pre-marshalled pace_rotary (see prepare_decode_step)."""
    args = _rotary_args(cfg, positions, freqs, q, k, q_out, k_out, magnitude, inverse, stream)
    return _prepared(LIB.pace_rotary, "pace_rotary", args, (cfg, positions, freqs, q, k, q_out, k_out))


# ------------------------------------------------------------------------------ cache

def cache_layout(cfg: CacheConfig) -> dict:
    """pace_cache_layout: cache_bytes, page_bytes, record_bytes, bits_per_value."""
    info = _CacheInfo()
    _check(LIB.pace_cache_layout(ctypes.byref(cfg._c), ctypes.byref(info)), "pace_cache_layout")
    return {f: getattr(info, f) for f, _ in _CacheInfo._fields_}


def _cache_io_args(cfg, cache, page_table, positions, k, v, stream):
    if positions.dim() != 2 or positions.shape[0] != cfg.B:
        raise ValueError(f"positions has shape {tuple(positions.shape)}, expected ({cfg.B}, T)")
    T = positions.shape[1]
    io = _io(cfg)
    kp, ks = _rows(k, "k", io, (cfg.B, T), cfg.Hkv, cfg.d)
    vp, vs = _rows(v, "v", io, (cfg.B, T), cfg.Hkv, cfg.d)
    return (ctypes.byref(cfg._c), _ptr(cache, "cache", torch.uint8, cfg._bytes),
            _ptr(page_table, "page_table", torch.int32, cfg.B * cfg.max_pages),
            _ptr(positions, "positions", torch.int32), T, kp, ks, vp, vs, _stream(stream))


def cache_write(cfg: CacheConfig, cache, page_table, positions, k, v, stream=None):
    """pace_cache_write.  cache uint8 [cache_bytes]; page_table int32 [B, max_pages]; positions
    int32 [B, T] (negative: skipped); k, v [B, T, Hkv, d]."""
    _call(LIB.pace_cache_write, "pace_cache_write", _cache_io_args(cfg, cache, page_table, positions, k, v, stream))


def cache_read(cfg: CacheConfig, cache, page_table, positions, k, v, stream=None):
    """pace_cache_read into k, v [B, T, Hkv, d] (zeros where a position is skipped)."""
    _call(LIB.pace_cache_read, "pace_cache_read", _cache_io_args(cfg, cache, page_table, positions, k, v, stream))


def prepare_cache_write(cfg: CacheConfig, cache, page_table, positions, k, v, stream=None):
    """Pre-marshalled pace_cache_write (see prepare_decode_step)."""
    args = _cache_io_args(cfg, cache, page_table, positions, k, v, stream)
    return _prepared(LIB.pace_cache_write, "pace_cache_write", args, (cfg, cache, page_table, positions, k, v))


# -------------------------------------------------------------------------- attention

def tree_bits(parents) -> np.ndarray:
    """pace_tree_bits: ancestor bits int32 [T, ceil(T / 32)] of one tree of drafted tokens
    (parents [T], -1 for the sequence itself, parents[i] < i), on the host."""
    p = np.ascontiguousarray(parents, dtype=np.int32)
    if p.ndim != 1:
        raise ValueError("parents must be one-dimensional")
    bits = np.zeros((len(p), (len(p) + 31) // 32), dtype=np.int32)
    _check(LIB.pace_tree_bits(p.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(p),
                              bits.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32))), "pace_tree_bits")
    return bits


def cache_attention_workspace_bytes(cfg: CacheConfig, T: int, max_len: int) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.pace_cache_attention_workspace_bytes(ctypes.byref(cfg._c), T, max_len, ctypes.byref(out)),
           "pace_cache_attention_workspace_bytes")
    return int(out.value)


def _attention_args(cfg, cache, page_table, q, ctx_lens, o, lse, tree, draft_lens, scale, max_len, workspace, stream):
    if q.dim() != 4:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected ({cfg.B}, T, {cfg.Hq}, {cfg.d})")
    T = q.shape[1]
    io = _io(cfg)
    qp, qs = _rows(q, "q", io, (cfg.B, T), cfg.Hq, cfg.d)
    words = (T + 31) // 32
    step = 0
    if tree is not None:
        if tree.dim() != 3 or tree.shape[0] not in (1, cfg.B) or tuple(tree.shape[1:]) != (T, words):
            raise ValueError(f"tree has shape {tuple(tree.shape)}, expected ({cfg.B} or 1, {T}, {words})")
        step = T * words if tree.shape[0] == cfg.B else 0
    if max_len is None:
        max_len = cfg.max_pages * cfg.page
    if scale is None:
        scale = 1.0 / math.sqrt(cfg.d)
    n_q = cfg.B * T * cfg.Hq
    return (ctypes.byref(cfg._c), _ptr(cache, "cache", torch.uint8, cfg._bytes),
            _ptr(page_table, "page_table", torch.int32, cfg.B * cfg.max_pages), qp, qs, T,
            _ptr(ctx_lens, "ctx_lens", torch.int32, cfg.B),
            _ptr(draft_lens, "draft_lens", torch.int32, cfg.B, optional=True),
            _ptr(tree, "tree", torch.int32, optional=True), step, scale, max_len,
            _ptr(o, "o", io, n_q * cfg.d), _ptr(lse, "lse", torch.float32, n_q, optional=True),
            _ptr(workspace, "workspace", torch.uint8, optional=True),
            workspace.numel() if workspace is not None else 0, _stream(stream))


def cache_attention(cfg: CacheConfig, cache, page_table, q, ctx_lens, o, lse=None, tree=None, draft_lens=None,
                    scale=None, max_len=None, workspace=None, stream=None):
    """pace_cache_attention.  q, o [B, T, Hq, d]; ctx_lens int32 [B]; tree int32
    [B or 1, T, ceil(T / 32)] of tree_bits rows (None: a chain); draft_lens int32 [B] or None;
    lse fp32 [B, T, Hq] or None; scale 1 / sqrt(d) by default; max_len (host, default the
    table's capacity) what the work is laid out for; workspace uint8 of
    cache_attention_workspace_bytes(cfg, T, max_len)."""
    _call(LIB.pace_cache_attention, "pace_cache_attention",
          _attention_args(cfg, cache, page_table, q, ctx_lens, o, lse, tree, draft_lens, scale, max_len, workspace, stream))


def prepare_cache_attention(cfg: CacheConfig, cache, page_table, q, ctx_lens, o, lse=None, tree=None, draft_lens=None,
                            scale=None, max_len=None, workspace=None, stream=None):
    """Pre-marshalled pace_cache_attention (see prepare_decode_step)."""
    args = _attention_args(cfg, cache, page_table, q, ctx_lens, o, lse, tree, draft_lens, scale, max_len, workspace, stream)
    return _prepared(LIB.pace_cache_attention, "pace_cache_attention", args,
                     (cfg, cache, page_table, q, ctx_lens, o, lse, tree, draft_lens, workspace))
