"""ctypes binding of the operators that serve drafted tokens through a hybrid stack (the C ABI
declared in include/pace_draft.h): the gated-delta layers' outputs of drafts, verification, the
accepted tokens' way into the layers, and cached entries moved to other places.

Argument marshalling only, as in `_lib`: the work is done by the HIP kernels of libpace.so.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from functools import cached_property

import torch

from ._cache import CacheConfig, _CacheCfg, _call, _prepared, _ptr, _stream
from ._lib import IO_BF16, IO_F32, LIB, LayerConfig, _Cfg, _check, layout

DRAFT_EXPORTS = ["pace_draft_step", "pace_draft_commit", "pace_draft_commit_workspace_bytes", "pace_draft_verify",
                 "pace_draft_verify_workspace_bytes", "pace_cache_move"]


class _VerifyCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "V", "prob_dtype")]


def _declare():
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L, V = ctypes.POINTER(_Cfg), ctypes.POINTER(_VerifyCfg)
    LIB.pace_draft_step.argtypes = [L, P, P, P, P, P, P, P, i32, P, P, i64, P, P]
    LIB.pace_draft_commit.argtypes = [L, P, P, P, P, P, P, i32, P, P, i32, P, sz, P]
    LIB.pace_draft_commit_workspace_bytes.argtypes = [L, i32, ctypes.POINTER(sz)]
    LIB.pace_draft_verify.argtypes = [V, P, i64, P, i64, P, P, i64, P, P, P, P, P, P, sz, P]
    LIB.pace_draft_verify_workspace_bytes.argtypes = [V, ctypes.POINTER(sz)]
    LIB.pace_cache_move.argtypes = [ctypes.POINTER(_CacheCfg), P, P, P, P, P, i64, P, i32, P]
    for name in DRAFT_EXPORTS:
        getattr(LIB, name).restype = ctypes.c_int


_declare()


def _at(t, name, dtype, numel):
    """_ptr of a required tensor, with one test where nothing is wrong."""
    try:
        if t.dtype is dtype and t.numel() == numel and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, name, dtype, numel)


# ------------------------------------------------------------------ gated-delta layers

_layers = {}


def _layer(cfg: LayerConfig):
    """(C configuration, state bytes, buffer bytes) of what a layer's configuration says now: worked out once for every
    set of values, as it takes longer than the rest of a call's host side."""
    bits = cfg.head_bits
    key = (cfg.B, cfg.Hv, cfg.Hk, cfg.dk, cfg.dv, cfg.group, cfg.asym, cfg.buf, cfg.bf16_io, cfg.dP, cfg.chunk,
           cfg.bf16_state, None if bits is None else tuple(bits))
    known = _layers.get(key)
    if known is None:
        sizes = layout(cfg)
        if len(_layers) >= 256:
            _layers.clear()
        known = _layers[key] = (cfg._c(), sizes["state_bytes"], sizes["buffer_bytes"])
    return known


def _layer_args(cfg: LayerConfig, state, buffer, k, v, a, beta):
    """(config, state, buffer), (k, v, a, beta), T of a call on drafts [B, T, ..]."""
    c, state_bytes, buffer_bytes = _layer(cfg)
    B, Hv, d, f32 = cfg.B, cfg.Hv, cfg.dk, torch.float32
    if a.dim() != 3 or a.shape[0] != B or a.shape[2] != Hv:
        raise ValueError(f"a has shape {tuple(a.shape)}, expected ({B}, T, {Hv})")
    T = a.shape[1]
    io = torch.bfloat16 if cfg.bf16_io else f32
    n = B * T
    return (c, (ctypes.byref(c), _at(state, "state", torch.uint8, state_bytes), _at(buffer, "buffer", torch.uint8, buffer_bytes)),
            (_at(k, "k", io, n * cfg.Hk * d), _at(v, "v", io, n * Hv * d), _at(a, "a", f32, n * Hv),
             _at(beta, "beta", f32, n * Hv)), T, io)


def _step_args(cfg, state, buffer, q, k, v, a, beta, o, tree, draft_lens, stream):
    c, head, tokens, T, io = _layer_args(cfg, state, buffer, k, v, a, beta)
    step, words = 0, (T + 31) // 32
    if tree is not None:
        if tree.dim() != 3 or tree.shape[0] not in (1, cfg.B) or tuple(tree.shape[1:]) != (T, words):
            raise ValueError(f"tree has shape {tuple(tree.shape)}, expected ({cfg.B} or 1, {T}, {words})")
        step = T * words if tree.shape[0] == cfg.B else 0
    n = cfg.B * T
    return (c, (*head, _at(q, "q", io, n * cfg.Hk * cfg.dk), *tokens, T,
                _ptr(draft_lens, "draft_lens", torch.int32, cfg.B, optional=True),
                _ptr(tree, "tree", torch.int32, optional=True), step, _at(o, "o", io, n * cfg.Hv * cfg.dv), _stream(stream)))


def draft_step(cfg: LayerConfig, state, buffer, q, k, v, a, beta, o, tree=None, draft_lens=None, stream=None):
    """pace_draft_step.  q, k [B, T, Hk, dk]; v, o [B, T, Hv, dv]; a, beta fp32 [B, T, Hv]; tree
    int32 [B or 1, T, ceil(T / 32)] of tree_bits rows (None: a chain); draft_lens int32 [B] or None."""
    _c, args = _step_args(cfg, state, buffer, q, k, v, a, beta, o, tree, draft_lens, stream)
    _call(LIB.pace_draft_step, "pace_draft_step", args)


def prepare_draft_step(cfg: LayerConfig, state, buffer, q, k, v, a, beta, o, tree=None, draft_lens=None, stream=None):
    """Pre-marshalled pace_draft_step (see prepare_decode_step)."""
    c, args = _step_args(cfg, state, buffer, q, k, v, a, beta, o, tree, draft_lens, stream)
    return _prepared(LIB.pace_draft_step, "pace_draft_step", args,
                     (c, state, buffer, q, k, v, a, beta, o, tree, draft_lens))


def draft_commit_workspace_bytes(cfg: LayerConfig, most: int) -> int:
    c, out = cfg._c(), ctypes.c_size_t(0)
    _check(LIB.pace_draft_commit_workspace_bytes(ctypes.byref(c), most, ctypes.byref(out)),
           "pace_draft_commit_workspace_bytes")
    return int(out.value)


def _commit_args(cfg, state, buffer, k, v, a, beta, nodes, counts, workspace, most, stream):
    c, head, tokens, T, _ = _layer_args(cfg, state, buffer, k, v, a, beta)
    if tuple(nodes.shape) != (cfg.B, T):
        raise ValueError(f"nodes has shape {tuple(nodes.shape)}, expected ({cfg.B}, {T})")
    return (c, (*head, *tokens, T, _at(nodes, "nodes", torch.int32, cfg.B * T), _at(counts, "counts", torch.int32, cfg.B),
                T if most is None else most, _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))


def draft_commit(cfg: LayerConfig, state, buffer, k, v, a, beta, nodes, counts, workspace, most=None, stream=None):
    """pace_draft_commit.  k, v, a, beta as of draft_step; nodes int32 [B, T], counts int32 [B] (of draft_verify);
    most: upper bound of the counts (host, default T); workspace uint8 of draft_commit_workspace_bytes(cfg, most)."""
    _c, args = _commit_args(cfg, state, buffer, k, v, a, beta, nodes, counts, workspace, most, stream)
    _call(LIB.pace_draft_commit, "pace_draft_commit", args)


def prepare_draft_commit(cfg: LayerConfig, state, buffer, k, v, a, beta, nodes, counts, workspace, most=None, stream=None):
    """Pre-marshalled pace_draft_commit (see prepare_decode_step)."""
    c, args = _commit_args(cfg, state, buffer, k, v, a, beta, nodes, counts, workspace, most, stream)
    return _prepared(LIB.pace_draft_commit, "pace_draft_commit", args,
                     (c, state, buffer, k, v, a, beta, nodes, counts, workspace))


# -------------------------------------------------------------------------- verification

@dataclass(frozen=True)
class VerifyConfig:
    """Python mirror of pace_verify_cfg."""
    B: int
    T: int
    V: int
    bf16_probs: bool = False

    @cached_property
    def _c(self):
        return _VerifyCfg(self.B, self.T, self.V, IO_BF16 if self.bf16_probs else IO_F32)


def draft_verify_workspace_bytes(cfg: VerifyConfig) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.pace_draft_verify_workspace_bytes(ctypes.byref(cfg._c), ctypes.byref(out)),
           "pace_draft_verify_workspace_bytes")
    return int(out.value)


def _probs(t, name, dtype, cfg):
    """(address, row stride) of probabilities [B, T, V] whose rows are evenly spaced."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (cfg.B, cfg.T, cfg.V):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(cfg.B, cfg.T, cfg.V)}")
    if t.is_contiguous():
        return t.data_ptr(), cfg.V
    s = t.stride()
    if cfg.V > 1 and s[2] != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    row = s[1] if cfg.T > 1 else s[0] if cfg.B > 1 else cfg.V
    if cfg.T > 1 and cfg.B > 1 and s[0] != cfg.T * row:
        raise ValueError(f"{name}: rows must be evenly spaced over the sequences")
    return t.data_ptr(), row


def _verify_args(cfg, target, tokens, parents, uniforms, nodes, counts, next_tokens, draft, draft_lens, workspace, stream):
    if workspace is None:
        raise ValueError("workspace is required: uint8 of draft_verify_workspace_bytes(cfg)")
    dtype = torch.bfloat16 if cfg.bf16_probs else torch.float32
    tp, ts = _probs(target, "target", dtype, cfg)
    dp, ds = _probs(draft, "draft", dtype, cfg) if draft is not None else (None, 0)
    step, n = 0, cfg.B * cfg.T
    if parents is not None:
        if parents.dim() != 2 or parents.shape[0] not in (1, cfg.B) or parents.shape[1] != cfg.T:
            raise ValueError(f"parents has shape {tuple(parents.shape)}, expected ({cfg.B} or 1, {cfg.T})")
        step = cfg.T if parents.shape[0] == cfg.B else 0
    i32 = torch.int32
    return (ctypes.byref(cfg._c), tp, ts, dp, ds, _at(tokens, "tokens", i32, n),
            _ptr(parents, "parents", i32, optional=True), step, _at(uniforms, "uniforms", torch.float32, n),
            _ptr(draft_lens, "draft_lens", i32, cfg.B, optional=True), _at(nodes, "nodes", i32, n),
            _at(counts, "counts", i32, cfg.B), _at(next_tokens, "next_tokens", i32, cfg.B),
            _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))


def draft_verify(cfg: VerifyConfig, target, tokens, parents, uniforms, nodes, counts, next_tokens, draft=None,
                 draft_lens=None, workspace=None, stream=None):
    """pace_draft_verify.  target, draft [B, T, V] (rows may be slices of longer ones; draft None: children were not
    drawn from probabilities); tokens int32 [B, T]; parents int32 [B or 1, T] (None: a chain); uniforms fp32 [B, T];
    out: nodes int32 [B, T], counts and next_tokens int32 [B]; workspace uint8 of draft_verify_workspace_bytes(cfg), which every
    call needs."""
    _call(LIB.pace_draft_verify, "pace_draft_verify",
          _verify_args(cfg, target, tokens, parents, uniforms, nodes, counts, next_tokens, draft, draft_lens, workspace, stream))


def prepare_draft_verify(cfg: VerifyConfig, target, tokens, parents, uniforms, nodes, counts, next_tokens, draft=None,
                         draft_lens=None, workspace=None, stream=None):
    """Pre-marshalled pace_draft_verify (see prepare_decode_step)."""
    args = _verify_args(cfg, target, tokens, parents, uniforms, nodes, counts, next_tokens, draft, draft_lens, workspace, stream)
    return _prepared(LIB.pace_draft_verify, "pace_draft_verify", args,
                     (cfg, target, tokens, parents, uniforms, nodes, counts, next_tokens, draft, draft_lens, workspace))


# ------------------------------------------------------------------------------- cache

def _move_args(cfg, cache, src_table, dst_table, start, counts, nodes, most, stream):
    if nodes is not None:
        if nodes.dim() != 2 or nodes.shape[0] != cfg.B:
            raise ValueError(f"nodes has shape {tuple(nodes.shape)}, expected ({cfg.B}, T)")
        most = nodes.shape[1] if most is None else most
        if most > nodes.shape[1]:
            raise ValueError(f"most is {most}, but nodes has rows of {nodes.shape[1]}")
    elif most is None:
        raise ValueError("most is required without nodes")
    pages = cfg.B * cfg.max_pages
    return (ctypes.byref(cfg._c), _at(cache, "cache", torch.uint8, cfg._bytes),
            _at(src_table, "src_table", torch.int32, pages), _at(dst_table, "dst_table", torch.int32, pages),
            _at(start, "start", torch.int32, cfg.B), _ptr(nodes, "nodes", torch.int32, optional=True),
            nodes.shape[1] if nodes is not None else 0, _at(counts, "counts", torch.int32, cfg.B), most, _stream(stream))


def cache_move(cfg: CacheConfig, cache, src_table, dst_table, start, counts, nodes=None, most=None, stream=None):
    """pace_cache_move.  The entry at start[b] + nodes[b, i], found through src_table, moves to start[b] + i through
    dst_table (int32 [B, max_pages] each), for i < counts[b]; start, counts int32 [B]; nodes int32 [B, T] (None: i itself); most:
    upper bound of the counts (host, default T)."""
    _call(LIB.pace_cache_move, "pace_cache_move",
          _move_args(cfg, cache, src_table, dst_table, start, counts, nodes, most, stream))


def prepare_cache_move(cfg: CacheConfig, cache, src_table, dst_table, start, counts, nodes=None, most=None, stream=None):
    """Pre-marshalled pace_cache_move (see prepare_decode_step)."""
    args = _move_args(cfg, cache, src_table, dst_table, start, counts, nodes, most, stream)
    return _prepared(LIB.pace_cache_move, "pace_cache_move", args,
                     (cfg, cache, src_table, dst_table, start, counts, nodes))
