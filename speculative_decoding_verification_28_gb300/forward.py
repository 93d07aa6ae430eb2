"""Binding of the forward-pass operators around a round: appending queries,
keys and values, attention over the cache, tree verification and the commit
of an accepted path.  As in api.py each function has the name of its C entry
point, takes CUDA tensors and raises on a negative return code; definitions
and layouts are in include/specverify.h.

Every function also takes stream= (default: the current stream of the tensors'
device), on which its outputs and scratch are allocated.  The tensors' device
is made current for the call.  Scratch that is not passed
in comes from a per-stream buffer; while a stream is being captured every call
gets a buffer of its own from the graph's memory (cleared inside the graph),
so captured graphs share none and may be replayed side by side.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _lib
from .api import _DT, _check, _need

FLAG_BAD_STATE, FLAG_BAD_TREE = 16, 32
MAX_NODES = 64
MAX_HEAD_DIM = 256


def _ptr(t):
    return None if t is None else t.data_ptr()


def _streamed(fn):
    """Runs fn with `stream` current, so that outputs and scratch it allocates
    belong to the stream that writes them."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)

    return call


class _On:
    """The current stream of the tensors' device, with that device current."""

    __slots__ = ("stream", "guard")

    def __init__(self, device):
        self.stream = torch.cuda.current_stream(device)
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


_scratch = {}


def _ws(given, kind, nbytes, device, stream, zero):
    """Scratch of at least nbytes for the current stream, cleared when new if
    the kernel needs it."""
    if given is not None:
        buf = getattr(given, "buf", given)
        _need(buf, torch.uint8, "workspace", device)
        return buf
    make = torch.zeros if zero else torch.empty
    if torch.cuda.is_current_stream_capturing():
        return make(nbytes, dtype=torch.uint8, device=device)
    key = kind, device.index, stream.cuda_stream
    buf = _scratch.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = _scratch[key] = make(nbytes, dtype=torch.uint8, device=device)
    return buf


def _cache(kv, layer):
    if kv.dim() != 6 or kv.shape[1] != 2:
        raise ValueError("kv must be [L, 2, N, H, S, D]")
    _need(kv, None, "kv")
    if kv.dtype not in _DT:
        raise ValueError(f"unsupported kv dtype {kv.dtype}")
    L, _, N, H, S, D = kv.shape
    if not 0 <= layer < L:
        raise ValueError(f"layer {layer} of {L}")
    return kv.device, L, N, H, S, D


def _out(t, shape, dtype, dev, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, dtype, name, dev, shape)
    return t


def _rows(idx, B, N, dev):
    _need(idx, torch.int32, "idx", dev, (B,))
    if idx is None and B > N:
        raise ValueError(f"{B} sequences in a cache of {N} rows: pass idx")


@_streamed
def spec_tree_plan(parent, n_nodes=None, mask=None, depth=None, flags=None):
    """parent [B, T] int32 -> (mask [B, T] int64 bit sets, depth [B, T] int32,
    flags [B] int32)."""
    B, T = parent.shape
    dev = parent.device
    _need(parent, torch.int32, "parent", dev)
    _need(n_nodes, torch.int32, "n_nodes", dev, (B,))
    mask = _out(mask, (B, T), torch.int64, dev, "mask")
    depth = _out(depth, (B, T), torch.int32, dev, "depth")
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    with _On(dev) as st:
        _check(_lib.load().spec_tree_plan(B, T, _ptr(parent), _ptr(n_nodes), _ptr(mask), _ptr(depth), _ptr(flags), st))
    return mask, depth, flags


def _append_common(qkv, kv, layer, inv_freq, q_weight, k_weight, lead):
    dev, L, N, H, S, D = _cache(kv, layer)
    _need(qkv, kv.dtype, "qkv", dev)
    heads = qkv.shape[-2]
    if qkv.dim() != lead + 2 or qkv.shape[-1] != D or heads <= 2 * H:
        raise ValueError(f"qkv must end in [Hq + 2 * {H}, {D}]")
    for w, nm in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        _need(w, kv.dtype, nm, dev, (D,))
    R = 0
    if inv_freq is not None:
        _need(inv_freq, torch.float32, "inv_freq", dev)
        R = 2 * inv_freq.numel()
        if R > D:
            raise ValueError(f"inv_freq turns {R} of {D} dimensions")
    return dev, (L, N, H, S, D), heads - 2 * H, R


@_streamed
def spec_append_round(qkv, kv, layer, length, pad, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                      interleaved=False, depth=None, n_nodes=None, idx=None, staged=None, q_out=None, flags=None):
    """qkv [B, T, Hq + 2H, D] of a round's nodes: per-head RMS norm of queries
    and keys, rotation, keys and values to the cache kv [L, 2, N, H, S, D] (or
    to staged [L, 2, B, H, T, D]).  pad None: 0.
    -> (q_out [B, T, Hq, D], flags [B] int32)."""
    dev, (L, N, H, S, D), Hq, R = _append_common(qkv, kv, layer, inv_freq, q_weight, k_weight, 2)
    B, T = qkv.shape[:2]
    _need(length, torch.int32, "length", dev, (B,))
    _need(pad, torch.int32, "pad", dev, (B,))
    _need(n_nodes, torch.int32, "n_nodes", dev, (B,))
    _need(depth, torch.int32, "depth", dev, (B, T))
    _need(staged, kv.dtype, "staged", dev, (L, 2, B, H, T, D))
    _rows(idx, B, N, dev)
    q_out = _out(q_out, (B, T, Hq, D), kv.dtype, dev, "q_out")
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    with _On(dev) as st:
        _check(_lib.load().spec_append_round(
            _ptr(qkv), _DT[kv.dtype], B, T, Hq, _ptr(kv), L, N, H, S, D, layer, _ptr(length), _ptr(pad), _ptr(idx),
            _ptr(n_nodes), _ptr(depth), _ptr(staged), _ptr(q_weight), _ptr(k_weight), eps, _ptr(inv_freq), R,
            1 if interleaved else 0, _ptr(q_out), _ptr(flags), st))
    return q_out, flags


@_streamed
def spec_append_prompt(qkv, kv, layer, cu, pad, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                       start=None, idx=None, q_out=None, flags=None):
    """spec_append_round for packed prompts: qkv [M, Hq + 2H, D], sequence b
    in rows cu[b] .. cu[b + 1] - 1 at positions start[b] ..
    -> (q_out [M, Hq, D], flags [B] int32)."""
    dev, (L, N, H, S, D), Hq, R = _append_common(qkv, kv, layer, inv_freq, q_weight, k_weight, 1)
    M, B = qkv.shape[0], cu.shape[0] - 1
    _need(cu, torch.int32, "cu", dev, (B + 1,))
    _need(pad, torch.int32, "pad", dev, (B,))
    _need(start, torch.int32, "start", dev, (B,))
    _rows(idx, B, N, dev)
    q_out = _out(q_out, (M, Hq, D), kv.dtype, dev, "q_out")
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    with _On(dev) as st:
        _check(_lib.load().spec_append_prompt(
            _ptr(qkv), _DT[kv.dtype], M, Hq, _ptr(kv), L, N, H, S, D, layer, B, _ptr(cu), _ptr(start), _ptr(pad),
            _ptr(idx), _ptr(q_weight), _ptr(k_weight), eps, _ptr(inv_freq), R, 1 if interleaved else 0, _ptr(q_out),
            _ptr(flags), st))
    return q_out, flags


def spec_attend_workspace_bytes(T, Hq, H, D):
    return int(_lib.load().spec_attend_workspace_bytes(int(T), int(Hq), int(H), int(D)))


@_streamed
def spec_attend_round(q, kv, layer, length, pad, tree_mask=None, n_nodes=None, idx=None, staged=None, scale=None,
                      out=None, flags=None, workspace=None):
    """Attention of a round's queries q [B, T, Hq, D] over the cached prefix
    and the nodes each may see (tree_mask [B, T] int64 bit sets; None: a
    chain).  scale None: 1 / sqrt(D).  workspace: zero-filled uint8 tensor of
    spec_attend_workspace_bytes.  -> (out [B, T, Hq, D], flags [B] int32)."""
    dev, L, N, H, S, D = _cache(kv, layer)
    _need(q, kv.dtype, "q", dev)
    B, T, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError(f"q must be [B, T, Hq, {D}]")
    _need(length, torch.int32, "length", dev, (B,))
    _need(pad, torch.int32, "pad", dev, (B,))
    _need(n_nodes, torch.int32, "n_nodes", dev, (B,))
    _need(tree_mask, torch.int64, "tree_mask", dev, (B, T))
    _need(staged, kv.dtype, "staged", dev, (L, 2, B, H, T, D))
    _rows(idx, B, N, dev)
    out = _out(out, (B, T, Hq, D), kv.dtype, dev, "out")
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    lib = _lib.load()
    on = _On(dev)
    with on as st:
        ws = _ws(workspace, "attend", lib.spec_attend_workspace_bytes(T, Hq, H, D), dev, on.stream, True)
        _check(lib.spec_attend_round(
            _ptr(q), _DT[kv.dtype], B, T, Hq, _ptr(kv), L, N, H, S, D, layer, _ptr(length), _ptr(pad), _ptr(idx),
            _ptr(n_nodes), _ptr(tree_mask), _ptr(staged), 1.0 / math.sqrt(D) if scale is None else scale, _ptr(out),
            _ptr(flags), _ptr(ws), ws.numel(), st))
    return out, flags


@_streamed
def spec_attend_prompt(q, kv, layer, cu, pad, start=None, idx=None, scale=None, out=None, flags=None):
    """Causal attention of packed prompts q [M, Hq, D] over the cache that
    spec_append_prompt filled.  -> (out [M, Hq, D], flags [B] int32)."""
    dev, L, N, H, S, D = _cache(kv, layer)
    _need(q, kv.dtype, "q", dev)
    M, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError(f"q must be [M, Hq, {D}]")
    B = cu.shape[0] - 1
    _need(cu, torch.int32, "cu", dev, (B + 1,))
    _need(pad, torch.int32, "pad", dev, (B,))
    _need(start, torch.int32, "start", dev, (B,))
    _rows(idx, B, N, dev)
    out = _out(out, (M, Hq, D), kv.dtype, dev, "out")
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    with _On(dev) as st:
        _check(_lib.load().spec_attend_prompt(
            _ptr(q), _DT[kv.dtype], M, Hq, _ptr(kv), L, N, H, S, D, layer, B, _ptr(cu), _ptr(start), _ptr(pad),
            _ptr(idx), 1.0 / math.sqrt(D) if scale is None else scale, _ptr(out), _ptr(flags), st))
    return out, flags


def spec_tree_workspace_bytes(B):
    return int(_lib.load().spec_tree_workspace_bytes(int(B)))


@_streamed
def spec_verify_tree(target_logits, tokens, parent, n_nodes=None, eos_id=-1, remaining=None, out_tokens=None,
                     path=None, n_accept=None, n_emit=None, flags=None, workspace=None):
    """Greedy verification of drafted trees: target_logits [B, T, V], tokens
    and parent [B, T] int32 -> (out_tokens [B, T], path [B, T], n_accept [B],
    n_emit [B], flags [B]) int32."""
    B, T, V = target_logits.shape
    dev = target_logits.device
    _need(target_logits, None, "target_logits", dev)
    if target_logits.dtype not in _DT:
        raise ValueError(f"unsupported logits dtype {target_logits.dtype}")
    _need(tokens, torch.int32, "tokens", dev, (B, T))
    _need(parent, torch.int32, "parent", dev, (B, T))
    _need(n_nodes, torch.int32, "n_nodes", dev, (B,))
    _need(remaining, torch.int32, "remaining", dev, (B,))
    out_tokens = _out(out_tokens, (B, T), torch.int32, dev, "out_tokens")
    path = _out(path, (B, T), torch.int32, dev, "path")
    n_accept = _out(n_accept, (B,), torch.int32, dev, "n_accept")
    n_emit = _out(n_emit, (B,), torch.int32, dev, "n_emit")
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    lib = _lib.load()
    on = _On(dev)
    with on as st:
        ws = _ws(workspace, "tree", max(256, lib.spec_tree_workspace_bytes(B)), dev, on.stream, False)
        _check(lib.spec_verify_tree(
            _ptr(target_logits), _DT[target_logits.dtype], B, T, V, _ptr(tokens), _ptr(parent), _ptr(n_nodes),
            int(eos_id), _ptr(remaining), _ptr(out_tokens), _ptr(path), _ptr(n_accept), _ptr(n_emit), _ptr(flags),
            _ptr(ws), ws.numel(), st))
    return out_tokens, path, n_accept, n_emit, flags


@_streamed
def spec_commit_tree(staged, kv, length, pad, path, n_emit, idx=None, flags=None):
    """Copy the accepted path's rows from staged [L, 2, B, H, T, D] to their
    slots in kv [L, 2, N, H, S, D].  length, pad: the round's.
    -> flags [B] int32."""
    dev, L, N, H, S, D = _cache(kv, 0)
    B, T = path.shape
    _need(staged, kv.dtype, "staged", dev, (L, 2, B, H, T, D))
    _need(length, torch.int32, "length", dev, (B,))
    _need(pad, torch.int32, "pad", dev, (B,))
    _need(path, torch.int32, "path", dev)
    _need(n_emit, torch.int32, "n_emit", dev, (B,))
    _rows(idx, B, N, dev)
    flags = _out(flags, (B,), torch.int32, dev, "flags")
    with _On(dev) as st:
        _check(_lib.load().spec_commit_tree(
            _ptr(staged), _ptr(kv), _DT[kv.dtype], L, B, T, N, H, S, D, _ptr(length), _ptr(pad), _ptr(path),
            _ptr(n_emit), _ptr(idx), _ptr(flags), st))
    return flags
