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
so captured graphs share none and may be replayed side by side.  After an attention
call that reported FLAG_TIMEOUT (never expected) spec_attend_reset makes a
stream's buffer good again.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from .api import _DT, _check, _need

FLAG_BAD_STATE, FLAG_BAD_TREE, FLAG_TIMEOUT = 16, 32, 64
MAX_NODES = 64
MAX_HEAD_DIM = 256
ATTEND_ZERO = 2048


# absent from builds without CUDA
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device_now = getattr(torch._C, "_cuda_getDevice", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)


def _streamed(fn):
    """Runs fn with `stream` current, so that outputs and scratch it allocates
    belong to the stream that writes them."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.device != stream.device:
                raise ValueError(f"stream on {stream.device}, a tensor on {t.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)

    return call


def _call(fn, dev, *args):
    """fn(*args, the current stream of dev), with dev the current device."""
    i = dev.index
    if _device_now() == i:
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(i))
    if rc:
        _check(rc)


def _at(t, dtype, name, dev, shape):
    """Address of a tensor that is what it has to be (None: null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _need(t, dtype, name, dev, shape)  # says what is wrong
    return t.data_ptr()


def _out(t, shape, dtype, dev, name, like=None):
    """t checked, or when None a new tensor; like: a checked tensor of the same
    kind, where there is one (allocations are half of a small call's time, and
    this one is shorter)."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else torch.empty_like(like)
    _at(t, dtype, name, dev, shape)
    return t


_scratch = {}


def _ws(given, kind, nbytes, device, head):
    """Scratch of at least nbytes for the current stream; when new, its first
    `head` bytes are cleared."""
    if given is not None:
        buf = getattr(given, "buf", given)
        _need(buf, torch.uint8, "workspace", device)
        return buf
    if _device_now() != device.index:
        with torch.cuda.device(device):
            return _ws(given, kind, nbytes, device, head)
    capturing = _capturing()
    if not capturing:
        key = kind, device.index, _raw_stream(device.index)
        buf = _scratch.get(key)
        if buf is not None and buf.numel() >= nbytes:
            return buf
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if head:
        buf[:head].zero_()
    if not capturing:
        _scratch[key] = buf
    return buf


def _cache(kv, layer, name="kv"):
    if kv.dim() != 6 or kv.shape[1] != 2:
        raise ValueError(f"{name} must be [L, 2, N, H, S, D]")
    if not kv.is_cuda or not kv.is_contiguous():
        _need(kv, None, name)
    if kv.dtype not in _DT:
        raise ValueError(f"unsupported {name} dtype {kv.dtype}")
    L, _, N, H, S, D = kv.shape
    if not 0 <= layer < L:
        raise ValueError(f"layer {layer} of {L}")
    return kv.device, L, N, H, S, D


def _rows(idx, B, N, dev):
    if idx is None and B > N:
        raise ValueError(f"{B} sequences in a cache of {N} rows: pass idx")
    return _at(idx, _I32, "idx", dev, (B,))


_I32 = torch.int32


@_streamed
def spec_tree_plan(parent, n_nodes=None, mask=None, depth=None, flags=None):
    """parent [B, T] int32 -> (mask [B, T] int64 bit sets, depth [B, T] int32,
    flags [B] int32)."""
    B, T = parent.shape
    dev = parent.device
    _need(parent, _I32, "parent", dev)
    n = _at(n_nodes, _I32, "n_nodes", dev, (B,))
    mask = _out(mask, (B, T), torch.int64, dev, "mask")
    depth = _out(depth, (B, T), _I32, dev, "depth")
    flags = _out(flags, (B,), _I32, dev, "flags")
    _call(_lib.load().spec_tree_plan, dev, B, T, parent.data_ptr(), n, mask.data_ptr(), depth.data_ptr(),
          flags.data_ptr())
    return mask, depth, flags


def _append_common(qkv, kv, layer, inv_freq, q_weight, k_weight, lead, name="kv"):
    dev, L, N, H, S, D = _cache(kv, layer, name)
    dt = kv.dtype
    shape = qkv.shape
    if len(shape) != lead + 2 or shape[-1] != D or shape[-2] <= 2 * H:
        raise ValueError(f"qkv must end in [Hq + 2 * {H}, {D}]")
    inv, R = None, 0
    if inv_freq is not None:
        _need(inv_freq, torch.float32, "inv_freq", dev)
        inv, R = inv_freq.data_ptr(), 2 * inv_freq.numel()
        if R > D:
            raise ValueError(f"inv_freq turns {R} of {D} dimensions")
    return (dev, dt, (L, N, H, S, D), shape[-2] - 2 * H, _at(qkv, dt, "qkv", dev, shape),
            _at(q_weight, dt, "q_weight", dev, (D,)), _at(k_weight, dt, "k_weight", dev, (D,)), inv, R)


@_streamed
def spec_append_round(qkv, kv, layer, length, pad, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                      interleaved=False, depth=None, n_nodes=None, idx=None, staged=None, q_out=None, flags=None):
    """qkv [B, T, Hq + 2H, D] of a round's nodes: per-head RMS norm of queries
    and keys, rotation, keys and values to the cache kv [L, 2, N, H, S, D] (or
    to staged [L, 2, B, H, T, D], where kv may be None: a prefix in pages, whose
    rows idx names).  pad None: 0.
    -> (q_out [B, T, Hq, D], flags [B] int32)."""
    paged = kv is None and staged is not None
    at, name = (staged, "staged") if paged else (kv, "kv")
    dev, dt, (L, N, H, S, D), Hq, x, qw, kw, inv, R = _append_common(qkv, at, layer, inv_freq, q_weight, k_weight, 2, name)
    B, T = qkv.shape[:2]
    if paged:  # the table's rows and lengths, which this call does not see: what it may count
        N, S = (2 ** 30 - 1) // H, 2 ** 31 - 257
    rows = B,
    length_at = _at(length, _I32, "length", dev, rows)
    q_out = _out(q_out, (B, T, Hq, D), dt, dev, "q_out")
    flags = _out(flags, rows, _I32, dev, "flags", length)
    _call(_lib.load().spec_append_round, dev, x, _DT[dt], B, T, Hq, None if paged else kv.data_ptr(), L, N, H, S, D, layer,
          length_at, _at(pad, _I32, "pad", dev, rows), _rows(idx, B, N, dev),
          _at(n_nodes, _I32, "n_nodes", dev, rows), _at(depth, _I32, "depth", dev, (B, T)),
          _at(staged, dt, "staged", dev, (L, 2, B, H, T, D)), qw, kw, eps, inv, R, 1 if interleaved else 0,
          q_out.data_ptr(), flags.data_ptr())
    return q_out, flags


@_streamed
def spec_append_prompt(qkv, kv, layer, cu, pad, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                       start=None, idx=None, q_out=None, flags=None):
    """spec_append_round for packed prompts: qkv [M, Hq + 2H, D], sequence b
    in rows cu[b] .. cu[b + 1] - 1 at positions start[b] ..
    -> (q_out [M, Hq, D], flags [B] int32)."""
    dev, dt, (L, N, H, S, D), Hq, x, qw, kw, inv, R = _append_common(qkv, kv, layer, inv_freq, q_weight, k_weight, 1)
    M, B = qkv.shape[0], cu.shape[0] - 1
    rows = B,
    q_out = _out(q_out, (M, Hq, D), dt, dev, "q_out")
    flags = _out(flags, rows, _I32, dev, "flags")
    _call(_lib.load().spec_append_prompt, dev, x, _DT[dt], M, Hq, kv.data_ptr(), L, N, H, S, D, layer, B,
          _at(cu, _I32, "cu", dev, (B + 1,)), _at(start, _I32, "start", dev, rows), _at(pad, _I32, "pad", dev, rows),
          _rows(idx, B, N, dev), qw, kw, eps, inv, R, 1 if interleaved else 0, q_out.data_ptr(), flags.data_ptr())
    return q_out, flags


_attend_bytes = {}  # spec_attend_workspace_bytes by its arguments


def spec_attend_workspace_bytes(T, Hq, H, D):
    return int(_lib.load().spec_attend_workspace_bytes(int(T), int(Hq), int(H), int(D)))


@_streamed
def spec_attend_reset(device=None):
    """After a spec_attend_round that reported FLAG_TIMEOUT: clears the head of
    the scratch kept for the current stream (or stream=) of the device (default:
    the current one), which every round on that stream reports FLAG_TIMEOUT for
    until then.  A workspace of one's own: workspace[:ATTEND_ZERO].zero_()."""
    i = None if device is None else torch.device(device).index
    i = _device_now() if i is None else i
    buf = _scratch.get(("attend", i, _raw_stream(i)))
    if buf is not None:
        buf[:ATTEND_ZERO].zero_()


@_streamed
def spec_attend_round(q, kv, layer, length, pad, tree_mask=None, n_nodes=None, idx=None, staged=None, scale=None,
                      out=None, flags=None, workspace=None):
    """Attention of a round's queries q [B, T, Hq, D] over the cached prefix
    and the nodes each may see (tree_mask [B, T] int64 bit sets; None: a
    chain).  scale None: 1 / sqrt(D).  workspace: uint8 tensor of
    spec_attend_workspace_bytes, its first ATTEND_ZERO bytes zero.  -> (out [B, T, Hq, D], flags [B] int32)."""
    dev, L, N, H, S, D = _cache(kv, layer)
    dt, shape = kv.dtype, q.shape
    B, T, Hq, Dq = shape
    if Dq != D:
        raise ValueError(f"q must be [B, T, Hq, {D}]")
    rows = B,
    q_at, length_at = _at(q, dt, "q", dev, shape), _at(length, _I32, "length", dev, rows)
    out = _out(out, shape, dt, dev, "out", q)
    flags = _out(flags, rows, _I32, dev, "flags", length)
    lib = _lib.load()
    need = _attend_bytes.get((T, Hq, H, D))
    if need is None:
        need = _attend_bytes[T, Hq, H, D] = lib.spec_attend_workspace_bytes(T, Hq, H, D)
    ws = _ws(workspace, "attend", need, dev, ATTEND_ZERO)
    _call(lib.spec_attend_round, dev, q_at, _DT[dt], B, T, Hq, kv.data_ptr(), L, N, H, S, D,
          layer, length_at, _at(pad, _I32, "pad", dev, rows), _rows(idx, B, N, dev),
          _at(n_nodes, _I32, "n_nodes", dev, rows), _at(tree_mask, torch.int64, "tree_mask", dev, (B, T)),
          _at(staged, dt, "staged", dev, (L, 2, B, H, T, D)), D ** -0.5 if scale is None else scale, out.data_ptr(),
          flags.data_ptr(), ws.data_ptr(), ws.numel())
    return out, flags


@_streamed
def spec_attend_prompt(q, kv, layer, cu, pad, start=None, idx=None, scale=None, out=None, flags=None):
    """Causal attention of packed prompts q [M, Hq, D] over the cache that
    spec_append_prompt filled.  -> (out [M, Hq, D], flags [B] int32)."""
    dev, L, N, H, S, D = _cache(kv, layer)
    dt, shape = kv.dtype, q.shape
    M, Hq, Dq = shape
    if Dq != D:
        raise ValueError(f"q must be [M, Hq, {D}]")
    B = cu.shape[0] - 1
    rows = B,
    q_at = _at(q, dt, "q", dev, shape)
    out = _out(out, shape, dt, dev, "out", q)
    flags = _out(flags, rows, _I32, dev, "flags")
    _call(_lib.load().spec_attend_prompt, dev, q_at, _DT[dt], M, Hq, kv.data_ptr(), L, N, H, S,
          D, layer, B, _at(cu, _I32, "cu", dev, (B + 1,)), _at(start, _I32, "start", dev, rows),
          _at(pad, _I32, "pad", dev, rows), _rows(idx, B, N, dev), D ** -0.5 if scale is None else scale,
          out.data_ptr(), flags.data_ptr())
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
    dev, dt = target_logits.device, target_logits.dtype
    _need(target_logits, None, "target_logits", dev)
    if dt not in _DT:
        raise ValueError(f"unsupported logits dtype {dt}")
    rows, nodes = (B,), (B, T)
    parent_at = _at(parent, _I32, "parent", dev, nodes)
    out_tokens = _out(out_tokens, nodes, _I32, dev, "out_tokens", parent)
    path = _out(path, nodes, _I32, dev, "path", parent)
    n_accept = _out(n_accept, rows, _I32, dev, "n_accept")
    n_emit = _out(n_emit, rows, _I32, dev, "n_emit", n_accept)
    flags = _out(flags, rows, _I32, dev, "flags", n_accept)
    lib = _lib.load()
    ws = _ws(workspace, "tree", 256 * B, dev, 0)  # at least what the call needs
    _call(lib.spec_verify_tree, dev, target_logits.data_ptr(), _DT[dt], B, T, V, _at(tokens, _I32, "tokens", dev, nodes),
          parent_at, _at(n_nodes, _I32, "n_nodes", dev, rows), int(eos_id),
          _at(remaining, _I32, "remaining", dev, rows), out_tokens.data_ptr(), path.data_ptr(), n_accept.data_ptr(),
          n_emit.data_ptr(), flags.data_ptr(), ws.data_ptr(), ws.numel())
    return out_tokens, path, n_accept, n_emit, flags


@_streamed
def spec_commit_tree(staged, kv, length, pad, path, n_emit, idx=None, flags=None):
    """Copy the accepted path's rows from staged [L, 2, B, H, T, D] to their
    slots in kv [L, 2, N, H, S, D].  length, pad: the round's.
    -> flags [B] int32."""
    dev, L, N, H, S, D = _cache(kv, 0)
    dt = kv.dtype
    B, T = path.shape
    rows = B,
    length_at = _at(length, _I32, "length", dev, rows)
    flags = _out(flags, rows, _I32, dev, "flags", length)
    _call(_lib.load().spec_commit_tree, dev, _at(staged, dt, "staged", dev, (L, 2, B, H, T, D)), kv.data_ptr(), _DT[dt],
          L, B, T, N, H, S, D, length_at, _at(pad, _I32, "pad", dev, rows),
          _at(path, _I32, "path", dev, (B, T)), _at(n_emit, _I32, "n_emit", dev, rows), _rows(idx, B, N, dev),
          flags.data_ptr())
    return flags
