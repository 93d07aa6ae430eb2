"""Binding of the paged 4-bit cache: pages forked, reserved, compacted and
copied, rows stored and loaded, attention of a round over them.  Names, checks,
streams and scratch are as in forward.py; definitions and layouts are in
include/specverify.h.
"""
from __future__ import annotations

import torch

from . import _lib
from .api import _DT, _need
from .forward import ATTEND_ZERO, _I32, _at, _call, _out, _streamed, _ws

Q4_GROUP = 32
PAGE_SIZES = (16, 32, 64, 128, 256)
_HALVES = (torch.bfloat16, torch.float16)


def q4_block_bytes(page, D):
    """Bytes of a block of a pool [L, 2, P, H, block]."""
    if page not in PAGE_SIZES or D < 1 or D % Q4_GROUP:
        raise ValueError(f"pages of {PAGE_SIZES} tokens and heads of a multiple of {Q4_GROUP}, not {page} and {D}")
    return page * 17 * D // 32


_page_of = {}  # tokens of a page by (bytes of a block, head size)


def _pool(pool, dev, H, D, layer, layers):
    """Checked pool -> (address, L, P, page)."""
    shape = pool.shape
    if len(shape) != 5 or shape[1] != 2 or shape[3] != H:
        raise ValueError(f"pool must be [L, 2, P, {H}, block]")
    at = _at(pool, torch.uint8, "pool", dev, shape)
    L, _, P, _, block = shape
    page = _page_of.get((block, D))
    if page is None:
        page = block * 32 // (17 * D) if D else 0
        if q4_block_bytes(page, D) != block:
            raise ValueError(f"a block of {block} bytes holds no whole number of tokens of heads of {D}")
        _page_of[block, D] = page
    if not 0 <= layer <= L - layers:
        raise ValueError(f"layers {layer} .. {layer + layers - 1} of {L}")
    return at, L, P, page


def _table(table, dev):
    """Checked table [R, MP] -> (address, R, MP)."""
    shape = table.shape
    if len(shape) != 2:
        raise ValueError("table must be [R, MP]")
    return _at(table, _I32, "table", dev, shape), shape[0], shape[1]


def _rows_of(given, B, most, dev, name):
    if given is None and B > most:
        raise ValueError(f"{B} sequences on {most} rows: pass {name}")
    return _at(given, _I32, name, dev, (B,))


def spec_page_workspace_bytes(B, MP, P):
    return int(_lib.load().spec_page_workspace_bytes(int(B), int(MP), int(P)))


_book_bytes = {}  # spec_page_workspace_bytes by its arguments


def _book(table, held, refs, B, workspace):
    """Checked table, held and refs -> (device, sizes, addresses, workspace)."""
    dev = table.device
    if not table.is_cuda:
        _need(table, None, "table")
    at, N, MP = _table(table, dev)
    P = refs.numel()
    held_at, refs_at = _at(held, _I32, "held", dev, (N,)), _at(refs, _I32, "refs", dev, (P,))
    need = _book_bytes.get((B, MP, P))
    if need is None:
        if B > 65535:
            raise ValueError(f"{B} sequences in a call")
        if len(_book_bytes) >= 4096:  # whoever has ever new sizes
            _book_bytes.clear()
        need = _book_bytes[B, MP, P] = spec_page_workspace_bytes(B, MP, P)
    return dev, (N, MP, P), (at, held_at, refs_at), _ws(workspace, "pages", need, dev, 0)


@_streamed
def spec_page_fork(table, held, refs, src, page, dst=None, length=None, flags=None, workspace=None):
    """Row dst[b] (None: b) of table [N, MP] becomes a fork of row src[b] (-1:
    nothing, the row is freed) with its pages for length[b] tokens (None: all).
    table, held [N] and refs [P] int32 are changed in place.  -> flags [B]."""
    B = src.shape[0]
    dev, (N, MP, P), book, ws = _book(table, held, refs, B, workspace)
    rows = B,
    src_at = _at(src, _I32, "src", dev, rows)
    flags = _out(flags, rows, _I32, dev, "flags", src)
    _call(_lib.load().spec_page_fork, dev, *book, N, MP, P, int(page), B, src_at, _rows_of(dst, B, N, dev, "dst"),
          _at(length, _I32, "length", dev, rows), flags.data_ptr(), ws.data_ptr(), ws.numel())
    return flags


@_streamed
def spec_page_reserve(table, held, refs, first, total, page, idx=None, copies=None, missing=None, flags=None,
                      workspace=None):
    """Pages for total[b] tokens in row idx[b] (None: b), of which those from
    first[b] on will be written and so are named by no other row.  missing: the
    pages that the pool lacked, where no row has got any (see spec_store_pages).
    -> (copies [B, 2] for spec_page_copy, missing [1], flags [B])."""
    B = first.shape[0]
    dev, (N, MP, P), book, ws = _book(table, held, refs, B, workspace)
    rows = B,
    first_at, total_at = _at(first, _I32, "first", dev, rows), _at(total, _I32, "total", dev, rows)
    copies = _out(copies, (B, 2), _I32, dev, "copies")
    if missing is None:
        missing = torch.empty(1, dtype=_I32, device=dev)
    missing_at = _at(missing, _I32, "missing", dev, (1,))
    if B == 0:  # for which the C call does nothing
        missing.zero_()
    flags = _out(flags, rows, _I32, dev, "flags", first)
    _call(_lib.load().spec_page_reserve, dev, *book, N, MP, P, int(page), B, first_at, total_at,
          _rows_of(idx, B, N, dev, "idx"), copies.data_ptr(), missing_at, flags.data_ptr(), ws.data_ptr(), ws.numel())
    return copies, missing, flags


@_streamed
def spec_page_compact(table, held, refs, moves=None, n_moves=None, workspace=None):
    """Live pages take the lowest numbers.  -> (moves [P, 2], n_moves [1]) for
    spec_page_copy."""
    dev, (N, MP, P), book, ws = _book(table, held, refs, 0, workspace)
    moves = _out(moves, (P, 2), _I32, dev, "moves")
    n_moves = _out(n_moves, (1,), _I32, dev, "n_moves")
    _call(_lib.load().spec_page_compact, dev, *book, N, MP, P, moves.data_ptr(), n_moves.data_ptr(), ws.data_ptr(),
          ws.numel())
    return moves, n_moves


@_streamed
def spec_page_copy(pool, pairs, n_pairs=None, err=None):
    """Copies whole pages of pool [L, 2, P, ...] (any contiguous tensor) by
    pairs [M, 2] (from, to; -1: none), the first n_pairs[0] of them.
    -> err [1]: pairs outside the pool."""
    shape = pool.shape
    if not pool.is_cuda or not pool.is_contiguous():
        _need(pool, None, "pool")
    if len(shape) < 4:
        raise ValueError("pool must be [L, 2, P, ...]")
    dev, L, two, P = pool.device, shape[0], shape[1], shape[2]
    if pairs.dim() != 2:
        raise ValueError("pairs must be [M, 2]")
    M = pairs.shape[0]
    pairs_at = _at(pairs, _I32, "pairs", dev, (M, 2))
    if err is None:
        err = torch.empty(1, dtype=_I32, device=dev)
    blocks = L * two * P
    _call(_lib.load().spec_page_copy, dev, pool.data_ptr(), L * two, P, pool.nbytes // blocks if blocks else 0, pairs_at, M,
          _at(n_pairs, _I32, "n_pairs", dev, (1,)), _at(err, _I32, "err", dev, (1,)))
    return err


def _rows16(t, name):
    shape = t.shape
    if len(shape) != 6 or shape[1] != 2:
        raise ValueError(f"{name} must be [L, 2, N, H, S, D]")
    if not t.is_cuda or not t.is_contiguous():
        _need(t, None, name)
    if t.dtype not in _HALVES:
        raise ValueError(f"unsupported {name} dtype {t.dtype}: bf16 or fp16")
    L, _, N, H, S, D = shape
    return t.device, L, N, H, S, D


@_streamed
def spec_store_pages(src, pool, table, pos, count, layer=0, slot=None, idx=None, row=None, path=None, flags=None,
                     missing=None):
    """Rows slot[b] + j (or + path[b, j]), j < count[b], of src [L, 2, N, H, S,
    D] row idx[b] -> positions pos[b] + j of table row row[b], layers layer ..
    of pool.  missing [1] of the reservation before it: where that is not 0,
    nothing is stored and all are flagged.  -> flags [B]."""
    dev, L, N, H, S, D = _rows16(src, "src")
    pool_at, Lp, P, page = _pool(pool, dev, H, D, layer, L)
    table_at, R, MP = _table(table, dev)
    B = pos.shape[0]
    rows = B,
    T = S if path is None else path.shape[-1]
    pos_at = _at(pos, _I32, "pos", dev, rows)
    flags = _out(flags, rows, _I32, dev, "flags", pos)
    _call(_lib.load().spec_store_pages_reserved, dev, src.data_ptr(), _DT[src.dtype], L, N, H, S, D, pool_at, Lp, P,
          page, layer, table_at, R, MP, B, T, pos_at, _at(count, _I32, "count", dev, rows),
          _at(slot, _I32, "slot", dev, rows), _rows_of(idx, B, N, dev, "idx"), _rows_of(row, B, R, dev, "row"),
          _at(path, _I32, "path", dev, (B, T)), _at(missing, _I32, "missing", dev, (1,)), flags.data_ptr())
    return flags


@_streamed
def spec_load_pages(pool, dst, table, pos, count, layer=0, slot=None, idx=None, row=None, flags=None):
    """Positions pos[b] + j, j < count[b], of table row row[b] -> rows slot[b] +
    j of dst [L, 2, N, H, S, D] row idx[b].  -> flags [B]."""
    dev, L, N, H, S, D = _rows16(dst, "dst")
    pool_at, Lp, P, page = _pool(pool, dev, H, D, layer, L)
    table_at, R, MP = _table(table, dev)
    B = pos.shape[0]
    rows = B,
    pos_at = _at(pos, _I32, "pos", dev, rows)
    flags = _out(flags, rows, _I32, dev, "flags", pos)
    _call(_lib.load().spec_load_pages, dev, pool_at, Lp, P, page, layer, dst.data_ptr(), _DT[dst.dtype], L, N,
          H, S, D, table_at, R, MP, B, S, pos_at, _at(count, _I32, "count", dev, rows),
          _at(slot, _I32, "slot", dev, rows), _rows_of(idx, B, N, dev, "idx"), _rows_of(row, B, R, dev, "row"),
          flags.data_ptr())
    return flags


_attend_bytes = {}  # spec_attend_pages_workspace_bytes by D, the only argument that it depends on


def spec_attend_pages_workspace_bytes(T, Hq, H, D):
    return int(_lib.load().spec_attend_pages_workspace_bytes(int(T), int(Hq), int(H), int(D)))


@_streamed
def spec_attend_pages(q, pool, layer, table, length, staged, tree_mask=None, n_nodes=None, idx=None, scale=None,
                      out=None, flags=None, workspace=None):
    """Attention of a round's queries q [B, T, Hq, D] over the prefix in pages
    (positions 0 .. length - 2 of table row idx[b]; None: b) and the nodes in
    staged [L, 2, B, H, T, D] that each may see.  -> (out [B, T, Hq, D], flags [B])."""
    dev, shape, dt = q.device, q.shape, q.dtype
    B, T, Hq, D = shape
    if staged.dim() != 6:
        raise ValueError("staged must be [L, 2, B, H, T, D]")
    H = staged.shape[3]
    if not q.is_cuda or not q.is_contiguous():
        _need(q, None, "q")
    if dt not in _HALVES:
        raise ValueError(f"unsupported q dtype {dt}: bf16 or fp16")
    pool_at, L, P, page = _pool(pool, dev, H, D, layer, 1)
    table_at, R, MP = _table(table, dev)
    rows = B,
    length_at = _at(length, _I32, "length", dev, rows)
    out = _out(out, shape, dt, dev, "out", q)
    flags = _out(flags, rows, _I32, dev, "flags", length)
    lib = _lib.load()
    need = _attend_bytes.get(D)
    if need is None:
        need = lib.spec_attend_pages_workspace_bytes(T, Hq, H, D)
        if need:
            _attend_bytes[D] = need
    ws = _ws(workspace, "attend", need, dev, ATTEND_ZERO)
    _call(lib.spec_attend_pages, dev, q.data_ptr(), _DT[dt], B, T, Hq, pool_at, L, P, H, page, D, layer,
          table_at, R, MP, length_at, _rows_of(idx, B, R, dev, "idx"), _at(n_nodes, _I32, "n_nodes", dev, rows),
          _at(tree_mask, torch.int64, "tree_mask", dev, (B, T)), _at(staged, dt, "staged", dev, (L, 2, B, H, T, D)),
          D ** -0.5 if scale is None else scale, out.data_ptr(), flags.data_ptr(), ws.data_ptr(), ws.numel())
    return out, flags
