"""Refusals of the entry points of the paged 4-bit cache, on the host (no GPU
needed): every call returns before any CUDA call."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_28_gb300 as sv


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_28_gb300 import _lib
    from speculative_decoding_verification_28_gb300 import build as libbuild

    libbuild.build()
    return _lib.load()


def at(x):
    return ctypes.c_void_p(x)


A, Q, POOL, OUT, ST, ODD, WS = (at(x) for x in (0x10000, 0x10000000, 0x100000000, 0x20000000, 0x30000000, 0x10001, 0x40000000))
MAX = (1 << 31) - 1


def store(lib, src=Q, dt=1, L=1, N=2, H=2, S=64, D=64, pool=POOL, Lp=2, P=9, page=16, layer=1, table=A, R=2, MP=4, B=2, T=5,
          pos=A, count=A, slot=None, idx=None, row=None, path=None, flags=None):
    return lib.spec_store_pages(src, dt, L, N, H, S, D, pool, Lp, P, page, layer, table, R, MP, B, T, pos, count, slot, idx, row,
                             path, flags, None)


def load(lib, src=Q, dt=1, L=1, N=2, H=2, S=64, D=64, pool=POOL, Lp=2, P=9, page=16, layer=1, table=A, R=2, MP=4, B=2, T=5,
         pos=A, count=A, slot=None, idx=None, row=None, flags=None):
    return lib.spec_load_pages(pool, Lp, P, page, layer, src, dt, L, N, H, S, D, table, R, MP, B, T, pos, count, slot, idx, row,
                            flags, None)


@pytest.mark.parametrize("call", [store, load])
def test_rows_refusals(lib, call):
    # layer 1 of the pool: 2 * 9 * 2 blocks of 544 bytes in
    inside = at(0x100000000 + 36 * 544)
    for kw in (dict(B=-1), dict(B=65536, N=65536, R=65536), dict(T=0), dict(T=-1), dict(T=MAX), dict(L=0), dict(L=2), dict(N=0),
               dict(S=0), dict(S=MAX), dict(H=0), dict(H=65536), dict(D=0), dict(D=48), dict(D=288), dict(Lp=0), dict(P=0),
               dict(P=(1 << 24) + 1), dict(page=8), dict(page=24), dict(page=512), dict(page=0), dict(page=-16),
               dict(layer=2), dict(layer=-1), dict(R=0), dict(MP=0), dict(MP=1 << 27), dict(src=None), dict(pool=None),
               dict(table=None), dict(pos=None), dict(count=None), dict(N=1), dict(R=1), dict(src=inside),
               dict(L=300, Lp=400, H=900)):
        assert call(lib, **kw) == -1, kw
    for dt in (0, 3, -1):
        assert call(lib, dt=dt) == -2
    for kw in (dict(src=at(0x10000008)), dict(pool=at(0x100000008)), dict(table=ODD), dict(pos=ODD), dict(count=ODD),
               dict(slot=ODD), dict(idx=ODD), dict(row=ODD), dict(flags=ODD)):
        assert call(lib, **kw) == -5, kw
    assert call(lib, B=0) == 0
    if call is store:
        assert call(lib, path=A, T=65) == -1
        assert call(lib, path=ODD) == -5


def test_book_refusals(lib):
    def fork(table=A, held=A, refs=A, N=4, MP=8, P=30, page=16, B=2, src=A, dst=None, length=None, flags=None, ws=WS,
             wsb=1 << 20):
        return lib.spec_page_fork(table, held, refs, N, MP, P, page, B, src, dst, length, flags, ws, wsb, None)

    def reserve(table=A, held=A, refs=A, N=4, MP=8, P=30, page=16, B=2, first=A, total=A, idx=None, copies=A, missing=A,
                flags=None, ws=WS, wsb=1 << 20):
        return lib.spec_page_reserve(table, held, refs, N, MP, P, page, B, first, total, idx, copies, missing, flags, ws, wsb,
                                     None)

    def compact(table=A, held=A, refs=A, N=4, MP=8, P=30, moves=A, n=A, ws=WS, wsb=1 << 20):
        return lib.spec_page_compact(table, held, refs, N, MP, P, moves, n, ws, wsb, None)

    for call in (fork, reserve, compact):
        for kw in (dict(table=None), dict(held=None), dict(refs=None), dict(N=0), dict(MP=0), dict(P=0), dict(MP=1 << 28),
                   dict(P=1 << 25)):
            assert call(**kw) == -1, kw
        for kw in (dict(ws=None), dict(wsb=64), dict(ws=ODD)):
            assert call(**kw) == -3, kw
        for kw in (dict(table=ODD), dict(held=ODD), dict(refs=ODD)):
            assert call(**kw) == -5, kw
    for call in (fork, reserve):
        for kw in (dict(B=-1), dict(B=65536), dict(B=5), dict(page=17), dict(page=0)):
            assert call(**kw) == -1, kw
        assert call(B=0) == 0
        assert call(flags=ODD) == -5
    assert fork(src=None) == -1
    for kw in (dict(src=ODD), dict(dst=ODD), dict(length=ODD)):
        assert fork(**kw) == -5
    for kw in (dict(first=None), dict(total=None), dict(copies=None), dict(missing=None)):
        assert reserve(**kw) == -1
    for kw in (dict(first=ODD), dict(total=ODD), dict(copies=ODD), dict(missing=ODD), dict(idx=ODD)):
        assert reserve(**kw) == -5
    for kw in (dict(moves=None), dict(n=None)):
        assert compact(**kw) == -1
    for kw in (dict(moves=ODD), dict(n=ODD)):
        assert compact(**kw) == -5
    assert lib.spec_page_workspace_bytes(-1, 4, 4) == 0 and lib.spec_page_workspace_bytes(3, 0, 4) == 0
    assert lib.spec_page_workspace_bytes(3, 4, 5) % 256 == 0


def test_copy_refusals(lib):
    def copy(pool=POOL, slabs=4, P=9, size=1088, pairs=A, M=3, n=None, err=None):
        return lib.spec_page_copy(pool, slabs, P, size, pairs, M, n, err, None)

    for kw in (dict(slabs=-1), dict(P=0), dict(size=0), dict(size=24), dict(size=8), dict(M=-1), dict(pool=None),
               dict(pairs=None), dict(P=1 << 25), dict(size=1 << 32), dict(slabs=MAX, size=1 << 20)):
        assert copy(**kw) == -1, kw
    for kw in (dict(pool=at(0x100000004)), dict(pairs=ODD), dict(n=ODD), dict(err=ODD)):
        assert copy(**kw) == -5, kw
    assert copy(M=0) == 0


def attend(lib, q=Q, dt=1, B=2, T=4, Hq=8, pool=POOL, L=2, P=9, H=2, page=16, D=64, layer=1, table=A, R=2, MP=4, length=A,
           idx=None, n=None, mask=None, staged=ST, scale=0.125, out=OUT, flags=None, ws=WS, wsb=1 << 30):
    return lib.spec_attend_pages(q, dt, B, T, Hq, pool, L, P, H, page, D, layer, table, R, MP, length, idx, n, mask, staged,
                                    scale, out, flags, ws, wsb, None)


def test_attend_refusals(lib):
    inside, in_nodes = at(0x100000000 + 36 * 544 + 32), at(0x30000000 + 4096)
    for kw in (dict(B=-1), dict(T=0), dict(T=65), dict(Hq=9), dict(Hq=0), dict(L=0), dict(layer=2), dict(layer=-1), dict(P=0),
               dict(H=0), dict(page=20), dict(D=32), dict(D=96), dict(D=256), dict(D=0), dict(R=0), dict(MP=0), dict(R=1),
               dict(MP=1 << 27), dict(q=None), dict(pool=None), dict(table=None), dict(length=None), dict(staged=None),
               dict(out=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=3e38), dict(out=Q), dict(out=inside), dict(out=in_nodes), dict(B=65537, R=65537),
               dict(B=60000, R=60000, MP=1 << 17)):
        assert attend(lib, **kw) == -1, kw
    for dt in (0, 9):
        assert attend(lib, dt=dt) == -2
    for kw in (dict(ws=None), dict(ws=at(0x40000010)), dict(wsb=16)):
        assert attend(lib, **kw) == -3, kw
    for kw in (dict(q=at(0x10000002)), dict(pool=at(0x100000008)), dict(out=at(0x20000004)), dict(staged=at(0x30000002)),
               dict(table=ODD), dict(length=ODD), dict(idx=ODD), dict(n=ODD), dict(mask=at(0x10004)), dict(flags=ODD)):
        assert attend(lib, **kw) == -5, kw
    assert attend(lib, B=0) == 0
    assert lib.spec_attend_pages_workspace_bytes(0, 8, 2, 64) == 0
    assert lib.spec_attend_pages_workspace_bytes(9, 32, 8, 128) % 256 == 0


def test_block_bytes():
    assert sv.q4_block_bytes(64, 128) == 64 * 68 and sv.q4_block_bytes(16, 32) == 272
    for page, D in ((8, 64), (48, 64), (64, 40), (64, 0)):
        with pytest.raises(ValueError):
            sv.q4_block_bytes(page, D)


def test_host_tensors_are_refused():
    pool = torch.zeros((1, 2, 3, 1, 544), dtype=torch.uint8)
    kv = torch.zeros((1, 2, 2, 1, 3, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    table, refs = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    calls = [lambda: sv.spec_page_fork(table, i, refs, i, 16),
             lambda: sv.spec_page_reserve(table, i, refs, i, i, 16),
             lambda: sv.spec_page_compact(table, i, refs),
             lambda: sv.spec_page_copy(pool, table),
             lambda: sv.spec_store_pages(kv, pool, table, i, i),
             lambda: sv.spec_load_pages(pool, kv, table, i, i),
             lambda: sv.spec_attend_pages(torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16), pool, 0, table, i, kv)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_nodes_without_a_cache(lib):
    from test_forward_boundary import ODD as odd
    from test_forward_boundary import ST, append_round

    # the checks of the cache are the staged block's then
    assert append_round(lib, kv=None) == -1
    for kw in (dict(q=None), dict(N=1), dict(S=0), dict(qkv=ST), dict(q=ST)):
        assert append_round(lib, kv=None, staged=ST, **kw) == -1, kw
    assert append_round(lib, kv=None, staged=odd) == -5
    assert append_round(lib, kv=None, staged=ST, B=0) == 0


def test_units_are_counted_with_their_starts(lib):
    # 288 million units of two tiles: ten tiles each are counted
    far = dict(q=at(1 << 44), out=at(1 << 45), staged=at(1 << 46))
    assert attend(lib, B=60000, R=60000, H=4800, Hq=4800, T=1, MP=1, page=16, L=1, layer=0, **far) == -1
    assert attend(lib, B=60000, R=60000, H=1200, Hq=1200, T=1, MP=1, page=16, L=1, layer=0, wsb=16, **far) == -3
