"""Refusals of the forward-pass entry points, on the host (no GPU needed):
every call returns before any CUDA call."""
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


A, Q, KV, OUT, ST, ODD = at(0x10000), at(0x10000000), at(0x100000000), at(0x20000000), at(0x30000000), at(0x10001)


def append_round(lib, qkv=Q, dt=1, B=2, T=4, Hq=8, kv=KV, L=2, N=2, H=2, S=64, D=64, layer=1, length=A, pad=A, idx=None,
                 n=None, depth=None, staged=None, qw=None, kw=None, eps=1e-6, inv=A, R=64, q=OUT, flags=None):
    return lib.spec_append_round(qkv, dt, B, T, Hq, kv, L, N, H, S, D, layer, length, pad, idx, n, depth, staged, qw, kw,
                                 eps, inv, R, 0, q, flags, None)


def test_append_round_refusals(lib):
    for kw in (dict(B=-1), dict(T=0), dict(T=65), dict(Hq=7), dict(Hq=0), dict(layer=2), dict(layer=-1), dict(D=257),
               dict(D=0), dict(S=0), dict(H=0), dict(L=0), dict(N=0), dict(qkv=None), dict(kv=None), dict(q=None),
               dict(length=None), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(R=63), dict(R=66),
               dict(R=-2), dict(inv=None), dict(N=1), dict(q=Q), dict(B=1 << 27, N=1 << 27)):
        assert append_round(lib, **kw) == -1, kw
    assert append_round(lib, dt=3) == -2
    for kw in (dict(qkv=ODD), dict(kv=ODD), dict(q=at(0x20000001)), dict(length=ODD), dict(pad=ODD), dict(idx=ODD),
               dict(n=ODD), dict(depth=ODD), dict(staged=ODD), dict(qw=ODD), dict(kw=ODD), dict(inv=ODD),
               dict(flags=ODD)):
        assert append_round(lib, **kw) == -5, kw
    assert append_round(lib, B=0) == 0


def append_prompt(lib, qkv=Q, dt=1, M=9, Hq=8, kv=KV, L=2, N=2, H=2, S=64, D=64, layer=1, B=2, cu=A, start=None, pad=None,
                  idx=None, eps=1e-6, inv=A, R=64, q=OUT, flags=None):
    return lib.spec_append_prompt(qkv, dt, M, Hq, kv, L, N, H, S, D, layer, B, cu, start, pad, idx, None, None, eps, inv, R,
                                  0, q, flags, None)


def test_append_prompt_refusals(lib):
    for kw in (dict(B=-1), dict(M=-1), dict(Hq=7), dict(layer=2), dict(D=300), dict(qkv=None), dict(cu=None),
               dict(kv=None), dict(N=1), dict(R=1), dict(inv=None), dict(q=Q), dict(M=1 << 29)):
        assert append_prompt(lib, **kw) == -1, kw
    assert append_prompt(lib, dt=-1) == -2
    for kw in (dict(cu=ODD), dict(start=ODD), dict(pad=ODD), dict(idx=ODD), dict(flags=ODD), dict(qkv=ODD)):
        assert append_prompt(lib, **kw) == -5, kw
    assert append_prompt(lib, B=0) == 0


def attend_round(lib, q=Q, dt=1, B=2, T=4, Hq=8, kv=KV, L=2, N=2, H=2, S=64, D=64, layer=0, length=A, pad=None, idx=None,
                 n=None, mask=None, staged=None, scale=0.125, out=OUT, flags=None, ws=ST, wsb=1 << 30):
    return lib.spec_attend_round(q, dt, B, T, Hq, kv, L, N, H, S, D, layer, length, pad, idx, n, mask, staged, scale, out,
                                 flags, ws, wsb, None)


def test_attend_round_refusals(lib):
    for kw in (dict(B=-1), dict(T=0), dict(T=65), dict(Hq=9), dict(layer=2), dict(D=257), dict(q=None), dict(kv=None),
               dict(out=None), dict(length=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=3e38), dict(N=1), dict(out=Q), dict(B=1 << 27, N=1 << 27),
               dict(B=65537, N=65537), dict(S=(1 << 31) - 1), dict(N=1 << 30)):
        assert attend_round(lib, **kw) == -1, kw
    assert attend_round(lib, dt=9) == -2
    for kw in (dict(ws=None), dict(ws=at(0x30000010)), dict(wsb=16)):
        assert attend_round(lib, **kw) == -3, kw
    for kw in (dict(q=ODD), dict(kv=ODD), dict(out=at(0x20000001)), dict(length=ODD), dict(pad=ODD), dict(idx=ODD),
               dict(n=ODD), dict(mask=at(0x10004)), dict(staged=ODD), dict(flags=ODD)):
        assert attend_round(lib, **kw) == -5, kw
    assert attend_round(lib, B=0) == 0
    assert lib.spec_attend_workspace_bytes(0, 8, 2, 64) == 0
    assert lib.spec_attend_workspace_bytes(9, 32, 8, 128) % 256 == 0


def attend_prompt(lib, q=Q, dt=1, M=9, Hq=8, kv=KV, L=2, N=2, H=2, S=64, D=64, layer=0, B=2, cu=A, start=None, pad=None,
                  idx=None, scale=0.125, out=OUT, flags=None):
    return lib.spec_attend_prompt(q, dt, M, Hq, kv, L, N, H, S, D, layer, B, cu, start, pad, idx, scale, out, flags, None)


def test_attend_prompt_refusals(lib):
    for kw in (dict(B=-1), dict(M=-2), dict(Hq=9), dict(layer=-1), dict(D=257), dict(q=None), dict(kv=None), dict(out=None),
               dict(cu=None), dict(scale=0.0), dict(N=1), dict(out=Q), dict(M=1 << 30), dict(B=65537, N=65537)):
        assert attend_prompt(lib, **kw) == -1, kw
    assert attend_prompt(lib, dt=4) == -2
    for kw in (dict(q=ODD), dict(cu=ODD), dict(start=ODD), dict(pad=ODD), dict(idx=ODD), dict(flags=ODD)):
        assert attend_prompt(lib, **kw) == -5, kw
    assert attend_prompt(lib, B=0) == 0


def test_tree_refusals(lib):
    def plan(B=2, T=4, parent=A, n=None, mask=A, depth=A, flags=None):
        return lib.spec_tree_plan(B, T, parent, n, mask, depth, flags, None)

    for kw in (dict(B=-1), dict(T=0), dict(T=65), dict(parent=None), dict(mask=None), dict(depth=None)):
        assert plan(**kw) == -1, kw
    for kw in (dict(parent=ODD), dict(n=ODD), dict(mask=at(0x10004)), dict(depth=ODD), dict(flags=ODD)):
        assert plan(**kw) == -5, kw
    assert plan(B=0) == 0

    def verify(x=Q, dt=1, B=2, T=4, V=100, tok=A, parent=A, n=None, rem=None, out=A, path=A, na=A, ne=A, ws=ST,
               wsb=1 << 20):
        return lib.spec_verify_tree(x, dt, B, T, V, tok, parent, n, -1, rem, out, path, na, ne, None, ws, wsb, None)

    for kw in (dict(B=-1), dict(T=0), dict(T=65), dict(V=0), dict(V=(1 << 31) - 1), dict(B=65536), dict(x=None), dict(tok=None), dict(parent=None),
               dict(out=None), dict(path=None), dict(na=None), dict(ne=None)):
        assert verify(**kw) == -1, kw
    assert verify(dt=5) == -2
    for kw in (dict(ws=None), dict(wsb=8), dict(ws=ODD)):
        assert verify(**kw) == -3, kw
    for kw in (dict(x=ODD), dict(tok=ODD), dict(parent=ODD), dict(n=ODD), dict(rem=ODD), dict(out=ODD), dict(path=ODD)):
        assert verify(**kw) == -5, kw
    assert verify(B=0) == 0

    def commit(st=Q, kv=KV, dt=1, L=2, B=2, T=4, N=2, H=2, S=64, D=64, length=A, pad=None, path=A, ne=A, idx=None,
               flags=None):
        return lib.spec_commit_tree(st, kv, dt, L, B, T, N, H, S, D, length, pad, path, ne, idx, flags, None)

    for kw in (dict(L=0), dict(B=-1), dict(T=65), dict(N=0), dict(H=0), dict(S=0), dict(D=0), dict(st=None), dict(kv=None),
               dict(length=None), dict(path=None), dict(ne=None), dict(N=1), dict(st=KV), dict(B=70000, N=70000)):
        assert commit(**kw) == -1, kw
    assert commit(dt=8) == -2
    for kw in (dict(st=ODD), dict(kv=ODD), dict(length=ODD), dict(pad=ODD), dict(path=ODD), dict(ne=ODD), dict(idx=ODD),
               dict(flags=ODD)):
        assert commit(**kw) == -5, kw
    assert commit(B=0) == 0


def test_host_tensors_are_refused():
    kv = torch.zeros((1, 2, 2, 1, 16, 8))
    q = torch.zeros((2, 3, 2, 8))
    ln = torch.tensor([3, 5], dtype=torch.int32)
    par = torch.tensor([[-1, 0, 0]] * 2, dtype=torch.int32)
    cu = torch.tensor([0, 2, 3], dtype=torch.int32)
    calls = [lambda: sv.spec_tree_plan(par),
             lambda: sv.spec_append_round(torch.zeros((2, 3, 4, 8)), kv, 0, ln, None, None),
             lambda: sv.spec_append_prompt(torch.zeros((3, 4, 8)), kv, 0, cu, None, None),
             lambda: sv.spec_attend_round(q, kv, 0, ln, None),
             lambda: sv.spec_attend_prompt(q[0], kv, 0, cu, None),
             lambda: sv.spec_verify_tree(torch.zeros((2, 3, 9)), par, par),
             lambda: sv.spec_commit_tree(torch.zeros((1, 2, 2, 1, 3, 8)), kv, ln, None, par, ln)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_overlaps_are_refused(lib):
    """What a call writes within what it reads: layer 1 of kv [2, 2, 2, 2, 64, 64]
    in 16 bits begins 65536 bytes in and is as long; a staged layer of 2 x 4
    nodes begins 4096 in and ends at 8192."""
    layer1, last, staged = 0x100000000 + 65536, 0x100000000 + 131072 - 2, 0x30000000
    for x in (layer1, last):
        assert append_round(lib, qkv=at(x)) == -1
        assert append_round(lib, q=at(x)) == -1
        assert append_prompt(lib, qkv=at(x)) == -1
        assert append_prompt(lib, q=at(x)) == -1
        assert attend_round(lib, out=at(x), layer=1) == -1
        assert attend_prompt(lib, out=at(x), layer=1) == -1
    for x in (staged + 4096, staged + 8192 - 2):
        st = at(staged)
        assert append_round(lib, qkv=at(x), staged=st) == -1
        assert append_round(lib, q=at(x), staged=st) == -1
        assert attend_round(lib, out=at(x), staged=st, layer=1) == -1
    big = 1 << 30  # sizes whose bytes pass 64 bits do not wrap around
    assert attend_round(lib, out=at(0x100000000 + big), L=big, S=big, N=big // 2, H=1, Hq=4, D=256) == -1
