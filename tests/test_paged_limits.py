"""Limits of the paged cache's entry points that the host sees (no GPU needed):
every call returns before any CUDA call."""
import pytest

from test_paged_boundary import A, ODD, POOL, Q, at, attend, lib, store  # noqa: F401


def store_reserved(lib, src=Q, dt=1, L=1, N=2, H=2, S=64, D=64, pool=POOL, Lp=2, P=9, page=16, layer=1, table=A, R=2, MP=4,
                   B=2, T=5, pos=A, count=A, slot=None, idx=None, row=None, path=None, missing=A, flags=None):
    return lib.spec_store_pages_reserved(src, dt, L, N, H, S, D, pool, Lp, P, page, layer, table, R, MP, B, T, pos, count,
                                         slot, idx, row, path, missing, flags, None)


@pytest.mark.parametrize("missing", [A, None])
def test_a_store_behind_a_reservation_refuses_what_a_store_refuses(lib, missing):  # noqa: F811
    inside = at(0x100000000 + 36 * 544)
    for kw in (dict(B=-1), dict(T=0), dict(L=0), dict(L=2), dict(H=65536), dict(D=48), dict(P=0), dict(page=24), dict(layer=2),
               dict(MP=1 << 27), dict(src=None), dict(pool=None), dict(table=None), dict(pos=None), dict(count=None),
               dict(N=1), dict(R=1), dict(src=inside), dict(path=A, T=65), dict(dt=0), dict(src=at(0x10000008)),
               dict(pos=ODD), dict(path=ODD), dict(flags=ODD), dict(B=0)):
        assert store_reserved(lib, missing=missing, **kw) == store(lib, **kw), kw
    assert store_reserved(lib, missing=ODD) == -5


def test_scales_that_fp16_scores_cannot_be_taken_to_base_2_with(lib):  # noqa: F811
    # 128 * 1.4427 times the scale has to be finite for fp16, the scale's 1.4427-fold for bf16
    assert attend(lib, dt=2, scale=1.9e36) == -1 and attend(lib, dt=2, scale=3e38) == -1
    assert attend(lib, dt=2, scale=1.8e36, wsb=16) == -3
    assert attend(lib, dt=1, scale=2e38, wsb=16) == -3 and attend(lib, dt=1, scale=3e38) == -1


def test_pages_copied_are_counted_by_the_chunks_of_a_launch(lib):  # noqa: F811
    """The last sizes within the limits get as far as the check of addresses, the next ones do not."""
    def copy(**kw):
        a = dict(pool=at(0x100000004), slabs=4, P=9, size=1088, M=3)
        a.update(kw)
        return lib.spec_page_copy(a["pool"], a["slabs"], a["P"], a["size"], A, a["M"], None, None, None)

    most = (1 << 31) - 1
    assert copy(slabs=most, size=464) == -5 and copy(slabs=most, size=480) == -1  # 10^12 bytes of a page
    assert copy(slabs=465, size=1 << 31) == -5 and copy(slabs=466, size=1 << 31) == -1
    assert copy(size=(1 << 31) + 16) == -1 and copy(P=1 << 24) == -5 and copy(M=1 << 24) == -5 and copy(M=(1 << 24) + 1) == -1
