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


def test_work_is_counted_by_what_tables_can_hold(lib):  # noqa: F811
    """B H ceil(T G / 8) (ceil(MP page / 64) + 9) below 2^31, whatever the lengths are."""
    far = dict(q=at(1 << 44), out=at(1 << 45), staged=at(1 << 46), L=1, layer=0, P=9, wsb=16)
    for B, H, G, T, page, MP in ((512, 8, 4, 8, 64, 112500), (1, 1, 1, 1, 256, (1 << 23) - 600), (4096, 2, 9, 7, 256, 1000),
                                 (60000, 8, 1, 64, 16, 4)):
        count = lambda mp: B * H * -(-T * G // 8) * (-(-mp * page // 64) + 9)  # noqa: E731, B023
        while count(MP + 64) < 1 << 31 and (MP + 64) * page <= (1 << 31) - 1 - 8192:
            MP += 64
        assert attend(lib, B=B, R=B, H=H, Hq=H * G, T=T, page=page, MP=MP, **far) == (-3 if count(MP) < 1 << 31 else -1)
        if (MP + 64) * page <= (1 << 31) - 1 - 8192:
            assert attend(lib, B=B, R=B, H=H, Hq=H * G, T=T, page=page, MP=MP + 64, **far) == -1
    assert attend(lib, **dict(far, MP=1 << 24, R=2, P=1 << 24)) == -3
    assert attend(lib, **dict(far, MP=(1 << 24) + 1)) == -1 and attend(lib, **dict(far, MP=4, P=(1 << 24) + 1)) == -1
    # one size of scratch for all rounds of a head size
    sizes = {lib.spec_attend_pages_workspace_bytes(T, Hq, H, 128) for T, Hq, H in ((1, 1, 1), (64, 64, 8), (9, 28, 4))}
    assert len(sizes) == 1
