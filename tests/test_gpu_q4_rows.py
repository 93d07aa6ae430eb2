"""Rows stored into 4-bit pages and loaded back, byte for byte against the
definition."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def values(g, shape, dtype):
    """rows of very different size, with ties, zeros, and what is not finite"""
    x = torch.randn(shape, generator=g) * torch.exp(4 * torch.randn((*shape[:-1], 1), generator=g))
    x = x.to(dtype)
    flat = x.view(-1, 32)
    flat[::7] = (torch.randint(-14, 15, (len(flat[::7]), 32), generator=g) / 2).to(dtype)  # multiples of s / 2
    flat[1::7, 0] = 7.0
    flat[2::29] = 0.0
    flat[5::29] = -0.0
    flat[8::29, 3] = float("nan")
    flat[9::29, 31] = float("-inf")
    flat[10::29] = 6e4 if dtype == torch.float16 else 1e30
    flat[11::29] = 1e-6
    flat[11::29, 5] = 3e-5
    flat[12::29] = 5.9e-8 if dtype == torch.float16 else 1e-38
    return x


def same(got, want):
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("page,D,H", [(16, 32, 1), (16, 64, 3), (32, 128, 2), (64, 96, 1), (128, 64, 2), (256, 256, 1)])
def test_store_a_run_of_slots(dt, page, D, H):
    g, rng = torch.Generator().manual_seed(1), np.random.default_rng(page)
    L, N, S, B, MP, Lp = 2, 5, 330, 4, 360 // page + 2, 4
    src = values(g, (L, 2, N, H, S, D), DT[dt])
    count, pos = np.array([0, 1, 65, 300]), np.array([3, 255, 17, 40])
    slot = np.array([330, 9, 100, 30])
    idx, row = rng.permutation(N)[:B], rng.permutation(6)[:B]
    table = ref.tables(rng, [MP] * 6, MP, 6 * MP + 3)
    P = 6 * MP + 3
    want = ref.empty_pool(Lp, P, H, page, D)
    got = want.cuda()
    f = sv.spec_store_pages(src.cuda(), got, table.cuda(), i32(pos).cuda(), i32(count).cuda(), layer=1, slot=i32(slot).cuda(),
                         idx=i32(idx).cuda(), row=i32(row).cuda())
    assert not f.any()
    for b in range(B):
        ref.put(want[1:3], page, D, table[row[b]], src[:, :, idx[b], :, slot[b]:slot[b] + count[b]], pos[b])
    same(got, want)
    # and back, into the other rows' slots left alone
    dst = torch.full((L, 2, N, H, S, D), 5.0, dtype=DT[dt])
    back = dst.cuda()
    f = sv.spec_load_pages(got, back, table.cuda(), i32(pos).cuda(), i32(count).cuda(), layer=1, slot=i32(slot).cuda(),
                        idx=i32(idx).cuda(), row=i32(row).cuda())
    assert not f.any()
    for b in range(B):
        dst[:, :, idx[b], :, slot[b]:slot[b] + count[b]] = ref.get(want[1:3], page, D, table[row[b]], count[b], pos[b]).to(DT[dt])
    odd = torch.isnan(dst)
    assert bool(odd.any()) and bool((torch.isnan(back.cpu()) == odd).all())
    same(back.nan_to_num(1.0), dst.nan_to_num(1.0))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,page,D", [(1, 16, 128), (26, 64, 128), (64, 32, 64), (9, 256, 32)])
def test_store_a_path(dt, T, page, D):
    g, rng = torch.Generator().manual_seed(T), np.random.default_rng(T)
    L, B, H, MP = 3, 7, 2, 5
    staged = values(g, (L, 2, B, H, T, D), DT[dt])
    count = rng.integers(0, T + 1, B)
    pos = rng.integers(0, MP * page - T, B)
    path = np.full((B, T), -1)
    for b in range(B):
        path[b, :count[b]] = np.sort(rng.permutation(T)[:count[b]])
    table = ref.tables(rng, [MP] * B, MP, B * MP)
    want = ref.empty_pool(L, B * MP, H, page, D)
    got = want.cuda()
    f = sv.spec_store_pages(staged.cuda(), got, table.cuda(), i32(pos).cuda(), i32(count).cuda(), path=i32(path).cuda())
    assert not f.any()
    for b in range(B):
        ref.put(want, page, D, table[b], staged[:, :, b][:, :, :, path[b, :count[b]]], pos[b])
    same(got, want)


def test_every_scale_and_code():
    """Groups whose largest value is each multiple of a scale's sixteenth, in
    both types: all bytes, all ties between them."""
    for dt in DT.values():
        top = np.concatenate([ref.SCALES[1:] * 7, (ref.SCALES[1:-1] + ref.SCALES[2:]) * 3.5, ref.SCALES[1:] * 7.4])
        top = torch.from_numpy(top).to(dt)
        frac = torch.arange(-16, 16) / 16.0
        x = (top.double()[:, None] * frac).to(dt).float()
        x[:, 0] = -top.float()
        n = len(x)
        S = n
        src = x.to(dt).view(1, 1, 1, 1, n, 32).expand(1, 2, 1, 1, n, 32).contiguous()
        MP = -(-S // 256)
        table = torch.arange(MP, dtype=torch.int32)[None]
        want = ref.empty_pool(1, MP, 1, 256, 32)
        got = want.cuda()
        zero = i32([0]).cuda()
        sv.spec_store_pages(src.cuda(), got, table.cuda(), zero, i32([n]).cuda())
        ref.put(want, 256, 32, table[0], src[:, :, 0])
        same(got, want)
        _, scales = ref.views(want, 256, 32)
        assert set(range(8, 220)) <= set(scales.flatten().tolist())


def test_flags_and_pages_outside_the_pool():
    L, B, H, T, D, page, MP = 1, 8, 1, 6, 64, 16, 3
    g = torch.Generator().manual_seed(3)
    src = torch.randn((L, 2, B, H, T, D), generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(B * MP, dtype=torch.int32).view(B, MP)
    P = B * MP
    pos = i32([0, -1, 43, 0, 0, 2147483647, 14, 0])
    count = i32([6, 3, 6, 7, -1, 1, 5, 6])
    slot = i32([0, 0, 0, 0, 0, 0, 0, 1])
    table[6, 1] = P
    pool = ref.empty_pool(L, P, H, page, D)
    got = pool.cuda()
    f = sv.spec_store_pages(src, got, table.cuda(), pos.cuda(), count.cuda(), slot=slot.cuda())
    assert [int(x) // 16 for x in f] == [0, 1, 1, 1, 1, 1, 1, 1]
    ref.put(pool, page, D, table[0], src[:, :, 0].cpu())
    ref.put(pool, page, D, table[6], src[:, :, 6, :, :2].cpu(), 14)  # those that have a page
    same(got, pool)
    back = torch.full_like(src, 3.0)
    f = sv.spec_load_pages(got, back, table.cuda(), pos.cuda(), count.cuda(), slot=slot.cuda())
    assert [int(x) // 16 for x in f] == [0, 1, 1, 1, 1, 1, 1, 1]
    assert (back[:, :, 1:6] == 3).all() and (back[:, :, 7] == 3).all() and (back[:, :, 6, :, 2:] == 3).all()
    same(back[:, :, 0].double(), ref.get(pool, page, D, table[0], 6))
    # repeated rows, rows and path entries out of range
    one, two = i32([0, 0]).cuda(), i32([2, 2]).cuda()
    for kw in (dict(row=i32([1, 1]).cuda()), dict(row=i32([-1, 8]).cuda()), dict(idx=i32([-1, 8]).cuda())):
        kw = {"row": i32([2, 3]).cuda(), "idx": i32([0, 0]).cuda(), **kw}
        got = pool.cuda()
        assert (sv.spec_store_pages(src, got, table.cuda(), one, two, **kw) == 16).all()
        same(got, pool)
    for bad in (-1, T, 2 ** 30):
        got = pool.cuda()
        path = i32([[0, bad, 0], [bad, 1, 0]]).cuda()
        assert (sv.spec_store_pages(src, got, table.cuda(), one, two, path=path) == 16).all()
        same(got, pool)
    keep = torch.full_like(src, 3.0)
    assert (sv.spec_load_pages(got, keep, table.cuda(), one, two, idx=i32([4, 4]).cuda()) == 16).all()
    assert (keep == 3).all()


def test_offsets_past_32_bits():
    """A pool of 4.6 GB: pages, layers and rows of it at its end."""
    L, P, H, D, page, B = 2, 131200, 4, 128, 32, 2
    pool = torch.zeros((L, 2, P, H, page * 68), dtype=torch.uint8, device="cuda")
    pool_small = ref.empty_pool(1, 4, H, page, D, 0)
    g = torch.Generator().manual_seed(4)
    src = torch.randn((1, 2, B, H, 40, D), generator=g).to(torch.float16)
    table, small = i32([[P - 1, P - 3], [P - 2, P - 4]]), i32([[3, 1], [2, 0]])
    pos, n = i32([0, 5]), i32([40, 33])
    f = sv.spec_store_pages(src.cuda(), pool, table.cuda(), pos.cuda(), n.cuda(), layer=1)
    assert not f.any()
    for b in range(B):
        ref.put(pool_small, page, D, small[b], src[:, :, b, :, :int(n[b])], int(pos[b]))
    same(pool[1:, :, P - 4:], pool_small)
    assert not pool[0].any() and not pool[1, :, :P - 4].any()
    back = torch.zeros_like(src).cuda()
    sv.spec_load_pages(pool, back, table.cuda(), pos.cuda(), n.cuda(), layer=1)
    same(back[0, :, 1, :, :33].double(), ref.get(pool_small, page, D, small[1], 33, 5)[0])
    moves = i32([[P - 1, 7], [P - 4, P - 5]]).cuda()
    sv.spec_page_copy(pool, moves)
    same(pool[:, :, 7], pool[:, :, P - 1].cpu())
    same(pool[:, :, P - 5], pool[:, :, P - 4].cpu())
