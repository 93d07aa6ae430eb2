"""Attention of rounds over pages of 4-bit keys and values, against its formula
in 64 bits on the values that the codes stand for."""
import numpy as np
import pytest
import torch

import forward_ref
import paged_ref as ref
import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
NAN = float("nan")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def cu_(x):
    return None if x is None else x.cuda()


def make(seed, dt, B, T, G, H, D, page, lens, tree=False, L=2, rows=0, scale=1.0, full=False):
    """Inputs of a round; every byte that nobody may read says NaN."""
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    lens = np.resize(np.asarray(lens), B)
    parent, n = forward_ref.random_trees(rng, B, T, full=full or not tree)
    mask = torch.from_numpy(forward_ref.plan(parent, n)[0]) if tree else None
    R = rows or B
    idx = rng.permutation(R)[:B] if rows else np.arange(B)
    MP = max(1, int(-(-lens.max() // page))) + 1
    pages = np.zeros(R, int)
    pages[idx] = -(-(lens - 1) // page)
    P = int(pages.sum()) + 2
    table = ref.tables(rng, pages, MP, P)
    pool = ref.empty_pool(L, P, H, page, D)
    for b in range(B):
        k = int(lens[b]) - 1
        if k:
            ref.put(pool, page, D, table[idx[b]], (torch.randn((L, 2, H, k, D), generator=g) * scale).to(DT[dt]))
    staged = torch.full((L, 2, B, H, T, D), NAN)
    for b in range(B):
        staged[:, :, b, :, :int(n[b])] = torch.randn((L, 2, H, int(n[b]), D), generator=g) * scale
    q = torch.randn((B, T, G * H, D), generator=g) * scale
    return dict(q=q.to(DT[dt]), pool=pool, table=table, length=i32(lens), staged=staged.to(DT[dt]), mask=mask,
                n=i32(n) if tree else None, idx=i32(idx) if rows else None)


def run(c, layer=1, scale=None, **kw):
    out = torch.full_like(c["q"], 7.0).cuda()
    return sv.spec_attend_pages(c["q"].cuda(), c["pool"].cuda(), layer, c["table"].cuda(), c["length"].cuda(),
                                   c["staged"].cuda(), tree_mask=cu_(c["mask"]), n_nodes=cu_(c["n"]), idx=cu_(c["idx"]),
                                   scale=scale, out=out, **kw)


def close(got, want, tol):
    real = ~torch.isnan(want)
    got = got.cpu().double()
    assert torch.isfinite(got[real]).all()
    off = ((got - want).abs() - tol)[real]
    assert off.numel() == 0 or float(off.max()) <= 0, (float(off.max()), float(tol[real].max()))


def check(c, layer=1, scale=None):
    o, flags = run(c, layer, scale)
    want, tol = ref.attend(c["q"], c["pool"], layer, c["table"], c["length"], c["staged"], c["mask"], c["n"], c["idx"],
                           scale)
    assert (flags == 0).all()
    close(o, want, tol)
    assert (o.cpu()[torch.isnan(want)] == 7.0).all()  # nodes past the last are left as they were


# prefix lengths around the ends of tiles and pages, none to long
LENS = [1, 2, 16, 17, 18, 33, 64, 65, 66, 129, 130, 257, 258, 390]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,H,D,page", [(1, 1, 1, 64, 16), (1, 4, 2, 128, 64), (1, 8, 1, 128, 256), (5, 1, 4, 64, 32),
                                          (2, 7, 2, 128, 16), (9, 4, 2, 128, 128), (16, 8, 1, 128, 32),
                                          (64, 1, 2, 64, 16), (33, 7, 1, 128, 64), (40, 5, 1, 64, 64)])
def test_chains(dt, T, G, H, D, page):
    check(make(1, dt, 7, T, G, H, D, page, LENS[T % 2::2]))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,H,D,page", [(2, 2, 2, 64, 16), (3, 2, 2, 128, 32), (13, 4, 2, 128, 64), (26, 7, 2, 128, 16),
                                          (64, 4, 1, 128, 128), (64, 7, 1, 64, 256)])
def test_trees(dt, T, G, H, D, page):
    check(make(2, dt, 7, T, G, H, D, page, LENS[T % 2::2], tree=True))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("G,H,T", [(71, 1, 3), (16, 2, 9), (130, 1, 1), (1, 9, 1), (3, 1, 64)])
def test_head_groups(dt, G, H, T):
    check(make(4, dt, 2, T, G, H, 64, 32, [200, 131]))


@pytest.mark.parametrize("page", ref.PAGES)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_a_table(page, D):
    check(make(5, "bf16", 5, 7, 4, 2, D, page, [1, 130, 300, 12, 257], rows=9))
    check(make(6, "f16", 5, 1, 4, 2, D, page, [1, 130, 300, 12, 257], rows=9))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,page", [(1, 8, 64), (1, 3, 16), (5, 3, 128), (9, 4, 32)])
def test_long_contexts_are_split(dt, T, G, page):
    check(make(7, dt, 2, T, G, 1, 128, page, [9000, 4100]), layer=0)


def test_many_short_sequences():
    check(make(8, "bf16", 700, 1, 2, 2, 64, 16, list(range(1, 60)), L=1), layer=0)
    check(make(9, "f16", 500, 3, 2, 1, 64, 32, list(range(1, 90)), L=1, tree=True), layer=0)


def test_scales_of_scores_and_queries():
    """Sharp and flat weights; rows of queries of very different size."""
    for dt in DT:
        c = make(10, dt, 3, 5, 3, 2, 128, 32, [300, 65, 20])
        check(c, scale=1.0)
        check(c, scale=1e-4)
        f = torch.exp2(torch.randint(-9, 4, c["q"].shape[:-1] + (1,), generator=torch.Generator().manual_seed(1)).float())
        c["q"] = (c["q"].float() * f).to(DT[dt])
        check(c)
        c["q"][0, 0] = 0.0
        check(c)
    c["q"] = torch.randn(c["q"].shape, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    c["staged"] = c["staged"].to(torch.bfloat16)
    for f in (2.0 ** 40, 2.0 ** -60):  # beyond fp16's range
        d = dict(c, q=(c["q"].float() * f).to(torch.bfloat16))
        check(d, scale=128 ** -0.5 / f)


def test_values_of_very_different_size():
    for dt, s in (("f16", 300.0), ("bf16", 2000.0), ("bf16", 1e-3), ("f16", 1e-3)):
        c = make(11, dt, 3, 4, 2, 2, 128, 16, [300, 65, 20], scale=s)
        check(c, scale=0.1 / (s * s))


def test_same_bits_again_and_whatever_the_buffers_held():
    c = make(12, "bf16", 6, 9, 4, 2, 128, 64, [2000, 700, 65, 1, 3000, 1500])
    a = run(c)[0]
    b = run(c)[0]
    assert torch.equal(a, b)
    ws = torch.full((sv.spec_attend_pages_workspace_bytes(9, 8, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:sv.ATTEND_ZERO].zero_()
    assert torch.equal(run(c, workspace=ws)[0], a)
    assert not ws[:sv.ATTEND_ZERO].any()


def test_rows_that_see_nothing_and_everything_masked():
    for dt in DT:
        c = make(13, dt, 3, 6, 3, 1, 64, 16, [1, 1, 40], tree=True, full=True)
        c["mask"][0, 2] = 0
        c["mask"][1] = 0
        c["mask"][2, 3] = 0  # the prefix alone
        check(c)
        o, _ = run(c)
        assert (o[0, 2] == 0).all() and (o[1] == 0).all()
        c["mask"][2] = -1  # bits past the nodes do not count
        c["n"][2] = 4
        check(c)
        c["n"][:] = 0
        o, flags = run(c)
        assert (o == 7).all() and not flags.any()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_what_is_not_finite_reaches_those_that_see_it(dt):
    T, G = 7, 3
    c = make(14, dt, 2, T, G, 1, 128, 32, [70, 1], tree=True, full=True)
    seen = [[int(m) >> a & 1 for a in range(T)] for m in c["mask"][0]]
    for value, layer in ((float("inf"), 1), (NAN, 1)):
        d = dict(c, staged=c["staged"].clone())
        d["staged"][layer, 1, 0, 0, 3, 77] = value
        d["staged"][layer, 1, 0, 0, 5, 2] = -value
        plain = dict(d, staged=d["staged"].nan_to_num(0.0, 0.0, 0.0))
        want, tol = ref.attend(plain["q"], plain["pool"], layer, plain["table"], plain["length"], plain["staged"], c["mask"],
                               c["n"])
        o = run(d, layer)[0].cpu().double()
        hit = torch.zeros_like(o, dtype=torch.bool)
        for i in range(T):
            hit[0, i, :, 77] |= bool(seen[i][3])
            hit[0, i, :, 2] |= bool(seen[i][5])
        assert torch.equal(torch.isfinite(o), ~hit)
        if value == float("inf"):
            assert (o[0, :, :, 77][hit[0, :, :, 77]] == value).all() and (o[0, :, :, 2][hit[0, :, :, 2]] == -value).all()
        assert float(((o - want).abs() - tol)[~hit].max()) <= 0
        # a key: the rows that see it have no result, the others theirs
        d = dict(c, staged=c["staged"].clone())
        d["staged"][layer, 0, 0, 0, 3, 5] = NAN
        o = run(d, layer)[0].cpu()
        for i in range(T):
            assert torch.isnan(o[0, i]).all() == bool(seen[i][3])
            assert torch.isfinite(o[0, i]).all() == (not seen[i][3])
        assert torch.isfinite(o[1]).all()


def test_a_group_that_is_not_finite_in_a_page():
    """One group of one key: that sequence's head is NaN; of one value: its 32 dimensions are."""
    c = make(15, "bf16", 2, 3, 2, 2, 128, 32, [70, 70])
    d = dict(c, pool=c["pool"].clone())
    _, scales = ref.views(d["pool"], 32, 128)
    scales[1, 0, c["table"][0, 1], 1, 7, 2] = 255
    o = run(d)[0].cpu()
    assert torch.isnan(o[0, :, 2:]).all() and torch.isfinite(o[0, :, :2]).all() and torch.isfinite(o[1]).all()
    d = dict(c, pool=c["pool"].clone())
    _, scales = ref.views(d["pool"], 32, 128)
    scales[1, 1, c["table"][0, 2], 0, 4, 3] = 255
    o = run(d)[0].cpu()
    assert torch.isnan(o[0, :, :2, 96:]).all() and torch.isfinite(o[0, :, :2, :96]).all()
    assert torch.isfinite(o[0, :, 2:]).all() and torch.isfinite(o[1]).all()


def test_flags():
    for T in (1, 9):
        c = make(16, "bf16", 8, T, 4, 2, 64, 16, [40, 17, 64, 30, 33, 100, 20, 18], rows=12)
        want, tol = ref.attend(c["q"], c["pool"], 1, c["table"], c["length"], c["staged"], idx=c["idx"])
        P, MP = c["pool"].shape[2], c["table"].shape[1]
        c["length"][0] = 0
        c["length"][1] = MP * 16 + 2
        c["idx"][2], c["idx"][3] = 12, -1
        c["table"][c["idx"][4], 1] = P
        c["table"][c["idx"][5], 2] = -1
        c["table"][c["idx"][7], 2:] = P + 5  # behind the prefix
        o, flags = run(c)
        assert [int(f) for f in flags] == [16] * 6 + [0] * 2
        assert (o[:4] == 7).all()
        close(o[6:], want[6:], tol[6:])
        c["n"] = i32([1, 1, 1, 1, 1, 1, T + 1, -1])
        assert [int(f) for f in run(c)[1]] == [16] * 8


@pytest.mark.parametrize("T,G", [(1, 8), (9, 4)])
def test_streams_and_graphs(T, G):
    """The same call on another stream, captured and replayed with other inputs,
    and two graphs side by side."""
    c = make(17, "bf16", 5, T, G, 2, 128, 64, [900, 33, 400, 1, 250])
    d = make(18, "bf16", 5, T, G, 2, 128, 64, [900, 33, 400, 1, 250])
    want = [run(x)[0] for x in (c, d)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = [{k: cu_(v) for k, v in x.items()} for x in (c, d)]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()

    def call(x, out, **kw):
        sv.spec_attend_pages(x["q"], x["pool"], 1, x["table"], x["length"], x["staged"], out=out, **kw)

    call(args[0], outs[0], stream=s)
    call(args[1], outs[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graphs = []
    for x, o in zip(args, outs):
        o.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(x, o)
        graphs.append(graph)
    for _ in range(5):
        for graph, stream in zip(graphs, (s, torch.cuda.current_stream())):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    for k in ("q", "pool", "table", "staged"):
        if args[0][k].shape == args[1][k].shape:
            args[0][k].copy_(args[1][k])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


def test_a_pool_past_32_bits():
    """Pages at the end of a layer of 5 GB, the second of two."""
    for T in (1, 9):
        c = make(19, "f16", 3, T, 4, 4, 128, 64, [900, 65, 400], L=1)
        P, H, block = c["pool"].shape[2:]
        big = 151000
        pool = torch.full((2, 2, big, H, block), 255, dtype=torch.uint8, device="cuda")
        pool[1, :, big - P:] = c["pool"][0].cuda()
        table = torch.where(c["table"] >= 0, c["table"] + (big - P), -1)
        staged = torch.cat([torch.full_like(c["staged"], NAN), c["staged"]])
        o, flags = sv.spec_attend_pages(c["q"].cuda(), pool, 1, table.cuda(), c["length"].cuda(), staged.cuda())
        want, tol = ref.attend(c["q"], c["pool"], 0, c["table"], c["length"], c["staged"])
        assert not flags.any()
        close(o, want, tol)
        del pool


def test_a_wait_that_gives_up_is_reported():
    from speculative_decoding_verification_28_gb300 import _lib

    c = make(20, "bf16", 4, 1, 4, 2, 64, 16, [40, 17, 64, 300])
    ws = torch.zeros(sv.spec_attend_pages_workspace_bytes(1, 8, 2, 64), dtype=torch.uint8, device="cuda")
    good = run(c, workspace=ws)[0]
    assert _lib.load().spec_attend_starve_next(100000) == 0
    assert (run(c, workspace=ws)[1] & sv.FLAG_TIMEOUT).all()
    assert (run(c, workspace=ws)[1] & sv.FLAG_TIMEOUT).all()  # until the head is cleared
    ws[:sv.ATTEND_ZERO].zero_()
    o, flags = run(c, workspace=ws)
    assert not flags.any() and torch.equal(o, good)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,D", [(3, 2, 64), (4, 4, 128), (7, 3, 64), (9, 7, 128), (9, 8, 64), (20, 7, 128)])
def test_values_that_are_not_finite_in_every_form(dt, T, G, D):
    """Rows that see a node whose value is not finite have it, the others what they would have without."""
    c = make(19, dt, 3, T, G, 2, D, 16, [130, 1, 17], tree=True, full=True)
    d = dict(c, staged=c["staged"].clone())
    at = [(b, h, b + 1 if b + 1 < T else 0, d) for b, h, d in ((0, 1, D - 3), (1, 0, 0), (2, 1, D // 2 - 1), (0, 0, D // 4))]
    for k, (b, h, node, dim) in enumerate(at):
        d["staged"][1, 1, b, h, node, dim] = (float("inf"), NAN, -float("inf"), float("inf"))[k]
    plain = dict(d, staged=d["staged"].nan_to_num(0.0, 0.0, 0.0))
    want, tol = ref.attend(plain["q"], plain["pool"], 1, plain["table"], plain["length"], plain["staged"], c["mask"], c["n"])
    o = run(d)[0].cpu().double()
    hit = torch.zeros_like(o, dtype=torch.bool)
    for b, h, node, dim in at:
        for i in range(T):
            hit[b, i, h * G:(h + 1) * G, dim] = bool(int(c["mask"][b, i]) >> node & 1)
    assert torch.equal(torch.isfinite(o), ~hit)
    assert float(((o - want).abs() - tol)[~hit].max()) <= 0


@pytest.mark.parametrize("T,G,D", [(4, 4, 128), (9, 4, 64), (20, 5, 128)])
def test_a_wait_that_gives_up_in_every_form(T, G, D):
    """Sequences whose units are cut over many CTAs; the call after it on a clean workspace is as if nothing had been."""
    from speculative_decoding_verification_28_gb300 import _lib

    c = make(21, "f16", 5, T, G, 2, D, 64, [1500, 17, 64, 3000, 1])
    ws = torch.zeros(sv.spec_attend_pages_workspace_bytes(T, 2 * G, 2, D), dtype=torch.uint8, device="cuda")
    good = run(c, workspace=ws)[0]
    assert _lib.load().spec_attend_starve_next(100000) == 0
    assert (run(c, workspace=ws)[1] & sv.FLAG_TIMEOUT).all()
    ws[:sv.ATTEND_ZERO].zero_()
    o, flags = run(c, workspace=ws)
    assert not flags.any() and torch.equal(o, good)
