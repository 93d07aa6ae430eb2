"""The forward-pass operators against their formulas in 64 bits: appending,
attention of rounds and prompts, tree verification, the commit of a path."""
import numpy as np
import pytest
import torch

import forward_ref as ref
import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def cu_(x):
    return None if x is None else x.cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def close(got, want, tol, name=""):
    real = ~torch.isnan(want)
    got = got.cpu().double()
    off = ((got - want).abs() - tol)[real]
    assert torch.isfinite(got[real]).all(), name
    assert off.numel() == 0 or float(off.max()) <= 0, (name, float(off.max()), float(tol[real].max()))


def round_case(seed, dtype, B, T, G, H, D, S, lens, L=2, tree=False, staged=False, pool=0, full=False):
    """Inputs of a round; every slot nobody sees holds NaN."""
    g, rng = gen(seed), np.random.default_rng(seed)
    lens = np.resize(np.asarray(lens), B)
    parent, n = ref.random_trees(rng, B, T, full=full or not tree)
    mask = torch.from_numpy(ref.plan(parent, n)[0]) if tree else None
    N = pool or B
    idx = i32(rng.permutation(N)[:B]) if pool else None
    room = S - (lens - 1) - (0 if staged else n)
    assert (room >= 0).all()
    pad = i32(rng.integers(0, room + 1)) if not pool else i32(np.zeros(B))
    kv = torch.full((L, 2, N, H, S, D), NAN)
    for b in range(B):
        r = b if idx is None else int(idx[b])
        p, e = int(pad[b]), int(pad[b]) + int(lens[b]) - 1 + (0 if staged else int(n[b]))
        kv[:, :, r, :, p:e] = torch.randn((L, 2, H, e - p, D), generator=g)
    kv = kv.to(dtype)
    st = None
    if staged:
        st = torch.full((L, 2, B, H, T, D), NAN)
        for b in range(B):
            st[:, :, b, :, :int(n[b])] = torch.randn((L, 2, H, int(n[b]), D), generator=g)
        st = st.to(dtype)
    q = randn(g, (B, T, G * H, D), dtype)
    return dict(q=q, kv=kv, length=i32(lens), pad=pad, mask=mask, n=i32(n) if tree else None, idx=idx, staged=st)


def run_round(c, layer=1, scale=None, **kw):
    out = torch.full_like(c["q"], 7.0).cuda()
    o, flags = sv.spec_attend_round(c["q"].cuda(), c["kv"].cuda(), layer, c["length"].cuda(), c["pad"].cuda(),
                                    tree_mask=cu_(c["mask"]), n_nodes=cu_(c["n"]), idx=cu_(c["idx"]),
                                    staged=cu_(c["staged"]), scale=scale, out=out, **kw)
    return o, flags


def check_round(c, layer=1, scale=None):
    o, flags = run_round(c, layer, scale)
    want, tol = ref.attend_round(c["q"], c["kv"], layer, c["length"], c["pad"], c["mask"], c["n"], c["idx"],
                                 c["staged"], scale)
    assert (flags == 0).all()
    close(o, want, tol)
    assert (o.cpu()[torch.isnan(want)] == 7.0).all()  # nodes past the last are left as they were


# prefix lengths around the tiles' ends, one token to long
LENS = [1, 2, 17, 64, 65, 66, 127, 128, 129, 130, 257, 385]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,G,H,D", [(1, 1, 1, 64), (1, 4, 2, 128), (5, 1, 4, 64), (9, 4, 2, 128), (16, 8, 1, 128),
                                     (64, 1, 2, 64), (33, 7, 1, 128), (40, 5, 2, 64)])
def test_attend_round_chain(dt, T, G, H, D):
    check_round(round_case(1, DT[dt], 6, T, G, H, D, 520, LENS[T % 2::2]))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,G,H,D", [(2, 2, 2, 64), (13, 4, 2, 128), (26, 7, 2, 128), (64, 4, 1, 128), (64, 7, 1, 64)])
@pytest.mark.parametrize("staged", [False, True])
def test_attend_round_tree(dt, T, G, H, D, staged):
    check_round(round_case(2, DT[dt], 6, T, G, H, D, 520, LENS[T % 2::2], tree=True, staged=staged))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 3, 36, 80, 96, 192, 255, 256])
def test_attend_round_any_head_size(dt, D):
    check_round(round_case(3, DT[dt], 3, 6, 3, 2, D, 150, [1, 70, 140], tree=True, staged=True))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,H,T", [(71, 1, 3), (16, 2, 9), (130, 1, 1), (1, 9, 1)])
def test_attend_round_head_groups(dt, G, H, T):
    check_round(round_case(4, DT[dt], 2, T, G, H, 64, 300, [200, 131]))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attend_round_in_a_pool(dt):
    check_round(round_case(5, DT[dt], 5, 7, 4, 2, 128, 400, [1, 130, 300, 12, 257], pool=9))
    check_round(round_case(6, DT[dt], 5, 7, 4, 2, 64, 400, [1, 130, 300, 12, 257], pool=9, tree=True, staged=True))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_attend_round_long_context_is_split(dt):
    # one sequence, one key head: its tiles go to many CTAs and are joined
    check_round(round_case(7, DT[dt], 1, 3, 2, 1, 64, 9000, [8991]), scale=0.2)
    check_round(round_case(8, DT[dt], 3, 20, 2, 2, 128, 2500, [2400, 1, 777], tree=True, staged=True))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,G,D", [(1, 1, 64), (3, 2, 128), (9, 4, 64), (20, 5, 128), (64, 4, 128), (64, 7, 64), (13, 3, 36)])
def test_attend_round_units_of_two_to_many_parts(dt, T, G, D):
    """Few units, cut every two tiles: parts from 2 on, joined in each of the ways there are."""
    check_round(round_case(40, DT[dt], 5, T, G, 2, D, 1400, [130, 250, 400, 700, 1250], tree=T > 1, staged=T > 1))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 80])
def test_attend_round_rows_that_see_nothing_give_zeros(dt, D):
    c = round_case(9, DT[dt], 4, 6, 2, 2, D, 200, [1, 1, 1, 150], tree=True, staged=True, full=True)
    c["mask"][0] = 0                       # no prefix, no node: all zeros
    c["mask"][1, ::2] = 0
    c["mask"][2, 3] = -1                   # bits past the nodes are ignored
    c["mask"][3] = 0                       # only the prefix
    o, flags = run_round(c)
    want, tol = ref.attend_round(c["q"], c["kv"], 1, c["length"], c["pad"], c["mask"], c["n"], c["idx"], c["staged"])
    close(o, want, tol)
    assert (o[0] == 0).all() and (o[1, ::2] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_attend_round_values_that_are_not_finite_stay_with_the_rows_that_see_them(dt):
    c = round_case(10, DT[dt], 1, 4, 2, 1, 64, 200, [140], tree=True, staged=True, full=True)
    c["mask"] = torch.tensor([[1, 3, 5, 9]])   # three children of the root
    c["staged"][1, 1, 0, 0, 2, 5] = float("inf")
    c["staged"][1, 1, 0, 0, 3, 6] = NAN
    c["staged"][1, 0, 0, 0, 3, 6] = NAN
    o, _ = run_round(c)
    want, tol = ref.attend_round(c["q"], c["kv"], 1, c["length"], c["pad"], c["mask"], c["n"], None, c["staged"])
    close(o[:, :2], want[:, :2], tol[:, :2])
    assert torch.isinf(o[0, 2, :, 5]).all() and torch.isnan(o[0, 3]).all()
    keep = [d for d in range(64) if d != 5]
    close(o[:, 2:3, :, keep], want[:, 2:3, :, keep], tol[:, 2:3, :, keep])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("big", [30.0, 1e-3])
def test_attend_round_large_and_small_scores(dt, big):
    c = round_case(11, DT[dt], 2, 5, 4, 2, 64, 400, [390, 200])
    c["q"] = (c["q"].float() * big).to(DT[dt])
    check_round(c)


def test_attend_round_flags_bad_state_and_leaves_its_output():
    c = round_case(12, torch.bfloat16, 8, 4, 2, 2, 64, 100, [10, 20, 30, 40, 50, 60, 70, 80], tree=True)
    c["n"][:] = 4
    c["length"][0] = 0
    c["pad"][1] = -1
    c["length"][2] = 2 ** 31 - 1
    c["pad"][3] = 2 ** 31 - 1
    c["n"][4] = 5
    c["n"][5] = -1
    o, flags = run_round(c)
    assert flags.tolist() == [16] * 6 + [0, 0]
    assert (o[:6] == 7).all() and not (o[6:] == 7).any()
    c["idx"] = i32([0, 1, 2, 3, 4, 5, 8, -1])
    o, flags = run_round(c)
    assert flags.tolist() == [16] * 8 and (o == 7).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attend_round_is_repeatable_and_can_be_captured(dt):
    c = round_case(13, DT[dt], 5, 9, 4, 2, 64, 1500, [1400, 3, 900, 128, 1])
    a, _ = run_round(c)
    d = {k: cu_(v) for k, v in c.items()}
    graphs, outs = [], []
    for _ in range(2):
        out = torch.zeros_like(d["q"])
        graphs.append(sv.RoundGraph(lambda: sv.spec_attend_round(d["q"], d["kv"], 1, d["length"], d["pad"], out=out)))
        outs.append(out)
    # two captured calls side by side share no scratch
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, a)
    # lengths are read on the device: a replay sees new ones
    d["length"].copy_(i32([7, 300, 1, 2, 1300]))
    graphs[0].replay()
    c["length"] = i32([7, 300, 1, 2, 1300])
    c["pad"], c["kv"] = torch.zeros(5, dtype=torch.int32), randn(gen(99), c["kv"].shape, DT[dt])
    d["pad"].copy_(c["pad"])
    d["kv"].copy_(c["kv"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], run_round(c)[0])


def test_attend_round_on_a_side_stream():
    c = round_case(14, torch.bfloat16, 3, 9, 4, 2, 128, 700, [600, 3, 128])
    a, _ = run_round(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d = {k: cu_(v) for k, v in c.items()}
    s.wait_stream(torch.cuda.current_stream())
    o, _ = sv.spec_attend_round(d["q"], d["kv"], 1, d["length"], d["pad"], stream=s)
    s.synchronize()
    assert torch.equal(o, a)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,G", [(2, 3), (5, 20)])
def test_attend_round_many_sequences(dt, T, G):
    # more sequences than a CTA has threads; some idle, some not valid
    g, rng = gen(17), np.random.default_rng(17)
    B, H, S, D = 777, 1, 24, 64
    lens, n = rng.integers(1, 18, B), rng.integers(0, T + 1, B)
    lens[::50] = 0
    kv = randn(g, (1, 2, B, H, S, D), DT[dt])
    q = randn(g, (B, T, G * H, D), DT[dt])
    out = torch.full_like(q, 7.0).cuda()
    o, flags = sv.spec_attend_round(q.cuda(), kv.cuda(), 0, i32(lens).cuda(), None, n_nodes=i32(n).cuda(), out=out)
    assert ((flags.cpu() == 16) == (i32(lens) == 0)).all()
    n[lens == 0] = 0
    want, tol = ref.attend_round(q, kv, 0, np.maximum(lens, 1), np.zeros(B, int), n=n)
    close(o, want, tol)
    assert (o.cpu()[torch.isnan(want)] == 7.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_attend_round_of_one_row_twice(dt):
    c = round_case(18, DT[dt], 4, 3, 4, 2, 128, 300, [200, 100, 30, 7], pool=4, tree=True, staged=True)
    c["idx"] = i32([2, 2, 0, 2])
    c["kv"] = randn(gen(19), c["kv"].shape, DT[dt])
    check_round(c)


def shifted(x):
    """The same values one element further into a buffer."""
    y = torch.zeros(x.numel() + 1, dtype=x.dtype, device=x.device)[1:].view(x.shape)
    return y.copy_(x)


@pytest.mark.parametrize("which", ["q", "kv", "staged", "out"])
def test_attend_round_buffers_of_element_alignment(which):
    c = round_case(20, torch.bfloat16, 3, 5, 2, 2, 64, 200, [150, 64, 3], tree=True, staged=True)
    d = {k: cu_(v) for k, v in c.items()}
    out = torch.zeros_like(d["q"])
    if which == "out":
        out = shifted(out)
    else:
        d[which] = shifted(d[which])
    o, flags = sv.spec_attend_round(d["q"], d["kv"], 1, d["length"], d["pad"], tree_mask=d["mask"], n_nodes=d["n"],
                                    staged=d["staged"], out=out)
    want, tol = ref.attend_round(c["q"], c["kv"], 1, c["length"], c["pad"], c["mask"], c["n"], None, c["staged"])
    close(o, want, tol)


def test_attend_round_offsets_past_32_bits():
    # the layer's slabs start more than 2^32 elements into the cache
    free, _ = torch.cuda.mem_get_info()
    N, H, S, D = 33, 2, 1 << 18, 128
    if free < 2 * N * H * S * D * 2 + (4 << 30):
        pytest.skip("not enough memory")
    kv = torch.empty((1, 2, N, H, S, D), dtype=torch.bfloat16, device="cuda")
    assert kv[0].numel() > 1 << 32
    g = gen(15)
    lens, pads = [300, 150], [S - 310, 5]
    q = randn(g, (2, 4, 4, D), torch.bfloat16)
    small = torch.zeros((1, 2, 2, H, 400, D), dtype=torch.bfloat16)
    for b, row in enumerate((N - 1, N - 2)):
        x = randn(g, (2, H, lens[b] + 3, D), torch.bfloat16)
        small[0, :, b, :, 5:5 + lens[b] + 3] = x
        kv[0, :, row, :, pads[b]:pads[b] + lens[b] + 3] = x.cuda()
    o, flags = sv.spec_attend_round(q.cuda(), kv, 0, i32(lens).cuda(), i32(pads).cuda(), idx=i32([N - 1, N - 2]).cuda())
    assert (flags == 0).all()
    want, tol = ref.attend_round(q, small, 0, lens, [5, 5])
    close(o, want, tol)


def test_attend_round_edges():
    kv = torch.zeros((1, 2, 3, 2, 40, 64), dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    o, flags = sv.spec_attend_round(torch.zeros((0, 3, 4, 64), dtype=torch.bfloat16, device="cuda"), kv, 0, e, e)
    assert o.shape == (0, 3, 4, 64) and flags.numel() == 0
    # every sequence idle
    c = round_case(16, torch.bfloat16, 2, 3, 2, 2, 64, 40, [10, 20], tree=True)
    c["n"][:] = 0
    o, flags = run_round(c)
    assert (o == 7).all() and (flags == 0).all()


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------
def prompt_case(seed, dtype, G, H, D, S, lens, past=None, pool=0, tail=0, L=1):
    g, rng = gen(seed), np.random.default_rng(seed)
    lens = np.asarray(lens)
    B = len(lens)
    past = np.zeros(B, np.int64) if past is None else np.asarray(past)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    N = pool or B
    idx = i32(rng.permutation(N)[:B]) if pool else None
    pad = i32(rng.integers(0, S - lens - past + 1))
    kv = torch.full((L, 2, N, H, S, D), NAN)
    for b in range(B):
        r, p, e = b if idx is None else int(idx[b]), int(pad[b]), int(pad[b] + lens[b] + past[b])
        kv[:, :, r, :, p:e] = torch.randn((L, 2, H, e - p, D), generator=g)
    q = randn(g, (int(cu[-1]) + tail, G * H, D), dtype)
    return dict(q=q, kv=kv.to(dtype), cu=i32(cu), pad=pad, start=i32(past), idx=idx)


def run_prompt(c, scale=None, layer=0):
    out = torch.full_like(c["q"], 7.0).cuda()
    return sv.spec_attend_prompt(c["q"].cuda(), c["kv"].cuda(), layer, c["cu"].cuda(), c["pad"].cuda(),
                                 start=cu_(c["start"]), idx=cu_(c["idx"]), scale=scale, out=out)


def check_prompt(c, scale=None, layer=0):
    o, flags = run_prompt(c, scale, layer)
    want, tol = ref.attend_prompt(c["q"], c["kv"], layer, c["cu"], c["pad"], c["start"], c["idx"], scale)
    assert (flags == 0).all()
    close(o, want, tol)
    assert (o.cpu()[torch.isnan(want)] == 7.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,H,D", [(1, 2, 64), (1, 1, 128), (2, 2, 128), (4, 1, 128), (7, 1, 64), (8, 1, 128), (5, 1, 80)])
def test_attend_prompt(dt, G, H, D):
    check_prompt(prompt_case(21, DT[dt], G, H, D, 300, [1, 0, 17, 130, 64, 65, 33, 129], tail=3))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("G,H,D", [(1, 2, 64), (4, 1, 128)])
def test_attend_prompt_longer_than_tiles(dt, G, H, D):
    check_prompt(prompt_case(22, DT[dt], G, H, D, 900, [513, 700]))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("G,H,D", [(1, 2, 64), (1, 1, 128), (4, 1, 128), (7, 1, 64)])
@pytest.mark.parametrize("lens,past", [((600, 3, 1300, 705), None), ((1, 1537), None), ((520, 811), (129, 0)),
                                       ((1, 0, 1, 1400), (0, 5, 700, 63))])
def test_attend_prompt_of_long_and_mixed_lengths(dt, G, H, D, lens, past):
    check_prompt(prompt_case(35, DT[dt], G, H, D, 1700, lens, past=past, tail=2))


@pytest.mark.parametrize("dt,G", [("bf16", 71), ("f16", 8)])
def test_attend_prompt_of_long_ones_with_many_heads_to_a_key_head(dt, G):
    check_prompt(prompt_case(38, DT[dt], G, 1, 64, 540, [514, 515][:1 if G > 8 else 2]))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_prompt_later_values_that_are_not_finite_in_a_long_one(dt, D):
    """Two rows of a tile's V, one of the tile after; the first is seen from
    row 600 on, the second from 640 (the end of a tile), the third from 645."""
    c = prompt_case(36, DT[dt], 2, 1, D, 900, [800])
    at = int(c["pad"][0])
    for pos, d, x in ((600, 3, float("-inf")), (640, 7, float("inf")), (645, D - 1, NAN)):
        c["kv"][0, 1, 0, 0, at + pos, d] = x
    o, _ = run_prompt(c)
    want, tol = ref.attend_prompt(c["q"], c["kv"], 0, c["cu"], c["pad"], c["start"])
    lo = 0
    hidden = []
    for pos, d, inf in ((600, 3, True), (640, 7, True), (645, D - 1, False), (800, 0, True)):
        keep = [x for x in range(D) if x not in hidden]
        close(o[lo:pos][..., keep], want[lo:pos][..., keep], tol[lo:pos][..., keep])
        if pos < 800:
            assert (torch.isinf if inf else torch.isnan)(o[pos:, :, d]).all()
            hidden.append(d)
        lo = pos


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_attend_prompt_in_pieces(dt):
    check_prompt(prompt_case(23, DT[dt], 4, 2, 64, 700, [40, 1, 129, 64], past=[300, 77, 128, 0], pool=6, tail=1))
    check_prompt(prompt_case(24, DT[dt], 3, 1, 128, 600, [100, 5], past=[450, 127]), scale=0.3)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G", [40, 71, 130])
def test_attend_prompt_many_heads_to_a_key_head(dt, G):
    check_prompt(prompt_case(25, DT[dt], G, 1, 64, 100, [20, 3, 40]))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attend_prompt_later_values_that_are_not_finite_reach_no_earlier_row(dt):
    c = prompt_case(26, DT[dt], 2, 1, 64, 200, [150])
    at = int(c["pad"][0])
    c["kv"][0, 1, 0, 0, at + 70, 3] = float("-inf")
    c["kv"][0, 0, 0, 0, at + 140, 3] = NAN
    o, _ = run_prompt(c)
    want, tol = ref.attend_prompt(c["q"], c["kv"], 0, c["cu"], c["pad"], c["start"])
    close(o[:70], want[:70], tol[:70])
    keep = [d for d in range(64) if d != 3]
    close(o[70:140][..., keep], want[70:140][..., keep], tol[70:140][..., keep])
    assert torch.isinf(o[70:140, :, 3]).all() and torch.isnan(o[140:]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attend_prompt_many_sequences(dt):
    rng = np.random.default_rng(30)
    check_prompt(prompt_case(30, DT[dt], 2, 2, 64, 40, rng.integers(0, 20, 100), past=rng.integers(0, 20, 100), pool=120))


def test_attend_prompt_element_alignment():
    c = prompt_case(31, torch.bfloat16, 2, 1, 128, 100, [40, 60])
    d = {k: cu_(v) for k, v in c.items()}
    o, _ = sv.spec_attend_prompt(shifted(d["q"]), d["kv"], 0, d["cu"], d["pad"])
    want, tol = ref.attend_prompt(c["q"], c["kv"], 0, c["cu"], c["pad"])
    close(o, want, tol)


def test_attend_prompt_flags():
    c = prompt_case(27, torch.bfloat16, 2, 2, 64, 100, [10, 20, 30, 40])
    c["pad"][0] = 91
    c["start"][1] = -1
    c["start"][2] = 2 ** 31 - 1
    o, flags = run_prompt(c)
    assert flags.tolist() == [16, 16, 16, 0]
    assert (o[:60] == 7).all() and not (o[60:] == 7).any()
    c = prompt_case(28, torch.bfloat16, 2, 2, 64, 100, [10, 20, 30, 40])
    c["cu"][2] = 5   # descends: nothing is taken
    o, flags = run_prompt(c)
    assert flags.tolist() == [16] * 4 and (o == 7).all()
    c = prompt_case(29, torch.bfloat16, 2, 2, 64, 100, [10, 20])
    c["cu"][2] = 31  # past the packed rows
    o, flags = run_prompt(c)
    assert flags.tolist() == [0, 16] and (o[10:] == 7).all()


def test_attend_prompt_edges():
    kv = torch.zeros((1, 2, 3, 2, 40, 64), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    o, flags = sv.spec_attend_prompt(q, kv, 0, z, z[:3])
    assert o.numel() == 0 and (flags == 0).all()


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------
def append_ref(qkv, H, pos, qw, kw, eps, inv_freq, inter):
    """qkv [n, heads, D] -> exact q, k, v"""
    Hq = qkv.shape[1] - 2 * H
    x = qkv.double()
    q = ref.turned(ref.normed(x[:, :Hq], qw, eps), pos, inv_freq, inter)
    k = ref.turned(ref.normed(x[:, Hq:Hq + H], kw, eps), pos, inv_freq, inter)
    return q, k, qkv[:, Hq + H:]


def freqs(R, base=1e4):
    return None if R == 0 else (1.0 / base ** (torch.arange(0, R, 2).double() / R)).float()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,H,D,R,inter,norm", [
    (4, 2, 128, 128, False, "qk"), (1, 3, 64, 64, False, ""), (7, 2, 128, 128, True, "q"), (2, 1, 64, 32, False, "k"),
    (3, 2, 80, 80, False, "qk"), (2, 2, 256, 256, False, "qk"), (2, 2, 128, 0, False, "qk"), (2, 2, 96, 64, True, "qk"),
    (9, 1, 3, 2, False, "k"), (5, 1, 1, 0, False, "q")])
@pytest.mark.parametrize("form", ["chain", "staged", "prompt", "pool"])
def test_append(dt, G, H, D, R, inter, norm, form):
    dtype, g, rng = DT[dt], gen(31), np.random.default_rng(31)
    L, layer, S, eps = 2, 1, 90, 1e-5
    qw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if "q" in norm else None
    kw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if "k" in norm else None
    inv = freqs(R)
    kwargs = dict(q_weight=cu_(qw), k_weight=cu_(kw), eps=eps, interleaved=inter)
    heads = G * H + 2 * H
    B = 4
    if form == "prompt":
        lens = [5, 0, 31, 1]
        cu = np.concatenate([[0], np.cumsum(lens)])
        qkv = randn(g, (int(cu[-1]) + 2, heads, D), dtype)
        kv = randn(g, (L, 2, B, H, S, D), dtype)
        start, pad = i32([3, 0, 40, 7]), i32([0, 5, 19, 82])
        kvd, qd = kv.cuda(), torch.full((qkv.shape[0], G * H, D), 7.0, dtype=dtype, device="cuda")
        _, flags = sv.spec_append_prompt(qkv.cuda(), kvd, layer, i32(cu).cuda(), pad.cuda(), cu_(inv), start=start.cuda(),
                                         q_out=qd, **kwargs)
        seqs = [(b, slice(int(cu[b]), int(cu[b + 1])), torch.arange(lens[b]) + int(start[b]), b,
                 int(pad[b]) + int(start[b])) for b in range(B)]
        qkv_of, q_of = (lambda b, s: qkv[s]), (lambda b, s: qd[s])
        left = [qd[int(cu[-1]):]]
        st = None
    else:
        T = 6
        parent, n = ref.random_trees(rng, B, T)
        depth = ref.plan(parent, n)[1] if form == "staged" else None
        if form == "chain":
            n = np.array([6, 3, 0, 1], np.int32)
        pool = 7 if form == "pool" else 0
        idx = i32([6, 0, 3, 2]) if pool else None
        qkv = randn(g, (B, T, heads, D), dtype)
        kv = randn(g, (L, 2, pool or B, H, S, D), dtype)
        length, pad = i32([1, 80, 33, 64]), i32([0, 4, 11, 20])
        st = randn(g, (L, 2, B, H, T, D), dtype) if form == "staged" else None
        kvd, std = kv.cuda(), cu_(st)
        qd = torch.full((B, T, G * H, D), 7.0, dtype=dtype, device="cuda")
        _, flags = sv.spec_append_round(qkv.cuda(), kvd, layer, length.cuda(), None if pool else pad.cuda(), cu_(inv),
                                        depth=cu_(None if depth is None else i32(depth)), n_nodes=i32(n).cuda(),
                                        idx=cu_(idx), staged=std, q_out=qd, **kwargs)
        if pool:
            pad[:] = 0
        seqs = [(b, slice(0, int(n[b])),
                 (torch.arange(int(n[b])) if depth is None else torch.from_numpy(depth[b, :n[b]]).long()) +
                 int(length[b]) - 1, b if idx is None else int(idx[b]), int(pad[b]) + int(length[b]) - 1)
                for b in range(B)]
        qkv_of, q_of = (lambda b, s: qkv[b, s]), (lambda b, s: qd[b, s])
        left = [qd[b, int(n[b]):] for b in range(B)]
    assert (flags == 0).all()
    for x in left:
        assert (x == 7).all()
    want_kv, tol_kv = kv.double(), torch.zeros(kv.shape, dtype=torch.float64)
    want_st = None if st is None else st.double()
    tol_st = None if st is None else torch.zeros_like(want_st)
    for b, s, pos, row, slot in seqs:
        q, k, v = append_ref(qkv_of(b, s), H, pos, qw, kw, eps, inv, inter)
        close(q_of(b, s), q, ref.append_tol(q, dtype), "q")
        m = len(pos)
        to, tl = (want_st[layer, :, b, :, :m], tol_st[layer, :, b, :, :m]) if st is not None else \
            (want_kv[layer, :, row, :, slot:slot + m], tol_kv[layer, :, row, :, slot:slot + m])
        to[0], to[1] = k.transpose(0, 1), v.double().transpose(0, 1)
        tl[0] = ref.append_tol(k, dtype).transpose(0, 1)
    close(kvd, want_kv, tol_kv, "kv")  # every other byte as it was
    if st is not None:
        close(std, want_st, tol_st, "staged")


@pytest.mark.parametrize("pos", [0, 4095, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 66])
def test_append_far_positions(pos):
    """Angles of far positions: fp32 queries stay within fp32 of the formula."""
    g = gen(32)
    D, inv = 64, freqs(64, 5e5)
    qkv = randn(g, (1, 4, 3, D), torch.float32)
    kv = torch.zeros((1, 2, 1, 1, 8, D), device="cuda")
    depth = i32([[0, 1, 2, 3]]) + max(0, pos - 4)
    st = torch.zeros((1, 2, 1, 1, 4, D), device="cuda")
    q, flags = sv.spec_append_round(qkv.cuda(), kv, 0, i32([1]).cuda(), None, inv.cuda(), depth=depth.cuda(), staged=st)
    want, k, v = append_ref(qkv[0], 1, depth[0].long(), None, None, 0, inv, False)
    close(q[0], want, ref.append_tol(want, torch.float32))
    close(st[0, 0, 0].transpose(0, 1), k, ref.append_tol(k, torch.float32))
    assert torch.equal(st[0, 1, 0].transpose(0, 1).cpu(), v)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_append_many_sequences(dt):
    """More prompts than a warp has lanes, into a pool, from an odd offset."""
    g, rng = gen(35), np.random.default_rng(35)
    B, N, S, D, H, Hq = 100, 130, 30, 64, 2, 4
    lens = rng.integers(0, 12, B)
    cu = np.concatenate([[0], np.cumsum(lens)])
    start, pad, idx = rng.integers(0, 9, B), rng.integers(0, 9, B), rng.permutation(N)[:B]
    qkv, kv = randn(g, (int(cu[-1]), Hq + 2 * H, D), DT[dt]), randn(g, (1, 2, N, H, S, D), DT[dt])
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DT[dt])
    want_kv, tol_kv = kv.double(), torch.zeros(kv.shape, dtype=torch.float64)
    want_q, tol_q = torch.zeros(int(cu[-1]), Hq, D).double(), torch.zeros(int(cu[-1]), Hq, D).double()
    for b in range(B):
        s, at = slice(int(cu[b]), int(cu[b + 1])), int(pad[b] + start[b])
        q, k, v = append_ref(qkv[s], H, torch.arange(lens[b]) + int(start[b]), w, w, 1e-6, freqs(D), False)
        want_q[s], tol_q[s] = q, ref.append_tol(q, DT[dt])
        want_kv[0, :, idx[b], :, at:at + lens[b]] = torch.stack([k, v.double()]).transpose(1, 2)
        tol_kv[0, 0, idx[b], :, at:at + lens[b]] = ref.append_tol(k, DT[dt]).transpose(0, 1)
    for move in (lambda x: x, shifted):
        kvd = move(kv.cuda())
        q, flags = sv.spec_append_prompt(move(qkv.cuda()), kvd, 0, i32(cu).cuda(), i32(pad).cuda(), freqs(D).cuda(),
                                         q_weight=w.cuda(), k_weight=w.cuda(), start=i32(start).cuda(), idx=i32(idx).cuda())
        assert (flags == 0).all()
        close(q, want_q, tol_q)
        close(kvd, want_kv, tol_kv)


@pytest.mark.parametrize("dt,D", [("f32", 128), ("f32", 32), ("bf16", 128), ("bf16", 64), ("f16", 256), ("f16", 128)])
@pytest.mark.parametrize("G,H,inter,norm,rot", [(3, 3, False, "qk", True), (1, 9, True, "q", True), (7, 1, False, "k", False)])
def test_append_many_tokens(dt, D, G, H, inter, norm, rot):
    """Tokens enough for a warp each; numbers of heads that leave a warp's last
    step, or its step itself, part empty."""
    g = gen(39)
    B, n, S = 5, 1001, 1010
    M, Hq = B * n, G * H
    qkv = randn(g, (M + 2, Hq + 2 * H, D), DT[dt])
    qw = randn(g, (D,), DT[dt]) if "q" in norm else None
    kw = randn(g, (D,), DT[dt]) if "k" in norm else None
    inv = freqs(D) if rot else None
    kv = torch.full((1, 2, B, H, S, D), 7.0, dtype=DT[dt], device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    pad = i32([0, 9, 3, 1, 7])
    q, flags = sv.spec_append_prompt(qkv.cuda(), kv, 0, cu, pad.cuda(), cu_(inv), q_weight=cu_(qw), k_weight=cu_(kw),
                                     interleaved=inter)
    assert (flags == 0).all()
    want, k, v = append_ref(qkv[:M], H, torch.arange(n).repeat(B), qw, kw, 1e-6, inv, inter)
    close(q[:M], want, ref.append_tol(want, DT[dt]))
    for b in range(B):
        p = int(pad[b])
        got = kv[0, :, b].cpu()
        wk = k[b * n:(b + 1) * n].transpose(0, 1)
        close(got[0, :, p:p + n], wk, ref.append_tol(wk, DT[dt]))
        assert torch.equal(got[1, :, p:p + n].double(), v[b * n:(b + 1) * n].transpose(0, 1).double())
        assert (got[:, :, :p] == 7).all() and (got[:, :, p + n:] == 7).all()


def test_append_extreme_heads():
    """All-zero heads, large and tiny ones, one that is not finite."""
    g = gen(33)
    D = 128
    qkv = randn(g, (5, 3, D), torch.float32)
    qkv[0] = 0
    qkv[1] *= 1e15
    qkv[2] *= 1e-15
    qkv[3, 0, 5] = float("inf")
    w = torch.ones(D)
    kv = torch.zeros((1, 2, 1, 1, 8, D), device="cuda")
    q, _ = sv.spec_append_prompt(qkv.cuda(), kv, 0, i32([0, 5]).cuda(), None, freqs(D).cuda(), q_weight=w.cuda(),
                                 k_weight=w.cuda(), eps=0.0 + 1e-6)
    want, k, v = append_ref(qkv, 1, torch.arange(5), w, w, 1e-6, freqs(D), False)
    for i in (0, 1, 2, 4):
        close(q[i], want[i], ref.append_tol(want[i], torch.float32))
    assert torch.isnan(q[3]).any()
    close(kv[0, 0, 0, :, :5].transpose(0, 1), k, ref.append_tol(k, torch.float32))


def test_append_flags_and_repeated_rows():
    g = gen(34)
    B, T, D, H = 5, 3, 64, 1
    qkv = randn(g, (B, T, 4, D), torch.bfloat16).cuda()
    kv = randn(g, (1, 2, 6, H, 20, D), torch.bfloat16).cuda()
    before = kv.clone()
    length, pad = i32([0, 18, 5, 5, 5]).cuda(), i32([0, 1, 0, 0, -2]).cuda()
    q = torch.full((B, T, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, flags = sv.spec_append_round(qkv, kv, 0, length, pad, None, q_out=q)
    assert flags.tolist() == [16, 16, 0, 0, 16]
    assert torch.equal(kv[:, :, [0, 1, 4, 5]], before[:, :, [0, 1, 4, 5]]) and (q[[0, 1, 4]] == 7).all()
    assert torch.equal(q[2:4], qkv[2:4, :, :2])
    kv.copy_(before)
    idx = i32([1, 4, 2, 2, 9]).cuda()
    _, flags = sv.spec_append_round(qkv, kv, 0, i32([5] * 5).cuda(), None, None, idx=idx, q_out=q)
    assert flags.tolist() == [0, 0, 16, 16, 16]
    assert torch.equal(kv[:, :, [0, 2, 3, 5]], before[:, :, [0, 2, 3, 5]])
    # staged nodes are written by sequence: the same row twice is fine
    st = torch.zeros((1, 2, B, H, T, D), dtype=torch.bfloat16, device="cuda")
    _, flags = sv.spec_append_round(qkv, kv, 0, i32([5] * 5).cuda(), None, None, idx=idx, staged=st)
    assert flags.tolist() == [0, 0, 0, 0, 16] and torch.equal(st[0, 1, :4, 0], qkv[:4, :, 3])
    cu = i32([0, 3, 2, 5, 5, 6]).cuda()
    kv.copy_(before)
    _, flags = sv.spec_append_prompt(qkv[:2].reshape(6, 4, D), kv, 0, cu, None, None)
    assert flags.tolist() == [16] * 5 and torch.equal(kv, before)


@pytest.mark.parametrize("D", [64, 80])
def test_append_flags_of_more_sequences_than_tokens(D):
    """Sequences without a token are flagged like the others."""
    g = gen(37)
    B, N = 300, 400
    lens = np.zeros(B, np.int64)
    lens[[7, 150, 299]] = 1
    cu = i32(np.concatenate([[0], np.cumsum(lens)])).cuda()
    idx = np.random.default_rng(37).permutation(N)[:B]
    idx[3] = idx[200]
    idx[299] = N
    qkv = randn(g, (3, 3, D), torch.bfloat16).cuda()
    kv = torch.zeros((1, 2, N, 1, 4, D), dtype=torch.bfloat16, device="cuda")
    _, flags = sv.spec_append_prompt(qkv, kv, 0, cu, None, None, idx=i32(idx).cuda())
    want = np.zeros(B, int)
    want[[3, 200, 299]] = 16
    assert flags.tolist() == want.tolist()
    wrote = torch.zeros(N, dtype=torch.bool)
    wrote[[int(idx[7]), int(idx[150])]] = True
    assert torch.equal((kv[0, 0, :, 0, 0] != 0).any(-1).cpu(), wrote)
    # a round's dead nodes as well
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    _, flags = sv.spec_append_round(randn(g, (B, 1, 3, D), torch.bfloat16).cuda(), kv, 0, n + 1, None, None,
                                    idx=i32(idx).cuda(), n_nodes=n)
    assert flags.tolist() == want.tolist()


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64])
def test_tree_plan(T):
    rng = np.random.default_rng(T)
    parent, n = ref.random_trees(rng, 40, T)
    n[0] = 0
    for b in range(40):
        parent[b, n[b]:] = 99  # not looked at
    want_m, want_d = ref.plan(parent, n)
    mask, depth, flags = sv.spec_tree_plan(i32(parent).cuda(), i32(n).cuda())
    assert (flags == 0).all()
    assert np.array_equal(mask.cpu().numpy(), want_m) and np.array_equal(depth.cpu().numpy(), want_d)


def test_verify_tree_from_an_odd_offset():
    x, tokens, parent, n = verify_case(45, "bf16", 5, 9, 1001, 0.9)
    d = shifted(x.cuda())
    got = sv.spec_verify_tree(d, i32(tokens).cuda(), i32(parent).cuda(), n_nodes=i32(n).cuda())
    want = sv.spec_verify_tree(x.cuda(), i32(tokens).cuda(), i32(parent).cuda(), n_nodes=i32(n).cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tree_plan_flags():
    parent = i32([[-1, 0, 1], [-1, 1, 0], [0, 0, 0], [-1, 0, -1], [-1, 0, 3], [-1, 0, 0], [-1, 0, 0]])
    mask, depth, flags = sv.spec_tree_plan(parent.cuda(), i32([3, 3, 3, 3, 3, 4, -1]).cuda())
    assert flags.tolist() == [0] + [32] * 6
    assert (mask[1:] == 0).all() and (depth[1:] == 0).all()


def verify_case(seed, dt, B, T, V, alpha, values="normal"):
    rng = np.random.default_rng(seed)
    parent, n = ref.random_trees(rng, B, T)
    x = torch.randn((B, T, V), generator=gen(seed))
    if values == "ties":
        x = (x * 2).round() / 2
    x = x.to(DT[dt])
    best = x.double().numpy().argmax(-1)
    tokens = rng.integers(0, V, (B, T))
    for b in range(B):
        for i in range(1, T):
            if rng.random() < alpha:
                tokens[b, i] = best[b, parent[b, i]]
    return x, tokens.astype(np.int32), parent, n


def check_verify(x, tokens, parent, n, eos=-1, rem=None):
    B, T, V = x.shape
    got = sv.spec_verify_tree(x.cuda(), i32(tokens).cuda(), i32(parent).cuda(), n_nodes=i32(n).cuda(), eos_id=eos,
                              remaining=cu_(None if rem is None else i32(rem)))
    out, path, na, ne, flags = (t.cpu().numpy() for t in got)
    assert (flags == 0).all()
    xs = x.double().numpy()
    for b in range(B):
        t, p, acc = ref.walk(xs[b], tokens[b], parent[b], int(n[b]), eos, 1 << 30 if rem is None else int(rem[b]))
        m = len(t)
        assert ne[b] == m and na[b] == acc, (b, ne[b], m)
        assert out[b, :m].tolist() == t and path[b, :m].tolist() == p
        assert (out[b, m:] == -1).all() and (path[b, m:] == -1).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,V,alpha", [(3, 1, 1, 0.5), (5, 9, 7, 0.9), (7, 26, 1000, 0.8), (4, 64, 32003, 0.95),
                                         (2, 13, 128256, 0.7), (40, 33, 255, 0.6)])
def test_verify_tree(dt, B, T, V, alpha):
    check_verify(*verify_case(41, dt, B, T, V, alpha))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_verify_tree_ties_stops_and_budgets(dt):
    x, tokens, parent, n = verify_case(42, dt, 30, 20, 50, 0.9, values="ties")
    check_verify(x, tokens, parent, n, eos=3)
    check_verify(x, tokens, parent, n, rem=np.arange(30) % 5 - 1)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_verify_tree_values_that_are_not_finite(dt):
    x, tokens, parent, n = verify_case(43, dt, 6, 12, 40000, 0.9)
    x[0, :, 31234] = NAN
    x[0, :, 39999] = NAN
    x[1] = float("-inf")
    x[2, :, 17] = float("inf")
    x[3, 0, :] = -0.0
    x[3, 0, 5] = 0.0
    tokens[1], tokens[0], tokens[2] = 0, 31234, 17
    check_verify(x, tokens, parent, n)


def test_verify_tree_flags():
    x, tokens, parent, n = verify_case(44, "f32", 4, 5, 100, 0.9)
    n[:] = [5, 6, -1, 5]
    parent[3, 2] = 2
    got = sv.spec_verify_tree(x.cuda(), i32(tokens).cuda(), i32(parent).cuda(), n_nodes=i32(n).cuda())
    assert got[4].tolist() == [0, 32, 32, 32] and got[3].tolist()[1:] == [0, 0, 0]
    assert (got[0][1:] == -1).all() and (got[1][1:] == -1).all()


def test_verify_tree_of_a_chain_is_the_chain_verification():
    from specgen import greedy_round_inputs

    B, k, V = 16, 5, 3000
    x, d = greedy_round_inputs(B, k, V, 0.7, 1.0, seed=5, dtype="f32")
    xt, dt = torch.from_numpy(x).cuda(), torch.from_numpy(d).cuda()
    want = sv.spec_verify_greedy(xt, dt, eos_id=3)
    tokens = torch.cat([torch.zeros((B, 1), dtype=torch.int32, device="cuda"), dt], 1)
    parent = torch.arange(-1, k, dtype=torch.int32, device="cuda").expand(B, k + 1).contiguous()
    got = sv.spec_verify_tree(xt, tokens, parent, eos_id=3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[1]) and torch.equal(got[3], want[2])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,H,L,pool", [(64, 3, 2, 0), (128, 4, 5, 9), (5, 1, 3, 0), (80, 2, 1, 7)])
def test_commit_tree(dt, D, H, L, pool):
    dtype, g, rng = DT[dt], gen(51), np.random.default_rng(51)
    B, T, S = 6, 10, 40
    st = randn(g, (L, 2, B, H, T, D), dtype)
    kv = randn(g, (L, 2, pool or B, H, S, D), dtype)
    ne = np.array([1, 10, 0, 3, 4, 2], np.int32)
    path = np.full((B, T), -1, np.int32)
    for b in range(B):
        path[b, :ne[b]] = np.sort(rng.choice(T, ne[b], replace=False))
    length, pad = i32([1, 31, 20, 5, 9, 30]), i32([0, 0, 3, 7, 1, 9])
    idx = i32(rng.permutation(pool)[:B]) if pool else None
    if pool:
        pad[:] = 0
    want = kv.clone()
    for b in range(B):
        row, slot = b if idx is None else int(idx[b]), int(pad[b] + length[b]) - 1
        want[:, :, row, :, slot:slot + ne[b]] = st[:, :, b][:, :, :, path[b, :ne[b]].astype(int)]
    kvd = kv.cuda()
    flags = sv.spec_commit_tree(st.cuda(), kvd, length.cuda(), pad.cuda(), i32(path).cuda(), i32(ne).cuda(), idx=cu_(idx))
    assert (flags == 0).all() and torch.equal(kvd.cpu(), want)


def test_commit_tree_flags():
    B, T, S, D = 8, 4, 20, 64
    g = gen(52)
    st, kv = randn(g, (1, 2, B, 1, T, D), torch.bfloat16).cuda(), randn(g, (1, 2, B, 1, S, D), torch.bfloat16).cuda()
    before = kv.clone()
    path = i32([[0, 1, 2, 3]] * B)
    path[0, 1] = 4
    path[1, 0] = -1
    args = [i32([5, 5, 0, 18, 5, 5, 5, 5]).cuda(), i32([0, 0, 0, 0, -1, 0, 0, 0]).cuda(), path.cuda(),
            i32([2, 1, 1, 4, 1, 5, -1, 0]).cuda()]
    flags = sv.spec_commit_tree(st, kv, *args)
    assert flags.tolist() == [16] * 7 + [0] and torch.equal(kv, before)
    good = [i32([5] * B).cuda(), None, i32([[0, 1, 2, 3]] * B).cuda(), i32([2] * B).cuda()]
    flags = sv.spec_commit_tree(st, kv, *good, idx=i32([0, 1, 2, 2, 4, 8, -1, 7]).cuda())
    assert flags.tolist() == [0, 0, 16, 16, 0, 16, 16, 0]
    for r in (2, 3, 5, 6):
        assert torch.equal(kv[:, :, r], before[:, :, r])


# ---------------------------------------------------------------------------
# all of them
# ---------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """Append, prompt attention and commit at the far end of a cache of more
    than 2^32 elements, and a walk over logits of more than 2^31."""
    free, _ = torch.cuda.mem_get_info()
    N, H, S, D = 33, 2, 1 << 18, 128
    if free < 2 * N * H * S * D * 2 + (8 << 30):
        pytest.skip("not enough memory")
    g = gen(60)
    kv = torch.empty((1, 2, N, H, S, D), dtype=torch.bfloat16, device="cuda")
    idx, pad, n = i32([N - 1, N - 2]), i32([S - 110, 3]), [100, 77]
    cu = i32([0, 100, 177])
    qkv = randn(g, (177, 4 + 2 * H, D), torch.bfloat16)
    q, flags = sv.spec_append_prompt(qkv.cuda(), kv, 0, cu.cuda(), pad.cuda(), None, idx=idx.cuda())
    assert (flags == 0).all() and torch.equal(q.cpu(), qkv[:, :4])
    small = torch.zeros((1, 2, 2, H, 120, D), dtype=torch.bfloat16)
    for b in range(2):
        x, p = qkv[cu[b]:cu[b + 1]], int(pad[b])
        small[0, 0, b, :, :n[b]] = x[:, 4:4 + H].transpose(0, 1)
        small[0, 1, b, :, :n[b]] = x[:, 4 + H:].transpose(0, 1)
        assert torch.equal(kv[0, :, int(idx[b]), :, p:p + n[b]].cpu(), small[0, :, b, :, :n[b]])
    o, flags = sv.spec_attend_prompt(q, kv, 0, cu.cuda(), pad.cuda(), idx=idx.cuda())
    want, tol = ref.attend_prompt(qkv[:, :4], small, 0, cu, i32([0, 0]), i32([0, 0]))
    assert (flags == 0).all()
    close(o, want, tol)
    st = randn(g, (1, 2, 2, H, 5, D), torch.bfloat16)
    path = i32([[0, 2, 4, -1, -1], [0, 1, -1, -1, -1]])
    flags = sv.spec_commit_tree(st.cuda(), kv, i32([101, 78]).cuda(), pad.cuda(), path.cuda(), i32([3, 2]).cuda(), idx=idx.cuda())
    assert (flags == 0).all()
    for b, rows in ((0, [0, 2, 4]), (1, [0, 1])):
        at = int(pad[b]) + n[b]
        assert torch.equal(kv[0, :, int(idx[b]), :, at:at + len(rows)].cpu(), st[0, :, b][:, :, rows])
    del kv
    B, T, V = 2, 64, 17_000_000
    x = torch.zeros((B, T, V), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    best = [[int(v) for v in torch.randint(0, V, (T,), generator=g)] for _ in range(B)]
    for b in range(B):
        for i in range(T):
            x[b, i, best[b][i]] = 1
    parent = i32([list(range(-1, T - 1))] * B)
    tokens = i32([[0] + r[:-1] for r in best])
    out, path, acc, emit, flags = sv.spec_verify_tree(x, tokens.cuda(), parent.cuda())
    assert (flags == 0).all() and emit.tolist() == [T] * B and acc.tolist() == [T - 1] * B
    assert out.tolist() == best and path.tolist() == [list(range(T))] * B


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_calls_on_two_streams_at_once(dt):
    """Two rounds of calls on streams of their own, and two captured ones
    replayed side by side, give what each gives alone."""
    cases = [round_case(61, DT[dt], 6, 9, 4, 2, 64, 900, [800, 500, 60, 700, 3, 350]),
             round_case(62, DT[dt], 3, 64, 4, 2, 128, 700, [600, 20, 333], tree=True, staged=True)]
    dev = [{k: cu_(v) for k, v in c.items()} for c in cases]
    g = gen(63)
    logits = randn(g, (7, 9, 5000), DT[dt]).cuda()
    parent = i32([list(range(-1, 8))] * 7).cuda()
    tokens = torch.cat([parent[:, :1], logits.float().argmax(-1).to(torch.int32)[:, :-1]], 1)

    def work(d):
        o, f = sv.spec_attend_round(d["q"], d["kv"], 1, d["length"], d["pad"], tree_mask=d["mask"], n_nodes=d["n"],
                                    staged=d["staged"], out=torch.zeros_like(d["q"]))
        return (o, f) + sv.spec_verify_tree(logits, tokens, parent)

    alone = [work(d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = [[], []]
    for _ in range(20):
        for i, (s, d) in enumerate(zip(streams, dev)):
            with torch.cuda.stream(s):
                got[i].append(work(d))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for r in got[i] for x, y in zip(r, alone[i]))
    graphs, outs = [], []
    for d in dev:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append([work(d) for _ in range(10)])
        graphs.append(gr)
    for _ in range(3):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for r in outs[i] for x, y in zip(r, alone[i]))
