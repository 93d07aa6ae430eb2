"""Masks and values that are not finite in the round kernels for more than 64
query rows a key head (one and two query tiles of the tensor cores), and through
CTAs that walk several units."""
import numpy as np
import pytest
import torch

import forward_ref as ref
import speculative_decoding_verification_28_gb300 as sv
from test_gpu_forward import DT, NAN, close, i32, round_case, run_round

pytestmark = pytest.mark.gpu
# rows a key head: 12 and 100 (one tile), 256 and 448 (two), 130 and 150 (two, the second nearly empty)
SHAPES = [(6, 2, 64), (20, 5, 128), (20, 5, 64), (64, 4, 128), (64, 4, 64), (64, 7, 128), (26, 5, 64), (50, 3, 128)]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,G,D", SHAPES)
def test_rows_that_see_nothing_give_zeros(dt, T, G, D):
    c = round_case(70, DT[dt], 5, T, G, 2, D, 340, [1, 1, 1, 150, 260], tree=True, staged=True, full=True)
    c["mask"][0] = 0                       # no prefix, no node: all zeros
    c["mask"][1, ::2] = 0
    c["mask"][2, T // 2:] = 0              # whole query tiles without a key
    c["mask"][3] = 0                       # only the prefix
    c["n"][2] = T - 1
    c["mask"][2, 0] = -1                   # bits past the nodes are ignored
    o, flags = run_round(c)
    want, tol = ref.attend_round(c["q"], c["kv"], 1, c["length"], c["pad"], c["mask"], c["n"], c["idx"], c["staged"])
    assert (flags == 0).all()
    close(o, want, tol)
    assert (o[0] == 0).all() and (o[1, ::2] == 0).all() and (o[2, T // 2:T - 1] == 0).all() and (o[2, T - 1] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("lens", [[140], [1], [128, 700, 1]])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(dt, T, G, D, lens):
    """Children of one root, each of which sees itself and the root: node x holds inf, y NaN (key and value)."""
    B = len(lens)
    c = round_case(71, DT[dt], B, T, G, 2, D, 800, lens, tree=True, staged=True, full=True)
    c["mask"] = (torch.ones(T, dtype=torch.int64) << torch.arange(T)).bitwise_or(torch.tensor(1)).repeat(B, 1)
    x, y = T // 2, T - 1
    c["staged"][1, 1, :, :, x, 5] = float("inf")
    c["staged"][1, 1, :, :, x, D - 1] = float("-inf")
    c["staged"][1, 1, :, :, y, 6] = NAN
    c["staged"][1, 0, :, :, y, 6] = NAN
    o, flags = run_round(c)
    want, tol = ref.attend_round(c["q"], c["kv"], 1, c["length"], c["pad"], c["mask"], c["n"], None, c["staged"])
    assert (flags == 0).all()
    rest = [i for i in range(T) if i not in (x, y)]
    close(o[:, rest], want[:, rest], tol[:, rest])
    assert (o[:, x, :, 5] == float("inf")).all() and (o[:, x, :, D - 1] == float("-inf")).all()
    assert torch.isnan(o[:, y]).all()
    keep = [d for d in range(D) if d not in (5, D - 1)]
    close(o[:, x][..., keep], want[:, x][..., keep], tol[:, x][..., keep])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,G,D", SHAPES)
def test_they_stay_with_their_sequence_where_a_cta_walks_many(dt, T, G, D):
    """More units than CTAs: sequences with and without such nodes follow one another in a CTA."""
    B, H, S = 420, 2, 24
    rng = np.random.default_rng(72)
    g = torch.Generator(device="cuda").manual_seed(72)
    dtype = DT[dt]
    lens = rng.integers(1, S + 1, B)
    kv = torch.randn((1, 2, B, H, S, D), generator=g, device="cuda").to(dtype)
    st = torch.randn((1, 2, B, H, T, D), generator=g, device="cuda").to(dtype)
    q = torch.randn((B, T, G * H, D), generator=g, device="cuda").to(dtype)
    mask = (torch.ones(T, dtype=torch.int64) << torch.arange(T)).bitwise_or(torch.tensor(1)).repeat(B, 1)
    def call(staged):
        out, flags = sv.spec_attend_round(q, kv, 0, i32(lens).cuda(), None, tree_mask=mask.cuda(), staged=staged)
        assert (flags == 0).all()
        return out

    clean = call(st)
    dirty = st.clone()
    odd = rng.random(B) < 0.4
    odd[:3] = [False, True, False]
    odd[-2:] = [True, False]
    for b in np.flatnonzero(odd):
        dirty[0, 1, b, :, int(rng.integers(1, T)), int(rng.integers(0, D))] = float("inf") if b % 2 else NAN
    out = call(dirty)
    bad = ~torch.isfinite(dirty[0, 1]).all(-1).all(1)  # [B, T] nodes
    assert torch.equal(out[~bad], clean[~bad])          # every other row, in every sequence, keeps its bits
    hit = out[bad]
    assert (~torch.isfinite(hit)).any(-1).all()
    # and nothing of it is left for the next call
    assert torch.equal(call(st), clean)
    # one clean sequence against the formula
    b = int(np.flatnonzero(~odd)[5])
    want, tol = ref.attend_round(q[b:b + 1].cpu(), kv[:, :, b:b + 1].cpu(), 0, lens[b:b + 1], [0], mask[b:b + 1], None, None,
                                 st[:, :, b:b + 1].cpu())
    close(out[b:b + 1], want, tol)
