"""Many keys of small weight beside one of weight 1: together they may be most
of a result that the large one's value (0) leaves out.

Weights in fp16 are held 2^11 times as large, with steps of 2^-24 below 2^-14,
so that each is off by up to u of itself, or by 2^-36: beside the bound of
forward_ref (u |exact| + A (u + 2 E + 2 (n + 64) u32)) a sum of n weights may be
off by n 2^-36 / l, l >= 1, times the values' largest (here 1); and an fp16
result below 2^-14 has steps of 2^-24."""
import math

import pytest
import torch

import speculative_decoding_verification_28_gb300 as sv
from test_gpu_forward import DT, i32

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def keys(dt, n, D, gap, S):
    """One key of score 0 and value 0, n - 1 of score -gap and value 1 (scale 1, queries e_0)."""
    kv = torch.zeros((1, 2, 1, 1, S, D), dtype=DT[dt], device="cuda")
    kv[0, 0, 0, 0, :, 0] = -gap
    kv[0, 0, 0, 0, 0, 0] = 0
    kv[0, 1, 0, 0, 1:] = 1
    return kv


def check(out, n, gap, dt):
    """out [rows, D] whose row i sees the first n[i] keys; the scores are the keys as stored (in bf16
    17.6875 is 17.75)"""
    gap = float(torch.tensor(gap).to(DT[dt]))
    w = math.exp(-gap)
    u = torch.finfo(DT[dt]).eps / 2
    for i, m in enumerate(n):
        small = (m - 1) * w
        want = small / (1 + small)
        weights = 0.0 if dt == "f32" else u
        tol = want * (u + weights + 2 * (gap * 72 * U32 + 2.0 ** -21) + 2 * (m + 64) * U32)
        if dt == "f16":
            tol += m * 2.0 ** -36 + 2.0 ** -25
        got = out[i].double()
        assert float((got - want).abs().max()) <= tol, (i, m, float(got[0]), want, tol)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("gap", [9.0, 15.0, 17.6875, 20.0])
@pytest.mark.parametrize("T,G,D", [(1, 4, 64), (9, 4, 128), (20, 5, 128), (64, 4, 64)])
def test_round(dt, gap, T, G, D):
    # the large key in the first tile, alone, and in the last
    n = 40000
    for flip in (False, True):
        kv = keys(dt, n, D, gap, n + T)
        if flip:
            kv[0, :, 0, 0, :n - 1] = kv[0, :, 0, 0, :n - 1].flip(1)
        q = torch.zeros((1, T, G, D), dtype=DT[dt], device="cuda")
        q[..., 0] = 1
        out, flags = sv.spec_attend_round(q, kv, 0, i32([n]).cuda(), None, scale=1.0)
        assert (flags == 0).all()
        for t in (0, T // 2, T - 1):
            check(out[0, t], [n + t] * G, gap, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("gap", [9.0, 17.6875])
@pytest.mark.parametrize("m,past", [(60, 9000), (700, 9000)])  # small units and large ones
@pytest.mark.parametrize("D", [64, 128])
def test_prompt(dt, gap, m, past, D):
    kv = keys(dt, past + m, D, gap, past + m)
    q = torch.zeros((m, 2, D), dtype=DT[dt], device="cuda")
    q[..., 0] = 1
    out, flags = sv.spec_attend_prompt(q, kv, 0, i32([0, m]).cuda(), None, start=i32([past]).cuda(), scale=1.0)
    assert (flags == 0).all()
    for h in (0, 1):
        check(out[:, h], [past + i + 1 for i in range(m)], gap, dt)
