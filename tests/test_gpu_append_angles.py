"""Rotation angles of far positions and large frequencies, to the last places.

A head whose pairs are (1, 0) turns into its cosines and sines.  Their error:
the library's sine and cosine of half turns, one unit in the last place of a
value up to 1 (2^-24); the correction's rounding (2^-25); the angle, 1e-8 turns
(2 pi 1e-8 = 6.3e-8).  The rotation itself is exact here: 1 c - 0 s."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_28_gb300 as sv

TOL = 2.0 ** -24 + 2.0 ** -25 + 2 * math.pi * 1e-8
PI = 31415926535897932384626433832795028841971693993751058209749445923078164062862090  # 10^79 pi
BITS = 200
INV = (10 ** 79 << BITS) // (2 * PI)  # 2^BITS / (2 pi)


def turns(pos, f):
    """Fraction of pos * f / (2 pi), exact to far below fp64's last place."""
    m, e = math.frexp(float(np.float32(f)))
    m, e = int(m * (1 << 24)), e - 24  # f = m 2^e
    x = int(pos) * m * INV
    x = x << e if e >= 0 else x >> -e
    return (x & ((1 << BITS) - 1)) / (1 << BITS)


def test_turns_of_plain_angles():
    for pos, f in ((1, 1.0), (3, 0.25), (10, 7.5)):
        x = pos * f / (2 * math.pi)
        assert abs(turns(pos, f) - (x - math.floor(x))) < 1e-14


FREQS = {"one": np.linspace(1.0, 0.7, 32), "small": 1e6 ** -(np.arange(32) / 32), "large": np.geomspace(1.5, 1000.0, 32)}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(FREQS))
@pytest.mark.parametrize("top", [4000, 4 * 10 ** 4, 10 ** 6, (1 << 22) + 1000, (1 << 24) - 1, (1 << 24) + 5000, 2 ** 31 - 66])
@pytest.mark.parametrize("D", [64, 66])  # a lane's vectors, and a warp a head
def test_append_angles_to_the_last_places(kind, top, D):
    rng = np.random.default_rng(top)
    B, T, R = 2, 64, 64
    inv = torch.from_numpy(FREQS[kind].astype(np.float32))
    pos = top - rng.integers(0, top // 3, (B, T))
    pos[0, 0] = top
    qkv = torch.zeros((B, T, 3, D))
    qkv[..., :R // 2] = 1
    kv = torch.zeros((1, 2, B, 1, 4, D), device="cuda")
    st = torch.zeros((1, 2, B, 1, T, D), device="cuda")
    q, flags = sv.spec_append_round(qkv.cuda(), kv, 0, torch.ones(B, dtype=torch.int32, device="cuda"), None, inv.cuda(),
                                    depth=torch.from_numpy(pos.astype(np.int32)).cuda(), staged=st)
    assert (flags == 0).all()
    frac = np.array([[[turns(p, f) for f in inv.tolist()] for p in row] for row in pos.tolist()]) * 2 * math.pi
    got = q[:, :, 0].cpu().double().numpy()
    assert np.abs(got[..., :R // 2] - np.cos(frac)).max() <= TOL
    assert np.abs(got[..., R // 2:R] - np.sin(frac)).max() <= TOL
    assert torch.equal(st[0, 0, :, 0], q[:, :, 0])
