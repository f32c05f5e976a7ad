"""Values at the edge in the attention layers' cache: infinities and NaN beside places that are
only copied, scales and scores far from one, and codes on a rounding tie.

Tolerances are derived where each test states them; u is the unit roundoff as in
test_attn_gpu.py (2^-24 fp32, 2^-8 bf16, 2^-11 fp16, 2^-22 for sums of tensor cores).
"""
import math

import numpy as np
import pytest
import torch

from test_attn_gpu import BF, F8, F32, attn, attn_problem, check_attn, new_pools, np64, rot_tables  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- places that are not rotated ------------------------------------------------


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("D,R", [(64, 0), (64, 16), (64, 48), (128, 0), (128, 32), (128, 96)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [9, 2500])
def test_append_copies_unrotated_places(attn, T, dt, D, R, interleaved):
    """Without a norm the places from R on are a copy, bit for bit: an infinity, a NaN or a
    negative zero among them stays where it is, in queries, keys and values."""
    Hq, Hkv = 4, 2
    g = torch.Generator().manual_seed(D + R)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dt)
    plain = x.clone()
    for t, value in ((0, float("inf")), (1, float("-inf")), (2, float("nan")), (3, -0.0)):
        for place in (R, R + 7, D - 1, D - 16):
            x[t, :, max(place, R)] = value
    x[4, :, R:] = -0.0
    x[5, :, R::2] = -0.0
    cos = sin = pos = None
    if R:
        cos, sin = (y.cuda() for y in rot_tables(3 * T, R))
        pos = torch.arange(T, dtype=torch.int32).cuda() * 3
    slots = torch.arange(T, dtype=torch.int32).cuda()

    def append(y):
        y = y.cuda()
        kc, vc, _, _ = new_pools(-(-T // 4), Hkv, 4, D, dt)
        q = attn.kv_append(y[:, :Hq], y[:, Hq: Hq + Hkv], y[:, Hq + Hkv:], slots, kc, vc, positions=pos,
                           cos=cos, sin=sin, interleaved=interleaved)
        back = [p.transpose(1, 2).reshape(-1, Hkv, D)[:T] for p in (kc, vc)]
        return torch.cat([q] + back, 1).cpu()

    got, want = append(x), append(plain)
    assert torch.equal(bits(got[..., :R]), bits(want[..., :R])) or R == 0     # rotated ones as without them
    kept, held = got[..., R:], x[..., R:]
    nan = torch.isnan(held)
    assert torch.equal(torch.isnan(kept), nan)
    assert torch.equal(bits(kept)[~nan], bits(held)[~nan])
