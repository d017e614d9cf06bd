"""Rotary positions of slow pairs, as stretched frequencies for long contexts have them, near the beginning: the sine of an angle far below
2^-32 of a turn's use is as good as the angle's 32-bit value.

Tolerance. The angle, a 64-bit fraction of a turn, is rounded to 32 bits (2^-24 of itself) and the sine is within two units of 2^-24 of its value: with the
product's rounding below 2^-21 of the result; then one rounding to the type."""
import math

import pytest
import torch

import cache_ref as ref
import swiglu_fp8_activation_gb300 as sgq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
def test_slow_pairs_at_near_positions(layout, inverse):
    R = 128
    freqs, _ = sgq.rope_frequencies(R, 500000.0, scaling="linear", stretch=64.0, device="cpu")
    pos = torch.tensor([1, 2, 3, 5, 17, 100, -1, -7])
    x = torch.zeros(len(pos), 2, R, dtype=BF16)
    first = (lambda h: slice(0, R // 2) if h == 0 else slice(R // 2, R)) if layout == "half" else (lambda h: slice(h, R, 2))
    x[:, 0, first(0)], x[:, 1, first(1)] = 1.0, -3.0                  # (1, 0) and (0, -3)
    got = sgq.rope(x.to(DEV), pos.to(DEV), freqs.to(DEV), layout=layout, inverse=inverse).cpu()
    turns = torch.tensor([[p * f / 2.0 ** 64 for f in freqs.tolist()] for p in pos.tolist()], dtype=torch.float64)
    turns = turns - turns.round()                                     # 53 bits of a product that no turn has passed by: exact to 2^-53
    angle = 2 * math.pi * turns * (-1 if inverse else 1)
    want = torch.zeros(x.shape, dtype=torch.float64)
    want[:, 0, first(0)], want[:, 0, first(1)] = angle.cos(), angle.sin()
    want[:, 1, first(0)], want[:, 1, first(1)] = 3 * angle.sin(), -3 * angle.cos()
    # of an angle near half a turn or a quarter, what is small is small beside 2^-24 of that turn
    near = (turns.abs() < 0.1).unsqueeze(1).repeat_interleave(2, 1)
    near = torch.cat((near, near), -1) if layout == "half" else near.repeat_interleave(2, -1)
    tol = 2.0 ** -21 * torch.where(near, want.abs(), 3.0)
    ref.check(got, want, tol + ref.rounding(want.abs() + tol, BF16))
