"""Angles of asm_rope at far positions, against exact arithmetic."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import paged_common as C
from long_prefix_attention_b200 import ops

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turn(p, f):
    """(cos, sin) of the angle p f: the turns are exact decimals, reduced to half a turn."""
    with localcontext() as ctx:
        ctx.prec = 75
        t = Decimal(int(p)) * Decimal(float(f)) / (2 * PI)
        t -= t.to_integral_value()
        a = float(2 * PI * t)
    return math.cos(a), math.sin(a)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rot", [128, 50])
def test_angles_are_exact_to_a_2_32nd_of_a_turn(dt, layout, rot):
    """Pairs (1, 0) become (cos, sin).  The angle is off by at most 2^-32 turns at any
    position; the sine and cosine of its rest (an eighth of a turn at most) take 2 ulp in
    fp32 (4 u of the result, with its rounding) and 2^-21 by the hardware for bf16; the
    result is rounded once."""
    d, u = 128, C.U[dt]
    rng = np.random.default_rng(3)
    pos = np.concatenate([[0, 1, -1, 2**31 - 1, -2**31, 2**30, 999983], rng.integers(2**30, 2**31, 60),
                          rng.integers(-2**31, 0, 30), rng.integers(0, 2**20, 20)])
    T = len(pos)
    f = C.freqs(rot, 500000.0)
    f[1] = 1.0 / 3.0
    ref = torch.tensor([[turn(p, x) for x in f.tolist()] for p in pos], dtype=torch.float64)
    x = torch.zeros(T, 1, d, dtype=dt, device="cuda")
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    x[..., i] = 1
    y = torch.empty_like(x)
    ops.asm_rope(x, torch.as_tensor(pos.astype(np.int32)).cuda(), f.cuda(), y, layout=layout)
    got = y.cpu().double()[:, 0]
    err = torch.stack([got[:, i], got[:, j]], -1) - ref
    bound = 2 * math.pi * 2.0 ** -32 + (4 * u if dt is torch.float32 else u) * ref.abs() + \
        (2.0 ** -21 if dt is torch.bfloat16 else 0.0)
    assert (err.abs() <= bound).all(), float((err.abs() / bound).max())
