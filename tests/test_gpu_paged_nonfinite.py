"""asm_shared_attention with infinities and NaN among the keys and values that
tokens do see."""
import math

import pytest
import torch

import paged_common as C
from test_gpu_paged import Batch

pytestmark = pytest.mark.gpu


def signed_queries(b):
    """Component 0 of every query: 2 for even tokens, -2 for odd ones."""
    t = torch.arange(b.q.shape[0])
    b.q[..., 0] = torch.where(t % 2 == 0, 2.0, -2.0).to(b.q.dtype)[:, None]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tok", [1, 6, 40, 100])
@pytest.mark.parametrize("where", ["prefix", "local"])
def test_an_infinite_key_in_every_column(dt, tok, where):
    """32 rows, each with one key of +inf, at place r of a unit that all its tokens
    see: a score of +inf makes the token's result NaN (inf - inf, as in the formula),
    one of -inf gives the key no weight, wherever the key lies and however many query
    rows share a tile (12 to 200; whole key lists of one worker and split ones)."""
    R, G, Hkv = 32, 2, 8
    if where == "prefix":
        b = Batch(dt, G * Hkv, Hkv, 64, 32, new=[tok] * R, seq=[tok] * R, goff=list(range(R + 1)), pre=[128] * R, seed=31)
    else:
        b = Batch(dt, G * Hkv, Hkv, 64, 32, new=[tok] * R, seq=[128 + tok] * R, seed=31)
    signed_queries(b)
    _, _, _, dot, cnt = b.ref()               # with finite keys: bounds the other keys' logits
    for r in range(R):
        page = int((b.ptable if where == "prefix" else b.table)[r, 0])
        b.kd[page, :, r, 0] = math.inf
    out, lse = b.run()
    ref, rl, a, _, _ = b.ref()
    o, z = out.cpu().double(), lse.cpu().double()
    even = torch.arange(R * tok) % 2 == 0
    assert torch.isnan(ref[even]).all() and torch.isfinite(ref[~even]).all()
    assert torch.isnan(o[even]).all() and not torch.isfinite(z[even]).any()
    odd = ~even
    eo, ez = C.attention_bounds(ref[odd], rl[odd], a[odd], dot[odd], cnt[odd], 64, b.dt)
    assert ((o[odd] - ref[odd]).abs() <= eo).all() and ((z[odd] - rl[odd]).abs() <= ez).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tok", [1, 6, 40, 100])
def test_scores_of_minus_infinity_alone(dt, tok):
    """Every key of +inf: tokens with a negative query component see scores of -inf
    alone, which is no key at all (0, -inf), the others NaN."""
    R = 30
    b = Batch(dt, 16, 8, 64, 32, new=[tok] * R, seq=[tok + 128] * R, goff=list(range(R + 1)), pre=[128] * R, seed=32)
    signed_queries(b)
    b.kd[..., 0] = math.inf
    out, lse = b.run()
    o, z = out.cpu(), lse.cpu()
    even = torch.arange(R * tok) % 2 == 0
    assert torch.isnan(o[even]).all() and not torch.isfinite(z[even]).any()
    assert (o[~even] == 0).all() and (z[~even] == -math.inf).all()
