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


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_in_a_very_long_key_list(d):
    """296 prefixes of 1.6 million keys (1024 keys of 8 pages, over and over), 32 query rows each, two whole
    lists per SM: infinite and NaN values in 8 places spread over the columns are found in time
    (the other warps' waits have a limit of about a second), and a value that only the last token of a row sees
    reaches it alone."""
    R, tok, G, S, reps = 296, 4, 8, 128, 1600
    b = Batch("bf16", G, 1, d, S, new=[tok] * R, seq=[tok] * R, goff=list(range(R + 1)), pre=[1024] * R, seed=33)
    pages = torch.as_tensor(b.ptable[0, :8])
    b.ptable = pages.repeat(reps).expand(R, 8 * reps).numpy().copy()
    b.pre = [1024 * reps] * R
    b.dev["prefix_table"] = torch.as_tensor(b.ptable, dtype=torch.int32).cuda()
    vals = torch.zeros(d)                  # what each column's sum becomes
    for i in range(8):
        c = i * (d // 8) + 3
        vals[c] = [math.inf, -math.inf, math.nan, math.inf][i % 4]
        b.vd[int(pages[i]), 0, 17 * i, c] = vals[c]
        if i == 7:                         # both signs: no number
            b.vd[int(pages[2]), 0, 1, c] = -math.inf
            vals[c] = math.nan
    last = int(b.table[5, 0])
    b.vd[last, 0, tok - 1, 0] = -math.inf  # the last token of row 5
    out, lse = b.run()
    o, z = out.cpu().double(), lse.cpu().double()
    t5 = 5 * tok + tok - 1
    assert (o[t5, :, 0] == -math.inf).all()
    o[t5, :, 0] = 0
    for c in range(d):
        if vals[c] != 0:
            assert (torch.isnan(o[..., c]).all() if math.isnan(vals[c]) else (o[..., c] == vals[c]).all()), c
            o[..., c] = 0
    assert torch.isfinite(o).all() and torch.isfinite(z).all()
    # rows 4 to 6 against the formula: the prefix's keys count `reps` times
    kp, vp = b.kd.cpu(), b.vd.cpu().nan_to_num(0, 0, 0)
    rows = slice(4, 7)
    q, tab = b.q[4 * tok:7 * tok], b.table[rows]
    off = [0, tok, 2 * tok, 3 * tok]
    base = b.ptable[rows, :8]
    po, pl, pa, pd, _ = C.attention(q, kp, vp, tab, off, [0] * 3, b.scale, [0, 1, 2, 3], [1024] * 3, base)
    lo, ll, la, ld, _ = C.attention(q, kp, vp, tab, off, [tok] * 3, b.scale)
    pl = pl + math.log(reps)
    rl = torch.logaddexp(pl, ll)
    wp, wl = torch.exp(pl - rl)[..., None], torch.exp(ll - rl)[..., None]
    ref, a = wp * po + wl * lo, wp * pa + wl * la
    keep = vals == 0
    cnt = torch.full((3 * tok,), 1024 * reps + tok)
    eo, ez = C.attention_bounds(ref, rl, a, torch.maximum(pd, ld), cnt, d, b.dt)
    got, gz = o[4 * tok:7 * tok], z[4 * tok:7 * tok]
    assert ((got - ref)[..., keep].abs() <= eo[..., keep])[..., 1:].all() and ((gz - rl).abs() <= ez).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tok", [1, 6, 40, 100])
@pytest.mark.parametrize("low", [32, 128])
def test_an_infinite_value_behind_a_weight_that_underflows(dt, tok, low):
    """Scores of -225 against others near 0: the weight is 0 in fp32, but the key is seen, and
    e^-225 times infinity is not finite, wherever the key lies and whatever shares its tile:
    alone among others, or in a run of `low` such keys (a warp's share of a unit, or a
    whole unit).  Columns and rows without such a value keep their results."""
    R = 32
    b = Batch(dt, 16, 8, 64, 32, new=[tok] * R, seq=[tok + 200] * R, goff=list(range(R + 1)), pre=[428] * R, seed=34)
    b.q[..., 0] = 30.0
    b.kd[..., 0] = 0.0
    places, odd = [], torch.arange(R * tok) // tok % 2 == 1
    for r in range(R):
        for i in range(4, 4 + low // 32):                                    # keys 128 .. 128 + low of the prefix
            b.kd[int(b.ptable[r, i]), :, :, 0] = -60.0
        places += [(int(b.ptable[r, 4]), 8, 33)]
        if r % 2 == 0:      # prefix keys 7 and 426, local keys 5 and 200, the first new one
            places += [(int(b.ptable[r, 0]), 7, 3), (int(b.ptable[r, 13]), 10, 11), (int(b.table[r, 0]), 5, 17),
                       (int(b.table[r, 6]), 8, 25)]
    for page, at, col in places:
        b.kd[page, :, at, 0] = -60.0
    clean, clse = b.run()
    for page, at, col in places:
        b.vd[page, :, at, col] = math.inf
    out, lse = b.run()
    assert torch.equal(lse, clse)
    finite, same = torch.isfinite(out).cpu(), (out == clean).cpu()
    assert not finite[..., 33].any().item()
    assert not finite[~odd][..., [3, 11, 17, 25]].any().item()
    keep = torch.ones(64, dtype=torch.bool)
    keep[33] = False
    assert same[odd][..., keep].all().item()
    keep[[3, 11, 17, 25]] = False
    assert same[..., keep].all().item()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("new,seq", [(1, 132), (6, 132), (20, 132), (40, 132), (70, 190), (100, 300)])
def test_a_nan_key_before_units_that_a_row_does_not_see(dt, new, seq):
    """The NaN of an early key reaches output and lse of every token, whether or not a later
    unit of its tile holds no key that it sees."""
    b = Batch(dt, 32, 8, 64, 32, new=[new] * 40, seq=[seq] * 40, seed=35)     # 320 lists: most are one worker's
    clean, clse = b.run()
    for r in range(10):
        b.kd[int(b.table[r, 0]), 1, 3, 5] = math.nan
    out, lse = b.run()
    nan = torch.zeros_like(lse, dtype=torch.bool)
    nan[:10 * new, 4:8] = True
    assert torch.isnan(out[nan]).all().item() and torch.isnan(lse[nan]).all().item()
    out[nan], lse[nan] = clean[nan], clse[nan]
    assert torch.equal(out, clean) and torch.equal(lse, clse)
