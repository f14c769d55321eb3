"""Paged serving calls on the GPU against their plain 64-bit forms."""
import math
import random

import numpy as np
import pytest
import torch

from long_prefix_attention_b200 import inputs, ops

import paged_common as C

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int64).astype(np.int32)).cuda()


# ------------------------------------------------------------------ pages --

def step_case(R, S, MP, seed, new_hi, ended=0.2, tight=False):
    rng = random.Random(seed)
    kv = [rng.choice([0, 1, S, S * MP, rng.randint(0, S * MP)]) if rng.random() < 0.3 else rng.randint(0, S * MP // 2)
          for _ in range(R)]
    new = [-rng.randint(1, 3) if rng.random() < ended else rng.choice([0, 1, 1, rng.randint(0, new_hi)])
           for _ in range(R)]
    held = sum(C.cdiv(k, S) for k in kv)
    need = sum(C.cdiv(k + n, S) - C.cdiv(k, S) for k, n in zip(kv, new) if n > 0)
    free = need // 2 if tight else need + 3
    F = max(1, held + free)
    ids = np.random.default_rng(seed).permutation(F)
    table = np.full((R, MP), -7)
    used = 0
    for r, k in enumerate(kv):
        n = C.cdiv(k, S)
        table[r, :n] = ids[used:used + n]
        used += n
    head = rng.randrange(F)
    pool = np.full(F, -9)
    pool[(head + np.arange(free)) % F] = ids[used:used + free]
    return kv, new, table, pool, head, free


def run_step(kv, new, base, table, pool, head, count, S, T, times=1, stream=None):
    R = len(kv)
    d = dict(kv_len=i32(kv), new_len=i32(new), pool=i32(pool), pool_state=i32([head, count, 5]), table=i32(table),
             seq_len=i32([77] * R), q_off=i32([77] * (R + 1)), row=i32([77] * T), pos=i32([77] * T),
             slot=i32([77] * T), pool_out=i32([77] * 3), pos_base=None if base is None else i32(base))
    for _ in range(times):
        ops.asm_page_step(page_size=S, **d)
    torch.cuda.synchronize()
    return {k: None if v is None else v.cpu().numpy() for k, v in d.items()}


def check_step(kv, new, base, table, pool, head, count, S, T, times=1):
    got = run_step(kv, new, base, table, pool, head, count, S, T, times)
    want = C.page_step(kv, new, base, table, pool, head, count, S, T)
    for k, w in zip(("seq_len", "q_off", "row", "pos", "slot", "pool_out"), want):
        assert np.array_equal(got[k], w), k
    assert np.array_equal(got["table"], table) and np.array_equal(got["pool"], pool)
    return got


@pytest.mark.parametrize("R,S,MP,new_hi", [(1, 16, 4, 40), (7, 128, 3, 90), (33, 64, 9, 300), (513, 32, 20, 60),
                                           (1000, 16, 40, 5), (4096, 16, 12, 9)])
@pytest.mark.parametrize("tight", [False, True])
def test_page_step_equals_a_host_allocator(R, S, MP, new_hi, tight):
    for seed in range(3):
        kv, new, table, pool, head, free = step_case(R, S, MP, 100 * R + seed, new_hi, tight=tight)
        n = sum(max(x, 0) for x in new)
        T = [n + 13, max(n - 5, 1), max(n, 1)][seed]   # padded, too short, exact
        base = None if seed == 0 else [31 * r for r in range(R)]
        check_step(kv, new, base, table, pool, head, free, S, T, times=1 + seed)


def test_page_step_at_the_edges():
    # nothing at all; every row ends; every row full; lengths outside the table are clamped
    S, MP = 16, 3
    empty = np.full((2, MP), -1)
    check_step([0, 0], [0, 0], None, empty.copy(), np.arange(4), 3, 4, S, 4)
    table = np.arange(6).reshape(2, MP)
    check_step([48, 33], [-1, -5], None, table.copy(), np.full(6, -1), 5, 0, S, 1)
    check_step([48, 33], [1, 15], None, table.copy(), np.full(6, -1), 5, 0, S, 20)
    check_step([-3, 1000], [2, -1], None, table.copy(), np.array([9, 9, 9, 9, 9, 5]), 5, 1, S, 3)
    # a row too long for its table asks for no page: 16 + 33 > 48
    table = np.array([[0, -1, -1], [1, -1, -1], [2, -1, -1]])
    got = check_step([16, 5, 16], [33, 3, 1], None, table, np.array([3, 4, -1, -1]), 0, 2, S, 40)
    assert got["seq_len"].tolist() == [16, 8, 17] and got["pool_out"].tolist() == [1, 1, 1]
    # a row that asks for more than there is keeps later rows that need pages out, not those that need none
    table = np.array([[0, -1, -1], [1, -1, -1], [2, -1, -1]])
    got = check_step([16, 5, 16], [32, 3, 1], None, table, np.array([3, -1, -1, -1]), 0, 1, S, 40)
    assert got["seq_len"].tolist() == [16, 8, 16] and got["pool_out"].tolist() == [0, 1, 2]
    # huge counts saturate without wrapping
    check_step([0] * 3, [2**31 - 1] * 3, None, np.full((3, MP), -1), np.arange(9), 0, 9, S, 5)


def test_page_step_has_no_tokens():
    R, S, MP = 3, 32, 4
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    seq, qo, out = i32([9] * R), i32([9] * (R + 1)), i32([9] * 3)
    ops.asm_page_step(i32([5, 6, 7]), i32([0, -1, 0]), i32([-1] * 8), i32([0, 0, 0]), S, i32([[1, -1, -1, -1]] * R),
                      seq, qo, z, z, z, out)
    assert seq.tolist() == [5, 0, 7] and qo.tolist() == [0] * 4 and out.tolist() == [0, 1, 0]


# ------------------------------------------------------------------- rope --

def heads(T, H, d, dt, seed, form="flat"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, d, generator=g).to(dt)
    if form == "flat":
        return x, x.cuda()
    if form == "packed":       # a slice of a wider projection
        w = torch.full((T, H + 2, d), math.nan, dtype=dt, device="cuda")
        w[:, 1:H + 1] = x.cuda()
        return x, w[:, 1:H + 1]
    if form == "heads":        # [H, T, d] seen as [T, H, d]
        return x, x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    odd = torch.full((T, H, d + 1), math.nan, dtype=dt, device="cuda")   # rows that are not 16-byte aligned
    odd[..., 1:] = x.cuda()
    return x, odd[..., 1:]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,H,d,rot,form", [(1, 1, 64, 64, "flat"), (3, 32, 128, 128, "flat"), (17, 5, 128, 64, "packed"),
                                            (40, 8, 64, 32, "heads"), (9, 3, 128, 2, "flat"), (11, 2, 64, 18, "packed"),
                                            (700, 7, 128, 128, "odd"), (2500, 9, 128, 96, "heads"),
                                            (3001, 32, 64, 64, "packed")])
def test_rope_matches_the_rotation(dt, layout, T, H, d, rot, form):
    dt = DT[dt]
    x, xd = heads(T, H, d, dt, T + H, form)
    g = torch.Generator().manual_seed(5)
    far = [1, 1000, 2**20, 2**31 - 1][T % 4]
    pos = torch.randint(-(far // 3), far, (T,), generator=g)
    f = C.freqs(rot, 10000.0)
    for inverse, ms in ((False, 1.0), (True, 1.37)):
        y = torch.full((T, H, d), math.nan, dtype=dt, device="cuda")
        ops.asm_rope(xd, i32(pos), f.cuda(), y, layout=layout, mscale=ms, inverse=inverse)
        ref = C.rotate(x.double(), pos, f, layout, ms, inverse)
        err = (y.cpu().double() - ref).abs()
        assert (err <= C.rope_bound(x, pos, f, layout, ms, dt, ref)).all()
        # in place gives the same bits
        z = xd.clone() if form == "flat" else xd
        ops.asm_rope(z, i32(pos), f.cuda(), z, layout=layout, mscale=ms, inverse=inverse)
        assert torch.equal(z, y)
        if form != "flat":
            x, xd = heads(T, H, d, dt, T + H, form)


def test_rope_takes_broadcast_heads_and_an_empty_batch():
    x = torch.randn(4, 1, 64, device="cuda")
    f = C.freqs(64, 1e4).cuda()
    pos = i32([3, 1, 4, 1])
    y, z = torch.empty(4, 6, 64, device="cuda"), torch.empty(4, 1, 64, device="cuda")
    ops.asm_rope(x.expand(4, 6, 64), pos, f, y)
    ops.asm_rope(x, pos, f, z)
    assert torch.equal(y, z.expand(4, 6, 64))
    e = torch.empty(0, 6, 64, device="cuda")
    ops.asm_rope(e, i32([]), f, e)


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_rope_is_the_gradient(layout):
    """<asm_rope(x), g> against autograd of the formula and against differences
    (the map is linear: a difference is exact up to rounding)."""
    T, H, d, rot, ms = 6, 3, 64, 48, 1.2
    x, g = (torch.randn(T, H, d, dtype=torch.float64, generator=torch.Generator().manual_seed(i)) for i in (1, 2))
    x, g = x.float().double(), g.float().double()
    pos, f = torch.randint(0, 100000, (T,)), C.freqs(rot, 10000.0)
    xr = x.clone().requires_grad_()
    (C.rotate(xr, pos, f, layout, ms) * g).sum().backward()
    got = torch.empty(T, H, d, device="cuda")
    ops.asm_rope(g.float().cuda(), i32(pos), f.cuda(), got, layout=layout, mscale=ms, inverse=True)
    bound = C.rope_bound(g, pos, f, layout, ms, torch.float32, xr.grad)
    assert ((got.cpu().double() - xr.grad).abs() <= bound).all()
    y0, y1 = torch.empty(T, H, d, device="cuda"), torch.empty(T, H, d, device="cuda")
    ops.asm_rope(x.float().cuda(), i32(pos), f.cuda(), y0, layout=layout, mscale=ms)
    for i in (0, 1, rot // 2, rot - 1, d - 1):
        e = x.clone()
        e[2, 1, i] += 1.0
        e = e.float()
        ops.asm_rope(e.cuda(), i32(pos), f.cuda(), y1, layout=layout, mscale=ms)
        step = float(e[2, 1, i].double() - x[2, 1, i])
        diff = (((y1 - y0).cpu().double()) * g).sum() / step
        slack = (4 * C.rope_bound(e, pos, f, layout, ms, torch.float32, y1.cpu().double()) * g.abs())[2, 1].sum()
        assert abs(float(diff) - float(xr.grad[2, 1, i])) <= float(slack)


@pytest.mark.parametrize("name,code", [("none", 0), ("linear", 1), ("base", 2), ("bands", 3), ("yarn", 4)])
@pytest.mark.parametrize("rot", [2, 64, 128])
def test_rope_frequencies(name, code, rot):
    f = torch.empty(rot // 2, dtype=torch.float64, device="cuda")
    lo, hi = (1.0, 32.0) if name == "yarn" else (1.0, 4.0)
    ops.asm_rope_freqs(f, 500000.0, scaling=code, factor=8.0, lo=lo, hi=hi, ctx=8192.0)
    ref = C.freqs(rot, 500000.0, name, 8.0, lo, hi, 8192.0)
    # a dozen operations in 64 bits, pow to 2 ulp of its argument's scaling by log(theta) < 14 (twice)
    assert ((f.cpu() - ref).abs() <= 64 * 2.0 ** -52 * ref).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,S,layout,form", [(1, 4, 1, 128, 128, 16, 0, "flat"), (37, 8, 8, 64, 32, 32, 1, "packed"),
                                                         (300, 8, 2, 128, 128, 128, 1, "packed"),
                                                         (65, 2, 1, 64, 10, 64, 0, "heads"), (130, 6, 3, 128, 64, 16, 0, "odd")])
def test_append_turns_and_stores(dt, T, Hq, Hkv, d, rot, S, layout, form):
    dt = DT[dt]
    (q, qd), (k, kd), (v, vd) = (heads(T, h, d, dt, i, form) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    n_pages = C.cdiv(T, S) + 4
    rng = np.random.default_rng(T)
    slot = rng.permutation(n_pages * S)[:T]
    if T > 5:
        slot[[1, 3]] = [-1, -(2**31)]
        slot[4] = n_pages * S           # one behind the last
        slot[5] = 2**31 - 1
    pos, f = torch.arange(T) + 70000, C.freqs(rot, 500000.0, "linear", 4.0)
    kp = torch.full((n_pages, Hkv, S, d), 7.0, dtype=dt, device="cuda")
    vp = torch.full_like(kp, 9.0)
    qo = torch.full((T, Hq, d), math.nan, dtype=dt, device="cuda")
    ops.asm_rope_append(qd, kd, vd, i32(pos), i32(slot), f.cuda(), qo, kp, vp, layout=layout, mscale=1.1)
    ref = C.rotate(q.double(), pos, f, layout, 1.1)
    assert ((qo.cpu().double() - ref).abs() <= C.rope_bound(q, pos, f, layout, 1.1, dt, ref)).all()
    rk = C.rotate(k.double(), pos, f, layout, 1.1)
    bk = C.rope_bound(k, pos, f, layout, 1.1, dt, rk)
    kc, vc = kp.cpu(), vp.cpu()
    seen = torch.zeros(n_pages, S, dtype=torch.bool)
    for t in range(T):
        s = int(slot[t])
        if 0 <= s < n_pages * S:
            seen[s // S, s % S] = True
            assert ((kc[s // S, :, s % S].double() - rk[t]).abs() <= bk[t]).all()
            assert torch.equal(vc[s // S, :, s % S], v[t])
    rest = ~seen[:, None, :].expand(n_pages, Hkv, S)
    assert (kc[rest] == 7).all() and (vc[rest] == 9).all()
    # q in place
    ops.asm_rope_append(qd, kd, vd, i32(pos), i32(slot), f.cuda(), qd, kp, vp, layout=layout, mscale=1.1)
    assert torch.equal(qd, qo)


# -------------------------------------------------------------- attention --

class Batch:
    """Pages, tables, queries and lengths of an attention call; everything
    outside the used places of the pages is NaN."""

    def __init__(self, dt, Hq, Hkv, d, S, new, seq, goff=None, pre=None, seed=0, pad=0, big=None, amp=1.5):
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.S, self.dt = Hq, Hkv, d, S, DT[dt]
        self.new, self.seq, self.goff, self.pre = new, seq, goff, pre
        self.q_off = np.concatenate([[0], np.cumsum(new)])
        self.T = int(self.q_off[-1]) + pad
        n_loc, n_pre = [C.cdiv(s, S) for s in seq], [C.cdiv(p, S) for p in (pre or [])]
        used = sum(n_loc) + sum(n_pre)
        self.n_pages = big or used + 3
        ids = np.random.default_rng(seed).permutation(used + 3) + (self.n_pages - used - 3)
        self.table = np.full((len(new), max(n_loc + [1]) + 1), 10**6)
        self.ptable = np.full((max(len(n_pre), 1), max(n_pre + [1])), -1)
        at = 0
        self.kd = torch.empty(self.n_pages, Hkv, S, d, dtype=self.dt, device="cuda")
        self.vd = torch.empty_like(self.kd)
        for x in (self.kd, self.vd):
            x[int(ids.min()):] = math.nan
        for tab, lens, counts in ((self.table, seq, n_loc), (self.ptable, pre or [], n_pre)):
            for r, (n, c) in enumerate(zip(lens, counts)):
                tab[r, :c] = ids[at:at + c]
                for p in range(c):
                    m = min(S, n - p * S)
                    for x in (self.kd, self.vd):
                        x[int(ids[at + p]), :, :m] = torch.randn(Hkv, m, d, generator=g).to(self.dt).cuda()
                at += c
        self.q = (amp * torch.randn(max(self.T, 1), Hq, d, generator=g)).to(self.dt)
        self.scale = 1 / math.sqrt(d)
        NG = 0 if goff is None else len(goff) - 1
        self.dev = dict(table=i32(self.table), prefix_table=i32(self.ptable) if NG else None)
        self.NG = NG

    def plan(self, stream=None):
        R, T = len(self.new), self.q.shape[0]
        n = ops.asm_shared_plan_size(R, self.NG, T, self.Hq, self.Hkv)
        plan = torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda")
        ops.asm_shared_plan(i32(self.q_off), i32(self.seq), self.dev["table"], T, self.Hq, self.Hkv, self.S, plan,
                            group_off=i32(self.goff) if self.NG else None,
                            prefix_len=i32(self.pre) if self.NG else None, prefix_table=self.dev["prefix_table"])
        return plan

    def ws(self):
        n = ops.asm_shared_attention_workspace_size(self.q.shape[0], self.Hq, self.Hkv, self.d)
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")   # the rest may hold anything: NaN here
        ws[:256] = 0
        return ws

    def run(self, err=0):
        plan, ws, q = self.plan(), self.ws(), self.q.cuda()
        out = torch.full_like(q, 55.0)
        lse = torch.full(q.shape[:2], 55.0, device="cuda")
        ops.asm_shared_attention(q, self.kd, self.vd, self.dev["table"], plan, self.scale, out, ws,
                                 prefix_table=self.dev["prefix_table"], lse_out=lse)
        assert ops.asm_workspace_error(ws) == err
        return out, lse

    def ref(self, lo=0):
        kp, vp = self.kd[lo:].cpu(), self.vd[lo:].cpu()
        return C.attention(self.q, kp, vp, self.table - lo, self.q_off, self.seq, self.scale, self.goff, self.pre,
                           self.ptable - lo)

    def check(self, lo=0):
        out, lse = self.run()
        ro, rl, a, dot, cnt = self.ref(lo)
        real = ~torch.isnan(rl[:, 0])
        o, z = out.cpu().double(), lse.cpu().double()
        assert (o[~real] == 55).all() and (z[~real] == 55).all()
        ro, rl, a, dot, cnt, o, z = (x[real] for x in (ro, rl, a, dot, cnt, o, z))
        eo, ez = C.attention_bounds(ro, rl, a, dot, cnt, self.d, self.dt)
        assert torch.equal(torch.isinf(z), torch.isinf(rl))
        fin = ~torch.isinf(rl)
        assert (o[~fin] == 0).all()
        assert ((z - rl)[fin].abs() <= ez[fin]).all(), float(((z - rl)[fin].abs() / ez[fin]).max())
        assert ((o - ro).abs() <= eo).all(), float(((o - ro).abs() / eo).max())
        return out, lse


CASES = {
    "one token, one key": dict(new=[1], seq=[1]),
    "decode, ragged": dict(new=[1] * 9, seq=[1, 2, 15, 16, 17, 127, 128, 129, 700]),
    "prefix only": dict(new=[1, 1, 1], seq=[0, 0, 0], goff=[0, 3], pre=[300]),
    "prefix and local": dict(new=[1] * 5, seq=[5, 130, 0, 64, 257], goff=[0, 5], pre=[513]),
    "groups, some rows alone": dict(new=[1, 2, 1, 3, 1, 1, 4], seq=[9, 40, 1, 300, 129, 77, 4], goff=[1, 3, 3, 6],
                                    pre=[129, 64, 1000]),
    "drafts": dict(new=[3, 8, 1, 5], seq=[3, 200, 64, 133], goff=[0, 4], pre=[100]),
    "prompt chunks": dict(new=[150, 1, 261], seq=[150, 400, 600], goff=[0, 3], pre=[260]),
    "no keys": dict(new=[2, 1, 3], seq=[0, 5, 2], goff=[1, 3], pre=[0]),
    "rows without tokens": dict(new=[0, 1, 0, 0, 2, 0], seq=[50, 50, 0, 7, 9, 0], goff=[0, 1, 6], pre=[40, 0]),
}


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("Hq,Hkv,d,S", [(4, 1, 64, 16), (4, 4, 128, 64), (16, 2, 128, 32), (4, 2, 64, 128)])
def test_shared_attention(dt, case, Hq, Hkv, d, S):
    Batch(dt, Hq, Hkv, d, S, seed=len(case), pad=2, **CASES[case]).check()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_shared_attention_splits_long_keys(dt):
    Batch(dt, 4, 1, 128, 64, new=[1, 1], seq=[3000, 37], goff=[0, 2], pre=[9000], seed=3).check()


def test_shared_attention_many_rows():
    rng = random.Random(1)
    seq = [rng.randint(1, 90) for _ in range(600)]
    Batch("bf16", 8, 2, 64, 16, new=[1] * 600, seq=seq, goff=[0, 100, 512], pre=[70, 33], seed=4).check()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 1)])
def test_shared_attention_mixes_segments(dt, Hq, Hkv):
    """More tiles than workers: key lists of one unit and of several, tall
    tiles and small ones, follow one another in one worker's range."""
    rng = random.Random(2)
    new = [rng.choice([1, 1, 1, 2, 5, 40, 70]) for _ in range(90)]
    seq = [n + rng.choice([0, 3, 100, 128, 200, 300, 700]) for n in new]
    Batch(dt, Hq, Hkv, 64, 32, new=new, seq=seq, goff=[4, 30, 33, 80], pre=[400, 90, 129], seed=13).check()


@pytest.mark.parametrize("d,S", [(64, 32), (128, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("n", [31, 32, 33, 47, 63, 64, 65, 96, 97])
def test_shared_attention_tile_heights(n, Hq, Hkv, d, S):
    """Query rows per tile around the limits of 32, 64 and 96, split over
    workers and not: rows of a group, and tokens of one row."""
    tok = C.cdiv(n, Hq // Hkv)
    Batch("bf16", Hq, Hkv, d, S, new=[1] * tok, seq=[3 + 2 * i for i in range(tok)], goff=[0, tok], pre=[3000], seed=n).check()
    Batch("bf16", Hq, Hkv, d, S, new=[tok, tok], seq=[tok + 100, tok], goff=[0, 2], pre=[70], seed=n, pad=1).check()
    Batch("bf16", Hq, Hkv, d, S, new=[tok], seq=[1500 + tok], seed=n).check()


def test_shared_attention_most_rows_and_groups():
    """4096 rows in 900 groups, some empty, some with tall rows between short ones."""
    rng = random.Random(3)
    new = [1] * 4096
    for r in (5, 700, 701, 2000):
        new[r] = 70
    new[9] = 0
    seq = [n + rng.randint(0, 6) for n in new]
    cuts = sorted(rng.randint(0, 4096) for _ in range(901))
    pre = [rng.randint(0, 20) for _ in range(900)]
    Batch("bf16", 2, 1, 64, 16, new=new, seq=seq, goff=cuts, pre=pre, seed=14).check()


def test_shared_attention_large_logits():
    """Scores of some hundreds: the running maximum moves far, weights underflow."""
    for dt in ("bf16", "f32"):
        Batch(dt, 4, 2, 128, 32, new=[1, 4, 140], seq=[300, 100, 500], goff=[0, 3], pre=[700], seed=5, amp=60.0).check()


def test_shared_attention_far_pages():
    """Pages more than 2^31 elements into the cache."""
    n = (2**31 // (2 * 64 * 128)) + 40
    b = Batch("bf16", 4, 2, 128, 64, new=[1, 3], seq=[200, 77], goff=[0, 2], pre=[150], seed=6, big=n)
    lo = n - 12
    assert b.table[b.table < 10**6].min() >= lo
    b.table = np.where(b.table >= 10**6, lo, b.table)
    b.check(lo)


def test_shared_attention_special_values():
    """An infinite score takes all the weight, a NaN reaches only the rows that see it."""
    for dt in ("f32", "bf16"):
        b = Batch(dt, 4, 2, 64, 16, new=[1, 1], seq=[40, 40], seed=7)
        pg = int(b.table[0, 1])
        b.vd[pg, 0, 3, 5] = math.inf
        b.vd[pg, 1, 2, 6] = math.nan
        out, lse = b.run()
        o = out.cpu()
        assert torch.isinf(o[0, :2, 5]).all() and torch.isnan(o[0, 2:, 6]).all()
        o[0, :2, 5], o[0, 2:, 6] = 0, 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("rows_per", [1, 3, 20, 40])
def test_infinite_values_stay_infinite(rows_per):
    """An infinite value anywhere in the keys a row sees (prefix or local) gives
    an infinite result in its column; one that it does not see gives nothing."""
    for dt in ("f32", "bf16"):
        b = Batch(dt, 4, 2, 64, 32, new=[rows_per] * 2, seq=[150 + rows_per] * 2, goff=[0, 2], pre=[200], seed=17)
        b.vd[int(b.ptable[0, 3]), 0, 7, 9] = -math.inf          # prefix key 103
        b.vd[int(b.table[0, 2]), 1, 1, 11] = math.inf           # local key 65 of row 0
        last = 149 + rows_per
        b.vd[int(b.table[1, last // 32]), 0, last % 32, 13] = math.inf   # the last new token of row 1
        out, lse = b.run()
        o, n = out.cpu(), rows_per
        assert torch.isfinite(lse).all()
        assert (o[:, :2, 9] == -math.inf).all()
        assert (o[:n, 2:, 11] == math.inf).all()
        assert (o[2 * n - 1, :2, 13] == math.inf).all()
        o[:, :2, 9], o[:n, 2:, 11], o[2 * n - 1, :2, 13] = 0, 0, 0
        assert torch.isfinite(o).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_later_token_never_reaches_an_earlier_one(dt):
    """Non-finite keys and values of a row's own later tokens stay out of the
    earlier tokens' results, in drafts and in long prompt chunks."""
    for new, seq, bad in (([6], [70], 67), ([200], [200], 150), ([300], [420], 300)):
        b = Batch(dt, 8, 2, 128, 32, new=new, seq=seq, goff=[0, 1], pre=[40], seed=8)
        o0, z0 = b.run()
        pg, at = int(b.table[0, bad // 32]), bad % 32
        b.vd[pg, :, at, ::3] = math.nan
        b.vd[pg, :, at, 1::3] = math.inf
        b.kd[pg, :, at, ::2] = math.nan
        o1, z1 = b.run()
        first = bad - (seq[0] - new[0])          # the token that is the bad key
        assert torch.equal(o0[:first], o1[:first]) and torch.equal(z0[:first], z1[:first])
        assert torch.isnan(o1[first:, :, 0]).all() and torch.isnan(z1[first:]).all()


def test_shared_attention_reports_bad_pages_and_foreign_plans():
    b = Batch("bf16", 4, 2, 128, 32, new=[1, 1], seq=[70, 70], seed=9)
    good, _ = b.run()
    b.dev["table"][0, 1] = b.n_pages
    out, _ = b.run(err=ops.ASM_ERR_INVALID_ARG)
    assert torch.equal(out[1], good[1])
    b.dev["table"][0, 1] = -5
    b.run(err=ops.ASM_ERR_INVALID_ARG)
    # a plan made for other heads
    b = Batch("bf16", 4, 2, 128, 32, new=[1, 1], seq=[70, 70], seed=9)
    plan = b.plan()
    ws, q = b.ws(), b.q.cuda()
    q2 = torch.cat([q, q], 1).contiguous()
    out = torch.full_like(q2, 3.0)
    big = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    big[:plan.numel()] = plan
    ws = torch.zeros(ops.asm_shared_attention_workspace_size(2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    ops.asm_shared_attention(q2, b.kd, b.vd, b.dev["table"], big, b.scale, out, ws)
    assert ops.asm_workspace_error(ws) == ops.ASM_ERR_INVALID_ARG and (out == 3).all()


def test_plan_survives_falling_offsets():
    """Offsets and lengths that make no sense are clamped: nothing is written
    outside the batch and nothing faults."""
    b = Batch("bf16", 4, 2, 64, 16, new=[3, 4, 2], seq=[30, 40, 20], goff=[0, 2, 3], pre=[30, 40], seed=10)
    b.table = np.where(b.table >= 10**6, b.table[0, 0], b.table)
    b.ptable = np.where(b.ptable < 0, b.ptable[0, 0], b.ptable)
    b.dev = dict(table=i32(b.table), prefix_table=i32(b.ptable))
    for qo, sl, go, pl in (([0, 9, 3, 9], [30, 40, 20], [0, 2, 3], [30, 40]),
                           ([5, 2, 900, -4], [10**9, -3, 20], [3, 0, 99], [10**9, -1]),
                           ([-9, -9, -9, -9], [1, 1, 1], [-1, -1, -1], [1, 1])):
        b.q_off, b.seq, b.goff, b.pre = np.array(qo), sl, go, pl
        plan, ws, q = b.plan(), b.ws(), b.q.cuda()
        out = torch.full_like(q, 55.0)
        ops.asm_shared_attention(q, b.kd, b.vd, b.dev["table"], plan, b.scale, out, ws,
                                 prefix_table=b.dev["prefix_table"])
        torch.cuda.synchronize()
        ops.asm_workspace_error(ws)


@pytest.mark.parametrize("tokens", [2**30, 2**27])
def test_a_plan_of_too_much_work_is_marked(tokens):
    """131072 new tokens of one row, 32 KV heads, behind 2^30 keys: 512 tiles x 32 x
    2^23 units of cost 4 are 3.7e9 per worker, above 2^31: the plan's first word, which
    the attention checks, is 0, and nothing is written behind the plan.  2^27 keys are
    an eighth of it, and planned."""
    T, H, S = 131072, 32, 128
    n = ops.asm_shared_plan_size(1, 1, T, H, H)
    plan = torch.full((n + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, T // S, dtype=torch.int32, device="cuda")
    ptable = torch.zeros(1, tokens // S, dtype=torch.int32, device="cuda")
    ops.asm_shared_plan(i32([0, T]), i32([T]), table, T, H, H, S, plan[:n], group_off=i32([0, 1]),
                        prefix_len=i32([tokens]), prefix_table=ptable)
    assert (int(plan[:4].cpu().numpy().view(np.int32)[0]) == 0) == (tokens == 2**30)
    assert (plan[n:] == 0x5a).all()


@pytest.mark.parametrize("tok", [8, 9, 12, 16, 17])
def test_a_later_token_never_reaches_an_earlier_draft(tok):
    """As above, for tiles of 32 to 68 query rows, the bad key in either half of a unit."""
    for seq, bad in ((tok + 60, tok + 55), (tok + 120, tok + 125 - 10)):
        b = Batch("bf16", 4, 1, 64, 32, new=[tok], seq=[seq], goff=[0, 1], pre=[40], seed=tok)
        o0, z0 = b.run()
        pg, at, first = int(b.table[0, bad // 32]), bad % 32, max(bad - (seq - tok), 0)
        b.vd[pg, :, at, ::3] = math.nan
        b.vd[pg, :, at, 1::3] = math.inf
        b.kd[pg, :, at, ::2] = math.nan
        o1, z1 = b.run()
        assert torch.equal(o0[:first], o1[:first]) and torch.equal(z0[:first], z1[:first])
        assert torch.isnan(o1[first:, :, 0]).all() and torch.isnan(z1[first:]).all()


def test_shared_attention_repeats_bit_for_bit():
    b = Batch("bf16", 8, 2, 128, 64, new=[1] * 20, seq=[100 + 7 * i for i in range(20)], goff=[0, 20], pre=[2000], seed=11)
    (o0, z0), (o1, z1) = b.run(), b.run()
    assert torch.equal(o0, o1) and torch.equal(z0, z1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_calls_at_once(dt):
    """Calls on two streams, with a workspace and a plan each, do not disturb one another."""
    both = [Batch(dt, 8, 2, 128, 32, new=[1] * 20, seq=[100 + 7 * i for i in range(20)], goff=[0, 20], pre=[1500], seed=21),
            Batch(dt, 4, 2, 128, 64, new=[150, 1, 5], seq=[400, 700, 60], goff=[0, 3], pre=[260], seed=22)]
    alone = [b.run() for b in both]
    ws, q, streams = [b.ws() for b in both], [b.q.cuda() for b in both], [torch.cuda.Stream() for _ in both]
    plans, outs = [b.plan() for b in both], [[torch.empty_like(x) for _ in range(8)] for x in q]
    torch.cuda.synchronize()
    for i in range(8):
        for j, b in enumerate(both):
            ops.asm_shared_attention(q[j], b.kd, b.vd, b.dev["table"], plans[j], b.scale, outs[j][i], ws[j],
                                     prefix_table=b.dev["prefix_table"], stream=streams[j])
    torch.cuda.synchronize()
    for j in (0, 1):
        assert ops.asm_workspace_error(ws[j]) == 0
        for o in outs[j]:
            assert torch.equal(o[:both[j].q_off[-1]], alone[j][0][:both[j].q_off[-1]])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_captured_steps_follow_the_lengths(dt):
    """One graph of plan and two layers, replayed with other lengths, and the
    same calls on a second stream at once with their own workspace."""
    b = Batch(dt, 8, 2, 128, 32, new=[1] * 6, seq=[300] * 6, goff=[0, 6], pre=[200], seed=12)
    q, seq, pre = b.q.cuda(), i32([300] * 6), i32([200])
    qo, go = i32(b.q_off), i32([0, 6])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    st = []
    for _ in range(2):
        st.append((torch.zeros_like(b.plan()), b.ws(), torch.empty_like(q), torch.empty_like(q)))

    def step(plan, ws, o1, o2, stream):
        ops.asm_shared_plan(qo, seq, b.dev["table"], 6, 8, 2, 32, plan, group_off=go, prefix_len=pre,
                            prefix_table=b.dev["prefix_table"], stream=stream)
        ops.asm_shared_attention(q, b.kd, b.vd, b.dev["table"], plan, b.scale, o1, ws,
                                 prefix_table=b.dev["prefix_table"], stream=stream)
        ops.asm_shared_attention(o1, b.kd, b.vd, b.dev["table"], plan, b.scale, o2, ws,
                                 prefix_table=b.dev["prefix_table"], stream=stream)

    torch.cuda.synchronize()
    graphs = []
    for x, s in zip(st, (s1, s2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step(*x, s)
        graphs.append(gr)
    for lens, p in (([300] * 6, 200), ([1, 17, 300, 128, 40, 5], 3), ([299] * 6, 0), ([64] * 6, 129)):
        seq.copy_(i32(lens))
        pre.copy_(i32([p]))
        torch.cuda.synchronize()
        for _ in range(3):
            for gr, s in zip(graphs, (s1, s2)):
                with torch.cuda.stream(s):
                    gr.replay()
        torch.cuda.synchronize()
        for x in st:
            assert ops.asm_workspace_error(x[1]) == 0
        b.seq, b.pre = lens, [p]
        want, _ = b.run()
        assert torch.equal(st[0][2], want) and torch.equal(st[1][2], want) and torch.equal(st[0][3], st[1][3])


# ------------------------------------------------------------ all together --

@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_serving_run(dt):
    """Two layers' worth of one request batch: a shared prompt prefix and the
    rows' prompts prefilled, then decode steps, then a row ends and its pages
    serve another: every output against dense causal attention over rotated
    keys in 64 bits."""
    dt_ = DT[dt]
    Hq, Hkv, d, S, MP, rot, layout = 8, 2, 64, 16, 8, 32, 1
    Lp, R, F = 75, 3, 40
    g = torch.Generator().manual_seed(0)
    freq = torch.empty(rot // 2, dtype=torch.float64, device="cuda")
    ops.asm_rope_freqs(freq, 10000.0, scaling=ops.ASM_ROPE_SCALE_LINEAR, factor=2.0)
    kp = torch.full((F, Hkv, S, d), math.nan, dtype=dt_, device="cuda")
    vp = torch.full_like(kp, math.nan)
    f = freq.cpu()

    def draw(T):
        return [torch.randn(T, h, d, generator=g).to(dt_) for h in (Hq, Hkv, Hkv)]

    # the prefix is row 0 of its own one-row table; its pages become the group's
    pool, state = i32(np.random.default_rng(0).permutation(F)), i32([7, F, 0])

    def page_step(kv, new, base, table, T):
        n = len(new)
        seq, qo, out = i32([0] * n), i32([0] * (n + 1)), i32([0] * 3)
        row, pos, slot = i32([0] * T), i32([0] * T), i32([0] * T)
        ops.asm_page_step(kv, i32(new), pool, state, S, table, seq, qo, row, pos, slot, out, pos_base=base)
        state.copy_(out)
        assert int(out[2]) == 0
        return seq, qo, pos, slot

    ptab = i32(np.full((1, MP), -1))
    seq, qo, pos, slot = page_step(i32([0]), [Lp], None, ptab, Lp)
    pq, pk, pv = draw(Lp)
    qr = torch.empty(Lp, Hq, d, dtype=dt_, device="cuda")
    ops.asm_rope_append(pq.cuda(), pk.cuda(), pv.cuda(), pos, slot, freq, qr, kp, vp, layout=layout)

    table, kv, base = i32(np.full((R, MP), -1)), i32([0] * R), i32([Lp] * R)
    hist = [[[], []] for _ in range(R)]       # rotated keys and values of each row, from the cache itself
    steps = [[20, 1, 37], [1, 1, 1], [1, 4, 1], [1, -1, 1], [2, 30, 1]]
    for new in steps:
        n_tok = sum(max(n, 0) for n in new)
        T = n_tok + 1                          # one padded token
        kv, qo, pos, slot = page_step(kv, new, base, table, T)
        q, k, v = draw(T)
        qr = torch.empty(T, Hq, d, dtype=dt_, device="cuda")
        ops.asm_rope_append(q.cuda(), k.cuda(), v.cuda(), pos, slot, freq, qr, kp, vp, layout=layout)
        rk = C.rotate(k.double(), pos.cpu(), f, layout)
        bound = C.rope_bound(k, pos.cpu(), f, layout, 1.0, dt_, rk)
        at = 0
        for r, n in enumerate(new):
            if n < 0:
                hist[r] = [[], []]
            for i in range(max(n, 0)):
                s = int(slot[at])
                assert int(pos[at]) == Lp + len(hist[r][0])
                cached = kp[s // S, :, s % S].cpu()
                assert ((cached.double() - rk[at]).abs() <= bound[at]).all()
                hist[r][0].append(cached)
                hist[r][1].append(v[at])
                at += 1
        n = ops.asm_shared_plan_size(R, 1, T, Hq, Hkv)
        plan = ops.alloc_workspace(n, "cuda", zero=False)
        ws = ops.alloc_workspace(ops.asm_shared_attention_workspace_size(T, Hq, Hkv, d), "cuda")
        go, pl = i32([0, R]), i32([Lp])
        ops.asm_shared_plan(qo, kv, table, T, Hq, Hkv, S, plan, group_off=go, prefix_len=pl, prefix_table=ptab)
        out = torch.full((T, Hq, d), 55.0, dtype=dt_, device="cuda")
        lse = torch.full((T, Hq), 55.0, device="cuda")
        ops.asm_shared_attention(qr, kp, vp, table, plan, 0.125, out, ws, prefix_table=ptab, lse_out=lse)
        assert ops.asm_workspace_error(ws) == 0
        pk64 = kp[ptab[0, :C.cdiv(Lp, S)].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :Lp].cpu().double()
        pv64 = pv.double().transpose(0, 1)
        at = 0
        for r, n in enumerate(new):
            for i in range(max(n, 0)):
                m = len(hist[r][0]) - n + i + 1
                kk = torch.cat([pk64, torch.stack(hist[r][0][:m], 1).double()], 1)
                vv = torch.cat([pv64, torch.stack(hist[r][1][:m], 1).double()], 1)
                qq = qr[at].cpu().double().view(Hkv, -1, d)
                s = torch.einsum("hgd,hkd->hgk", qq, kk) * 0.125
                z = torch.logsumexp(s, 2)
                p = torch.exp(s - z[..., None])
                ref = torch.einsum("hgk,hkd->hgd", p, vv).reshape(Hq, d)
                a = torch.einsum("hgk,hkd->hgd", p, vv.abs()).reshape(1, Hq, d)
                dot = (torch.einsum("hgd,hkd->hgk", qq.abs(), kk.abs()) * 0.125).amax(2).reshape(1, Hq)
                eo, ez = C.attention_bounds(ref[None], z.reshape(1, Hq), a, dot, torch.tensor([kk.shape[1]]), d, dt_)
                assert ((out[at].cpu().double() - ref).abs() <= eo[0]).all()
                assert ((lse[at].cpu().double() - z.reshape(Hq)).abs() <= ez[0]).all()
                at += 1
        assert (out[at:] == 55).all() and (lse[at:] == 55).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_memory_state_joins_paged_local_tokens(dt):
    """The memory's retrieved state (asm_decode_step without local tokens)
    merged with asm_shared_attention over local pages equals asm_decode_step
    over the same tokens in contiguous caches."""
    cfg = dict(inputs.CONFIGS[1], dtype=dt, Hq=8, Hkv=2)
    lens = [1, 37, 100, 64]
    ins = inputs.decode_inputs(cfg, B=4, K=200, T=100, local_len=lens)
    dv = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in ins.items()}
    B, Hq, d = dv["q"].shape
    Hkv, S = 2, 32

    def decode(T, local):
        ws = ops.alloc_workspace(ops.asm_decode_workspace_size(B, Hq, Hkv, 200, T, d, dv["q"].dtype), "cuda")
        out, lse = torch.empty_like(dv["q"]), torch.empty(B, Hq, device="cuda")
        ops.asm_decode_step(dv["q"], dv["centroids"], dv["a_bar"], dv["logz_bar"], dv["k_cache"][:, :, :T].contiguous(),
                            dv["v_cache"][:, :, :T].contiguous(), i32(local), ins["scale"], out, ws, lse_out=lse)
        return out, lse

    want, want_lse = decode(100, lens)
    got, lse = decode(1, [0] * B)
    n = sum(C.cdiv(x, S) for x in lens)
    kp = torch.full((n, Hkv, S, d), math.nan, dtype=dv["q"].dtype, device="cuda")
    vp = torch.full_like(kp, math.nan)
    table, at = np.full((B, 4), -1), 0
    for b, x in enumerate(lens):
        for p in range(C.cdiv(x, S)):
            m = min(S, x - p * S)
            kp[at, :, :m] = dv["k_cache"][b, :, p * S:p * S + m]
            vp[at, :, :m] = dv["v_cache"][b, :, p * S:p * S + m]
            table[b, p] = at
            at += 1
    plan = ops.alloc_workspace(ops.asm_shared_plan_size(B, 0, B, Hq, Hkv), "cuda", zero=False)
    ws = ops.alloc_workspace(ops.asm_shared_attention_workspace_size(B, Hq, Hkv, d), "cuda")
    ops.asm_shared_plan(i32(range(B + 1)), i32(lens), i32(table), B, Hq, Hkv, S, plan)
    loc, loc_lse = torch.empty_like(dv["q"]), torch.empty(B, Hq, device="cuda")
    ops.asm_shared_attention(dv["q"], kp, vp, i32(table), plan, ins["scale"], loc, ws, lse_out=loc_lse)
    ops.asm_merge_states(got, lse, loc, loc_lse)
    assert ops.asm_workspace_error(ws) == 0
    # both sides hold the parity rule of the decode tests; the merge rounds its inputs and its result once more
    u = C.U[dv["q"].dtype]
    tol = (2e-2 if dt == "bf16" else 1e-4) + 3 * u * float(want.abs().max())
    assert float((got - want).abs().max()) <= tol
    assert float((lse - want_lse).abs().max()) <= (2e-2 if dt == "bf16" else 1e-4)
