"""Paged serving calls without a GPU: arguments are refused with the
documented status before any CUDA call, and the plan's and the workspace's
sizes cover what the kernels address."""
import ctypes
import math

import pytest
import torch

from long_prefix_attention_b200 import _lib, build, ops

import paged_common as C

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NULL = None


def at(i, off=0):
    """Distinct fake addresses, 1 GiB apart, never dereferenced."""
    return ctypes.c_void_p((i + 1) * (1 << 30) + off)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def page_step(lib, **kw):
    a = dict(kv=at(0), new=at(1), base=at(2), R=4, S=16, MP=8, table=at(3), pool=at(4), state=at(5), F=64, T=10,
             seq=at(6), qoff=at(7), row=at(8), pos=at(9), slot=at(10), pout=at(11))
    a.update(kw)
    return lib.asm_page_step(a["kv"], a["new"], a["base"], a["R"], a["S"], a["MP"], a["table"], a["pool"], a["state"],
                             a["F"], a["T"], a["seq"], a["qoff"], a["row"], a["pos"], a["slot"], a["pout"], None)


def test_page_step_refusals(lib):
    for kw in (dict(kv=NULL), dict(new=NULL), dict(table=NULL), dict(pool=NULL), dict(state=NULL), dict(seq=NULL),
               dict(qoff=NULL), dict(pout=NULL), dict(row=NULL), dict(slot=at(10, 2)), dict(base=at(2, 1)),
               dict(R=0), dict(T=-1), dict(F=0), dict(MP=0), dict(F=1 << 27), dict(MP=1 << 27),
               dict(seq=at(0)), dict(pout=at(5)), dict(seq=at(1, 12)), dict(slot=at(2))):
        assert page_step(lib, **kw) == INVALID, kw
    assert page_step(lib, S=24) == UNSUPPORTED
    assert page_step(lib, S=256) == UNSUPPORTED
    assert page_step(lib, R=4097) == UNSUPPORTED


def test_page_step_refuses_a_table_or_ring_within_other_arrays(lib):
    for kw in (dict(seq=at(3, 4)), dict(pout=at(4, 8)), dict(slot=at(3, 124)), dict(kv=at(3)), dict(new=at(4)),
               dict(base=at(3, 16)), dict(state=at(4, 252)), dict(table=at(4, 128)), dict(pool=at(3, 64))):
        assert page_step(lib, **kw) == INVALID, kw


def rope(lib, **kw):
    a = dict(x=at(0), xt=512, xh=128, T=5, H=4, d=128, dt=1, pos=at(1), f=at(2), rot=128, lay=0, ms=1.0, inv=0, y=at(3),
             yt=512, yh=128)
    a.update(kw)
    return lib.asm_rope(a["x"], a["xt"], a["xh"], a["T"], a["H"], a["d"], a["dt"], a["pos"], a["f"], a["rot"], a["lay"],
                        a["ms"], a["inv"], a["y"], a["yt"], a["yh"], None)


def test_rope_refusals(lib):
    for kw in (dict(x=NULL), dict(y=NULL), dict(pos=NULL), dict(f=NULL), dict(f=at(2, 4)), dict(rot=0), dict(rot=130),
               dict(rot=7), dict(lay=2), dict(dt=2), dict(H=0), dict(T=-1), dict(ms=math.nan), dict(ms=math.inf),
               dict(xt=-1), dict(yt=128), dict(yh=0), dict(yh=64, yt=512), dict(x=at(0, 1)),
               dict(y=at(0), yt=1024), dict(y=at(0), yh=256, yt=1024)):
        assert rope(lib, **kw) == INVALID, kw
    assert rope(lib, d=96) == UNSUPPORTED
    assert rope(lib, T=0) == 0


def test_rope_freqs_refusals(lib):
    f = lib.asm_rope_freqs
    assert f(NULL, 64, 1e4, 0, 1.0, 1.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 63, 1e4, 0, 1.0, 1.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 130, 1e4, 0, 1.0, 1.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 64, 1.0, 0, 1.0, 1.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 64, 1e4, 5, 1.0, 1.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 64, 1e4, 1, 0.5, 1.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 64, 1e4, 3, 2.0, 4.0, 4.0, 8192.0, None) == INVALID
    assert f(at(0), 64, 1e4, 4, 2.0, 1.0, 4.0, 0.0, None) == INVALID


def append(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), T=5, Hq=8, Hkv=2, d=128, dt=1, pos=at(3), slot=at(4), f=at(5), rot=128, lay=0,
             ms=1.0, qo=at(6), ot=1024, kp=at(7), vp=at(8), n=4, S=16)
    a.update(kw)
    return lib.asm_rope_append(a["q"], 1024, 128, a["k"], 256, 128, a["v"], 256, 128, a["T"], a["Hq"], a["Hkv"],
                               a["d"], a["dt"], a["pos"], a["slot"], a["f"], a["rot"], a["lay"], a["ms"], a["qo"],
                               a["ot"], 128, a["kp"], a["vp"], a["n"], a["S"], None)


def test_rope_append_refusals(lib):
    for kw in (dict(k=NULL), dict(v=NULL), dict(slot=NULL), dict(kp=NULL), dict(vp=at(8, 8)), dict(n=0), dict(n=1 << 27),
               dict(Hkv=0), dict(Hq=0), dict(rot=126 + 4), dict(vp=at(7)), dict(vp=at(7, 1024)), dict(ot=512),
               dict(qo=at(0), ot=2048)):
        assert append(lib, **kw) == INVALID, kw
    assert append(lib, S=8) == UNSUPPORTED
    assert append(lib, d=80) == UNSUPPORTED
    assert append(lib, T=0) == 0


def plan(lib, **kw):
    a = dict(qo=at(0), sl=at(1), go=at(2), pl=at(3), R=4, NG=2, T=100, Hq=8, Hkv=2, S=16, MP=8, MPP=8, plan=at(4),
             nb=1 << 24)
    a.update(kw)
    return lib.asm_shared_plan(a["qo"], a["sl"], a["go"], a["pl"], a["R"], a["NG"], a["T"], a["Hq"], a["Hkv"], a["S"],
                               a["MP"], a["MPP"], a["plan"], a["nb"], None)


def attn(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), n=64, S=16, t=at(3), MP=8, pt=at(4), MPP=8, plan=at(5), pb=1 << 24, R=4, NG=2,
             T=100, Hq=8, Hkv=2, d=128, scale=0.1, dt=1, out=at(6), lse=at(7), ws=at(8), wb=1 << 29)
    a.update(kw)
    return lib.asm_shared_attention(a["q"], a["k"], a["v"], a["n"], a["S"], a["t"], a["MP"], a["pt"], a["MPP"],
                                    a["plan"], a["pb"], a["R"], a["NG"], a["T"], a["Hq"], a["Hkv"], a["d"], a["scale"],
                                    a["dt"], a["out"], a["lse"], a["ws"], a["wb"], None)


def test_shared_attention_refusals(lib):
    need = lib.asm_shared_plan_size(4, 2, 100, 8, 2)
    assert need > 0
    for kw in (dict(qo=NULL), dict(sl=NULL), dict(go=NULL), dict(pl=NULL), dict(R=0), dict(NG=-1), dict(T=0),
               dict(Hkv=3), dict(MP=0), dict(MPP=0), dict(MP=1 << 28)):
        assert plan(lib, **kw) == INVALID, kw
    for kw in (dict(R=4097), dict(NG=4097), dict(T=(1 << 24) + 1), dict(Hq=32), dict(S=20)):
        assert plan(lib, **kw) == UNSUPPORTED, kw
    assert plan(lib, nb=need - 1) == WORKSPACE and plan(lib, plan=NULL) == WORKSPACE
    wneed = lib.asm_shared_attention_workspace_size(100, 8, 2, 128)
    for kw in (dict(q=NULL), dict(k=at(1, 8)), dict(v=NULL), dict(t=NULL), dict(pt=NULL), dict(out=NULL),
               dict(lse=at(7, 2)), dict(n=0), dict(n=1 << 28), dict(dt=2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.nan), dict(scale=math.inf), dict(out=at(0)), dict(out=at(0, 2048)), dict(T=0)):
        assert attn(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(S=512), dict(Hq=32), dict(R=5000)):
        assert attn(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(pb=need - 1), dict(plan=NULL), dict(ws=NULL), dict(wb=wneed - 1)):
        assert attn(lib, **kw) == WORKSPACE, kw
    assert lib.asm_shared_plan_size(4, 2, 100, 9, 2) == 0
    assert lib.asm_shared_attention_workspace_size(100, 8, 2, 96) == 0


def test_binding_refuses_host_tensors_and_other_types():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.asm_page_step(i, i, i, i, 16, i.view(1, 4), i, i, i, i, i, i)
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        ops.asm_rope(x, i, torch.zeros(32, dtype=torch.float64), x)
    with pytest.raises(ValueError):
        ops.asm_shared_attention(x, x, x, i, i, 1.0, x, i)
    with pytest.raises(TypeError):
        ops._i32("f", i.long())


def test_key_lists_are_at_most_2_to_30(lib):
    """A unit's last key plus one unit stays within int32."""
    assert plan(lib, MP=(1 << 26) + 1) == INVALID and plan(lib, MPP=(1 << 26) + 1) == INVALID
    assert attn(lib, MP=(1 << 26) + 1) == INVALID and attn(lib, MPP=(1 << 26) + 1) == INVALID
    # the limit itself passes on to the next check
    assert plan(lib, MP=1 << 26, MPP=1 << 26, nb=16) == WORKSPACE
    assert attn(lib, MP=1 << 26, MPP=1 << 26, pb=16) == WORKSPACE


def plan_tiles(new, old, pre, cuts, G):
    """The tiles of a plan, (query rows per KV head, units) each, as the plan
    kernel lays them out: prefix tiles over the runs of rows of up to 128 query
    rows, then every row's own, which hold the prefix too where the row has
    more."""
    single, dual = 128 // G, 256 // G

    def split(n):
        return [] if n <= 0 else [n] if n <= single else [min(dual, n - i) for i in range(0, n, dual)]

    group = [next((g for g in range(len(pre)) if cuts[g] <= r < cuts[g + 1]), None) for r in range(len(new))]
    tiles, run, at = [], 0, None
    runs = []
    for r, g in enumerate(group):
        if g is None or new[r] > single:
            at = None
            continue
        if at != g:
            runs.append([g, 0])
            at = g
        runs[-1][1] += new[r]
    for g, n in runs:
        tiles += [(t * G, C.cdiv(pre[g], 128)) for t in split(n)]
    for r, n in enumerate(new):
        done = 0
        for t in split(n):
            done += t
            both = C.cdiv(pre[group[r]], 128) if n > single and group[r] is not None else 0
            tiles.append((t * G, both + C.cdiv(old[r] + done, 128)))
    return tiles


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_the_plans_bounds_hold(lib, G):
    """For random lengths: the tiles, the partial rows and the segments never
    exceed what the size functions provide for, and the workers' ranges take
    every unit once."""
    import random
    rng = random.Random(G)
    Hkv, workers = 4, 148
    Hq = G * Hkv
    unit_cost = lambda rows: 4 if rows > 128 else 2          # noqa: E731
    head_cost = lambda rows: 4 if rows > 128 else 2          # noqa: E731
    for _ in range(150):
        R, NG = rng.randint(1, 60), rng.randint(0, 4)
        new = [rng.choice([0, 1, 1, 3, rng.randint(0, 900)]) for _ in range(R)]
        old = [rng.choice([0, 100, 9000]) for _ in range(R)]
        pre = [rng.choice([0, 1, 300, 40000]) for _ in range(NG)]
        cuts = sorted(rng.randint(0, R) for _ in range(NG + 1))
        T = max(1, sum(new))
        tiles = plan_tiles(new, old, pre, cuts, G)
        assert len(tiles) <= min(R, T) + min(NG, T) + 4 * C.cdiv(T * G, 256)
        cost = [head_cost(r) + unit_cost(r) * u if u else 0 for r, u in tiles]
        W = Hkv * sum(cost)
        size = max(C.cdiv(W, workers), 4 if any(r > 128 for r, _ in tiles) else 2)
        assert sum((c // size + 2) * Hkv * r for (r, u), c in zip(tiles, cost) if u) <= \
            4 * T * Hq + (workers + 1) * 256
        c0 = 0
        for (r, u), c in zip(tiles, cost):
            for _ in range(Hkv):
                who = [(c0 + head_cost(r) + unit_cost(r) * k) // size for k in range(u)]
                if who:
                    assert who[-1] < workers and who[-1] - who[0] + 1 <= c // size + 2
                    # no worker between the first and the last goes without a unit
                    assert sorted(set(who)) == list(range(who[0], who[-1] + 1))
                c0 += c


def test_the_quintic_exponential():
    """A quarter of the softmax exponentials runs on the FMA pipe
    (csrc/shared_attn_tc.cu, exp2_poly_x2): the same steps in fp32, a fused
    multiply-add as an exact product and one rounding, stay within the 2^-20
    the attention bounds count."""
    import numpy as np
    f32 = np.float32
    co = [f32(x) for x in (0.001327647245, 0.009675540961, 0.05550713092, 0.2402212024, 0.693146944, 1.000000119)]
    t = np.linspace(-100.0, 20.0, 600_001).astype(f32)
    y = (t + f32(12582912.0)).astype(f32)
    n = (y - f32(12582912.0)).astype(f32)
    fr = (t.astype(np.float64) - n.astype(np.float64)).astype(f32)
    p = np.full_like(fr, co[0])
    for c in co[1:]:
        p = (p.astype(np.float64) * fr.astype(np.float64) + float(c)).astype(f32)
    bits = (p.view(np.uint32) + (y.view(np.uint32) << np.uint32(23))).astype(np.uint32)
    got, ref = bits.view(f32).astype(np.float64), np.exp2(t.astype(np.float64))
    assert (np.abs(got - ref) / ref).max() < 2.0 ** -20 / 2


def test_shared_attention_refuses_outputs_within_other_arrays(lib):
    """Tiles of a call read their inputs and the partial states while others write."""
    ws = lib.asm_shared_attention_workspace_size(100, 8, 2, 128)
    pl = lib.asm_shared_plan_size(4, 2, 100, 8, 2)
    out_n, lse_n, kv_n = 100 * 8 * 128 * 2, 100 * 8 * 4, 64 * 2 * 16 * 128 * 2
    for kw in (dict(out=at(1)), dict(out=at(2, kv_n - 16)), dict(out=at(3)), dict(out=at(4, 48)), dict(out=at(5, pl - 16)),
               dict(out=at(8)), dict(lse=at(0)), dict(lse=at(1, 64)), dict(lse=at(2)), dict(lse=at(3, 4)), dict(lse=at(4)),
               dict(lse=at(5)), dict(lse=at(6)), dict(lse=at(6, out_n - 4)), dict(lse=at(8, 256)), dict(ws=at(0)),
               dict(ws=at(1, 16)), dict(ws=at(2)), dict(ws=at(3)), dict(ws=at(4)), dict(ws=at(5)), dict(ws=at(6)),
               dict(ws=at(7)), dict(out=at(9), ws=at(9, out_n - 16)), dict(out=at(9), lse=at(9, out_n - 4))):
        assert attn(lib, **kw) == INVALID, {k: hex(v.value) for k, v in kw.items()}
    for kw in (dict(qo=at(4)), dict(sl=at(4, 256)), dict(go=at(4, pl - 16)), dict(pl=at(4, 512)), dict(plan=at(1))):
        assert plan(lib, **kw) == INVALID, kw
    assert lse_n and ws


def test_rope_append_refuses_caches_within_other_arrays(lib):
    cache = 4 * 16 * 2 * 128 * 2
    for kw in (dict(q=at(7)), dict(k=at(7, 256)), dict(v=at(8, cache - 2)), dict(qo=at(8)), dict(pos=at(7)), dict(slot=at(8, 4)),
               dict(f=at(7, 64)), dict(kp=at(1, 2 * 4 * 256)), dict(vp=at(2, 256))):
        assert append(lib, **kw) == INVALID, kw


def tiles_provided(plan_bytes, T):
    """Tiles of 64 bytes between the workers' first tiles (256 + 4096 bytes) and the token map
    (8 bytes a token, 256-byte aligned) of a plan of that size."""
    return ((plan_bytes - 8 * T) // 256 * 256 - 4352) // 64


def partial_rows_provided(ws_bytes, d):
    """Partial rows (two floats of statistics, d of output) that surely fit a workspace of
    that size, its error word and two alignments apart."""
    return (ws_bytes - 256 - 2 * 255) // (8 + 4 * d)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_the_size_functions_cover_the_plan(lib, G):
    """For random lengths, the tiles of the plan and the rows of its partial states fit what
    asm_shared_plan_size and asm_shared_attention_workspace_size return."""
    import random
    rng = random.Random(50 + G)
    Hkv, workers = 4, 148               # without a GPU the library sizes for 148 multiprocessors
    Hq = G * Hkv
    tightest = 0.0
    for _ in range(300):
        R, NG = rng.randint(1, 60), rng.randint(0, 4)
        new = [rng.choice([0, 1, 1, 3, rng.randint(0, 900), 128 // G, 128 // G + 1]) for _ in range(R)]
        old = [rng.choice([0, 100, 9000]) for _ in range(R)]
        pre = [rng.choice([0, 1, 300, 40000]) for _ in range(NG)]
        cuts = sorted(rng.randint(0, R) for _ in range(NG + 1))
        T = max(1, sum(new))
        tiles = plan_tiles(new, old, pre, cuts, G)
        have = tiles_provided(lib.asm_shared_plan_size(R, NG, T, Hq, Hkv), T)
        assert len(tiles) <= have
        tightest = max(tightest, len(tiles) / have)
        cost = [(4 if r > 128 else 2) * (u + 1) if u else 0 for r, u in tiles]
        size = max(C.cdiv(Hkv * sum(cost), workers), 4 if any(r > 128 for r, _ in tiles) else 2)
        need = sum((c // size + 2) * Hkv * r for (r, u), c in zip(tiles, cost) if u)
        for d in (64, 128):
            assert need <= partial_rows_provided(lib.asm_shared_attention_workspace_size(T, Hq, Hkv, d), d)
    assert tightest > 0.3               # the bound is not checked against thin air
