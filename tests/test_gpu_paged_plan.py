"""The plan of asm_shared_attention read back, and lengths that make no sense."""
import random

import numpy as np
import pytest
import torch

import paged_common as C
from long_prefix_attention_b200 import ops
from test_gpu_paged import Batch, i32
from test_paged_cpu import partial_rows_provided, plan_tiles, tiles_provided

pytestmark = pytest.mark.gpu

# csrc/shared.cuh: Header, first[1024], Tile
HEADER = np.dtype([(k, "<i4") for k in ("magic", "R", "NG", "T", "Hq", "Hkv", "S", "max_pages", "max_prefix_pages", "workers",
                                        "ntiles", "range")] + [("W", "<i8"), ("inv", "<f8")])
TILE = np.dtype([(k, "<i4") for k in ("tok0", "ntok", "group", "row", "pre_keys", "keys", "base", "units", "direct", "cap")] +
                [("cost0", "<i8"), ("row0", "<i8"), ("pad", "<i4", 2)])
FIRST, TILES = 256, 256 + 4 * 1024


def clamped(q_off, seq, goff, pre, R, T, table_keys, prefix_keys):
    """The documented rule: offsets raised to the largest before them, all within their limits."""
    def rise(x, hi):
        return np.maximum.accumulate(np.clip(np.asarray(x, dtype=np.int64), 0, hi))
    return rise(q_off, T), np.clip(seq, 0, table_keys), rise(goff, R), np.clip(pre, 0, prefix_keys)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_the_plan_holds_every_unit_once(G):
    """Tiles, costs, partial rows, the workers' first tiles and the token map of plans for random
    lengths against the host's model, and within what the size functions provide."""
    rng = random.Random(G)
    Hkv, S = 4, 16
    Hq = G * Hkv
    for it in range(30):
        R, NG = rng.randint(1, 60), rng.randint(1, 4)
        new = [rng.choice([0, 1, 1, 3, rng.randint(0, 900)]) for _ in range(R)]
        old = [rng.choice([0, 100, 9000]) for _ in range(R)]
        pre = [rng.choice([0, 1, 300, 40000]) for _ in range(NG)]
        cuts = sorted(rng.randint(0, R) for _ in range(NG + 1))
        T = max(1, sum(new)) + rng.choice([0, 7])
        seq = [a + b for a, b in zip(new, old)]
        n = ops.asm_shared_plan_size(R, NG, T, Hq, Hkv)
        buf = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        q_off = np.concatenate([[0], np.cumsum(new)])
        ops.asm_shared_plan(i32(q_off), i32(seq), torch.zeros(R, 700, dtype=torch.int32, device="cuda"), T, Hq, Hkv, S,
                            buf[:n], group_off=i32(cuts), prefix_len=i32(pre),
                            prefix_table=torch.zeros(NG, 3000, dtype=torch.int32, device="cuda"))
        assert (buf[n:] == 0x5a).all().item()
        raw = buf[:n].cpu().numpy()
        h = raw[:HEADER.itemsize].view(HEADER)[0]
        want = plan_tiles(new, old, pre, cuts, G)
        assert (h["R"], h["NG"], h["T"], h["ntiles"]) == (R, NG, T, len(want)) and len(want) <= tiles_provided(n, T)
        t = raw[TILES:TILES + TILE.itemsize * len(want)].view(TILE)
        assert [(int(x["ntok"]) * G, int(x["units"])) for x in t] == want
        unit = np.where(t["ntok"] * G > 128, 4, 2).astype(np.int64)
        cost = np.where(t["units"] > 0, unit * (t["units"].astype(np.int64) + 1), 0)      # a head costs as much as a unit
        assert (t["cost0"] == np.concatenate([[0], np.cumsum(cost)])[:-1]).all() and h["W"] == Hkv * cost.sum()
        size, workers = int(h["range"]), int(h["workers"])
        assert size >= 1 and workers * size >= h["W"]
        # partial rows: a tile's end before the next one's begin
        rows = np.where(t["units"] > 0, t["cap"].astype(np.int64) * Hkv * t["ntok"] * G, 0)
        assert (t["row0"] == np.concatenate([[0], np.cumsum(rows)])[:-1]).all()
        ws = ops.asm_shared_attention_workspace_size(T, Hq, Hkv, 64)
        assert rows.sum() <= partial_rows_provided(ws, 64)
        for x, c, u in zip(t, cost, unit):
            for g in range(Hkv) if x["units"] else ():
                c0 = int(x["cost0"]) * Hkv + g * int(c)
                who = (c0 + u * (1 + np.arange(x["units"], dtype=np.int64))) // size
                assert who[-1] < workers and who[-1] - who[0] + 1 <= x["cap"]
        first = raw[FIRST:FIRST + 4 * workers].view("<i4")
        ends = (t["cost0"] + cost) * Hkv
        for w in range(workers):
            if w * size < h["W"]:
                assert first[w] == np.searchsorted(ends, w * size, side="right")
        tok = raw[TILES + (tiles_provided(n, T)) * TILE.itemsize:].view("<i4")[:2 * T].reshape(T, 2)
        group = [next((g for g in range(NG) if cuts[g] <= r < cuts[g + 1]), -1) for r in range(R)]
        row = np.repeat(np.arange(R), new)
        for i in range(T):
            a, b = (int(v) for v in tok[i])
            if i >= len(row):
                assert (a, b) == (-1, -1)
                continue
            x, r = t[a], int(row[i])
            assert x["row"] == r and x["tok0"] <= i < x["tok0"] + x["ntok"]
            short = new[r] <= 128 // G
            assert (b >= 0) == (short and group[r] >= 0)
            if b >= 0:
                y = t[b]
                assert y["group"] == group[r] and y["tok0"] <= i < y["tok0"] + y["ntok"] and y["keys"] == 0
            assert x["direct"] == int(group[r] < 0 or pre[group[r]] == 0 or not short)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_lengths_that_make_no_sense_are_clamped(dt):
    """Falling and negative offsets, lengths past the tables: the results are those of the
    documented rule, and nothing behind out, lse, plan and workspace is written."""
    R, S, pages = 3, 16, 5
    base = Batch(dt, 4, 2, 64, S, new=[3, 4, 2], seq=[30, 40, 20], goff=[0, 2, 3], pre=[30, 40], seed=10)
    g = torch.Generator().manual_seed(1)
    for x in (base.kd, base.vd):
        x.copy_(torch.randn(x.shape, generator=g).to(base.dt))
    rng = random.Random(7)
    base.table = np.array([[rng.randrange(base.n_pages) for _ in range(pages)] for _ in range(R)])
    base.ptable = np.array([[rng.randrange(base.n_pages) for _ in range(pages + 1)] for _ in range(2)])
    base.dev = dict(table=i32(base.table), prefix_table=i32(base.ptable))
    T = base.q.shape[0]
    odd = [-2**31, -5, -1, 0, 1, 2, 3, 5, 8, 9, 12, 79, 80, 81, 900, 2**31 - 1]
    cases = [([0, 9, 3, 9], [30, 40, 20], [0, 2, 3], [30, 40]), ([5, 2, 900, -4], [10**9, -3, 20], [3, 0, 99], [10**9, -1]),
             ([-9, -9, -9, -9], [1, 1, 1], [-1, -1, -1], [1, 1])]
    cases += [tuple([rng.choice(odd) for _ in range(n)] for n in (4, 3, 3, 2)) for _ in range(40)]
    for qo, sl, go, pl in cases:
        n_plan = ops.asm_shared_plan_size(R, 2, T, 4, 2)
        n_ws = ops.asm_shared_attention_workspace_size(T, 4, 2, 64)
        plan = torch.full((n_plan + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        ws = torch.full((n_ws + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        out = torch.full((T + 2, 4, 64), 55.0, dtype=base.dt, device="cuda")
        lse = torch.full((T + 2, 4), 55.0, device="cuda")
        ops.asm_shared_plan(i32(qo), i32(sl), base.dev["table"], T, 4, 2, S, plan[:n_plan], group_off=i32(go),
                            prefix_len=i32(pl), prefix_table=base.dev["prefix_table"])
        ops.asm_shared_attention(base.q.cuda(), base.kd, base.vd, base.dev["table"], plan[:n_plan], base.scale, out[:T],
                                 ws[:n_ws], prefix_table=base.dev["prefix_table"], lse_out=lse[:T])
        assert ops.asm_workspace_error(ws[:n_ws]) == 0
        assert (plan[n_plan:] == 0x5a).all().item() and (ws[n_ws:] == 0x5a).all().item()
        q_off, seq, goff, pre = clamped(qo, sl, go, pl, R, T, pages * S, (pages + 1) * S)
        ro, rl, a, dot, cnt = C.attention(base.q, base.kd.cpu(), base.vd.cpu(), base.table, q_off, seq, base.scale,
                                          goff, pre, base.ptable)
        o, z = out.cpu().double(), lse.cpu().double()
        real = torch.zeros(T + 2, dtype=torch.bool)
        real[:T] = ~torch.isnan(rl[:, 0])
        assert real.sum() == q_off[-1] - q_off[0]
        assert (o[~real] == 55).all() and (z[~real] == 55).all()
        keep = real[:T]
        ro, rl, a, dot, cnt, o, z = ro[keep], rl[keep], a[keep], dot[keep], cnt[keep], o[real], z[real]
        eo, ez = C.attention_bounds(ro, rl, a, dot, cnt, 64, base.dt)
        fin = ~torch.isinf(rl)
        assert torch.equal(torch.isinf(z), ~fin) and (o[~fin] == 0).all()
        assert ((z - rl)[fin].abs() <= ez[fin]).all() and ((o - ro).abs() <= eo).all()
