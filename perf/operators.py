"""Workloads of the serving operators around the attention-state memory.

Four operators of a decode or prefill step whose requests keep their local
tokens in pages and share long prefixes:

* ``pages``:  page tables and slot maps of a step, from the request lengths;
* ``rope``:   rotary positions of one tensor of heads (and their inverse);
* ``append``: rotary positions of q and k, and k, v written to their pages;
* ``attn``:   attention of a ragged batch over the prefixes its rows share
              (each read once for all its rows) and over each row's own pages.

``listed()`` names fixed cases, ``draw`` makes more of the same ranges,
``prepare`` the inputs of one, ``run`` one pass (plain torch, or the library's
calls when ``own`` is true), ``work`` its unavoidable bytes and operations and
``exact`` its result from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a small batch: latency only
        dict(name="pages-decode-r16", op="pages", rows=16, tokens=16, page=64, max_pages=64, new_lo=1, new_hi=1,
             ended=0.0, tight=False, lens=1),
        # a busy server's step: decode rows, prompt chunks of hundreds of tokens, rows that end, a pool that runs
        # short, and a padded token batch
        dict(name="pages-mixed-r1500", op="pages", rows=1500, tokens=40000, page=16, max_pages=513, new_lo=1,
             new_hi=700, ended=0.1, tight=True, lens=2),
        # the queries of a 16-row decode step of one LLaMA-3.1-8B layer
        dict(name="rope-decode-t16", op="rope", tokens=16, heads=32, d=128, rot=128, layout="half", inverse=False,
             scaling="bands", far=131072, dt="bf16", packed=False),
        # keys un-rotated (or their gradient) at positions up to a million, half of the head rotated
        dict(name="rope-inverse-t32785", op="rope", tokens=32785, heads=8, d=128, rot=64, layout="pairs",
             inverse=True, scaling="yarn", far=1 << 20, dt="f32", packed=False),
        # a 64-row decode step: q, k, v are views of one packed projection
        dict(name="append-decode-t64", op="append", tokens=64, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="bands", far=40000, page=64, hole=0.0, dt="bf16", packed=True),
        # prompt chunks of 8191 tokens in all; a few tokens have no slot
        dict(name="append-prefill-t8191", op="append", tokens=8191, hq=32, hkv=8, d=128, rot=128, layout="pairs",
             scaling="linear", far=70000, page=16, hole=0.01, dt="bf16", packed=True),
        # the smallest attention: one token, one short prefix, a handful of local tokens
        dict(name="attn-tiny-f32", op="attn", hq=2, hkv=1, d=64, page=16, rows=1, groups=1, alone=0.0, pre_lo=512,
             pre_hi=512, old_lo=15, old_hi=15, new_lo=1, new_hi=1, dt="f32", lens=3),
        # 16 decode rows of a LLaMA-3.1-8B layer behind one 16384-token prefix, ragged local lengths
        dict(name="attn-decode-r16-p16384", op="attn", hq=32, hkv=8, d=128, page=64, rows=16, groups=1, alone=0.0,
             pre_lo=16384, pre_hi=16384, old_lo=0, old_hi=4095, new_lo=1, new_hi=1, dt="bf16", lens=4),
        # 64 decode rows, a 32768-token prefix, 8192 local tokens each: the local pages bound it
        dict(name="attn-decode-r64-p32768", op="attn", hq=32, hkv=8, d=128, page=64, rows=64, groups=1, alone=0.0,
             pre_lo=32768, pre_hi=32768, old_lo=8191, old_hi=8191, new_lo=1, new_hi=1, dt="bf16", lens=5),
        # several short prefixes, some rows with none, 1 to 8 drafted tokens a row to verify, small pages
        dict(name="attn-verify-r40-g3", op="attn", hq=16, hkv=16, d=64, page=16, rows=40, groups=3, alone=0.2,
             pre_lo=301, pre_hi=5003, old_lo=0, old_hi=1500, new_lo=1, new_hi=8, dt="bf16", lens=6),
        # prompt chunks behind a long prefix: the tensor cores bound it
        dict(name="attn-prefill-r6-p16384", op="attn", hq=32, hkv=8, d=128, page=64, rows=6, groups=1, alone=0.0,
             pre_lo=16384, pre_hi=16384, old_lo=0, old_hi=1000, new_lo=257, new_hi=511, dt="bf16", lens=7),
        # fp32 storage, a handful of rows
        dict(name="attn-decode-r8-f32", op="attn", hq=8, hkv=2, d=128, page=32, rows=8, groups=2, alone=0.0,
             pre_lo=4000, pre_hi=4097, old_lo=100, old_hi=700, new_lo=1, new_hi=2, dt="f32", lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "rope", "append", "attn", "attn"])
    if op == "pages":
        rows = _log(rng, 1, 2000)
        hi = rng.choice([1, 1, 8, 700])
        return dict(op=op, rows=rows, tokens=min(40000, rows * max(1, hi // 2) + rng.randint(0, 64)),
                    page=rng.choice([16, 32, 64, 128]), max_pages=rng.randint(40, 513), new_lo=rng.choice([0, 1]),
                    new_hi=hi, ended=rng.choice([0.0, 0.1, 0.3]), tight=rng.random() < 0.3, lens=rng.randint(10, 10**6))
    if op in ("rope", "append"):
        d = rng.choice([64, 128])
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        c = dict(op=op, d=d, rot=rot, layout=rng.choice(["half", "pairs"]),
                 scaling=rng.choice(["none", "linear", "base", "bands", "yarn"]), far=_log(rng, 100, 1 << 20),
                 dt=rng.choice(["bf16", "bf16", "f32"]), packed=rng.random() < 0.5)
        if op == "rope":
            c.update(tokens=_log(rng, 1, 30000), heads=rng.choice([1, 2, 5, 8]) if rng.random() < 0.5 else 32,
                     inverse=rng.random() < 0.5)
            if c["heads"] == 32:
                c["tokens"] = min(c["tokens"], 8000)
        else:
            hkv = rng.choice([1, 2, 4, 8])
            c.update(tokens=_log(rng, 1, 8191), hkv=hkv, hq=hkv * rng.choice([1, 2, 4]),
                     page=rng.choice([16, 32, 64, 128]), hole=rng.choice([0.0, 0.05]))
        return c
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    hq = min(hq, 32)
    d = rng.choice([64, 128])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    groups = rng.choice([0, 1, 1, 2, 4])
    kind = rng.choice(["decode", "decode", "verify", "prefill"])
    if dt == "f32":
        rows, pre, old = _log(rng, 1, 12), _log(rng, 30, 4096), _log(rng, 1, 700)
        new = {"decode": 1, "verify": 4, "prefill": 60}[kind]
    else:
        rows = _log(rng, 1, 64) if kind != "prefill" else _log(rng, 1, 6)
        pre, old = _log(rng, 60, 32768), _log(rng, 1, 8191)
        new = {"decode": 1, "verify": 8, "prefill": 450}[kind]
        if kind == "prefill":
            pre, old = min(pre, 16384), min(old, 1000)
    return dict(op=op, hq=hq, hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]), rows=rows, groups=groups,
                alone=rng.choice([0.0, 0.0, 0.3]), pre_lo=max(1, pre // 2), pre_hi=pre, old_lo=rng.randint(0, old),
                old_hi=old, new_lo=1, new_hi=new, dt=dt, lens=rng.randint(10, 10**6))


# ---------------------------------------------------- lengths and layouts --

def _cdiv(a, b):
    return -(-a // b)


def _page_lens(case):
    """Host lengths of a ``pages`` case: cached tokens, new tokens (-1: the row ends), free pages."""
    rng = random.Random(case["lens"])
    R, ps, MP = case["rows"], case["page"], case["max_pages"]
    kv, new, left = [], [], case["tokens"]
    for _ in range(R):
        kv.append(rng.randint(0, min(4000, MP * ps)))
        if rng.random() < case["ended"]:
            new.append(-1)
            continue
        n = rng.randint(case["new_lo"], case["new_hi"])
        if case["new_hi"] > 8 and rng.random() < 0.9:
            n = min(n, 1)                      # most rows decode, some bring a prompt chunk
        n = min(n, left)
        left -= n
        new.append(n)
    held = sum(_cdiv(k, ps) for k in kv)
    need = sum(_cdiv(k + n, ps) - _cdiv(k, ps) for k, n in zip(kv, new) if n > 0)
    free = max(1, need * 2 // 3) if case["tight"] else need + 7
    return kv, new, held, free


def _attn_lens(case):
    """Host lengths of an ``attn`` case: prefix lengths, rows per group, old and new tokens per row."""
    rng = random.Random(case["lens"])
    R, NG = case["rows"], case["groups"]
    pre = [rng.randint(case["pre_lo"], case["pre_hi"]) for _ in range(NG)]
    shared = R - int(R * case["alone"]) if NG else 0
    cuts = sorted(rng.randint(0, shared) for _ in range(max(0, NG - 1)))
    goff = [0] + cuts + [shared] if NG else [0]
    old = [rng.randint(case["old_lo"], case["old_hi"]) for _ in range(R)]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(R)]
    return pre, goff, old, new


def _freqs(case, dev):
    """Angle per position of each rotated pair, 64 bits, and the factor on cos and sin."""
    rot = case["rot"]
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=dev)
    theta, factor, ctx = 500000.0, 8.0, 8192.0
    kind = case["scaling"]
    if kind == "base":
        theta = theta * factor ** (rot / max(rot - 2, 1))
    f = theta ** (-i / rot)
    if kind == "linear":
        f = f / factor
    if kind == "bands":
        wl = 2 * math.pi / f
        lo, hi = 1.0, 4.0
        s = ((ctx / wl - lo) / (hi - lo)).clamp(0, 1)
        f = (1 - s) * f / factor + s * f
    if kind == "yarn":
        def dim(turns):
            return rot * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64, device=dev) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    return f, (0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0)


# ---------------------------------------------------------------- prepare --

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = _PREPARE[case["op"]](case, seed, g, dev)
    st["case"] = case
    if own:
        _attach(st)
    return st


def _i32(x, dev):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(dev)


def _prep_pages(case, seed, g, dev):
    R, ps, MP, T = case["rows"], case["page"], case["max_pages"], case["tokens"]
    kv, new, held, free = _page_lens(case)
    rng = np.random.default_rng(seed)
    F = held + free
    ids = rng.permutation(F).astype(np.int32)
    table = np.full((R, MP), -1, np.int32)
    at = 0
    for r in range(R):
        n = _cdiv(kv[r], ps)
        table[r, :n] = ids[at:at + n]
        at += n
    head = int(rng.integers(0, F))
    pool = np.full(F, -1, np.int32)
    pool[(head + np.arange(free)) % F] = ids[at:]
    return dict(kv_len=_i32(kv, dev), new_len=_i32(new, dev), pos_base=_i32(rng.integers(0, 33000, R), dev),
                pool=_i32(pool, dev), pool_state=_i32([head, free, 0], dev), table=_i32(table, dev),
                seq_len=torch.empty(R, dtype=torch.int32, device=dev),
                q_off=torch.empty(R + 1, dtype=torch.int32, device=dev),
                row=torch.empty(T, dtype=torch.int32, device=dev), pos=torch.empty(T, dtype=torch.int32, device=dev),
                slot=torch.empty(T, dtype=torch.int32, device=dev),
                pool_out=torch.empty(3, dtype=torch.int32, device=dev))


def _heads(g, dev, T, H, d, dt):
    return torch.randn(T, H, d, generator=g, device=dev).to(dt)


def _prep_rope(case, seed, g, dev):
    T, H, d, dt = case["tokens"], case["heads"], case["d"], _DT[case["dt"]]
    x = _heads(g, dev, T, H + 3, d, dt)[:, 1:H + 1] if case["packed"] else _heads(g, dev, T, H, d, dt)
    f, ms = _freqs(case, dev)
    pos = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
    return dict(x=x, pos=pos, freq=f, mscale=ms, y=torch.empty(T, H, d, dtype=dt, device=dev))


def _prep_append(case, seed, g, dev):
    T, Hq, Hkv, d, ps, dt = case["tokens"], case["hq"], case["hkv"], case["d"], case["page"], _DT[case["dt"]]
    if case["packed"]:
        qkv = _heads(g, dev, T, Hq + 2 * Hkv, d, dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (_heads(g, dev, T, h, d, dt) for h in (Hq, Hkv, Hkv))
    n_pages = _cdiv(T, ps) + 3
    rng = np.random.default_rng(seed)
    pages = rng.permutation(n_pages)
    start = int(rng.integers(0, ps))
    t = np.arange(T) + start
    slot = pages[t // ps] * ps + t % ps
    slot[rng.random(T) < case["hole"]] = -1
    f, ms = _freqs(case, dev)
    far = max(0, case["far"] - T)
    return dict(q=q, k=k, v=v, pos=_i32(far + np.arange(T), dev), slot=_i32(slot, dev), freq=f, mscale=ms,
                q_out=torch.empty(T, Hq, d, dtype=dt, device=dev),
                k_pages=torch.zeros(n_pages, Hkv, ps, d, dtype=dt, device=dev),
                v_pages=torch.zeros(n_pages, Hkv, ps, d, dtype=dt, device=dev))


def _prep_attn(case, seed, g, dev):
    Hq, Hkv, d, ps, dt = case["hq"], case["hkv"], case["d"], case["page"], _DT[case["dt"]]
    pre, goff, old, new = _attn_lens(case)
    R, NG = case["rows"], case["groups"]
    loc = [a + b for a, b in zip(old, new)]
    n_pre, n_loc = [_cdiv(x, ps) for x in pre], [_cdiv(x, ps) for x in loc]
    used = sum(n_pre) + sum(n_loc)
    n_pages = used + 5
    rng = np.random.default_rng(seed)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((R, max(n_loc) + 2), -1, np.int32)
    ptable = np.full((max(NG, 1), max(n_pre + [1])), -1, np.int32)
    at = 0
    for j, n in enumerate(n_pre):
        ptable[j, :n] = ids[at:at + n]
        at += n
    for r, n in enumerate(n_loc):
        table[r, :n] = ids[at:at + n]
        at += n
    T = sum(new)
    k = torch.empty(n_pages, Hkv, ps, d, dtype=dt, device=dev)
    v = torch.empty(n_pages, Hkv, ps, d, dtype=dt, device=dev)
    step = max(1, (1 << 26) // (Hkv * ps * d))
    for a in range(0, n_pages, step):           # drawn in pieces: the fp32 draws stay small
        for x in (k, v):
            m = min(step, n_pages - a)
            x[a:a + m] = torch.randn(m, Hkv, ps, d, generator=g, device=dev).to(dt)
    q = (1.5 * torch.randn(T, Hq, d, generator=g, device=dev)).to(dt)
    return dict(q=q, k_pages=k, v_pages=v, table=_i32(table, dev), ptable=_i32(ptable, dev) if NG else None,
                q_off=_i32(np.concatenate([[0], np.cumsum(new)]), dev), seq_len=_i32(loc, dev),
                group_off=_i32(goff, dev) if NG else None, prefix_len=_i32(pre, dev) if NG else None,
                scale=1.0 / math.sqrt(d), pre=pre, goff=goff, old=old, new=new,
                out=torch.zeros(T, Hq, d, dtype=dt, device=dev),
                lse=torch.zeros(T, Hq, dtype=torch.float32, device=dev))


_PREPARE = dict(pages=_prep_pages, rope=_prep_rope, append=_prep_append, attn=_prep_attn)


def _attach(st):
    """What a user of the library keeps beside the inputs: for attention, the
    step's plan (shared by all layers) and the workspace."""
    from long_prefix_attention_b200 import ops
    st["ops"] = ops
    c = st["case"]
    st["layout"] = ops.ASM_ROPE_HALF if c.get("layout") == "half" else ops.ASM_ROPE_PAIRS
    if c["op"] == "attn":
        T = st["q"].shape[0]
        NG = c["groups"]
        st["plan"] = ops.alloc_workspace(ops.asm_shared_plan_size(c["rows"], NG, T, c["hq"], c["hkv"]), "cuda",
                                         zero=False)
        st["ws"] = ops.alloc_workspace(ops.asm_shared_attention_workspace_size(T, c["hq"], c["hkv"], c["d"]), "cuda")
        ops.asm_shared_plan(st["q_off"], st["seq_len"], st["table"], T, c["hq"], c["hkv"], c["page"], st["plan"],
                            group_off=st["group_off"], prefix_len=st["prefix_len"], prefix_table=st["ptable"])


# -------------------------------------------------------------------- run --

def run(st):
    return _RUN[st["case"]["op"], own](st)


def _own_pages(st):
    st["ops"].asm_page_step(st["kv_len"], st["new_len"], st["pool"], st["pool_state"], st["case"]["page"], st["table"],
                            st["seq_len"], st["q_off"], st["row"], st["pos"], st["slot"], st["pool_out"],
                            pos_base=st["pos_base"])
    return [st[k] for k in ("table", "pool", "seq_len", "q_off", "row", "pos", "slot", "pool_out")]


def _plain_pages(st):
    kv, new = st["kv_len"].long(), st["new_len"].long()
    ps, dev = st["case"]["page"], kv.device
    table, pool = st["table"], st["pool"]
    (R, MP), T, F = table.shape, st["row"].shape[0], pool.shape[0]
    head, count = st["pool_state"][0].long(), st["pool_state"][1].long()
    n = new.clamp(min=0)
    off = torch.cumsum(n, 0)
    held = (kv + ps - 1) // ps
    fits = (off <= T) & (kv + n <= MP * ps)
    need = torch.where(fits, (kv + n + ps - 1) // ps - held, 0)
    incl = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (incl <= count))
    give = torch.where(ok, need, 0)
    base = torch.cumsum(give, 0)                         # granted pages end here (rows granted in order)
    seq = torch.where(new < 0, 0, torch.where(ok, kv + n, kv))
    back = torch.where(new < 0, held, 0)
    bend = torch.cumsum(back, 0)
    # new table entries
    j = torch.arange(MP, device=dev)[None]
    rel = j - held[:, None]
    hit = (rel >= 0) & (rel < give[:, None])
    take = (head + (base - give)[:, None] + rel) % F
    table.copy_(torch.where(hit, pool[take], table))
    # pages of ended rows, in row order, behind the free ones
    hit = j < back[:, None]
    put = (head + count + (bend - back)[:, None] + j) % F
    pool[put[hit]] = table[hit]
    # the tokens' rows, positions and slots
    t = torch.arange(T, device=dev)
    row = torch.searchsorted(off, t, right=True)
    real = row < R
    r = row.clamp(max=R - 1)
    i = kv[r] + t - (off - n)[r]
    page = table[r, (i // ps).clamp(max=MP - 1)].long()
    good = real & ok[r]
    slot = torch.where(good, page * ps + i % ps, -1)
    pos = torch.where(real, st["pos_base"].long()[r] + i, 0)
    q_off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), off]).clamp(max=T)
    refused = (~ok & (n > 0)).sum()
    out = torch.stack([(head + base[-1]) % F, count - base[-1] + bend[-1], refused])
    return [table, pool] + [x.to(torch.int32) for x in (seq, q_off, torch.where(real, row, -1), pos, slot, out)]


def _rotate(x, cos, sin, rot, layout):
    """x [T, H, d] in the arithmetic type, cos and sin [T, 1, rot / 2]."""
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _cos_sin(st):
    ang = st["pos"].double()[:, None, None] * st["freq"]
    c, s = torch.cos(ang) * st["mscale"], torch.sin(ang) * st["mscale"]
    return c.float(), (-s if st["case"].get("inverse") else s).float()


def _plain_rope(st):
    c = st["case"]
    cos, sin = _cos_sin(st)
    st["y"].copy_(_rotate(st["x"].float(), cos, sin, c["rot"], c["layout"]))
    return st["y"]


def _own_rope(st):
    c = st["case"]
    st["ops"].asm_rope(st["x"], st["pos"], st["freq"], st["y"], layout=st["layout"], mscale=st["mscale"],
                       inverse=c["inverse"])
    return st["y"]


def _plain_append(st):
    c, ps = st["case"], st["case"]["page"]
    cos, sin = _cos_sin(st)
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, c["rot"], c["layout"]))
    k = _rotate(st["k"].float(), cos, sin, c["rot"], c["layout"]).to(st["k"].dtype)
    keep = torch.nonzero(st["slot"] >= 0)[:, 0]
    s = st["slot"][keep].long()
    st["k_pages"][s // ps, :, s % ps] = k[keep]
    st["v_pages"][s // ps, :, s % ps] = st["v"][keep]
    return [st["q_out"], st["k_pages"], st["v_pages"]]


def _own_append(st):
    st["ops"].asm_rope_append(st["q"], st["k"], st["v"], st["pos"], st["slot"], st["freq"], st["q_out"],
                              st["k_pages"], st["v_pages"], layout=st["layout"], mscale=st["mscale"])
    return [st["q_out"], st["k_pages"], st["v_pages"]]


def _span(pages, ids, n):
    """The first n tokens of the listed pages: [Hkv, n, d] in 32 bits."""
    x = pages[ids.long()]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n].float()


def _plain_attn(st):
    """Row by row scores over the local pages, group by group over the prefix
    (its keys gathered once for all rows), joined by the softmax statistics."""
    c, ps = st["case"], st["case"]["page"]
    Hq, Hkv, d = c["hq"], c["hkv"], c["d"]
    G = Hq // Hkv
    T = st["q"].shape[0]
    q = (st["q"].float() * st["scale"]).view(T, Hkv, G, d).transpose(0, 1)         # [Hkv, T, G, d]
    m = torch.full((2, Hkv, T, G), -math.inf, device=q.device)
    z = torch.zeros(2, Hkv, T, G, device=q.device)
    o = torch.zeros(2, Hkv, T, G, d, device=q.device)

    def part(w, a, b, k, v, bar):
        s = torch.matmul(q[:, a:b].reshape(Hkv, (b - a) * G, d), k.transpose(1, 2))
        if bar is not None:
            s = s.masked_fill(bar, -math.inf)
        mx = s.amax(2)
        p = torch.exp(s - mx[..., None])
        m[w, :, a:b], z[w, :, a:b] = mx.view(Hkv, b - a, G), p.sum(2).view(Hkv, b - a, G)
        o[w, :, a:b] = torch.matmul(p, v).view(Hkv, b - a, G, d)

    starts = np.concatenate([[0], np.cumsum(st["new"])]).tolist()
    for j, n in enumerate(st["pre"]):
        a, b = starts[st["goff"][j]], starts[st["goff"][j + 1]]
        if b > a and n > 0:
            ids = st["ptable"][j, :_cdiv(n, ps)]
            k, v = _span(st["k_pages"], ids, n), _span(st["v_pages"], ids, n)
            step = max(1, (1 << 28) // (Hq * n))
            for x in range(a, b, step):
                part(0, x, min(b, x + step), k, v, None)
    for r, (old, new) in enumerate(zip(st["old"], st["new"])):
        a, n = starts[r], old + new
        ids = st["table"][r, :_cdiv(n, ps)]
        bar = None
        if new > 1:
            seen = old + torch.arange(new, device=q.device).repeat_interleave(G)
            bar = torch.arange(n, device=q.device)[None] > seen[:, None]
        part(1, a, a + new, _span(st["k_pages"], ids, n), _span(st["v_pages"], ids, n), bar)
    mm = torch.maximum(m[0], m[1])
    w = torch.exp(m - mm)
    zz = w[0] * z[0] + w[1] * z[1]
    res = (w[0][..., None] * o[0] + w[1][..., None] * o[1]) / zz[..., None]
    st["out"].copy_(res.transpose(0, 1).reshape(T, Hq, d))
    st["lse"].copy_((mm + torch.log(zz)).transpose(0, 1).reshape(T, Hq))
    return [st["out"], st["lse"]]


def _own_attn(st):
    st["ops"].asm_shared_attention(st["q"], st["k_pages"], st["v_pages"], st["table"], st["plan"], st["scale"],
                                   st["out"], st["ws"], prefix_table=st["ptable"], lse_out=st["lse"])
    return [st["out"], st["lse"]]


_RUN = {("pages", False): _plain_pages, ("pages", True): _own_pages, ("rope", False): _plain_rope,
        ("rope", True): _own_rope, ("append", False): _plain_append, ("append", True): _own_append,
        ("attn", False): _plain_attn, ("attn", True): _own_attn}


# ------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "pages":
        kv, new, held, free = _page_lens(case)
        need = sum(_cdiv(k + n, case["page"]) - _cdiv(k, case["page"]) for k, n in zip(kv, new) if n > 0)
        back = sum(_cdiv(k, case["page"]) for k, n in zip(kv, new) if n < 0)
        taken = min(need, free)
        # lengths and bases in, lengths and offsets out, three words a token, one read and one write a moved page
        return dict(bytes=4 * (5 * case["rows"] + 3 * case["tokens"] + 2 * (taken + back) + 8),
                    flops=case["rows"] * 8 + case["tokens"] * 4)
    es = _ES[case["dt"]]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["d"]
        return dict(bytes=2 * n * es + 4 * case["tokens"] + 4 * case["rot"],
                    flops=3 * case["tokens"] * case["heads"] * case["rot"])
    if op == "append":
        n = case["tokens"] * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return dict(bytes=2 * n * es + 8 * case["tokens"] + 4 * case["rot"],
                    flops=3 * case["tokens"] * (case["hq"] + case["hkv"]) * case["rot"])
    pre, goff, old, new = _attn_lens(case)
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    tok = starts[-1]
    keys = sum(n for j, n in enumerate(pre) if goff[j + 1] > goff[j]) + sum(old) + tok
    pairs = sum(n * (starts[goff[j + 1]] - starts[goff[j]]) for j, n in enumerate(pre))
    pairs += sum(o * n + n * (n + 1) // 2 for o, n in zip(old, new))
    return dict(bytes=2 * keys * case["hkv"] * case["d"] * es + tok * case["hq"] * (2 * case["d"] * es + 4),
                flops=4 * pairs * case["hq"] * case["d"])


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](case, st)


def _exact_pages(case, st):
    """One row after another, as a host allocator would."""
    kv, new, base = (st[k].tolist() for k in ("kv_len", "new_len", "pos_base"))
    table, pool = st["table"].cpu().numpy().copy(), st["pool"].cpu().numpy().copy()
    head, count, _ = st["pool_state"].tolist()
    (R, MP), T, F, ps = table.shape, case["tokens"], len(pool), case["page"]
    row, pos, slot = np.full(T, -1, np.int32), np.zeros(T, np.int32), np.full(T, -1, np.int32)
    q_off, seq = [0], []
    taken, asked, refused, returned, at = 0, 0, 0, [], 0
    for r in range(R):
        if new[r] < 0:
            returned += table[r, :_cdiv(kv[r], ps)].tolist()
            seq.append(0)
            q_off.append(min(at, T))
            continue
        end = at + new[r]
        held, want = _cdiv(kv[r], ps), _cdiv(kv[r] + new[r], ps)
        ok = end <= T and want <= MP
        if ok:
            asked += want - held
            ok = want == held or asked <= count
        if ok:
            for p in range(held, want):
                table[r, p] = pool[(head + taken) % F]
                taken += 1
        elif new[r] > 0:
            refused += 1
        seq.append(kv[r] + new[r] if ok else kv[r])
        for i in range(new[r]):
            if at + i < T:
                x = kv[r] + i
                row[at + i], pos[at + i] = r, base[r] + x
                if ok:
                    slot[at + i] = table[r, x // ps] * ps + x % ps
        at = end
        q_off.append(min(at, T))
    for i, p in enumerate(returned):
        pool[(head + count + i) % F] = p
    res = [table, pool, seq, q_off, row, pos, slot, [(head + taken) % F, count - taken + len(returned), refused]]
    dev = st["table"].device
    return [_i32(x, dev) for x in res]


def _exact_turn(x, st):
    """Complex rotation of every pair, 64 bits."""
    c = st["case"]
    rot = c["rot"]
    sign = -1.0 if c.get("inverse") else 1.0
    ang = st["pos"].double()[:, None, None] * st["freq"] * sign
    w = torch.polar(torch.full_like(ang, st["mscale"]), ang)
    x = x.double()
    if c["layout"] == "half":
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * w
        body = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * w
        body = torch.view_as_real(z).flatten(-2)
    return torch.cat([body, x[..., rot:]], -1)


def _exact_rope(case, st):
    return _exact_turn(st["x"], st)


def _exact_append(case, st):
    ps = case["page"]
    k, v = _exact_turn(st["k"], st), st["v"].double()
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    slot = st["slot"].long()
    keep = slot >= 0
    s = slot[keep]
    kp[s // ps, :, s % ps] = k[keep]
    vp[s // ps, :, s % ps] = v[keep]
    return [_exact_turn(st["q"], st), kp, vp]


def _exact_attn(case, st):
    """Every token of every row over its whole key list, one softmax, 64 bits."""
    G, ps = case["hq"] // case["hkv"], case["page"]
    pre, goff, old, new = st["pre"], st["goff"], st["old"], st["new"]
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r in range(case["rows"]):
        j = next((x for x in range(len(pre)) if goff[x] <= r < goff[x + 1]), None)
        n, np_ = old[r] + new[r], pre[j] if j is not None else 0
        at_key = torch.arange(n, device="cuda")
        where_l = st["table"][r].long()[at_key // ps], at_key % ps
        if j is not None:
            at_pre = torch.arange(np_, device="cuda")
            where_p = st["ptable"][j].long()[at_pre // ps], at_pre % ps
        for h in range(case["hkv"]):
            k, v = st["k_pages"][:, h], st["v_pages"][:, h]
            ks, vs = k[where_l], v[where_l]
            if j is not None:
                ks, vs = torch.cat([k[where_p], ks]), torch.cat([v[where_p], vs])
            ks, vs = ks.double(), vs.double()
            qs = st["q"][at:at + new[r], h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,kd->tgk", qs, ks) * st["scale"]
            seen = np_ + old[r] + torch.arange(new[r], device="cuda")
            s.masked_fill_((torch.arange(np_ + n, device="cuda")[None] > seen[:, None])[:, None], -math.inf)
            zz = torch.logsumexp(s, 2)
            lse[at:at + new[r], h * G:(h + 1) * G] = zz
            out[at:at + new[r], h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", torch.exp(s - zz[..., None]), vs)
        at += new[r]
    return [out, lse]


_EXACT = dict(pages=_exact_pages, rope=_exact_rope, append=_exact_append, attn=_exact_attn)
