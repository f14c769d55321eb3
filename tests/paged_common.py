"""Plain 64-bit forms of the paged serving calls, and the error bounds the
tests hold the kernels to.

Bounds count roundings: a value rounded to t is off by at most u(t) =
finfo(t).eps / 2 relative to itself.
"""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def cdiv(a, b):
    return -(-a // b)


def page_step(kv, new, base, table, pool, head, count, S, T):
    """One row after another, as a host allocator would (numpy, in place on
    table and pool).  Returns seq_len, q_off, row, pos, slot, pool_out."""
    (R, MP), F = table.shape, len(pool)
    row, pos, slot = np.full(T, -1), np.zeros(T, int), np.full(T, -1)
    q_off, seq, back = [0], [], []
    taken = asked = refused = at = 0
    for r in range(R):
        k = min(max(int(kv[r]), 0), MP * S)
        if new[r] < 0:
            back += [int(x) for x in table[r, :cdiv(k, S)]]
            seq.append(0)
            q_off.append(min(at, T))
            continue
        n = int(new[r])
        end, held, want = at + n, cdiv(k, S), cdiv(k + n, S)
        ok = end <= T and k + n <= MP * S
        if ok:
            asked += want - held
            ok = want == held or asked <= count
        if ok:
            for p in range(held, want):
                table[r, p] = pool[(head + taken) % F]
                taken += 1
        elif n:
            refused += 1
        seq.append(k + n if ok else k)
        for i in range(min(n, max(T - at, 0))):
            x = k + i
            row[at + i], pos[at + i] = r, x + (0 if base is None else int(base[r]))
            if ok:
                slot[at + i] = table[r, x // S] * S + x % S
        at = end
        q_off.append(min(at, T))
    back = back[:F - count]
    for i, p in enumerate(back):
        pool[(head + count + i) % F] = p
    return (np.array(seq), np.array(q_off), row, pos, slot,
            np.array([(head + taken) % F, count - taken + len(back), refused]))


def freqs(rot, theta, scaling="none", factor=1.0, lo=1.0, hi=4.0, ctx=8192.0):
    """Angle per position, pair by pair in Python floats."""
    out = []
    for i in range(rot // 2):
        th = theta * factor ** (rot / (rot - 2 if rot > 2 else 1)) if scaling == "base" else theta
        f = th ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            w = min(1.0, max(0.0, (ctx * f / (2 * math.pi) - lo) / (hi - lo)))
            f = w * f + (1 - w) * f / factor
        elif scaling == "yarn":
            def at(turns):
                return rot * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(at(hi)), 0), min(math.ceil(at(lo)), rot - 1)
            w = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f = w * f / factor + (1 - w) * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, pos, freq, layout, mscale=1.0, inverse=False):
    """x [T, H, d] fp64; layout 0 half, 1 pairs."""
    rot = 2 * len(freq)
    ang = pos.double()[:, None, None] * freq
    c, s = torch.cos(ang) * mscale, torch.sin(ang) * (-mscale if inverse else mscale)
    y = x.clone()
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., i], x[..., j]
    y[..., i] = a * c - b * s
    y[..., j] = b * c + a * s
    return y


def rope_bound(x, pos, freq, layout, mscale, dtype, ref):
    """Two products of one rounding each and their sum (3 u32), the sine (2^-21
    absolute by the hardware for bf16 storage, 2^-23 by sincospi), the angle's
    2^-32 turns and the frequency's 2^-53 p f -- each times |a| + |b| of the
    pair -- and the result's one rounding."""
    rot = 2 * len(freq)
    xa = x.double().abs()
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    ang = pos.double().abs()[:, None, None] * freq.abs()
    e = 3 * 2.0 ** -24 + (2.0 ** -21 if dtype == torch.bfloat16 else 2.0 ** -23) + 2 * math.pi * 2.0 ** -32 + \
        2.0 ** -51 * ang
    s = (xa[..., i] + xa[..., j]) * e * abs(mscale)
    out = torch.zeros_like(xa)
    out[..., i], out[..., j] = s, s
    return out + U[dtype] * ref.abs() + 1e-37


def attention(q, kp, vp, table, q_off, seq, scale, group_off=None, pre_len=None, ptable=None):
    """Token by token and KV head by KV head over the whole key list, fp64 on
    the CPU.  Returns out, lse (NaN where no row has the token), and for the
    bounds a = sum_j softmax_j |v_j| and dot = max_j scale sum_i |q_i k_ji|."""
    T, Hq, d = q.shape
    _, Hkv, S, _ = kp.shape
    G = Hq // Hkv
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    a, dot = torch.zeros_like(out), torch.zeros_like(lse)
    cnt = torch.zeros(T, dtype=torch.long)
    NG = 0 if group_off is None else len(group_off) - 1

    def span(ids, n):
        x = torch.arange(n)
        pg = torch.as_tensor([int(v) for v in ids])[x // S] if n else torch.zeros(0, dtype=torch.long)
        return kp[pg, :, x % S].double(), vp[pg, :, x % S].double()       # [n, Hkv, d]

    for r in range(len(seq)):
        j = next((g for g in range(NG) if group_off[g] <= r < group_off[g + 1]), None)
        K, V = span(table[r], int(seq[r]))
        if j is not None:
            pk, pv = span(ptable[j], int(pre_len[j]))
        n = int(q_off[r + 1]) - int(q_off[r])
        for i in range(n):
            t, see = int(q_off[r]) + i, min(max(int(seq[r]) - n + i + 1, 0), int(seq[r]))
            k, v = K[:see], V[:see]
            if j is not None:
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            cnt[t] = k.shape[0]
            if k.shape[0] == 0:
                out[t], lse[t] = 0.0, -math.inf
                continue
            qq = q[t].double().view(Hkv, G, d)
            s = torch.einsum("hgd,khd->hgk", qq, k) * scale
            lse[t] = torch.logsumexp(s, 2).reshape(Hq)
            p = torch.exp(s - torch.logsumexp(s, 2, keepdim=True))
            out[t] = torch.einsum("hgk,khd->hgd", p, v).reshape(Hq, d)
            a[t] = torch.einsum("hgk,khd->hgd", p, v.abs()).reshape(Hq, d)
            dot[t] = (torch.einsum("hgd,khd->hgk", qq.abs(), k.abs()) * scale).amax(2).reshape(Hq)
    return out, lse, a, dot, cnt


def attention_bounds(ref, lse, a, dot, cnt, d, dtype):
    """A logit is a sum of d products in fp32 (2 u32 a term, the tensor cores
    may truncate) and one scaling: e = (2 d + 4) u32 dot; its exponential adds
    4 u32 |its argument| (at most 2 dot + |lse|) and 2^-20.  The sums of n weights
    and products add n u32 (the longest chain of additions), the joins 8 u32.
    bf16 storage rounds each weight of the products once more (u_bf16 a).
    The result is rounded once."""
    u = U[torch.float32]
    w = (2 * d + 4) * u * dot + 4 * u * (2 * dot + lse.nan_to_num(0, 0, 0).abs()) + 2.0 ** -20
    acc = (cnt.double() * u + 8 * u)[:, None]
    e_lse = w + acc + 4 * u * lse.nan_to_num(0, 0, 0).abs()
    e_out = a * (2 * w + 2 * acc + (U[torch.bfloat16] if dtype == torch.bfloat16 else 0.0))[..., None] + \
        U[dtype] * ref.abs()
    return e_out + 1e-30, e_lse
