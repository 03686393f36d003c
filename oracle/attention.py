"""Softmax attention of a hybrid model's attention layers in fp64 (numpy), from the definitions:
causal attention over whole prompts and its gradients, the paged cache's plan, its 8-bit encoding
(e4m3 with one power-of-two scale per page and head) and one-token attention over it.

Plain and slow; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_FLOOR = -60


def f64(x):
    if hasattr(x, "detach"):
        import torch
        x = x.detach().to("cpu", torch.float64).numpy()
    return np.asarray(x, dtype=np.float64)


def sequences(lead, cu):
    """[(first token, last token + 1)] over the flattened token axis."""
    if cu is None:
        B, T = lead
        return [(b * T, (b + 1) * T) for b in range(B)]
    cu = [int(c) for c in cu]
    return list(zip(cu[:-1], cu[1:]))


def prompt(q, k, v, cu=None, scale=None, dout=None):
    """Causal attention: dict with out, lse and, where dout is given, dq, dk, dv; and the sums of
    magnitudes that rounding bounds need: pv = sum p |v|, s_abs = the largest scale sum |q| |k|, and
    with dout p_do = sum p |dout| and, per query (_k) and per key (_q), scale sum x |k| or scale sum
    x |q| for x = |ds| (ds), x = p sum |dout| |v| (dov) and x = p sum |dout| pv (dpv)."""
    q, k, v = f64(q), f64(k), f64(v)
    lead, (Hq, d), Hk = q.shape[:-2], q.shape[-2:], k.shape[-2]
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else float(scale)
    n = int(np.prod(lead))
    q2, k2, v2 = q.reshape(n, Hq, d), k.reshape(n, Hk, d), v.reshape(n, Hk, d)
    r = {x: np.zeros((n, Hq, d)) for x in ("out", "pv")}
    r["lse"] = np.zeros((n, Hq))
    s_abs = 0.0
    top = lambda x: float(np.abs(np.nan_to_num(x)).max(initial=0.0))
    longest = max([b - a for a, b in sequences(lead, cu)])
    r["amp"] = G * longest * top(v2)
    if dout is not None:
        r["amp"] += G * longest * (1 + 2 * scale * max(top(q2), top(k2)) * d * top(v2)) * top(f64(dout))
        do2 = f64(dout).reshape(n, Hq, d)
        r |= {x: np.zeros((n, Hq, d)) for x in ("dq", "ds_k", "dov_k", "dpv_k")}
        r |= {x: np.zeros((n, Hk, d)) for x in ("dk", "dv", "p_do", "ds_q", "dov_q", "dpv_q")}
    for a, b in sequences(lead, cu):
        if b <= a:
            continue
        dead = np.triu(np.ones((b - a, b - a), bool), 1)
        for h in range(Hq):
            g = h // G
            s = scale * q2[a:b, h] @ k2[a:b, g].T
            s_abs = max(s_abs, float((scale * np.abs(q2[a:b, h]) @ np.abs(k2[a:b, g]).T).max()))
            s[dead] = -np.inf
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(-1, keepdims=True)
            p = e / z
            o = p @ v2[a:b, g]
            r["out"][a:b, h], r["lse"][a:b, h] = o, (m + np.log(z))[:, 0]
            r["pv"][a:b, h] = p @ np.abs(v2[a:b, g])
            if dout is None:
                continue
            do = do2[a:b, h]
            ds = p * (do @ v2[a:b, g].T - (do * o).sum(-1, keepdims=True))
            r["dq"][a:b, h] = scale * ds @ k2[a:b, g]
            r["dk"][a:b, g] += scale * ds.T @ q2[a:b, h]
            r["dv"][a:b, g] += p.T @ do
            r["p_do"][a:b, g] += p.T @ np.abs(do)
            sums = dict(ds=np.abs(ds), dov=p * (np.abs(do) @ np.abs(v2[a:b, g]).T),
                        dpv=p * (np.abs(do) * r["pv"][a:b, h]).sum(-1, keepdims=True))
            for x, y in sums.items():
                r[x + "_k"][a:b, h] = scale * y @ np.abs(k2[a:b, g])
                r[x + "_q"][a:b, g] += scale * y.T @ np.abs(q2[a:b, h])
    for x in [x for x in r if x != "amp"]:
        r[x] = r[x].reshape(*lead, *r[x].shape[1:])
    r["s_abs"] = s_abs
    return r


def plan(lens, added, table, free_list, free_head, page, rows):
    """The plan of one step as lists, request by request; the table is copied."""
    lens, added = [int(x) for x in lens], [int(x) for x in added]
    table = np.array(table, dtype=np.int64, copy=True)
    free = [int(x) for x in free_list]
    N, width = table.shape
    none = dict(cu_seqlens=[0] * (N + 1), slots=[-1] * rows, positions=[-1] * rows, lens=list(lens),
                free_head=int(free_head), table=table)
    if not 0 <= free_head <= len(free):
        return none | dict(status=[4, 0])
    for r in range(N):
        if lens[r] < 0 or added[r] < 0 or lens[r] + added[r] > width * page:
            return none | dict(status=[2, r])
    total = sum(added)
    if total > rows:
        return none | dict(status=[3, total - rows])
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, added))
    if need > len(free) - free_head:
        return none | dict(status=[1, need - (len(free) - free_head)])
    head, cu, slots, positions = int(free_head), [0], [], []
    for r in range(N):
        for pos in range(lens[r], lens[r] + added[r]):
            if pos % page == 0:
                table[r, pos // page] = free[head]
                head += 1
            slots.append(int(table[r, pos // page]) * page + pos % page)
            positions.append(pos)
        cu.append(len(slots))
    pad = [-1] * (rows - total)
    return dict(cu_seqlens=cu, slots=slots + pad, positions=positions + pad,
                lens=[a + b for a, b in zip(lens, added)], free_head=head, table=table, status=[0, 0])


def decode_e4m3(b):
    """The value of each e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities."""
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x = np.where((e == 15) & (m == 7), np.nan, x)
    return np.where(b & 128, -x, x)


_TABLE = decode_e4m3(np.arange(127))  # 0 .. 448, ascending


def encode_e4m3(x):
    """Nearest e4m3 byte, ties to the even mantissa, magnitudes above 448 (infinity too) to 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_TABLE, a), 1, 126)
    lo = hi - 1
    below, above = a - _TABLE[lo], _TABLE[hi] - a
    pick = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    pick = np.where(np.isnan(x), 127, pick)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_of(amax):
    """The least 2^e, e >= -60, with amax <= 448 2^e (infinity as the largest fp32)."""
    amax = min(float(amax), float(np.finfo(np.float32).max))
    e = SCALE_FLOOR
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, slots, cache, scale):
    """New rows x [rows, Hk, d] into cache bytes [P, Hk, page, d] and scale [P, Hk] (copied)."""
    x, cache, scale = f64(x), np.array(cache, copy=True), f64(scale).copy()
    page = cache.shape[2]
    slots = [int(s) for s in slots]
    t = 0
    while t < len(slots):
        if not 0 <= slots[t] < cache.shape[0] * page:
            t += 1
            continue
        u = t + 1
        while u < len(slots) and slots[u] == slots[u - 1] + 1 and slots[u] % page:
            u += 1
        pg, off = divmod(slots[t], page)
        for h in range(x.shape[1]):
            top = np.abs(x[t:u, h])
            new = scale_of(np.max(np.where(np.isnan(top), 0.0, top)))
            if off:
                old, new = scale[pg, h], max(new, scale[pg, h])
                if new != old:
                    cache[pg, h, :off] = encode_e4m3(decode_e4m3(cache[pg, h, :off]) * (old / new))
            cache[pg, h, off:off + u - t] = encode_e4m3(x[t:u, h] / new)
            scale[pg, h] = new
        t = u
    return cache, scale


def decode(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale=None):
    """One-token attention; also sum p |v| per output and the largest scale sum |q| |k|."""
    q, ks, vs = f64(q), f64(k_scale), f64(v_scale)
    N, Hq, d = q.shape
    P, Hk, page, _ = k_cache.shape
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else float(scale)
    out, pv, s_abs = np.zeros((N, Hq, d)), np.zeros((N, Hq, d)), 0.0
    for n in range(N):
        L = max(0, min(int(lens[n]), table.shape[1] * page))
        at = [(int(table[n, j // page]), j % page) for j in range(L)]
        at = [(p, o) for p, o in at if 0 <= p < P]
        if not at:
            continue
        pg, of = (np.array(z) for z in zip(*at))
        for h in range(Hk):
            K = decode_e4m3(k_cache[pg, h, of]) * ks[pg, h][:, None]
            V = decode_e4m3(v_cache[pg, h, of]) * vs[pg, h][:, None]
            for g in range(h * G, (h + 1) * G):
                s = scale * K @ q[n, g]
                s_abs = max(s_abs, float((scale * np.abs(K) @ np.abs(q[n, g])).max()))
                e = np.exp(s - s.max())
                p = e / e.sum()
                out[n, g], pv[n, g] = p @ V, p @ np.abs(V)
    return out, pv, s_abs
