"""One-token attention over the 8-bit cache, per (request, head, element): the definition in fp64 with the sums that
a bound on the kernel's rounding needs, that bound, and the rounding of its weights by itself.

In the kernel's frame the weight of token j is y_j = exp2(log2(e) s_j + log2 vs_j - M), M the least whole number at or
above the largest exponent: out = sum y_j V8_j / sum (y_j / vs_j).  Products take 2^15 y_j, rounded to fp16 (bf16 calls)
or to a sum of two fp16 (fp32 calls): off by 2^-11 (2^-22) of itself, and by 2^-25 where it falls below fp16's
normal numbers.  The largest 2^15 y_j is at least 2^14, so that floor is 2^-39 of the largest weight, and no
weight is off by more than itself.
"""
import numpy as np

from oracle import attention as oa
from tests import attn_bounds as ab

FRAME = 15
FLOOR = 2.0 ** -25 / 2.0 ** (FRAME - 1)


def sums(q, kc, vc, ks, vs, table, lens, scale=None):
    """[(n, h, dict of arrays)] for every query head of a request with tokens."""
    q, ks, vs = oa.f64(q), oa.f64(ks), oa.f64(vs)
    N, Hq, d = q.shape
    P, Hk, page, _ = kc.shape
    scale = d ** -0.5 if scale is None else float(scale)
    for n in range(N):
        L = max(0, min(int(lens[n]), table.shape[1] * page))
        j = np.arange(L)
        pg, of = np.asarray(table)[n][j // page], j % page
        on = (pg >= 0) & (pg < P)
        pg, of = pg[on], of[on]
        if not len(pg):
            continue
        for h in range(Hq):
            g = h // (Hq // Hk)
            K = oa.decode_e4m3(kc[pg, g, of]) * ks[pg, g][:, None]
            s = scale * K @ q[n, h]
            yield n, h, dict(s=s, V8=oa.decode_e4m3(vc[pg, g, of]), vs=vs[pg, g],
                             s_abs=scale * np.abs(K) @ np.abs(q[n, h]),
                             q_abs=scale * np.abs(K).sum(1) * np.abs(q[n, h]).max())


def softmax(x):
    e = np.exp(x["s"] - x["s"].max())
    return e / e.sum()


def bound(x, dtype, d, chain):
    """(result, bound) of one head; chain: tokens that one warp adds up."""
    p, V8, vs = softmax(x), np.abs(x["V8"]), x["vs"]
    out = p @ (x["V8"] * vs[:, None])
    z = p * vs
    top = z.max()
    # a score: products of d terms, each addition with at least single precision; q to 2^-22 (fp32 calls), and to
    # 2^-33 of the head's largest; four factors and the shifts by log2 vs and M; exp2 to 2^-22
    lg = np.abs(np.log2(vs))
    far = np.log2(np.maximum(z / top, 2.0 ** -200))
    part = 2.0 ** -22 if dtype == "f32" else 0.0
    e = (x["s_abs"] * (d * 2.0 ** -23 + 4 * 2.0 ** -24 + part) + 2.0 ** -33 * x["q_abs"]
         + np.log(2) * 2.0 ** -24 * (3 * lg + np.abs(far) + FRAME + 1) + 2.0 ** -22)
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    pv = z @ V8
    floor = np.minimum(FLOOR * top, z) @ V8
    # products are added up a token at a time at worst, the sum eight tokens apart; then four warps and the splits
    add = chain * 2.0 ** -23 + (chain / 8 + 64) * 2.0 ** -24
    err = (z * (e + w)) @ V8 + pv * (p @ e) + floor + add * pv
    return out, 1.02 * (ab.U[dtype] * np.abs(out) + err) + 1e-37


def rounded(x, parts, frame=FRAME):
    """The result with weights rounded as the kernel rounds them, all else in fp64 (frame None: the largest weight at 1)."""
    t = x["s"] * np.log2(np.e) + np.log2(x["vs"])
    y = np.exp2(t - t.max()) if frame is None else np.exp2(t - np.ceil(t.max()) + frame)
    w = y.astype(np.float16).astype(np.float64)
    if parts == 2:
        w += (y - w).astype(np.float16).astype(np.float64)
    return (w @ x["V8"]) / (y / x["vs"]).sum()


def chain(lens, N, Hq, d, workspace):
    """Tokens a warp adds up: every fourth tile of 32 of a split."""
    splits = max(1, workspace // (N * Hq * (d + 4) * 4))
    per = -(-(-(-int(max(lens)) // 32)) // splits)
    return 32 * -(-per // 4)


def compare(got, q, kc, vc, ks, vs, table, lens, dtype, chain, scale=None):
    got, seen = oa.f64(got), np.zeros(q.shape[:2], bool)
    for n, h, x in sums(q, kc, vc, ks, vs, table, lens, scale):
        want, b = bound(x, dtype, q.shape[-1], chain)
        ab.check(f"request {n}, head {h}", got[n, h], want, b)
        seen[n, h] = True
    assert not got[~seen].any()


# ---- contexts ------------------------------------------------------------------------------------

def sink(lens, at, gap, Hk, G, d, page, seed, dtype):
    """Contexts whose token `at` has a score about `gap` powers of two above the others' and a value of 0."""
    import torch
    r = np.random.RandomState(seed)
    q = torch.from_numpy(r.randn(len(lens), Hk * G, d)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    q[:] = q[:, :1]  # every head of a request asks the same, so that one sink serves all
    table, used = np.full((len(lens), max(-(-int(x) // page) for x in lens) + 1), -1), 0
    x, y, slots = [], [], []
    for n, L in enumerate(lens):
        blocks = -(-int(L) // page)
        table[n, :blocks] = used + r.permutation(blocks)
        used += blocks
        k, v = r.randn(L, Hk, d) * 0.02, r.randn(L, Hk, d)
        i = at if at >= 0 else L + at
        q0 = q[n, 0].double().numpy()
        k[i], v[i] = q0 * gap * np.log(2) * d ** 0.5 / (q0 @ q0), 0.0
        x.append(k)
        y.append(v)
        j = np.arange(L)
        slots.append(table[n][j // page] * page + j % page)
    kc, vc = (np.zeros((used, Hk, page, d), np.uint8) for _ in range(2))
    slots = np.concatenate(slots)
    kc, ks = oa.append(np.concatenate(x), slots, kc, np.zeros((used, Hk)))
    vc, vs = oa.append(np.concatenate(y), slots, vc, np.zeros((used, Hk)))
    return q, kc, vc, ks, vs, table
