"""Bounds on bf16 gradients of rows whose D_i is formed as sum_j p_ij (dout_i . v_j), the first 256 of a sequence: as
tests/attn_bounds.py, but without the rounding of out (and of the weights that made it) in D."""
import numpy as np
import torch

from tests import attn_bounds as ab


def backward(r, d, n, G):
    """Bounds on dq, dk, dv; n: keys that a row sees at most."""
    u = w = ab.U["bf16"]
    ep = 2 * ab.weight_error(r["s_abs"], d, n) + 2.0 ** -22 * (1 + np.abs(r["lse"]).max() + r["s_abs"])
    dd = ep + (n + 2 * d + 4) * 2.0 ** -24  # weights, products of d terms, the sum over the keys
    res = []
    for name, side, m in (("dq", "_k", n), ("dk", "_q", G * n)):
        res.append(u * np.abs(r[name]) + (w + m * 2.0 ** -24) * r["ds" + side]
                   + (ep + 2 * d * 2.0 ** -24) * r["dov" + side] + (ep + dd) * r["dpv" + side])
    dv = u * np.abs(r["dv"]) + (w + ep + G * n * 2.0 ** -24) * r["p_do"]
    return [1.02 * x + 2.0 ** -126 * r["amp"] for x in (*res, dv)]


def near(lead, Hq, Hk, d, seed):
    """Values that lie near one another and small scores: ds is small beside D, whose rounding then shows."""
    g = torch.Generator().manual_seed(seed)
    r = lambda h, s: s * torch.randn(*lead, h, d, generator=g)
    k0, v0 = torch.randn(d, generator=g), torch.randn(d, generator=g)
    return tuple(x.bfloat16() for x in (r(Hq, 0.02), k0 + r(Hk, 0.1), v0 + r(Hk, 0.004), r(Hq, 1.0)))
