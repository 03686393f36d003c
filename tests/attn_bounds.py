"""Element-wise bounds on the rounding error of the attention kernels, from the arithmetic they document.

u: half a step of the result's type.  r: rounding of the softmax weights (and of ds) for the products
they enter, half a bf16 step in bf16 calls, none in fp32 calls.  A score is a sum of d exact products
in fp32: off by at most d 2^-24 sum |q| |k| scale, and a few roundings of its size more for the scaling
and the shift by the maximum; exp2 is off by 2^-22; a sum of n positive terms in fp32 by n 2^-24.
Second-order terms: 2 %.

exp2 gives 0 below 2^-126 (the smallest normal number): a weight may be off by that much whatever its
size, which a result sees times what stands beside the weight, summed over the weights (amp).
"""
import numpy as np

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def weight_error(s_abs, d, n):
    """Relative error of a softmax weight before it is rounded for a product."""
    return (2 * (d + 8) * s_abs + 2 * n) * 2.0 ** -24 + 2.0 ** -21


def forward(r, dtype, d, n):
    """(bound on out, bound on lse); n: the longest sequence."""
    u, w = U[dtype], U["bf16"] if dtype == "bf16" else 0.0
    e = weight_error(r["s_abs"], d, n)
    out = u * np.abs(r["out"]) + (w + e + n * 2.0 ** -24) * r["pv"]
    return 1.02 * out + 2.0 ** -126 * r["amp"], e + 2.0 ** -22 * (1 + np.abs(r["lse"]))


def backward(r, dtype, d, n, G):
    """Bounds on dq, dk, dv, computed from the kernel's own out and lse."""
    u, w = U[dtype], U["bf16"] if dtype == "bf16" else 0.0
    e = weight_error(r["s_abs"], d, n)
    # a weight from lse: both its score and lse are off
    ep = 2 * e + 2.0 ** -22 * (1 + np.abs(r["lse"]).max() + r["s_abs"])
    # D_i = dout . out: out is off by its rounding and by the forward's bound, both below pv
    dd = u + w + e + (n + 2 * d) * 2.0 ** -24
    res = []
    for name, side, m in (("dq", "_k", n), ("dk", "_q", G * n)):
        acc = m * 2.0 ** -24
        res.append(u * np.abs(r[name]) + (w + acc) * r["ds" + side] + (ep + 2 * d * 2.0 ** -24) * r["dov" + side]
                   + (ep + dd) * r["dpv" + side])
    dv = u * np.abs(r["dv"]) + (w + ep + G * n * 2.0 ** -24) * r["p_do"]
    return [1.02 * x + 2.0 ** -126 * r["amp"] for x in (*res, dv)]


def decode(out, pv, s_abs, dtype, d, n):
    """Bound on one-token attention over the cache: weights rounded to fp16 (2^-11) in bf16 calls, to the
    sum of two fp16 (2^-22, and 2^-25 of the largest weight) in fp32 calls; q in fp32 calls to the sum
    of two fp16 (2^-22); a weight below 2^-14 of the largest has an absolute error of 2^-25 of it."""
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    q = 0.0 if dtype == "bf16" else 2.0 ** -22 * s_abs
    e = weight_error(s_abs, d, n) + 2 * q
    return 1.02 * (U[dtype] * np.abs(out) + (w + e + n * 2.0 ** -24) * pv) + 1e-37


def check(name, got, want, bound):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    over = np.abs(got - want) / bound
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[at] <= 1, f"{name}: {over[at]:.2f} of its bound at {at}: {got[at]} for {want[at]}"
