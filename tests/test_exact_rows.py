"""The bound of tests/exact_rows.py refuses gradients whose D comes from out rounded to bf16 (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests import exact_rows as er


def inputs(T, d, seed):
    return er.near((1, T), 2, 1, d, seed)


def dq_from(q, k, v, do, rounded):
    """dq with ds rounded to bf16, D from out rounded to bf16 or from the weights, the rest in fp64."""
    r = oa.prompt(q, k, v, dout=do)
    q, k, v, do = (oa.f64(x)[0] for x in (q, k, v, do))
    T, Hq, d = q.shape
    bf = lambda x: torch.from_numpy(x).bfloat16().double().numpy()
    dq = np.zeros_like(q)
    for h in range(Hq):
        s = q[:, h] @ k[:, 0].T * d ** -0.5
        s[np.triu(np.ones((T, T), bool), 1)] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        o = p @ v[:, 0]
        D = (do[:, h] * (bf(o) if rounded else o)).sum(-1, keepdims=True)
        dq[:, h] = bf(p * (do[:, h] @ v[:, 0].T - D)) @ k[:, 0] * d ** -0.5
    return bf(dq)[None], r


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 3, 8, 40, 200])
def test_bound(T, d):
    data = inputs(T, d, T)
    for rounded in (False, True):
        dq, r = dq_from(*data, rounded)
        over = np.abs(dq - r["dq"]) / er.backward(r, d, T, 2)[0]
        assert (over.max() > 1) == rounded, over.max()
