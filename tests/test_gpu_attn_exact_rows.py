"""bf16 gradients of the first 256 rows of a sequence, within the bounds of a D that the rounding of out does not touch
(tests/exact_rows.py)."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests import attn_bounds as ab
from tests import exact_rows as er

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def inputs(lead, Hq, Hk, d, seed, kind):
    if kind == "near":
        return er.near(lead, Hq, Hk, d, seed)
    g = torch.Generator().manual_seed(seed)
    r = lambda h: torch.randn(*lead, h, d, generator=g).bfloat16()
    return r(Hq), r(Hk), r(Hk), r(Hq)


def grads(q, k, v, do, cu=None):
    import linear_attention_sequence_rule_b200 as gdn
    dev = [x.cuda() for x in (q, k, v, do)]
    cud = None if cu is None else cu.cuda()
    out, lse = gdn.attn_fwd(*dev[:3], cu_seqlens=cud)
    got = gdn.attn_bwd(*dev[:3], out, lse, dev[3], cu_seqlens=cud)
    gdn.device_status()
    return [oa.f64(x) for x in got]


@pytest.mark.parametrize("kind", ["near", "any"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 64, 129, 200, 256])
def test_sequences_of_such_rows_alone(T, d, kind):
    q, k, v, do = inputs((3, T), 4, 2, d, T + d, kind)
    r = oa.prompt(q, k, v, dout=do)
    for name, x, b in zip(("dq", "dk", "dv"), grads(q, k, v, do), er.backward(r, d, T, 2)):
        ab.check(name, x, r[name], b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[300, 1, 700], [257, 1000, 2]])
def test_the_first_rows_of_longer_sequences(lengths, d):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    q, k, v, do = inputs((sum(lengths),), 2, 1, d, 7, "near")
    dq = grads(q, k, v, do, cu)[0]
    for a, L in zip(cu.tolist(), lengths):
        for n in (1, 2, 4, 16, 64, 256):  # dq of a row needs no row behind it
            n = min(n, L)
            rows = slice(a, a + n)
            r = oa.prompt(q[rows], k[rows], v[rows], cu=[0, n], dout=do[rows])
            ab.check("dq", dq[rows], r["dq"], er.backward(r, d, n, 2)[0])
