"""One-token attention's softmax weights: contexts in which most of the weight lies on a token that has little or
nothing to say, and pages whose value scales lie far apart, within bounds of each request and head
(tests/decode_bounds.py)."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests import decode_bounds as db

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check(q, kc, vc, ks, vs, table, lens, dtype, scale=None):
    import linear_attention_sequence_rule_b200 as gdn
    q = q.to(DT[dtype])
    N, Hq, d = q.shape
    dev = [torch.from_numpy(c).cuda() for c in (kc, vc)]
    sc = [torch.from_numpy(np.asarray(s)).float().cuda() for s in (ks, vs)]
    out = gdn.attn_decode(q.cuda(), *dev, *sc, i32(table), i32(lens), scale=scale)
    gdn.device_status()
    ws = gdn.gdn_attn_decode_workspace_bytes(N, Hq, kc.shape[1], d, kc.shape[2], table.shape[1], gdn._DT[DT[dtype]])
    db.compare(out, q, kc, vc, ks, vs, table, lens, dtype, db.chain(lens, N, Hq, d, ws), scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [0, 10, 14, 18, 22, 26, 32, 45])
def test_sink_in_front_of_a_long_context(gap, dtype):
    q, *cache, table = db.sink([8192], 0, gap, 1, 2, 64, 64, 1, dtype)
    check(q, *cache, table, [8192], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,G", [(64, 16, 3), (128, 32, 9), (128, 128, 1), (128, 64, 17)])
@pytest.mark.parametrize("at", [0, 77, -1])
def test_sink_anywhere(at, d, page, G, dtype):
    lens = [900, 131, 78, 1500]
    q, *cache, table = db.sink(lens, at, 23, 1, G, d, page, 2, dtype)
    check(q, *cache, table, lens, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sinks_of_contexts_that_are_not_split(dtype):
    import linear_attention_sequence_rule_b200 as gdn
    n, Hk = 70, 8
    lens = [int(x) for x in np.random.RandomState(3).randint(1, 260, n)]
    q, *cache, table = db.sink(lens, 0, 24, Hk, 1, 64, 64, 3, dtype)
    assert gdn.gdn_attn_decode_workspace_bytes(n, Hk, Hk, 64, 64, table.shape[1], gdn._DT[DT[dtype]]) == 0
    check(q, *cache, table, lens, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("far", [8, 16, 24])
def test_one_page_of_large_values(far, dtype):
    """A page whose scale is 2^far of the others' for the sake of one channel, in which the others are 0."""
    d, page, L = 64, 16, 600
    r = np.random.RandomState(far)
    P = -(-L // page)
    x, y = r.randn(L, 1, d) * 0.3, r.randn(L, 1, d)
    y[160:176, :, :-1], y[160:176, :, -1] = 0.0, 2.0 ** far
    empty = np.zeros((P, 1, page, d), np.uint8)
    kc, ks = oa.append(x, np.arange(L), empty, np.zeros((P, 1)))
    vc, vs = oa.append(y, np.arange(L), empty, np.zeros((P, 1)))
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(4)).to(DT[dtype])
    check(q, kc, vc, ks, vs, np.arange(P)[None], [L], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_page_of_zeros_beside_others(dtype):
    """Values of 0 have the least scale, 2^-60: their tokens still carry their weight in the sum."""
    d, page, L = 64, 32, 320
    r = np.random.RandomState(5)
    P = L // page
    x, y = r.randn(L, 1, d) * 0.3, r.randn(L, 1, d)
    y[64:128] = 0.0
    empty = np.zeros((P, 1, page, d), np.uint8)
    kc, ks = oa.append(x, np.arange(L), empty, np.zeros((P, 1)))
    vc, vs = oa.append(y, np.arange(L), empty, np.zeros((P, 1)))
    assert (vs[2:4] == 2.0 ** -60).all()
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(6)).to(DT[dtype])
    check(q, kc, vc, ks, vs, np.arange(P)[None], [L], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32), (128, 128)])
def test_few_tokens(d, page, dtype):
    """Contexts short enough that a bound sees the second half of an fp32 call's weights."""
    lens = [1, 2, 3, 5, 8, 13, 16, 17, 21, 32, 33, 40]
    q, *cache, table = db.sink(lens, 0, 2, 2, 3, d, page, 7, dtype)
    check(q, *cache, table, lens, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 7, 8, 9, 16, 17, 40])
def test_shared_heads(G, dtype):
    lens, page, d = [70, 333], 64, 128
    r = np.random.RandomState(G)
    P = 9
    table = r.permutation(P)[:8].reshape(2, 4)
    table = np.concatenate([table, np.full((2, 2), -1)], 1)
    lens[1] = 250
    cache = []
    for _ in range(2):
        c = r.randint(0, 127, (P, 2, page, d)) | (r.randint(0, 2, (P, 2, page, d)) << 7)
        cache.append((c.astype(np.uint8), 2.0 ** r.randint(-9, -5, (P, 2))))
    q = torch.randn(2, 2 * G, d, generator=torch.Generator().manual_seed(G)).to(DT[dtype])
    (kc, ks), (vc, vs) = cache
    check(q, kc, vc, ks, vs, table, lens, dtype, scale=0.01)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_frames_rise_and_fall(dtype):
    """Exponents that rise and fall over the context by fractions of a power of two, below and above 0."""
    d, page, L = 64, 32, 700
    r = np.random.RandomState(8)
    P = -(-L // page)
    y = r.randn(L, 1, d) * 2.0 ** r.randint(-3, 3, (L, 1, 1))
    q = torch.ones(1, 2, d) * torch.tensor([1.0, -1.0]).view(1, 2, 1)
    x = np.zeros((L, 1, d))
    x[:, 0, :4] = (np.linspace(-6, 6, L) + 0.3 * r.randn(L))[:, None]
    empty = np.zeros((P, 1, page, d), np.uint8)
    kc, ks = oa.append(x, np.arange(L), empty, np.zeros((P, 1)))
    vc, vs = oa.append(y, np.arange(L), empty, np.zeros((P, 1)))
    check(q, kc, vc, ks, vs, np.arange(P)[None], [L], dtype, scale=1.0)
