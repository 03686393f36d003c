"""Causal softmax attention over whole prompts and its gradients against the fp64 oracle, within bounds
that follow from the kernels' arithmetic (tests/attn_bounds.py)."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests import attn_bounds as ab

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def inputs(lead, Hq, Hk, d, dtype, seed, peak=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, s=1.0: (s * torch.randn(*lead, h, d, generator=g)).to(DT[dtype])
    return r(Hq, peak), r(Hk), r(Hk), r(Hq)


def cu_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)


def run(q, k, v, do, cu=None, scale=None):
    import linear_attention_sequence_rule_b200 as gdn
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    cud = None if cu is None else cu.cuda()
    out, lse = gdn.attn_fwd(qd, kd, vd, cu_seqlens=cud, scale=scale)
    grads = gdn.attn_bwd(qd, kd, vd, out, lse, dod, cu_seqlens=cud, scale=scale)
    gdn.device_status()
    return [oa.f64(x) for x in (out, lse, *grads)]


def compare(q, k, v, do, dtype, cu=None, scale=None, got=None, rows=slice(None)):
    got = run(q, k, v, do, cu, scale) if got is None else got
    r = oa.prompt(q[rows], k[rows], v[rows], cu=cu, scale=scale, dout=do[rows])
    n = max([b - a for a, b in oa.sequences(q.shape[:-2], cu)])
    d, G = q.shape[-1], q.shape[-2] // k.shape[-2]
    bo, bl = ab.forward(r, dtype, d, n)
    bounds = [bo, bl, *ab.backward(r, dtype, d, n, G)]
    for name, x, b in zip(("out", "lse", "dq", "dk", "dv"), got, bounds):
        ab.check(name, x[rows], r[name], b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 300, 513])
def test_dense_lengths(T, d, dtype):
    q, k, v, do = inputs((2, T), 2, 1, d, dtype, seed=T + d)
    compare(q, k, v, do, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (3, 1), (12, 4), (10, 2), (8, 1)])
def test_shared_heads(Hq, Hk, dtype):
    q, k, v, do = inputs((1, 190), Hq, Hk, 64, dtype, seed=Hq)
    compare(q, k, v, do, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [0, 1, 0, 2, 0], [129, 64, 1, 300, 0, 128, 5], [256, 256], [7] * 40,
                                     [640, 17, 383]])
def test_packed(lengths, d, dtype):
    q, k, v, do = inputs((sum(lengths),), 4, 2, d, dtype, seed=len(lengths) + d)
    compare(q, k, v, do, dtype, cu=cu_of(lengths))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B", [128, 129, 300, 1025, 2500])
def test_packed_many_sequences(B, dtype):
    lengths = np.random.RandomState(B).randint(0, 9, B)
    lengths[[1, B // 2, B - 2]] = [200, 333, 129]
    q, k, v, do = inputs((int(lengths.sum()) + 2,), 2, 1, 64, dtype, seed=B)
    n = int(lengths.sum())
    compare(q, k, v, do, dtype, cu=cu_of(lengths), rows=slice(0, n))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_calls_on_two_streams_at_once(dtype):
    import linear_attention_sequence_rule_b200 as gdn
    cases, alone = [], []
    for i, (lead, Hq, Hk, d) in enumerate([((2, 700), 6, 2, 64), ((1, 1100), 4, 1, 128)]):
        q, k, v, do = (x.cuda() for x in inputs(lead, Hq, Hk, d, dtype, seed=20 + i))
        out, lse = gdn.attn_fwd(q, k, v)
        cases.append((q, k, v, out, lse, do))
        alone.append((out, lse, *gdn.attn_bwd(*cases[-1])))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], []
    for _ in range(5):
        for c, w, st in zip(cases, alone, streams):
            got.append((w, (*gdn.attn_fwd(*c[:3], stream=st), *gdn.attn_bwd(*c, stream=st))))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, x in got for a, b in zip(w, x))
    gdn.device_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_peaked_softmax_and_scale(dtype):
    # scores of +-60 and more: the running maximum moves far, most weights underflow
    q, k, v, do = inputs((1, 400), 2, 2, 128, dtype, seed=3, peak=6.0)
    k[:, ::7] *= 4
    compare(q, k, v, do, dtype, scale=0.25)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rising_and_falling_scores(dtype):
    # each key scores above (below) all before it: every block moves (keeps) the maximum
    T, d = 700, 64
    q, k, v, do = inputs((2, T), 1, 1, d, dtype, seed=4)
    q[..., 0], k[..., 0] = 8.0, 0.0
    ramp = torch.arange(T, dtype=torch.float32) / 8
    k[0, :, 0, 0], k[1, :, 0, 0] = ramp.to(k.dtype), (-ramp).to(k.dtype)
    compare(q, k, v, do, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_prompt(dtype):
    q, k, v, do = inputs((1, 2500), 2, 1, 128, dtype, seed=5)
    compare(q, k, v, do, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_neighbours_and_rows_behind_stay_apart(dtype, d):
    """Sequences whose rows are NaN, and NaN rows behind the last sequence, reach no other sequence;
    rows behind the last one are not written."""
    import linear_attention_sequence_rule_b200 as gdn
    lengths, tail = [70, 33, 129, 5, 200], 37
    cu = cu_of(lengths)
    n = sum(lengths)
    q, k, v, do = inputs((n + tail,), 4, 2, d, dtype, seed=6)
    bad = [slice(70, 103), slice(232, 237), slice(n, n + tail)]
    for x in (q, k, v, do):
        for b in bad:
            x[b] = float("nan")
    dev = [x.cuda() for x in (q, k, v, do)]
    mark = lambda t: torch.full_like(t, 7.0)
    out, lse = mark(dev[0]), torch.full((n + tail, 4), 7.0, device="cuda")
    gdn.attn_fwd(*dev[:3], cu_seqlens=cu.cuda(), out=out, lse=lse)
    grads = [mark(dev[0]), mark(dev[1]), mark(dev[2])]
    gdn.attn_bwd(*dev[:3], out, lse, dev[3], cu_seqlens=cu.cuda(), dq=grads[0], dk=grads[1], dv=grads[2])
    gdn.device_status()
    for t in (out, lse, *grads):
        assert bool((t[n:] == 7.0).all())
    got = [oa.f64(x) for x in (out, lse, *grads)]
    at = 0
    for i, L in enumerate(lengths):
        if i not in (1, 3):
            rows = slice(at, at + L)
            compare(q, k, v, do, dtype, cu=torch.tensor([0, L]), got=got, rows=rows)
        at += L


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph(dtype):
    import linear_attention_sequence_rule_b200 as gdn
    lengths = [130, 0, 700, 64]
    q, k, v, do = (x.cuda() for x in inputs((sum(lengths),), 6, 2, 64, dtype, seed=8))
    cu = cu_of(lengths).cuda()
    out, lse = gdn.attn_fwd(q, k, v, cu_seqlens=cu)
    eager = (out, lse, *gdn.attn_bwd(q, k, v, out, lse, do, cu_seqlens=cu))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, l2 = gdn.attn_fwd(q, k, v, cu_seqlens=cu, stream=side)
    again = (o2, l2, *gdn.attn_bwd(q, k, v, o2, l2, do, cu_seqlens=cu, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, again))
    held = [torch.zeros_like(x) for x in eager]
    need = gdn.gdn_attn_bwd_workspace_bytes(4, q.shape[0], 6, 2, 64, 1, gdn._DT[q.dtype])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.attn_fwd(q, k, v, cu_seqlens=cu, out=held[0], lse=held[1])
        gdn.attn_bwd(q, k, v, held[0], held[1], do, cu_seqlens=cu, dq=held[2], dk=held[3], dv=held[4], workspace=ws)
    for _ in range(2):
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))
    gdn.device_status()


def test_results_for_a_given_stream_take_no_memory_that_another_still_writes():
    import linear_attention_sequence_rule_b200 as gdn
    q, k, v, do = (x.cuda() for x in inputs((1, 300), 4, 4, 64, "bf16", seed=12))
    out, lse = gdn.attn_fwd(q, k, v)
    want = (out, lse, *gdn.attn_bwd(q, k, v, out, lse, do))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(int(2e7))  # the writes of memory that is free again are still to come
    for x in want * 2:
        torch.full_like(x, 7.0)
    torch.empty(gdn.gdn_attn_bwd_workspace_bytes(1, 300, 4, 4, 64, 0, 0), dtype=torch.uint8, device="cuda").fill_(9)
    got = (*gdn.attn_fwd(q, k, v, stream=side), *gdn.attn_bwd(q, k, v, out, lse, do, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gradients_are_the_forwards_differences():
    """fp32: the directional derivative from attn_bwd against a central difference of attn_fwd."""
    import linear_attention_sequence_rule_b200 as gdn
    q, k, v, do = (x.cuda() for x in inputs((1, 150), 4, 2, 64, "f32", seed=9))
    out, lse = gdn.attn_fwd(q, k, v)
    grads = gdn.attn_bwd(q, k, v, out, lse, do)
    g = torch.Generator("cuda").manual_seed(10)
    h = 2.0 ** -7
    for i, x in enumerate((q, k, v)):
        dirn = torch.randn(x.shape, generator=g, device="cuda")
        move = lambda s: [y + s * dirn if j == i else y for j, y in enumerate((q, k, v))]
        f = lambda s: (gdn.attn_fwd(*move(s))[0].double() * do.double()).sum()
        diff, want = float(f(h) - f(-h)) / (2 * h), float((grads[i].double() * dirn.double()).sum())
        # truncation h^2 / 6 times a third derivative of order the sum's size; fp32 out rounding / h
        size = float((do.double().abs() * out.double().abs()).sum())
        assert abs(diff - want) <= size * (h * h + 2.0 ** -20 / h), (i, diff, want, size)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_pack_and_optional_results(dtype):
    import linear_attention_sequence_rule_b200 as gdn
    e = torch.empty(0, 2, 64, dtype=DT[dtype], device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = gdn.attn_fwd(e, e, e, cu_seqlens=cu)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    q, k, v, do = inputs((1, 80), 2, 2, 64, dtype, seed=11)
    dev = [x.cuda() for x in (q, k, v)]
    out = torch.empty_like(dev[0])
    rc = gdn.gdn_attn_fwd(*(x.data_ptr() for x in dev), out.data_ptr(), None, 1, 80, 2, 2, 64, None,
                          gdn._DT[DT[dtype]], 0.125, torch.cuda.current_stream().cuda_stream)
    assert rc == gdn.GDN_OK, gdn.gdn_last_error()
    assert torch.equal(out, gdn.attn_fwd(*dev)[0])
