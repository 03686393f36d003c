"""Pins of the attention oracle (oracle/attention.py): a hand-worked case, limits known in closed form,
gradients against central differences of the forward, the e4m3 code against its published corner
values and torch's conversion, and the cache's write against its own definition."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa


def rnd(shape, seed):
    return np.random.RandomState(seed).randn(*shape)


def test_two_tokens_by_hand():
    # one head, d = 1, scale 1: scores 0 | 0, ln 3
    q = np.array([[[[1.0]], [[1.0]]]])
    k = np.array([[[[0.0]], [[math.log(3.0)]]]])
    v = np.array([[[[4.0]], [[8.0]]]])
    r = oa.prompt(q, k, v, scale=1.0, dout=np.array([[[[1.0]], [[1.0]]]]))
    # row 0 sees token 0; row 1 has weights 1/4, 3/4: 1 + 6 = 7
    assert np.allclose(r["out"].ravel(), [4.0, 7.0], atol=1e-15)
    assert np.allclose(r["lse"].ravel(), [0.0, math.log(4.0)], atol=1e-15)
    # ds of row 1: 1/4 (4 - 7), 3/4 (8 - 7) = -3/4, 3/4
    assert np.allclose(r["dq"].ravel(), [0.0, 0.75 * math.log(3.0)], atol=1e-15)
    assert np.allclose(r["dk"].ravel(), [-0.75, 0.75], atol=1e-15)
    assert np.allclose(r["dv"].ravel(), [1.25, 0.75], atol=1e-15)


def test_equal_keys_average_and_heads_share():
    q, v = rnd((1, 5, 4, 3), 1), rnd((1, 5, 2, 3), 2)
    k = np.ones((1, 5, 2, 3))
    r = oa.prompt(q, k, v)
    for h in range(4):
        want = np.cumsum(v[0, :, h // 2], 0) / np.arange(1, 6)[:, None]
        assert np.allclose(r["out"][0, :, h], want, atol=1e-14)


def test_packed_is_each_sequence_alone():
    cu = [0, 3, 3, 4, 9]
    q, k, v, do = rnd((9, 4, 5), 3), rnd((9, 2, 5), 4), rnd((9, 2, 5), 5), rnd((9, 4, 5), 6)
    r = oa.prompt(q, k, v, cu=cu, dout=do)
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        one = oa.prompt(q[None, a:b], k[None, a:b], v[None, a:b], dout=do[None, a:b])
        for x in ("out", "lse", "dq", "dk", "dv"):
            assert np.allclose(r[x][a:b], one[x][0], atol=1e-14)


def test_gradients_are_the_forwards_differences():
    cu = [0, 4, 7]
    x = dict(q=rnd((7, 4, 3), 7), k=rnd((7, 2, 3), 8), v=rnd((7, 2, 3), 9))
    do = rnd((7, 4, 3), 10)
    r = oa.prompt(**x, cu=cu, scale=0.7, dout=do)
    h = 1e-6
    for name, got in (("q", r["dq"]), ("k", r["dk"]), ("v", r["dv"])):
        for at in np.ndindex(*x[name].shape):
            y = {z: w.copy() for z, w in x.items()}
            y[name][at] += h
            up = (oa.prompt(**y, cu=cu, scale=0.7)["out"] * do).sum()
            y[name][at] -= 2 * h
            down = (oa.prompt(**y, cu=cu, scale=0.7)["out"] * do).sum()
            assert abs((up - down) / (2 * h) - got[at]) < 1e-7


def test_e4m3_code():
    assert oa.decode_e4m3(0x7e) == 448.0 and oa.decode_e4m3(0x38) == 1.0 and oa.decode_e4m3(0x01) == 2.0 ** -9
    assert np.isnan(oa.decode_e4m3(0x7f)) and oa.decode_e4m3(0x80) == 0.0 and oa.decode_e4m3(0x08) == 2.0 ** -6
    every = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    want = every.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oa.decode_e4m3(every.numpy()), want, equal_nan=True)
    x = np.concatenate([rnd((4000,), 11) * 100, rnd((4000,), 12) * 1e-2, want[np.isfinite(want)]])
    mid = np.sort(want[np.isfinite(want)])
    x = np.clip(np.concatenate([x, (mid[1:] + mid[:-1]) / 2]), -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oa.decode_e4m3(oa.encode_e4m3(x)), oa.decode_e4m3(got))
    assert oa.encode_e4m3(np.inf) == 0x7e and oa.encode_e4m3(-np.inf) == 0xfe and oa.encode_e4m3(np.nan) & 0x7f == 0x7f


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.1, 1), (224.0, -1), (0.0, -60), (1e-30, -60), (1.0, -8),
                                    (1.75, -8), (1.7500001, -7), (float("inf"), 120)])
def test_scale_is_the_least_power_of_two(amax, e):
    assert oa.scale_of(amax) == 2.0 ** e


def test_append_keeps_what_is_held_and_grows_the_scale():
    x = rnd((6, 1, 4), 13)
    x[3:] *= 100
    cache, scale = np.zeros((3, 1, 4, 4), np.uint8), np.full((3, 1), 7.0)
    c1, s1 = oa.append(x[:3], [4, 5, 6], cache, scale)           # page 1, offsets 0..2
    c2, s2 = oa.append(x[3:], [7, 0, -1], c1, s1)                # page 1's last token, page 0's first
    assert s1[1, 0] < s2[1, 0] and s2[2, 0] == 7.0
    for t, (pg, of) in enumerate([(1, 0), (1, 1), (1, 2), (1, 3), (0, 0)]):
        got = oa.decode_e4m3(c2[pg, 0, of]) * s2[pg, 0]
        # half a step of e4m3 (2^-4 relative), twice for a row rounded twice, and half the least step
        assert np.all(np.abs(got - x[t, 0]) <= 2 * 2.0 ** -4 * np.abs(x[t, 0]) + 2.0 ** -10 * s2[pg, 0])


def test_plan_takes_pages_in_order_and_refuses_whole():
    table = np.array([[9, -1, -1], [8, -1, -1], [-1, -1, -1]])
    r = oa.plan([3, 4, 0], [2, 1, 5], table, [20, 21, 22, 23, 24], 1, 4, 10)
    assert r["status"] == [0, 0] and r["cu_seqlens"] == [0, 2, 3, 8] and r["free_head"] == 5
    assert r["table"].tolist() == [[9, 21, -1], [8, 22, -1], [23, 24, -1]]
    assert r["slots"] == [39, 84, 88, 92, 93, 94, 95, 96, -1, -1] and r["positions"][:3] == [3, 4, 4]
    assert oa.plan([3, 4, 0], [2, 1, 5], table, [20, 21, 22, 23], 1, 4, 10)["status"] == [1, 1]
    assert oa.plan([3, 4, 0], [2, 9, 5], table, [20] * 9, 1, 4, 99)["status"] == [2, 1]
    assert oa.plan([3, 4, 0], [2, 1, 5], table, [20] * 9, 1, 4, 7)["status"] == [3, 1]
    assert oa.plan([3, 4, 0], [2, 1, 5], table, [20] * 9, 10, 4, 10)["status"] == [4, 0]


def test_decode_is_the_prompts_last_row():
    page, lens = 4, [6, 0, 1]
    k, v = rnd((3, 8, 2, 5), 14), rnd((3, 8, 2, 5), 15)
    kc, ks = np.zeros((7, 2, page, 5), np.uint8), np.ones((7, 2))
    vc, vs = kc.copy(), ks.copy()
    table = np.array([[3, 1], [-1, -1], [6, -1]])
    for n in range(3):
        slots = [int(table[n, j // page]) * page + j % page for j in range(lens[n])]
        kc, ks = oa.append(k[n, :lens[n]], slots, kc, ks)
        vc, vs = oa.append(v[n, :lens[n]], slots, vc, vs)
    q = rnd((3, 4, 5), 16)
    out, _, _ = oa.decode(q, kc, vc, ks, vs, table, lens)
    assert not out[1].any()
    for n in (0, 2):
        at = [(int(table[n, j // page]), j % page) for j in range(lens[n])]
        K = np.array([oa.decode_e4m3(kc[p, :, o]) * ks[p][:, None] for p, o in at])
        V = np.array([oa.decode_e4m3(vc[p, :, o]) * vs[p][:, None] for p, o in at])
        full = oa.prompt(np.repeat(q[n][None, None], lens[n], 1), K[None], V[None])["out"][0, -1]
        assert np.allclose(out[n], full, atol=1e-13)
