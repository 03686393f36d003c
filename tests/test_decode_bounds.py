"""The bound on one-token attention (tests/decode_bounds.py) accepts weights rounded as the kernel documents it and
refuses coarser ones: a largest weight of 1, and one fp16 in place of two (CPU only)."""
import numpy as np
import pytest

from tests import decode_bounds as db


def over(data, dtype, parts, frame, chain=32, scale=None):
    """The largest error of a result with so rounded weights, in bounds."""
    worst = 0.0
    for _, _, x in db.sums(*data, scale=scale):
        want, b = db.bound(x, dtype, data[0].shape[-1], chain)
        worst = max(worst, float((np.abs(db.rounded(x, parts, frame) - want) / b).max()))
    return worst


def data(lens, at, gap, dtype, seed=1, page=16, d=64):
    q, kc, vc, ks, vs, table = db.sink(lens, at, gap, 1, 1, d, page, seed, dtype)
    return q, kc, vc, ks, vs, table, lens


@pytest.mark.parametrize("dtype,parts", [("bf16", 1), ("f32", 2)])
@pytest.mark.parametrize("gap", [0, 8, 14, 18, 22, 26, 34, 45])
def test_the_frame_holds_what_stands_beside_a_sink(gap, dtype, parts):
    assert over(data([4000], 0, gap, dtype), dtype, parts, db.FRAME, chain=1024) <= 1


@pytest.mark.parametrize("gap", [22, 24, 26, 30])
def test_a_largest_weight_of_one_does_not(gap):
    assert over(data([4000], 0, gap, "f32"), "f32", 2, None, chain=1024) > 1
    if gap >= 26:
        assert over(data([4000], 0, gap, "bf16"), "bf16", 1, None, chain=1024) > 1


@pytest.mark.parametrize("seed", range(3))
def test_one_half_in_place_of_two_is_too_coarse_for_fp32(seed):
    d = data([2, 5, 9, 17, 33], 0, 2, "f32", seed=seed)
    assert over(d, "f32", 2, db.FRAME) <= 1
    assert over(d, "f32", 1, db.FRAME) > 1
