"""Attention over an e4m3 paged cache with block scales of every size that the
interface allows, in each of the kernels: few rows of a key head, one tile of
128 rows, several of them.

Bounds.  x is a score in log2 with its values' scale added, P = 2^(x - m + 6)
rounded to fp16: by 2^-11 of it, and by 2^-25 where it is below 2^-14.  The
largest P is 2^-2 at least (m is raised once some x exceeds it by 8), so the
second adds up to n 2^-23 of the largest |V| over n keys.  A score's fp32 dot
product is off by some 2^-22 of |q| |k|; O by twice that factor.  O's own
rounding comes on top, and where the outputs are fp16 their subnormal half step.
"""
import math

import numpy as np
import pytest
import torch

import ops_ref as R
import test_kv8 as K8

pytestmark = pytest.mark.gpu

# query rows of a key head: the kernel for few, one tile of the other, several items of it
SQ = {"few": 3, "one tile": 30, "many": 150}
D = 128


def draw(rows, lens=(384, 200), seed=9, block=16, spread=0.0):
    return K8.draw((2, 4, 2, SQ[rows], D, 64, 6, block, "bf16", True, lens), seed=seed, spread=spread, nan=False)


def check(st, scale=1 / math.sqrt(D), floor=0.0, rounded=0.0, causal=True):
    o, lse = K8.call(st, causal, scale)
    o, lse = R.f64(o), R.f64(lse)
    ro, rl = R.attend_paged(R.f64(st["q"]), R.f64(st["kp"]), R.f64(st["vp"]), R.f64(st["ks"]), R.f64(st["vs"]),
                            st["lens"].numpy(), st["table"].numpy(), causal, scale)
    assert not np.isnan(o).any() and not np.isnan(lse).any()
    dead = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), dead) and (lse[dead] < 0).all() and (o[dead] == 0).all()
    q, n = R.f64(st["q"]), int(st["lens"].max())
    group = q.shape[1] // st["kp"].shape[2]
    err = np.zeros(q.shape[:3])
    vmax = np.zeros(q.shape[:3])
    for e in range(q.shape[0]):
        pages = st["table"][e].numpy()
        pages = pages[(pages >= 0) & (pages < st["kp"].shape[0])]
        for h in range(q.shape[1]):
            ks, vs = (R.f64(st[x])[pages, h // group].max(initial=0.0) for x in ("ks", "vs"))
            err[e, h] = (2.0 ** -22 + rounded) * abs(scale) * np.linalg.norm(q[e, h], axis=-1) * ks * 448 * math.sqrt(D)
            vmax[e, h] = vs * np.abs(R.f64(st["vp"])[pages, :, h // group]).max(initial=0.0)
    off = np.abs(lse[~dead] - rl[~dead])
    assert (off <= err[~dead] + 2.0 ** -20 * (1 + np.abs(rl[~dead]))).all(), off.max()
    bound = R.HALF_STEP[torch.bfloat16] * np.abs(ro) + ((2.0 ** -11 + rounded + n * 2.0 ** -23 + 2 * err) * vmax)[..., None] + floor
    assert (np.abs(o - ro) <= bound).all(), (np.abs(o - ro) - bound).max()
    # and as a whole the roundings of P are independent: O is as good as its own type
    for e in range(q.shape[0]):
        for h in range(q.shape[1]):
            assert np.linalg.norm((o - ro)[e, h]) <= 2 ** -7 * np.linalg.norm(ro[e, h]) + floor * math.sqrt(o[e, h].size)
    return o, lse


# what V's products lose below 2^-24 of the scale that they enter with, which is 2^-64 at least, times 448 / 2
LOST = 2.0 ** (-64 - 25 + 9)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("vs", [2.0 ** -127, 2.0 ** -130, 2.0 ** -149, 2.0 ** -126 / 448, 2.0 ** -100, 2.0 ** -70])
def test_values_of_tiny_scales_among_others(rows, vs):
    """One tile of 128 tokens of them, between tiles of ordinary scales."""
    st = draw(rows)
    for e in range(2):
        st["vs"][st["table"][e, 2:4].long()] = float(np.float32(vs))
    check(st, floor=LOST)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("vs", [2.0 ** -130, 2.0 ** -126, 2.0 ** -90, 2.0 ** -60, 2.0 ** -30])
def test_all_values_of_small_scales(rows, vs):
    st = draw(rows)
    st["vs"][:] = float(np.float32(vs))
    check(st, floor=LOST)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("vs", [2.0 ** 60, 2.0 ** 119, 2.0 ** 126 * 1.5, 2.0 ** 127])
def test_all_values_of_large_scales(rows, vs):
    """Values of 1 at most, so that their products with the scale are finite."""
    st = draw(rows)
    st["vp"] = (st["vp"].float() / 448).to(torch.float8_e4m3fn)
    st["vs"][:] = float(np.float32(vs))
    check(st)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("ks", [2.0 ** -140, 2.0 ** -126, 2.0 ** -60])
def test_keys_of_tiny_scales(rows, ks):
    """Scores of (almost) nothing: the mean of the values."""
    st = draw(rows)
    st["ks"][:] = float(np.float32(ks))
    check(st)
    st = draw(rows)
    for e in range(2):
        st["ks"][st["table"][e, 2:4].long()] = float(np.float32(ks))
    check(st)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("vs", [2.0 ** -64, 2.0 ** -31, 1.0, 2.0 ** 90])
def test_lse_does_not_depend_on_the_values_scale(rows, vs):
    """Scores of 0: the LSE of n keys is log n.  Up to 512 of them: log2 n is
    below 9, so its half step is 2^-21 at most, the mantissa's logarithm is off
    by 2^-24, the product with ln 2 by 2^-22, and each of the sum's parts by
    2^-23 of itself: below 2^-20 together."""
    st = draw(rows)
    st["ks"][:] = 0.0
    st["vs"][:] = vs
    _, lse = K8.call(st, True)
    for e, n in enumerate(st["lens"].tolist()):
        seen = n - SQ[rows] + 1 + np.arange(SQ[rows])
        assert (np.abs(R.f64(lse)[e] - np.log(np.maximum(seen, 1)))[:, seen > 0] <= 2.0 ** -20).all()


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("vs", [2.0 ** -64, 2.0 ** -40, 2.0 ** -25, 1.0, 2.0 ** 60, 2.0 ** 119])
@pytest.mark.parametrize("zeros", [[0], [3], [5], [2, 3], [0, 1, 4, 5]], ids=str)
def test_zeros_among_values_of_one_scale(rows, vs, zeros):
    """Pages whose blocks have a V scale of 0: keys with a weight, and no
    value.  Two pages of 64 tokens are a whole tile of 128."""
    st = draw(rows)
    st["vp"] = (st["vp"].float() / 448).to(torch.float8_e4m3fn)
    st["vs"][:] = vs
    for e in range(2):
        st["vs"][st["table"][e, zeros].long()] = 0.0
    check(st)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("vs", [2.0 ** -64, 2.0 ** -40, 2.0 ** -25, 1.0, 2.0 ** 60])
def test_pages_outside_the_pool_among_values_of_one_scale(rows, vs):
    st = draw(rows)
    st["vs"][:] = vs
    st["ks"] *= 2.0 ** -20
    st["q"] *= 2.0 ** 10
    st["table"][0, 1], st["table"][0, 2], st["table"][0, 3] = -1, 10 ** 6, -(2 ** 31)
    st["table"][1, 0] = 2 ** 31 - 1
    check(st)


@pytest.mark.parametrize("rows", SQ)
def test_nothing_but_zeros(rows):
    """O is 0 and the LSE what the scores say."""
    st = draw(rows)
    st["vs"][:] = 0.0
    o, _ = check(st)
    assert (o == 0).all()
    st = draw(rows)
    st["table"][:] = -1
    o, lse = check(st)
    assert (o == 0).all()
    seen = 200 - SQ[rows] + 1 + np.arange(SQ[rows])
    assert np.abs(lse[1] - np.log(np.maximum(seen, 1)))[:, seen > 0].max() < 1e-5


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("gap", [-60.0, -20.0, 20.0, 60.0])
def test_zeros_whose_scores_are_far_from_the_others(rows, gap):
    """Keys of zero values that outweigh the others by 2^gap, or the reverse."""
    st = draw(rows)
    st["vs"][:] = 2.0 ** -20
    st["q"] = torch.ones_like(st["q"])
    kp = st["kp"].float() * 2.0 ** -8
    st["ks"][:] = 1.0
    for e in range(2):
        far = st["table"][e, 2:4].long()
        kp[far] = math.copysign(1.0, gap)
        st["ks"][far] = 2.0 ** -7 * abs(gap) * math.log(2)
        st["vs"][far] = 0.0
    st["kp"] = kp.to(torch.float8_e4m3fn)
    check(st, scale=1.0)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("low", [-100, -64, -36, 0])
def test_scales_of_values_as_far_apart_as_they_may_be(rows, low):
    """2^96 between one page's values and the next one's, two pages' and the
    next two's: the keys of the small ones keep their weights.  (2^-100 counts as 2^-64.)"""
    for step in (1, 2):
        st = draw(rows)
        st["vp"] = (st["vp"].float() / 448).to(torch.float8_e4m3fn)
        for e in range(2):
            for i in range(6):
                st["vs"][int(st["table"][e, i])] = 2.0 ** (max(low, -64) + 96 if i // step % 2 else low)
        check(st, floor=LOST)


@pytest.mark.parametrize("rows", SQ)
def test_a_scale_of_minus_zero_is_a_scale_of_zero(rows):
    st = draw(rows)
    st["vs"][:, :, 1] = 0.0
    st["ks"][:, :, 2] = 0.0
    want = K8.call(st, True)
    st["vs"][:, :, 1] = -0.0
    st["ks"][:, :, 2] = -0.0
    got = K8.call(st, True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
