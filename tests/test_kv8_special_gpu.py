"""Attention over an e4m3 paged cache: special inputs in each of its kernels
(few rows of a key head, one tile of 128 rows, several items of 256), with the
bounds of test_kv8_scales_gpu."""
import math

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
import ops_ref as R
import test_kv8 as K8
from test_kv8_scales_gpu import D, SQ, check, draw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("scale", [-0.3, -1e-3, 0.0, 2.0, 1e-30])
def test_scales_of_the_scores(rows, scale):
    check(draw(rows, seed=5), scale)


@pytest.mark.parametrize("rows", SQ)
@pytest.mark.parametrize("causal", [True, False])
def test_block_scales_within_fifteen_binary_orders_of_the_largest(rows, causal):
    """Powers of two, block by block: in every kernel keys and values are exact."""
    st = draw(rows, seed=6)
    g = torch.Generator().manual_seed(3)
    for name, top in (("ks", -5), ("vs", 0)):
        st[name] = torch.exp2(torch.randint(top - 15, top + 1, st[name].shape, generator=g).float())
    check(st, causal=causal)


@pytest.mark.parametrize("rows", SQ)
def test_block_scales_from_tiny_to_huge_and_zero(rows):
    """Beyond that the kernel for many rows loses what is below 2^-25 of a
    tile's largest scale: nothing beside the row's largest value."""
    st = draw(rows, seed=9)
    g = torch.Generator().manual_seed(1)
    st["vs"] = torch.exp2(torch.randint(-40, 40, st["vs"].shape, generator=g).float())
    st["ks"] = torch.exp2(torch.randint(-30, -4, st["ks"].shape, generator=g).float())
    st["vs"][:, :, 1] = 0.0
    st["ks"][:, :, 2] = 0.0
    o, lse = K8.call(st, True)
    (ro, rl), _, _ = K8.reference(st, True, 1 / math.sqrt(D))
    # sums over 80 binary orders: each row by its own size.  Keys lose at most 2^-25 of the largest scale 2^-5, against
    # 128 values of q: a score moves by 2^-29.  Values: P's 2^-11, what is lost below 2^-25 of a tile's largest scale
    # (whose weight may be small) and bf16's 2^-8.
    row = np.abs(ro).max(-1, keepdims=True)
    assert (np.abs(R.f64(o) - ro) <= row * 2.0 ** -7).all()
    assert np.abs(R.f64(lse) - rl)[np.isfinite(rl)].max() <= 2.0 ** -16


@pytest.mark.parametrize("rows", SQ)
def test_scales_that_are_no_powers_of_two(rows):
    """In the kernel for many rows a value is rounded twice, with its ratio to
    the tile's largest scale and in the product: by 2^-10 at most."""
    st = draw(rows, seed=21, spread=1.0)
    g = torch.Generator().manual_seed(2)
    for n in ("ks", "vs"):
        st[n] = st[n] * (torch.rand(st[n].shape, generator=g) * 0.5 + 0.5)
    st["ks"] /= st["ks"].max() * 32  # scores of an ordinary size
    check(st, rounded=0.0 if rows == "few" else 2.0 ** -10)


@pytest.mark.parametrize("rows", SQ)
def test_rows_of_queries_far_apart_in_size(rows):
    """bf16 queries from 2^-130 to 2^30 in one batch, and within a row; an
    infinity or a NaN stays in its row."""
    st = K8.draw((1, 8, 2, SQ[rows], D, 64, 4, 16, "bf16", True, (250,)), seed=31, spread=0.0, nan=False)
    st["ks"] *= 2.0 ** -6
    st["q"][0, 0] *= 2.0 ** -30
    st["q"][0, 1] = 0
    st["q"][0, 2, :, 0] *= 2.0 ** -20
    st["q"][0, 3] = st["q"][0, 3] * 2.0 ** -130
    st["q"][0, 4, ::2] *= 2.0 ** 12
    check(st)
    clean, clean_lse = K8.call(st, True)
    last = SQ[rows] - 1
    st["q"][0, 5, 0, 3], st["q"][0, 6, 1, 3], st["q"][0, 7, last, 9] = float("inf"), float("nan"), -float("inf")
    o, lse = K8.call(st, True)
    bad = torch.zeros((8, SQ[rows]), dtype=torch.bool)
    bad[5, 0] = bad[6, 1] = bad[7, last] = True
    assert o[0][bad].isnan().all() and lse[0, 6, 1].isnan()
    assert torch.equal(o[0][~bad], clean[0][~bad]) and torch.equal(lse[0][~bad], clean_lse[0][~bad])


@pytest.mark.parametrize("rows", SQ)
def test_fp16_queries_of_the_largest_and_smallest_sizes(rows):
    st = K8.draw((2, 4, 2, SQ[rows], D, 64, 6, 16, "fp16", True, (384, 200)), seed=13, spread=0.0, nan=False)
    st["ks"][:] = 2.0 ** -22
    st["q"][:, 0] = (st["q"][:, 0].float() * 15000).clamp(-65504, 65504).half()
    st["q"][:, 1] *= 2.0 ** -14  # subnormal
    K8.check(*K8.call(st, True), st, True, 1 / math.sqrt(D))


@pytest.mark.parametrize("rows", SQ)
def test_graphs_with_new_lengths_and_two_streams(rows):
    st = draw(rows, seed=17)
    g = {n: t.to(DEV) for n, t in st.items()}
    args = (g["q"], g["kp"], g["vp"], g["ks"], g["vs"], g["lens"], g["table"])
    want = af.attn_fwd_kvcache_paged_fp8(*args, causal=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [af.attn_fwd_kvcache_paged_fp8(*args, causal=True, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = af.attn_fwd_kvcache_paged_fp8(*args, causal=True)
    for lens in ((1, 0), (0, 384), (129, 128), (1000, -5), (384, 200)):
        g["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        again = af.attn_fwd_kvcache_paged_fp8(*args, causal=True)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
        check({**st, "lens": torch.tensor(lens, dtype=torch.int32)})


@pytest.mark.parametrize("case", [
    (70, 2, 1, 1, 64, 16, 5, 16, "bf16", True, tuple((11 * i) % 81 for i in range(70))),      # more requests than a warp has lanes
    (40, 2, 1, 26, 64, 16, 8, 16, "fp16", True, tuple((13 * i) % 129 for i in range(40))),    # the same, many rows
    (34, 1, 1, 300, 128, 32, 12, 32, "bf16", True, tuple((37 * i) % 385 for i in range(34))),
    (2, 4, 1, 2100, 64, 64, 40, 64, "bf16", True, (2500, 2099)),                              # more items of a head than lanes
    (2, 4, 1, 2100, 64, 64, 5, 64, "fp16", False, (320, 0)),
], ids=lambda c: "_".join(map(str, c[:10])))
def test_more_requests_and_items_than_lanes(case):
    K8.test_matches_the_definition(case)
