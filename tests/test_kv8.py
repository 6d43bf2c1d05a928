"""Attention over an e4m3 paged cache with a scale for each block of tokens
and head, against the fp64 definition; what lies behind the lengths and outside
the pages is NaN throughout; the refusals (on the CPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import ops_ref as R

gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

# b, h, h_kv, sq, d, page, pages, block, dtype, causal, lens
CASES = [
    (1, 1, 1, 1, 128, 16, 1, 16, "bf16", True, (1,)),
    (1, 8, 1, 1, 128, 64, 8, 16, "bf16", True, (500,)),
    (4, 8, 8, 1, 64, 128, 3, 32, "fp16", True, (384, 1, 0, 129)),
    (3, 32, 8, 1, 128, 256, 8, 64, "bf16", True, (2048, 17, 700)),
    (2, 6, 2, 5, 64, 16, 40, 16, "fp16", True, (640, 3)),              # rows that see no key
    (2, 4, 2, 9, 128, 48, 7, 16, "bf16", False, (300, -2)),            # a length below zero
    (1, 4, 1, 33, 128, 32, 20, 32, "fp16", True, (5000,)),             # a length past the capacity
    (2, 16, 1, 1, 64, 128, 4, 128, "bf16", False, (511, 512)),
    (1, 32, 4, 1, 128, 128, 9, 128, "fp16", True, (1111,)),
    (2, 2, 2, 200, 128, 64, 5, 64, "bf16", True, (300, 150)),          # a chunk longer than its cache
    (1, 6, 3, 130, 64, 128, 4, 16, "fp16", True, (490,)),
    (1, 2, 1, 300, 128, 256, 3, 32, "bf16", False, (650,)),
    (5, 3, 3, 2, 128, 16, 12, 16, "bf16", True, (0, 0, 0, 0, 0)),      # nothing cached
    (2, 8, 2, 11, 128, 48, 9, 16, "fp16", True, (430, 25)),            # 44 rows: three tiles of 16
    (3, 2, 1, 25, 64, 16, 30, 16, "bf16", True, (480, 0, 24)),         # 50 rows, one Q tile; no or too few keys
    (2, 4, 2, 90, 128, 16, 40, 16, "bf16", True, (640, 89)),           # 180 rows, pages of 16
    (2, 6, 2, 120, 64, 96, 7, 32, "fp16", False, (600, 1)),            # 360 rows
    (1, 2, 2, 700, 128, 128, 11, 128, "fp16", True, (1400,)),          # items that several CTAs share
    (40, 2, 1, 1, 64, 64, 3, 64, "bf16", True, tuple((7 * i) % 193 for i in range(40))),
]


def draw(case, seed=11, spread=1.0, nan=True):
    b, h, hkv, sq, d, page, pages, block, dt, causal, lens = case
    g = torch.Generator().manual_seed(seed + 5 * h + sq)
    n = b * pages + 2
    q = torch.randn((b, h, sq, d), generator=g).to(DT[dt])
    kp, ks = R.random_pool(n, page, hkv, d, block, seed, spread)
    vp, vs = R.random_pool(n, page, hkv, d, block, seed + 1, spread)
    table = torch.randperm(n, generator=g)[:b * pages].reshape(b, pages).to(torch.int32)
    st = dict(q=q, kp=kp, vp=vp, ks=ks, vs=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32))
    if nan:  # behind the lengths, and in pages of no request
        used = torch.zeros((n, page), dtype=torch.bool)
        for e in range(b):
            ln = min(max(int(lens[e]), 0), pages * page)
            for p in range(pages):
                used[int(table[e, p]), :max(0, min(page, ln - p * page))] = True
        for pool in (kp, vp):
            pool.view(torch.uint8)[~used] = 0x7F
        dead = ~used.view(n, page // block, block).any(2)
        for sc in (ks, vs):
            sc.transpose(1, 2)[dead] = float("nan")
    return st


def call(st, causal, scale=None, **kw):
    g = {n: t.to(DEV) for n, t in st.items()}
    o, lse = af.attn_fwd_kvcache_paged_fp8(g["q"], g["kp"], g["vp"], g["ks"], g["vs"], g["lens"], g["table"],
                                           causal=causal, scale=scale, **kw)
    torch.cuda.synchronize()
    assert af.status()[0] == 0
    return o, lse


def reference(st, causal, scale):
    kp, vp = (np.nan_to_num(R.f64(st[n])) for n in ("kp", "vp"))
    ks, vs = (np.nan_to_num(R.f64(st[n])) for n in ("ks", "vs"))
    return R.attend_paged(R.f64(st["q"]), kp, vp, ks, vs, st["lens"].numpy(), st["table"].numpy(), causal, scale), vp, vs


def check(o, lse, st, causal, scale):
    (ro, rl), vp, vs = reference(st, causal, scale)
    t = st["q"].dtype
    o, lse = R.f64(o), R.f64(lse)
    assert not np.isnan(o).any() and not np.isnan(lse).any()
    dead = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), dead) and (lse[dead] < 0).all() and (o[dead] == 0).all()
    # The weights: a score of size x has an fp32 dot product's error, some 2^-22 of the sum of its terms'
    # sizes (at most |q||k|); each P has that error and one fp16 rounding (2^-11, or
    # 2^-25 of the largest).  So LSE is off by at most the largest score's error, and O by that and 2^-11, of
    # the largest |V|; its own rounding comes on top.
    q, b = R.f64(st["q"]), o.shape[0]
    kmax = np.nan_to_num(R.f64(st["ks"])).max() * 448 * math.sqrt(o.shape[-1])
    err = 2.0 ** -22 * np.abs(scale) * np.linalg.norm(q, axis=-1) * kmax
    assert (np.abs(lse[~dead] - rl[~dead]) <= err[~dead] + 2.0 ** -20 * (1 + np.abs(rl[~dead]))).all()
    vmax = vs.max() * 448
    bound = R.HALF_STEP[t] * np.abs(ro) + (2.0 ** -11 + 2 * err[..., None]) * vmax + 2.0 ** -25
    worst = np.abs(o - ro) - bound
    assert (worst <= 0).all(), worst.max()
    # and as a whole: the roundings of P are independent, so the result is as good as its own type's
    rel = np.linalg.norm(o - ro) / max(np.linalg.norm(ro), 1e-30)
    assert rel <= 2 * R.HALF_STEP[t], rel


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c[:10])))
def test_matches_the_definition(case):
    st = draw(case)
    d, causal = case[4], case[9]
    o, lse = call(st, causal)
    check(o, lse, st, causal, 1 / math.sqrt(d))


@gpu
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_scales_of_the_scores(scale):
    st = draw(CASES[4], seed=5)
    check(*call(st, True, scale), st, True, scale)


@gpu
def test_block_scales_from_tiny_to_huge_and_zero():
    case = (2, 4, 2, 3, 128, 64, 6, 16, "bf16", True, (384, 200))
    st = draw(case, seed=9, nan=False)
    g = torch.Generator().manual_seed(1)
    st["vs"] = torch.exp2(torch.randint(-60, 60, st["vs"].shape, generator=g).float())
    st["ks"] = torch.exp2(torch.randint(-20, -4, st["ks"].shape, generator=g).float())
    st["vs"][:, :, 1] = 0.0
    st["ks"][:, :, 2] = 0.0
    o, lse = call(st, True)
    (ro, rl), _, _ = reference(st, True, 1 / math.sqrt(128))
    # sums over 120 binary orders: each row by its own size
    row = np.abs(ro).max(-1, keepdims=True)
    assert (np.abs(R.f64(o) - ro) <= row * 2.0 ** -7).all()
    assert np.abs(R.f64(lse) - rl).max() <= 2.0 ** -16


@gpu
def test_scales_that_are_no_powers_of_two():
    case = CASES[3]
    st = draw(case, seed=21, nan=False)
    g = torch.Generator().manual_seed(2)
    for n in ("ks", "vs"):
        st[n] = st[n] * (torch.rand(st[n].shape, generator=g) * 0.5 + 0.5)
    check(*call(st, True), st, True, 1 / math.sqrt(128))


@gpu
def test_rows_of_queries_far_apart_in_size():
    """bf16 queries from 2^-30 to 2^30 in one batch, and within a row."""
    case = (1, 8, 2, 2, 128, 64, 4, 16, "bf16", True, (250,))
    st = draw(case, seed=31, nan=False)
    st["ks"] *= 2.0 ** -6
    st["q"][0, 0] *= 2.0 ** -30
    st["q"][0, 1] = 0
    st["q"][0, 2, :, 0] *= 2.0 ** -20
    st["q"][0, 3] = st["q"][0, 3] * 2.0 ** -130
    check(*call(st, True), st, True, 1 / math.sqrt(128))
    st["q"][0, 5, 0, 3] = float("inf")
    st["q"][0, 6, 1, 3] = float("nan")
    o, lse = call(st, True)
    o, lse = R.f64(o), R.f64(lse)
    assert np.isnan(o[0, 5, 0]).all() and np.isnan(o[0, 6, 1]).all() and np.isnan(lse[0, 6, 1])
    st["q"][0, 5, 0, 3] = st["q"][0, 6, 1, 3] = 0
    keep = np.ones((8, 2), dtype=bool)
    keep[5, 0] = keep[6, 1] = False
    (ro, rl), _, _ = reference(st, True, 1 / math.sqrt(128))
    assert np.abs(lse[0] - rl[0])[keep].max() < 1e-4 and np.isfinite(o[0][keep]).all()


@gpu
def test_pages_outside_the_pool_read_as_zeros():
    case = (2, 4, 2, 1, 64, 32, 8, 32, "fp16", True, (250, 100))
    st = draw(case, seed=41, nan=False)
    st["table"][0, 2], st["table"][0, 7], st["table"][1, 0] = -1, 10 ** 6, -(2 ** 31)
    check(*call(st, True), st, True, 1 / math.sqrt(64))


@gpu
def test_without_lse_outputs_given_and_workspace_reused():
    case = CASES[3]
    st = draw(case)
    g = {n: t.to(DEV) for n, t in st.items()}
    lib = binding.load()
    b, h, sq, d = g["q"].shape
    need = af.kvcache_paged_fp8_workspace_bytes(b, h, 8, sq, d)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    args = (g["q"], g["kp"], g["vp"], g["ks"], g["vs"], g["lens"], g["table"])
    o1, l1 = af.attn_fwd_kvcache_paged_fp8(*args, causal=True, workspace=ws)
    o2, l2 = torch.empty_like(o1), torch.empty_like(l1)
    af.attn_fwd_kvcache_paged_fp8(*args, causal=True, workspace=ws, o=o2, lse=l2)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    o3 = torch.empty_like(o1)
    rc = lib.attn_fwd_kvcache_paged_fp8(*(t.data_ptr() for t in args), o3.data_ptr(), None, b, h, 8, sq,
                                        g["kp"].shape[0], 256, 8, 64, d, 1, float(1 / math.sqrt(d)), 1, ws.data_ptr(), need,
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(o1, o3)


@gpu
def test_two_streams_and_graphs_with_new_lengths():
    st = draw(CASES[3], nan=False)
    g = {n: t.to(DEV) for n, t in st.items()}
    args = (g["q"], g["kp"], g["vp"], g["ks"], g["vs"], g["lens"], g["table"])
    want = af.attn_fwd_kvcache_paged_fp8(*args, causal=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s in streams:
            got.append(af.attn_fwd_kvcache_paged_fp8(*args, causal=True, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = af.attn_fwd_kvcache_paged_fp8(*args, causal=True)
    for lens in ((1, 2000, 0), (2048, 17, 700)):
        g["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        st["lens"] = torch.tensor(lens, dtype=torch.int32)
        check(o, lse, st, True, 1 / math.sqrt(128))


@gpu
def test_queries_of_one_head_do_not_depend_on_their_neighbours():
    """A key that only later queries see takes no part in the earlier ones,
    whatever it holds: NaN in the last cached tokens."""
    for case in ((1, 2, 1, 4, 128, 64, 4, 16, "bf16", True, (203,)), (1, 3, 3, 40, 64, 64, 4, 16, "fp16", True, (203,)),
                 (1, 4, 2, 40, 128, 64, 4, 16, "fp16", True, (203,)), (1, 1, 1, 190, 64, 64, 4, 32, "bf16", True, (203,))):
        st = draw(case, seed=51, nan=False)
        sq, n = case[3], 203
        clean = call(st, True)
        for name in ("kp", "vp"):
            bad = {k: v.clone() for k, v in st.items()}
            page, row = int(st["table"][0, (n - 2) // 64]), (n - 2) % 64  # seen by the last two queries
            bad[name].view(torch.uint8)[page, row, :, 7] = 0x7F
            o, _ = call(bad, True)
            assert torch.equal(o[:, :, :sq - 2], clean[0][:, :, :sq - 2])
            assert torch.isnan(o[:, :, sq - 2:]).any(-1).all()


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


BUF = ctypes.create_string_buffer(4096)
P = ctypes.addressof(BUF) + (-ctypes.addressof(BUF)) % 256


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), -3), (dict(dtype=2), -4), (dict(b=-1), -2), (dict(h=3), -2), (dict(h_kv=0), -2), (dict(h_kv=-1), -2),
    (dict(sq=1 << 31), -2), (dict(page=40), -2), (dict(block=0), -2), (dict(block=24), -2), (dict(block=128), -2),
    (dict(num_pages=1 << 28), -2), (dict(pages=1 << 26), -2), (dict(scale=math.nan), -5), (dict(q=None), -1),
    (dict(q=P + 8), -6), (dict(ks=None), -1), (dict(ks=P + 2), -6), (dict(lens=None), -1), (dict(table=P + 1), -6),
    (dict(ws=None), -1), (dict(ws=P + 4), -6), (dict(ws_bytes=100), -2), (dict(lse=P + 1), -6),
    (dict(h=1 << 15, h_kv=1, sq=1 << 20), -2),
])
def test_refusals(lib, kw, code):
    a = dict(q=P, kp=P, vp=P, ks=P, vs=P, lens=P, table=P, o=P, lse=None, b=1, h=4, h_kv=2, sq=1, num_pages=4, page=64,
             pages=2, block=16, d=64, scale=0.1, dtype=1, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    rc = lib.attn_fwd_kvcache_paged_fp8(a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["lens"], a["table"], a["o"],
                                        a["lse"], a["b"], a["h"], a["h_kv"], a["sq"], a["num_pages"], a["page"],
                                        a["pages"], a["block"], a["d"], 1, a["scale"], a["dtype"], a["ws"],
                                        a["ws_bytes"], None)
    assert rc == code and lib.attn_last_error()


@pytest.mark.parametrize("o", [P, P + 64, P - 64, (1 << 32) + 1024, (1 << 33) - 16])
def test_an_output_over_an_input_is_refused(lib, o):
    q, kp, vp = P, 1 << 32, 1 << 33
    rc = lib.attn_fwd_kvcache_paged_fp8(q, kp, vp, P, P, P, P, o, None, 1, 4, 2, 1, 4, 64, 2, 16, 64, 1, 0.1, 1, P, 1 << 40,
                                        None)
    assert rc == -2 and b"overlaps" in lib.attn_last_error()


def test_nothing_to_do_and_workspace(lib):
    for kw in (dict(b=0), dict(h=0), dict(sq=0)):
        n = dict(b=1, h=2, sq=1)
        n.update(kw)
        assert lib.attn_fwd_kvcache_paged_fp8(*[None] * 9, n["b"], n["h"], 2, n["sq"], 4, 64, 2, 16, 64, 1, 0.1, 1, None,
                                              0, None) == 0
    assert lib.attn_fwd_kvcache_paged_fp8_workspace_bytes(1, 2, 1, 1, 96) == -3
    assert lib.attn_fwd_kvcache_paged_fp8_workspace_bytes(-1, 2, 1, 1, 64) == -2
    assert lib.attn_fwd_kvcache_paged_fp8_workspace_bytes(1, 2, 1, 1, 64) > 0


@gpu
def test_binding_refusals():
    st = {n: t.to(DEV) for n, t in draw(CASES[3], nan=False).items()}
    names = ("q", "kp", "vp", "ks", "vs", "lens", "table")
    bad = [dict(q=st["q"].float()), dict(kp=st["kp"].view(torch.uint8)), dict(ks=None), dict(lens=st["lens"].long()),
           dict(table=st["table"][:1]), dict(ks=st["ks"][:, :4]), dict(vs=st["vs"].half()), dict(q=st["q"][0]),
           dict(q=st["q"].expand(3, 32, 1, 128)[:, ::2]), dict(lens=st["lens"].cpu()), dict(vp=st["vp"][:4])]
    for kw in bad:
        a = {**st, **kw}
        with pytest.raises(af.AttnError):
            af.attn_fwd_kvcache_paged_fp8(*(a[n] for n in names))
    with pytest.raises(af.AttnError):
        af.attn_fwd_kvcache_paged_fp8(*(st[n] for n in names), workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
