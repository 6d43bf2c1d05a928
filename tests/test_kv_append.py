"""Append of rotated keys and of values to a paged cache, in 16 bits and in
e4m3 with a scale for each block of tokens and head, against the fp64
definition row by row; the refusals (on the CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import ops_ref as R

gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

# b, heads, s_new, d, page, pages, block (0: 16 bits), rot, interleaved, dtype, lens, news
CASES = [
    (3, 2, 1, 128, 16, 4, 16, 128, False, "bf16", (0, 17, 63), None),
    (2, 8, 1, 64, 128, 2, 128, 64, True, "fp16", (127, 128), None),
    (4, 3, 40, 128, 64, 3, 32, 64, False, "fp16", (0, 31, 190, 192), None),   # dropped past the capacity
    (3, 5, 70, 64, 32, 5, 16, 32, True, "bf16", (-4, 33, 100), (70, 0, 13)),   # padded
    (2, 1, 200, 128, 256, 2, 64, 128, True, "bf16", (5, 300), (200, 500)),
    (2, 2, 130, 128, 128, 3, 128, 16, False, "fp16", (100, 1000), (-3, 130)),
    (2, 4, 33, 64, 64, 2, 64, 0, False, "bf16", (64, 1), None),                # no rotation
    (3, 7, 9, 128, 16, 4, 0, 128, False, "bf16", (0, 17, 60), None),
    (2, 32, 50, 64, 48, 3, 0, 48, True, "fp16", (40, -1), (50, 20)),
    (2, 3, 5, 128, 128, 1, 0, 0, False, "fp16", (3, 126), None),
]


def draw(case, seed=3):
    b, h, s, d, page, pages, block, rot, il, dt, lens, news = case
    g = torch.Generator().manual_seed(seed + s * 7 + h)
    n = b * pages + 2
    x = torch.randn((b, s, 2 * h, d), generator=g)
    x *= torch.exp(1.5 * torch.randn((b, s, 2 * h, 1), generator=g))  # blocks whose scale has to grow
    x = x.to(DT[dt])
    st = dict(k_new=x[:, :, :h].transpose(1, 2), v_new=x[:, :, h:].transpose(1, 2))
    st["table"] = torch.randperm(n, generator=g)[:b * pages].reshape(b, pages).to(torch.int32)
    st["lens"] = torch.tensor(lens, dtype=torch.int32)
    st["news"] = None if news is None else torch.tensor(news, dtype=torch.int32)
    st["cos"], st["sin"] = R.tables(page * pages, rot) if rot else (None, None)
    if block:
        st["k_pool"], st["k_scale"] = R.random_pool(n, page, h, d, block, seed)
        st["v_pool"], st["v_scale"] = R.random_pool(n, page, h, d, block, seed + 1)
    else:
        st["k_pool"], st["v_pool"] = (torch.randn((n, page, h, d), generator=g).to(DT[dt]) for _ in range(2))
        st["k_scale"] = st["v_scale"] = None
    return st


def to_dev(st):
    return {n: None if t is None else (t.to(DEV) if t.is_contiguous() else
                                       torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device=DEV).copy_(t))
            for n, t in st.items()}


def call(g, il, stream=None):
    af.attn_kvcache_append_paged(g["k_new"], g["v_new"], g["k_pool"], g["v_pool"], g["lens"], g["table"], cos=g["cos"],
                                 sin=g["sin"], interleaved=il, k_scale=g["k_scale"], v_scale=g["v_scale"],
                                 new_seqlens=g["news"], stream=stream)


def reference(st, block, il):
    return R.append_paged(R.f64(st["k_new"]), R.f64(st["v_new"]), R.f64(st["k_pool"]), R.f64(st["v_pool"]),
                          R.f64(st["k_scale"]), R.f64(st["v_scale"]), st["lens"].numpy(),
                          None if st["news"] is None else st["news"].numpy(), st["table"].numpy(), R.f64(st["cos"]),
                          R.f64(st["sin"]), il, block)


def check(g, st, block, il):
    kp, vp, ks, vs = reference(st, block, il)
    if block:
        # a rotated value has three fp32 roundings, which can move a value that lies within 2^-22 of
        # the middle between two e4m3 values to its other neighbour: a few in a million
        assert np.array_equal(R.f64(g["k_scale"]), ks) and np.array_equal(R.f64(g["v_scale"]), vs)
        got = R.f64(g["k_pool"])
        off = got != kp
        assert off.mean() <= 1e-4, off.sum()
        assert (np.abs(got - kp) <= 2.0 ** -3 * np.abs(kp) + 2.0 ** -9).all()
        assert np.array_equal(R.f64(g["v_pool"]), vp)
    else:
        t = g["k_pool"].dtype
        got = R.f64(g["k_pool"])
        row = np.abs(kp).max(-1, keepdims=True)
        assert (np.abs(got - kp) <= R.HALF_STEP[t] * np.abs(kp) + 2.0 ** -22 * row + 2.0 ** -25).all()
        assert np.array_equal(R.f64(g["v_pool"]), vp)


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_append(case):
    st = draw(case)
    g = to_dev(st)
    call(g, case[8])
    check(g, st, case[6], case[8])
    assert torch.equal(g["lens"].cpu(), st["lens"]) and torch.equal(g["table"].cpu(), st["table"])


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_equal_the_formula_step_by_step_in_fp32(interleaved, dt):
    """Each product and each sum rounded: no difference in any bit."""
    b, h, s, d, page, pages, rot, block = 2, 5, 250, 128, 64, 4, 96, 32
    g = torch.Generator().manual_seed(41)
    k = torch.randn((b, h, s, d), generator=g).to(DT[dt]).to(DEV)
    cos, sin = (t.to(DEV) for t in R.tables(page * pages, rot))
    table = torch.arange(b * pages, dtype=torch.int32, device=DEV).reshape(b, pages)
    lens = torch.zeros(b, dtype=torch.int32, device=DEV)
    x = k.float()
    i = torch.arange(rot // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, sn = cos[:s], sin[:s]
    want = x.clone()
    p0, p1 = x[..., first] * c, x[..., second] * sn
    want[..., first] = p0 - p1
    p0, p1 = x[..., second] * c, x[..., first] * sn
    want[..., second] = p0 + p1

    def tokens(pool):
        return pool.reshape(b, page * pages, h, d)[:, :s].transpose(1, 2)

    kp, vp = (torch.zeros((b * pages, page, h, d), dtype=DT[dt], device=DEV) for _ in range(2))
    af.attn_kvcache_append_paged(k, k, kp, vp, lens, table, cos, sin, interleaved)
    assert torch.equal(tokens(kp), want.to(DT[dt]))
    kp, vp = (torch.zeros((b * pages, page, h, d), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((b * pages, h, page // block), device=DEV) for _ in range(2))
    af.attn_kvcache_append_paged(k, k, kp, vp, lens, table, cos, sin, interleaved, ks, vs)
    scale = ks.transpose(1, 2).reshape(b, page * pages // block, h).repeat_interleave(block, 1)[:, :s].transpose(1, 2)[..., None]
    assert torch.equal(tokens(kp).float(), (want / scale).to(torch.float8_e4m3fn).float())


@gpu
@pytest.mark.parametrize("block", [0, 16])
def test_pages_outside_the_pool_are_not_written(block):
    case = (2, 2, 40, 64, 32, 3, block, 64, False, "bf16", (0, 20), None)
    st = draw(case)
    st["table"][0, 1], st["table"][1, 0], st["table"][1, 2] = -1, 8, 2 ** 31 - 1
    g = to_dev(st)
    call(g, False)
    check(g, st, block, False)


@gpu
def test_values_that_are_not_finite_and_blocks_of_zeros():
    case = (1, 2, 32, 64, 32, 2, 16, 0, False, "bf16", (0,), None)
    st = draw(case)
    v = st["v_new"].contiguous().clone()
    v[0, 0, 3, 5], v[0, 0, 4, 6], v[0, 0, 5, 7] = float("inf"), -float("inf"), float("nan")
    v[0, 1, :16] = 0.0
    st["v_new"] = v
    g = to_dev(st)
    call(g, False)
    pg = int(st["table"][0, 0])
    got = g["v_pool"].float()[pg]
    assert got[3, 0, 5] == 448 and got[4, 0, 6] == -448 and torch.isnan(got[5, 0, 7])
    assert (got[:16, 1] == 0).all() and g["v_scale"][pg, 1, 0] == 2.0 ** -64
    kp, vp, ks, vs = reference(st, 16, False)
    assert np.array_equal(R.f64(g["v_scale"]), vs) and np.array_equal(R.f64(g["v_pool"]), vp, equal_nan=True)


@gpu
@pytest.mark.parametrize("block", [16, 64])
def test_one_token_at_a_time_stands_for_the_same_values(block):
    """Token by token a block's scale grows as needed; at the end it is the
    one of a single append, and the values agree to e4m3's step (a stored value
    is rounded again only below e4m3's smallest normal)."""
    case = (2, 3, 70, 128, 128, 1, block, 128, False, "bf16", (0, 9), None)
    st = draw(case)
    one, steps = to_dev(st), to_dev(st)
    call(one, False)
    for t in range(70):
        step = dict(steps)
        step["k_new"], step["v_new"] = steps["k_new"][:, :, t:t + 1], steps["v_new"][:, :, t:t + 1]
        step["lens"] = steps["lens"] + t
        call(step, False)
    for name in ("k", "v"):
        assert torch.equal(one[name + "_scale"], steps[name + "_scale"])
        a, b = one[name + "_pool"].float(), steps[name + "_pool"].float()
        assert ((a - b).abs() <= a.abs() * 2.0 ** -4 + 2.0 ** -9).all()


@gpu
def test_another_stream_and_a_graph():
    case = CASES[3]
    st = draw(case)
    g = to_dev(st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(g, case[8], stream=side)
    side.synchronize()
    check(g, st, case[6], case[8])
    g = to_dev(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(g, case[8])
    for n in ("k_pool", "v_pool"):
        g[n].view(torch.uint8).copy_(st[n].to(DEV).view(torch.uint8))
    graph.replay()
    graph.replay()  # the same rows in the same places: nothing changes
    torch.cuda.synchronize()
    check(g, st, case[6], case[8])


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


BUF = ctypes.create_string_buffer(1 << 16)
P = ctypes.addressof(BUF) + (-ctypes.addressof(BUF)) % 256
S3 = ctypes.c_int64 * 3


@pytest.mark.parametrize("kw,code", [
    (dict(page=24), -2), (dict(page=0), -2), (dict(pages=0), -2), (dict(num_pages=0), -2), (dict(num_pages=1 << 30), -2),
    (dict(block=8), -2), (dict(block=48, page=48), -2), (dict(block=64), -2), (dict(block=0), -2), (dict(d=96), -3),
    (dict(dtype=3), -4), (dict(b=-1), -2), (dict(s=-1), -2), (dict(s=1 << 30, b=4), -2), (dict(rot=8), -2),
    (dict(sin=None), -1), (dict(table_len=63), -2), (dict(k_new=None), -1), (dict(k_new=P + 8), -6), (dict(lens=None), -1),
    (dict(lens=P + 2), -6), (dict(news=P + 1), -6), (dict(ks=None), -1), (dict(st=(128, 64, 12)), -6), (dict(st=None), -1),
    (dict(k_new=P + 16384), -2), (dict(v_pool=P + 16384 + 64), -2), (dict(table=P + 2), -6), (dict(vs=None), -1),
])
def test_refusals(lib, kw, code):
    a = dict(k_new=P, v_new=P + 1024, k_pool=P + 16384, v_pool=P + 32768, ks=P + 2048, vs=P + 2048, lens=P + 3328, news=None,
             table=P + 3328, cos=P + 4096, sin=P + 4096, st=(128, 64, 64), b=1, h=1, s=2, num_pages=4, page=32, pages=2,
             block=16, d=64, rot=64, table_len=64, dtype=1)
    a.update(kw)
    st = None if a["st"] is None else S3(*a["st"])
    rc = lib.attn_kvcache_append_paged(a["k_new"], a["v_new"], a["k_pool"], a["v_pool"], a["ks"], a["vs"], a["lens"],
                                       a["news"], a["table"], a["cos"], a["sin"], st, S3(128, 64, 64), a["b"], a["h"],
                                       a["s"], a["num_pages"], a["page"], a["pages"], a["block"], a["d"], a["rot"],
                                       a["table_len"], 0, a["dtype"], None)
    assert rc == code and lib.attn_last_error()


def test_nothing_to_append(lib):
    for kw in (dict(b=0), dict(h=0), dict(s=0)):
        n = dict(b=1, h=1, s=1)
        n.update(kw)
        assert lib.attn_kvcache_append_paged(*[None] * 13, n["b"], n["h"], n["s"], 4, 32, 2, 16, 64, 0, 0, 0, 1, None) == 0


@gpu
def test_binding_refusals():
    st = to_dev(draw(CASES[0]))
    bad = [dict(v_new=st["v_new"].half()), dict(k_scale=None), dict(k_pool=st["k_pool"].view(torch.uint8)),
           dict(lens=st["lens"].long()), dict(table=st["table"][:2]), dict(k_scale=st["k_scale"][:, :1]),
           dict(k_scale=None, v_scale=None), dict(news=st["lens"][:2]), dict(v_pool=st["v_pool"][:, :, :1]),
           dict(cos=st["cos"][:5]), dict(v_scale=st["v_scale"].double()), dict(k_pool=st["k_pool"].cpu())]
    for kw in bad:
        with pytest.raises(af.AttnError):
            call({**st, **kw}, False)
