"""RMS norm of queries and keys with the rotary rotation, and its gradients,
against the fp64 definition; the definition's gradients against differences;
the refusals (on the CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import ops_ref as R

gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)

# b, h, h_kv, s, d, rot, interleaved, dtype, layout
CASES = [
    (1, 1, 1, 1, 128, 128, False, "bf16", "dense"),
    (2, 32, 8, 1, 128, 128, False, "bf16", "fused"),
    (3, 5, 3, 7, 64, 64, False, "fp16", "fused"),
    (2, 9, 1, 33, 128, 64, False, "fp16", "fused"),
    (1, 2, 2, 130, 64, 32, True, "bf16", "dense"),
    (2, 16, 16, 65, 128, 128, True, "fp16", "fused"),
    (4, 3, 2, 50, 128, 16, False, "bf16", "packed"),
    (3, 17, 4, 101, 64, 48, True, "fp16", "packed"),
    (2, 4, 4, 300, 64, 16, True, "bf16", "fused"),
]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def draw(case, seed=1):
    b, h, hkv, s, d, rot, il, dt, layout = case
    g = torch.Generator().manual_seed(seed + 31 * s + h)
    t = DT[dt]
    if layout == "packed":
        x = torch.randn((b * s, h + 2 * hkv, d), generator=g).to(t)
        q, k = x[:, :h], x[:, h:h + hkv]
        pos = torch.cat([torch.arange(s, dtype=torch.int32)] * b)
    else:
        x = torch.randn((b, s, h + 2 * hkv, d), generator=g).to(t)
        q, k = x[:, :, :h].transpose(1, 2), x[:, :, h:h + hkv].transpose(1, 2)
        if layout == "dense":
            q, k = q.contiguous(), k.contiguous()
        pos = torch.randint(0, 400, (b, s), generator=g, dtype=torch.int32)
    wq, wk = ((torch.rand(d, generator=g) + 0.5).to(t) for _ in range(2))
    cos, sin = R.tables(400, rot)
    gq, gk = (torch.randn(u.shape, generator=g).to(t) for u in (q, k))
    return dict(q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, pos=pos, gq=gq, gk=gk, il=il)


def on_gpu(st):
    """To the device with the strides kept (views of one storage)."""
    def move(t):
        if not torch.is_tensor(t):
            return t
        return t.to(DEV) if t.is_contiguous() else torch.empty_strided(t.size(), t.stride(), dtype=t.dtype,
                                                                       device=DEV).copy_(t)
    return {n: move(t) for n, t in st.items()}


def as_tokens(t):
    """[b, h, s, d] or [total, h, d] as fp64 [tokens, heads, d]."""
    a = R.f64(t)
    return a.transpose(0, 2, 1, 3).reshape(-1, a.shape[1], a.shape[3]) if a.ndim == 4 else a


def close(got, ref, t, rows_of=None, what=""):
    """One rounding to the type, and the fp32 arithmetic: a dozen roundings
    of values no larger than the row's largest (2^-24 each), with rsqrt's two
    ulp: 2^-19 of the row's largest covers it.  fp16's subnormal half step: 2^-25."""
    got, bound = as_tokens(got), R.HALF_STEP[t] * np.abs(ref) + 2.0 ** -25
    row = np.abs(rows_of if rows_of is not None else ref).max(-1, keepdims=True)
    bad = np.abs(got - ref) > bound + 2.0 ** -19 * row
    assert not bad.any(), f"{what}: {bad.sum()} values off, worst {np.abs(got - ref).max():.3e}"


def reference(st, case, eps=1e-6):
    pos = st["pos"].numpy().reshape(-1)
    cos, sin = R.f64(st["cos"]), R.f64(st["sin"])
    out = [R.norm_rope(as_tokens(st[n]), R.f64(st[w]), cos, sin, pos, eps, st["il"]) for n, w in (("q", "wq"), ("k", "wk"))]
    back = [R.norm_rope_bwd(as_tokens(st[g]), as_tokens(st[n]), R.f64(st[w]), cos, sin, pos, eps, st["il"])
            for g, n, w in (("gq", "q", "wq"), ("gk", "k", "wk"))]
    return out, back


def test_the_definitions_gradients_are_its_differences():
    rng = np.random.default_rng(5)
    x, w, g = rng.normal(size=(6, 3, 64)), rng.normal(size=64), rng.normal(size=(6, 3, 64))
    cos, sin = (R.f64(t) for t in R.tables(10, 32))
    pos = np.array([0, 3, 9, -1, 10, 5])
    for il in (False, True):
        f = lambda a, b: (R.norm_rope(a, b, cos, sin, pos, 1e-6, il) * g).sum()  # noqa: E731
        dx, dw = R.norm_rope_bwd(g, x, w, cos, sin, pos, 1e-6, il)
        for _ in range(20):
            e, ew = rng.normal(size=x.shape), rng.normal(size=64)
            h = 1e-6
            diff = (f(x + h * e, w + h * ew) - f(x - h * e, w - h * ew)) / (2 * h)
            assert abs(diff - (dx * e).sum() - (dw * ew).sum()) < 1e-6 * (1 + abs(diff))


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    st = draw(case)
    g = on_gpu(st)
    q, k = af.attn_qk_norm_rope(g["q"], g["k"], g["wq"], g["wk"], g["cos"], g["sin"], g["pos"], interleaved=st["il"])
    (rq, rk), _ = reference(st, case)
    assert q.is_contiguous() and k.is_contiguous()
    close(q, rq, q.dtype, what="q")
    close(k, rk, k.dtype, what="k")
    assert torch.equal(g["q"].cpu(), st["q"]) and torch.equal(g["k"].cpu(), st["k"])


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    st = draw(case)
    g = on_gpu(st)
    dq, dk, dwq, dwk = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], g["q"], g["k"], g["wq"], g["wk"], g["cos"], g["sin"],
                                                g["pos"], interleaved=st["il"])
    _, ((rq, rwq), (rk, rwk)) = reference(st, case)
    for got, ref, n, name in ((dq, rq, "gq", "q"), (dk, rk, "gk", "k")):
        close(got, ref, got.dtype, what="d" + name)
    for got, ref, gg, x, w in ((dwq, rwq, "gq", "q", "wq"), (dwk, rwk, "gk", "k", "wk")):
        # |dw| sums: each term has some ten fp32 roundings, and so has each of the partial sums it passes through
        n = as_tokens(st[x]) / np.sqrt((as_tokens(st[x]) ** 2).mean(-1, keepdims=True) + 1e-6)
        pos = st["pos"].numpy().reshape(-1)
        dy = R.rotate(as_tokens(st[gg]), R.f64(st["cos"])[pos][:, None], -R.f64(st["sin"])[pos][:, None], st["il"])
        bound = (np.abs(dy * n).sum((0, 1)) + 1e-6) * 2.0 ** -24 * 200
        assert (np.abs(R.f64(got) - ref) <= bound).all()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_backward_without_eps_when_heads_do_not_fill_a_unit(d):
    gen = torch.Generator().manual_seed(17)
    q, gq = (torch.randn(1, 3, 5, d, generator=gen).to(torch.bfloat16) for _ in range(2))
    k, gk = (torch.randn(1, 1, 5, d, generator=gen).to(torch.bfloat16) for _ in range(2))
    w = torch.ones(d, dtype=torch.bfloat16)
    dq, dk, dwq, dwk = af.attn_qk_norm_rope_bwd(*(t.cuda() for t in (gq, gk, q, k, w, w)), eps=0.0)
    for dx, dw, g, x in ((dq, dwq, gq, q), (dk, dwk, gk, k)):
        x, g = as_tokens(x), as_tokens(g)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True))
        n = x * r
        close(dx, r * (g - n * (g * n).mean(-1, keepdims=True)), dx.dtype, rows_of=r * g)
        # each of 15 terms and of their sums has some ten fp32 roundings
        bound = (np.abs(g * n).sum((0, 1)) + 1e-6) * 2.0 ** -24 * 200
        assert (np.abs(R.f64(dw) - (g * n).sum((0, 1))) <= bound).all()


@gpu
@pytest.mark.parametrize("norm,turn", [(False, True), (True, False)])
def test_norm_alone_and_rotation_alone(norm, turn):
    case = (2, 6, 2, 40, 128, 96, False, "bf16", "fused")
    st = draw(case)
    g = on_gpu(st)
    w = (g["wq"], g["wk"]) if norm else (None, None)
    cs = (g["cos"], g["sin"]) if turn else (None, None)
    pos = st["pos"].numpy().reshape(-1)
    cos, sin = (R.f64(st["cos"]), R.f64(st["sin"])) if turn else (None, None)
    q, k = af.attn_qk_norm_rope(g["q"], g["k"], *w, *cs, g["pos"] if turn else None)
    dq, dk, dwq, dwk = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], g["q"], g["k"], *w, *cs, g["pos"] if turn else None)
    for got, back, dw, n, gn, wn in ((q, dq, dwq, "q", "gq", "wq"), (k, dk, dwk, "k", "gk", "wk")):
        ww = R.f64(st[wn]) if norm else None
        close(got, R.norm_rope(as_tokens(st[n]), ww, cos, sin, pos, 1e-6, False), got.dtype)
        ref, _ = R.norm_rope_bwd(as_tokens(st[gn]), as_tokens(st[n]), ww, cos, sin, pos, 1e-6, False)
        close(back, ref, got.dtype)
        assert (dw is None) == (not norm)


@gpu
def test_positions_by_default_shared_and_outside_the_tables():
    case = (3, 4, 2, 20, 64, 64, False, "fp16", "fused")
    st = draw(case)
    g = on_gpu(st)
    args = (g["q"], g["k"], g["wq"], g["wk"], g["cos"], g["sin"])
    a = af.attn_qk_norm_rope(*args)
    b = af.attn_qk_norm_rope(*args, torch.arange(20, dtype=torch.int32, device=DEV))
    c = af.attn_qk_norm_rope(*args, torch.arange(20, dtype=torch.int32, device=DEV).expand(3, 20))
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))
    af.binding.status_clear()
    pos = st["pos"].clone()
    pos[0, 3], pos[2, 19], pos[1, 0] = -1, -(2 ** 31), 7
    g["q"][0, :, 3] = float("nan")  # padding may hold anything
    st["q"][0, :, 3] = 0.0
    q, _ = af.attn_qk_norm_rope(*args, pos.to(DEV))
    assert af.status()[0] == 0
    ref = R.norm_rope(as_tokens(st["q"]), R.f64(st["wq"]), R.f64(st["cos"]), R.f64(st["sin"]), pos.numpy().reshape(-1),
                      1e-6, False)
    close(q, ref, q.dtype)
    assert (q[0, :, 3] == 0).all() and (q[2, :, 19] == 0).all()
    dq, dk, dwq, _ = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], *args, pos.to(DEV))
    assert (dq[0, :, 3] == 0).all() and (dk[2, :, 19] == 0).all() and torch.isfinite(dwq).all()
    pos[1, 5] = 400  # one past the end of the tables
    q, _ = af.attn_qk_norm_rope(*args, pos.to(DEV))
    assert (q[1, :, 5] == 0).all() and af.status()[0] == 4
    af.binding.status_clear()


@gpu
def test_in_place_and_into_slices():
    case = (2, 6, 2, 40, 128, 128, False, "bf16", "fused")
    st = draw(case)
    g = on_gpu(st)
    tail = (g["wq"], g["wk"], g["cos"], g["sin"], g["pos"])
    want = af.attn_qk_norm_rope(g["q"], g["k"], *tail)
    grads = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], g["q"], g["k"], *tail)
    fused = torch.full((2, 40, 10, 128), 7.0, dtype=torch.bfloat16, device=DEV)  # the projection's gradient
    dq, dk = fused[:, :, :6].transpose(1, 2), fused[:, :, 6:8].transpose(1, 2)
    again = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], g["q"], g["k"], *tail, dq=dq, dk=dk)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)) and (fused[:, :, 8:] == 7).all()
    af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], g["q"], g["k"], *tail, dq=g["gq"], dk=g["gk"])
    assert torch.equal(g["gq"], grads[0]) and torch.equal(g["gk"], grads[1])
    af.attn_qk_norm_rope(g["q"], g["k"], *tail, q_out=g["q"], k_out=g["k"])
    assert torch.equal(g["q"], want[0]) and torch.equal(g["k"], want[1])


@gpu
def test_equal_calls_give_equal_bits_and_graphs_replay():
    case = (2, 32, 8, 700, 128, 128, False, "bf16", "fused")
    g = on_gpu(draw(case))
    tail = (g["q"], g["k"], g["wq"], g["wk"], g["cos"], g["sin"], g["pos"])
    first = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], *tail)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], *tail, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = af.attn_qk_norm_rope(*tail)
        back = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], *tail)
    g["q"].copy_(g["q"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    now = af.attn_qk_norm_rope(*tail)
    nback = af.attn_qk_norm_rope_bwd(g["gq"], g["gk"], *tail)
    assert all(torch.equal(a, b) for a, b in zip(out + back, now + nback))


@gpu
@pytest.mark.parametrize("shape", [(0, 4, 2, 5), (2, 4, 2, 0), (2, 0, 2, 5), (2, 4, 0, 5)])
def test_empty_axes(shape):
    b, h, hkv, s = shape
    q = torch.randn((b, h, s, 64), device=DEV).half()
    k = torch.randn((b, hkv, s, 64), device=DEV).half()
    w = torch.ones(64, device=DEV).half()
    cos, sin = (t.to(DEV) for t in R.tables(16, 64))
    qo, ko = af.attn_qk_norm_rope(q, k, w, w, cos, sin)
    dq, dk, dwq, dwk = af.attn_qk_norm_rope_bwd(q, k, q, k, w, w, cos, sin)
    assert qo.shape == q.shape and ko.shape == k.shape
    assert torch.isfinite(qo).all() and torch.isfinite(dk).all()
    if q.numel() == 0:
        assert (dwq == 0).all()
    if k.numel() == 0:
        assert (dwk == 0).all()


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


BUF = ctypes.create_string_buffer(8192)
P = ctypes.addressof(BUF) + (-ctypes.addressof(BUF)) % 256
S3 = ctypes.c_int64 * 3


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), -3), (dict(dtype=2), -4), (dict(b=-1), -2), (dict(s=1 << 31), -2), (dict(b=1 << 20, s=1 << 20), -2),
    (dict(eps=-1.0), -5), (dict(eps=float("nan")), -5), (dict(rot=0), -2), (dict(rot=24), -2), (dict(rot=80), -2),
    (dict(table_len=0), -2), (dict(sin=None), -1), (dict(cos=P + 4), -6), (dict(q=None), -1), (dict(q=P + 8), -6),
    (dict(qs=(1024, 64, 68)), -6), (dict(qs=(-8, 64, 64)), -6), (dict(os=(1024, 64, 32)), -2), (dict(pos=P + 2), -6),
    (dict(pos=None, table_len=3), -2), (dict(pos_b=-1), -2), (dict(q_out=P), -2), (dict(w=P + 2), -6),
    (dict(b=1 << 12, s=1 << 12, h=1 << 10), -2),
])
def test_refusals(lib, kw, code):
    a = dict(q=P, w=P, cos=P, sin=P, pos=P, q_out=P + 4096, qs=(1024, 64, 128), os=(1024, 256, 64), b=1, h=2, hkv=0, s=4,
             d=64, rot=64, table_len=16, pos_b=0, eps=1e-6, dtype=1)
    a.update(kw)
    rc = lib.attn_qk_norm_rope(a["q"], None, a["w"], None, a["cos"], a["sin"], a["pos"], a["q_out"], None, S3(*a["qs"]),
                               None, S3(*a["os"]), None, a["b"], a["h"], a["hkv"], a["s"], a["d"], a["rot"],
                               a["table_len"], a["pos_b"], 0, a["eps"], a["dtype"], None)
    assert rc == code and lib.attn_last_error()


def test_backward_refusals(lib):
    assert lib.attn_qk_norm_rope_bwd_workspace_bytes(96) == -3
    need = lib.attn_qk_norm_rope_bwd_workspace_bytes(64)
    st = S3(512, 256, 64)

    def call(w=P, dw=P + 64, ws=P, ws_bytes=need, g=P):
        return lib.attn_qk_norm_rope_bwd(g, None, P, None, w, None, None, None, None, P + 4096, None, dw, None, st, None,
                                         st, None, st, None, 1, 2, 0, 4, 64, 0, 0, 0, 0, 1e-6, 1, ws, ws_bytes, None)
    assert call(w=None) == -1       # a gradient of no weight
    assert call(ws=None) == -1 and call(ws=P + 4) == -6 and call(ws_bytes=need - 1) == -2
    assert call(dw=P + 2) == -6 and call(g=None) == -1 and call(g=P + 8) == -6


def test_backward_in_place_with_other_strides_is_refused(lib):
    need = lib.attn_qk_norm_rope_bwd_workspace_bytes(64)

    def call(g, x, dx, gs, xs):
        return lib.attn_qk_norm_rope_bwd(g, None, x, None, P, None, None, None, None, dx, None, P + 64, None, S3(*gs), None,
                                         S3(*xs), None, S3(512, 256, 64), None, 1, 2, 0, 4, 64, 0, 0, 0, 0, 1e-6, 1, P,
                                         need, None)
    assert call(P, P + 4096, P, (512, 64, 128), (512, 256, 64)) == -2    # over its output's gradient
    assert call(P + 4096, P, P, (512, 256, 64), (512, 64, 128)) == -2    # over its input


@gpu
def test_binding_refusals():
    q = torch.zeros((2, 4, 8, 64), device=DEV).half()
    k = torch.zeros((2, 2, 8, 64), device=DEV).half()
    cos, sin = (t.to(DEV) for t in R.tables(16, 64))
    bad = [
        dict(k=k.bfloat16()), dict(k=k[:, :, :4]), dict(q=q.transpose(2, 3)), dict(q=q.float(), k=k.float()),
        dict(q_weight=torch.ones(64, device=DEV)), dict(q_weight=torch.ones(32, device=DEV).half()), dict(cos=None),
        dict(cos=cos.double()), dict(positions=torch.zeros(8, device=DEV)),
        dict(positions=torch.zeros((2, 7), dtype=torch.int32, device=DEV)),
        dict(q=q[0].transpose(0, 1), k=k[0].transpose(0, 1)), dict(q_out=q.float()), dict(q=q.cpu()),
        dict(q=torch.zeros((2, 4, 8, 72), device=DEV).half()[..., :64][..., ::1].as_strided((2, 4, 8, 64), (2304, 576, 71, 1))),
    ]
    for kw in bad:
        a = dict(q=q, k=k, cos=cos, sin=sin)
        a.update(kw)
        with pytest.raises(af.AttnError):
            af.attn_qk_norm_rope(a.pop("q"), a.pop("k"), **a)
