"""The expanded form of latent attention and its gradients against their
definitions in 64 bits, and their refusals."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import latent_ref as L
import ops_ref as R

gpu = pytest.mark.gpu
SCALE = 192 ** -0.5

# heads, queries of each sequence, keys of each, causal, type
CASES = [
    (1, (1,), (1,), True, "bf16"),
    (2, (128,), (128,), True, "fp16"),
    (3, (300,), (300,), False, "fp16"),
    (2, (513,), (513,), True, "bf16"),
    (2, (1, 129, 64, 257), (1, 129, 64, 257), True, "bf16"),
    (1, (200, 5), (333, 200), True, "fp16"),          # keys that were there before
    (2, (200, 130), (100, 1), True, "bf16"),          # queries that see no key
    (2, (0, 70, 0), (50, 70, 0), True, "bf16"),       # sequences without queries, without keys
    (1, (70, 30), (0, 40), False, "fp16"),
    (5, (65,), (700,), False, "bf16"),
    (1, (900,), (130,), False, "bf16"),
    (17, (40, 20), (40, 20), True, "fp16"),
    (1, tuple((37 * i) % 150 for i in range(70)), tuple((53 * i) % 140 for i in range(70)), True, "bf16"),  # many sequences
    (2, tuple(i % 4 for i in range(1100)), tuple(i % 3 for i in range(1100)), False, "fp16"),
    (1, (0,) * 40 + (300,) + (0,) * 40, (7,) * 40 + (400,) + (0,) * 40, True, "bf16"),
]


def make(case, seed=3):
    h, nq, nk, causal, dt = case
    t = L.DTYPES[dt]
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(nq), sum(nk)
    q = torch.randn((tq, h, L.KEY + 8), generator=g).to(t)[..., :L.KEY]
    up = torch.randn((tk, h, 2 * 128), generator=g).to(t)
    kr = torch.randn((tk, L.TOKEN), generator=g).to(t)[:, L.LATENT:]
    gr = torch.randn((tq, h, L.VALUE), generator=g).to(t)
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32) for n in (nq, nk)]
    return q, up[..., :128], kr, up[..., 128:], gr, cu


def on_gpu(t):
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


def call(q, kn, kr, v, cu, case, **kw):
    return (on_gpu(q), on_gpu(kn), on_gpu(kr), on_gpu(v)), (cu[0].cuda(), cu[1].cuda(), max(case[1]), max(case[2]))


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c)[:60])
def test_forward_and_gradients(case):
    q, kn, kr, v, gr, cu = make(case)
    causal, half = case[3], R.HALF_STEP[q.dtype]
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=causal)
    f = [L.f64(t) for t in (q, kn, kr, v)]
    want, wlse, absolute, size = L.expanded(*f, cu[0].numpy(), cu[1].numpy(), causal, SCALE)
    bound = L.output_error(want, absolute, size.T, half, 12)
    L.check(o, want, bound, "O")
    L.check(lse, wlse, L.score_error(size, 12) + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(wlse), wlse, 0))), "LSE")

    got = af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=causal)
    ref = L.expanded_grads(*f, L.f64(gr), cu[0].numpy(), cu[1].numpy(), causal, SCALE, half, bound)
    for name, t, like in zip(("dq", "dk_nope", "dk_rope", "dv"), got, (q, kn, kr, v)):
        assert t.shape == like.shape and t.dtype == q.dtype
        L.check(t, *ref[name], name)


def test_the_formula_against_differences():
    """The gradients' formula above, in 64 bits, against differences of the outputs along random directions."""
    case = (2, (20, 7), (30, 7), True, "bf16")
    q, kn, kr, v, gr, cu = make(case)
    f = [L.f64(t) for t in (q, kn, kr, v)]
    cu = [c.numpy() for c in cu]
    ref = L.expanded_grads(*f, L.f64(gr), *cu, True, SCALE, 0.0, np.zeros(gr.shape))
    rng = np.random.default_rng(1)
    for i, name in enumerate(("dq", "dk_nope", "dk_rope", "dv")):
        step = rng.standard_normal(f[i].shape)
        loss = [(L.expanded(*[x + e * step if k == i else x for k, x in enumerate(f)], *cu, True, SCALE)[0] * L.f64(gr)).sum()
                for e in (1e-5, -1e-5)]
        assert abs((loss[0] - loss[1]) / 2e-5 - (ref[name][0] * step).sum()) < 1e-6 * np.abs(ref[name][0] * step).sum()


@gpu
def test_gradients_against_differences():
    """The kernels' gradients along random directions against differences of the outputs in 64 bits."""
    case = (3, (150, 40), (150, 60), True, "fp16")
    q, kn, kr, v, gr, cu = make(case, seed=9)
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=True)
    got = af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=True)
    f, c = [L.f64(t) for t in (q, kn, kr, v)], [x.numpy() for x in cu]
    want, _, absolute, size = L.expanded(*f, *c, True, SCALE)
    ref = L.expanded_grads(*f, L.f64(gr), *c, True, SCALE, 2.0 ** -11, L.output_error(want, absolute, size.T, 2.0 ** -11, 12))
    rng = np.random.default_rng(2)
    for i, name in enumerate(("dq", "dk_nope", "dk_rope", "dv")):
        step = rng.choice([-1.0, 1.0], f[i].shape)
        loss = [(L.expanded(*[x + e * step if k == i else x for k, x in enumerate(f)], *c, True, SCALE)[0] * L.f64(gr)).sum()
                for e in (1e-5, -1e-5)]
        diff = (loss[0] - loss[1]) / 2e-5
        # each value within its bound, in whichever direction
        assert abs((L.f64(got[i]) * step).sum() - diff) <= ref[name][1].sum() + 1e-6 * np.abs(ref[name][0]).sum()


@gpu
def test_equal_calls_give_equal_bits():
    case = (6, (700, 33), (700, 33), True, "bf16")
    q, kn, kr, v, gr, cu = make(case)
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=True)
    a, b = (af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=True) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("causal", [False, True])
def test_many_calls_in_a_row(causal):
    """Small calls queued behind one another, whose warps run at uneven paces: no wait gives up, and all give equal bits."""
    case = (4, (320,), (1024,), causal, "fp16")
    q, kn, kr, v, gr, cu = make(case)
    ins, packed = call(q, kn, kr, v, cu, case)
    gr = on_gpu(gr)
    binding.status_clear()
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=causal)
    first = af.attn_bwd_latent(*ins, o, gr, lse, *packed, causal=causal)
    for _ in range(200):
        got = [af.attn_bwd_latent(*ins, o, gr, lse, *packed, causal=causal) for _ in range(20)]
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, first))
    assert binding.status()[0] == 0


@gpu
def test_given_outputs_between_one_another():
    """o and the gradients into views of larger tensors; nothing else of those is written."""
    case = (4, (130, 3), (200, 3), True, "bf16")
    q, kn, kr, v, gr, cu = make(case, seed=17)
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=True)
    plain = af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=True)
    t = dict(dtype=q.dtype, device="cuda")
    wide = torch.full((133, 4, 160), 5.0, **t)
    l2 = torch.empty_like(lse)
    o2, got = af.attn_fwd_latent(*ins, *packed, causal=True, o=wide[..., 16:144], lse=l2)
    assert got is l2 and torch.equal(o2, o) and torch.equal(l2, lse) and (wide[..., :16] == 5).all() and (wide[..., 144:] == 5).all()
    dup, dc, dq = torch.full((203, 4, 264), 5.0, **t), torch.full((203, 576), 5.0, **t), torch.full((133, 5, 192), 5.0, **t)
    ws = torch.empty(af.bwd_latent_workspace_bytes(4, 133, 203), dtype=torch.uint8, device="cuda")
    out = af.attn_bwd_latent(*ins, o2, on_gpu(gr), lse, *packed, causal=True, dq=dq[:, :4], dk_nope=dup[..., :128],
                             dk_rope=dc[:, 512:], dv=dup[..., 128:256], workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(out, plain))
    assert (dup[..., 256:] == 5).all() and (dc[:, :512] == 5).all() and (dq[:, 4] == 5).all()


@gpu
def test_sequences_outside_the_totals_are_left():
    """A sequence whose offsets are no part of the tensors is skipped, its neighbours are not."""
    case = (2, (60, 50), (60, 50), True, "bf16")
    q, kn, kr, v, gr, cu = make(case, seed=23)
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=True)
    good = af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=True)
    bad = [torch.tensor([0, 60, 110, 200], dtype=torch.int32, device="cuda")] * 2
    o2, l2 = torch.full_like(o, 3.0), torch.full_like(lse, 3.0)
    af.attn_fwd_latent(*ins, *bad, 60, 60, causal=True, o=o2, lse=l2)
    assert torch.equal(o2, o) and torch.equal(l2, lse)
    out = af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *bad, 60, 60, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(out, good))
    none = [torch.tensor([0, 60, -5], dtype=torch.int32, device="cuda")] * 2
    o2, l2 = torch.full_like(o, 3.0), torch.full_like(lse, 3.0)
    af.attn_fwd_latent(*ins, *none, 60, 60, causal=True, o=o2, lse=l2)
    assert torch.equal(o2[:60], o[:60]) and (o2[60:] == 3).all() and (l2[:, 60:] == 3).all()


@gpu
@pytest.mark.parametrize("nq,nk", [((5, 200), (0, 0)), ((0, 0), (5, 200))], ids=["no keys", "no queries"])
def test_nothing_on_one_side(nq, nk):
    """No keys in any sequence: outputs and gradients of the queries are zero; no queries: those of the keys."""
    case = (2, nq, nk, True, "bf16")
    q, kn, kr, v, gr, cu = make(case, seed=25)
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = torch.full(gr.shape, 3.0, dtype=q.dtype, device="cuda"), torch.full((2, sum(nq)), 3.0, device="cuda")
    af.attn_fwd_latent(*ins, *packed, causal=True, o=o, lse=lse)
    assert (o == 0).all() and torch.isneginf(lse).all()
    out = [torch.full(t.shape, 3.0, dtype=q.dtype, device="cuda") for t in (q, kn, kr, v)]
    af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=True, dq=out[0], dk_nope=out[1], dk_rope=out[2], dv=out[3])
    assert all((t == 0).all() for t in out)


@gpu
@pytest.mark.parametrize("scale", [2.0, -0.5, 0.0])
def test_scales(scale):
    case = (2, (200,), (200,), True, "fp16")
    q, kn, kr, v, gr, cu = make(case, seed=29)
    ins, packed = call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=True, scale=scale)
    f, c = [L.f64(t) for t in (q, kn, kr, v)], [x.numpy() for x in cu]
    want, wlse, absolute, size = L.expanded(*f, *c, True, scale)
    bound = L.output_error(want, absolute, size.T, 2.0 ** -11, 12)
    L.check(o, want, bound, "O")
    L.check(lse, wlse, L.score_error(size, 12) + 2.0 ** -20 * (1 + np.abs(wlse)), "LSE")
    got = af.attn_bwd_latent(*ins, o, on_gpu(gr), lse, *packed, causal=True, scale=scale)
    ref = L.expanded_grads(*f, L.f64(gr), *c, True, scale, 2.0 ** -11, bound)
    for name, t in zip(ref, got):
        L.check(t, *ref[name], name)


@gpu
def test_what_lies_behind_a_sequence():
    """NaN in the next sequence's tokens, which a tile brings along, reaches nothing of this one's."""
    case = (2, (70, 60), (90, 60), True, "bf16")
    q, kn, kr, v, gr, cu = make(case, seed=37)
    res = []
    for bad in (False, True):
        ins, packed = call(q, kn, kr, v, cu, case)
        g = on_gpu(gr)
        if bad:
            for t in (*ins[1:], ):
                t[90:] = float("nan")
            ins[0][70:] = float("nan")
            g[70:] = float("inf")
        o, lse = af.attn_fwd_latent(*ins, *packed, causal=True)
        d = af.attn_bwd_latent(*ins, o, g, lse, *packed, causal=True)
        res.append((o[:70], lse[:, :70], d[0][:70], d[1][:90], d[2][:90], d[3][:90]))
    assert all(torch.equal(x, y) and x.isfinite().all() for x, y in zip(*res))


# ------------------------------------------------------------------ refusals, on the CPU (no call here reaches a launch)

I2 = ctypes.c_int64 * 2
AT = {n: i << 28 for i, n in enumerate(("q", "kn", "kr", "v", "o", "g", "lse", "dq", "dkn", "dkr", "dv", "cu", "ws"), 1)}


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


def fwd(lib, **kw):
    a = dict(AT, qs=(2 * 192, 192), ks=(2 * 128, 128), rs=64, vs=(2 * 128, 128), os=(2 * 128, 128), batch=1, h=2, tq=10, tk=12, mq=10,
             mk=12, scale=0.1, dt=1, cuk=AT["cu"])
    a.update(kw)
    return lib.attn_fwd_latent(a["q"], a["kn"], a["kr"], a["v"], a["o"], a["lse"], a["cu"], a["cuk"], I2(*a["qs"]), I2(*a["ks"]), a["rs"],
                               I2(*a["vs"]), I2(*a["os"]), a["batch"], a["h"], a["tq"], a["tk"], a["mq"], a["mk"], 1, a["scale"], a["dt"],
                               None)


BAD = [
    (dict(q=None), -1), (dict(kn=None), -1), (dict(kr=None), -1), (dict(v=None), -1), (dict(cu=None), -1),
    (dict(q=AT["q"] + 8), -6), (dict(v=AT["v"] + 2), -6), (dict(lse=AT["lse"] + 2), -6), (dict(cu=AT["cu"] + 1), -6),
    (dict(batch=-1), -2), (dict(h=-1), -2), (dict(tq=-1), -2), (dict(mq=11), -2), (dict(mk=13), -2), (dict(tq=1 << 31, mq=1), -2),
    (dict(dt=5), -4), (dict(scale=float("nan")), -5), (dict(batch=1 << 28), -2), (dict(batch=1 << 20, h=1 << 11), -2),
]


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(o=None), -1), (dict(o=AT["o"] + 8), -6), (dict(qs=(0, 192)), -6), (dict(ks=(256, -128)), -6), (dict(rs=63), -6),
    (dict(os=(2 * 128, 120)), -2), (dict(os=(128, 128)), -2), (dict(o=AT["q"] + 16), -2), (dict(o=AT["kr"] - 32), -2),
], ids=str)
def test_forward_refused(lib, kw, code):
    assert fwd(lib, **kw) == code, lib.attn_last_error()
    assert lib.attn_last_error()


def bwd(lib, **kw):
    a = dict(AT, batch=1, h=2, tq=10, tk=12, mq=10, mk=12, scale=0.1, dt=1, bytes=1 << 30, st=None)
    a.update(kw)
    st = {"q": (384, 192), "kn": (256, 128), "kr": (64, 0), "v": (256, 128), "o": (256, 128), "g": (256, 128), "dq": (384, 192),
          "dkn": (256, 128), "dkr": (64, 0), "dv": (256, 128)}
    st.update(a["st"] or {})
    flat = (ctypes.c_int64 * 20)(*[x for pair in st.values() for x in pair])
    return lib.attn_bwd_latent(a["q"], a["kn"], a["kr"], a["v"], a["o"], a["g"], a["lse"], a["dq"], a["dkn"], a["dkr"], a["dv"], a["cu"],
                               a["cu"], flat, a["batch"], a["h"], a["tq"], a["tk"], a["mq"], a["mk"], 1, a["scale"], a["dt"], a["ws"],
                               a["bytes"], None)


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(o=None), -1), (dict(g=None), -1), (dict(lse=None), -1), (dict(dq=None), -1), (dict(dkr=None), -1), (dict(ws=None), -1),
    (dict(ws=AT["ws"] + 8), -6), (dict(bytes=64), -2), (dict(dv=AT["dkn"]), -2), (dict(dv=AT["dkn"] + 64), -2), (dict(dq=AT["q"]), -2),
    (dict(dkr=AT["dq"] + 16), -2), (dict(st={"dv": (256, 64)}), -2), (dict(st={"dkr": (32, 0)}), -2), (dict(st={"g": (256, 0)}), -6),
    (dict(dv=AT["dkn"] + 256, st={"dkn": (512, 256), "dv": (512, 128)}), -2),
], ids=str)
def test_backward_refused(lib, kw, code):
    assert bwd(lib, **kw) == code, lib.attn_last_error()
    assert lib.attn_last_error()


def test_parts_of_one_gradient_are_apart(lib):
    """dk_nope and dv as the halves of one tensor's rows are no overlap: what is refused then is the lack of a GPU, if anything."""
    if torch.cuda.is_available():
        pytest.skip("the call would run")
    rc = bwd(lib, dv=AT["dkn"] + 256, st={"dkn": (512, 256), "dv": (512, 256)})
    assert rc in (-7, -8), lib.attn_last_error()


@pytest.mark.parametrize("kw", [dict(batch=0), dict(h=0), dict(mq=0, tq=0)], ids=str)
def test_nothing_to_do(lib, kw):
    assert fwd(lib, q=None, kn=None, v=None, o=None, **kw) == 0
    if "mq" not in kw:
        assert bwd(lib, q=None, kn=None, v=None, dq=None, ws=None, **kw) == 0


def test_workspace(lib):
    assert lib.attn_bwd_latent_workspace_bytes(3, 100, 77) == 1280 + 3 * 77 * 64 * 4
    assert lib.attn_bwd_latent_workspace_bytes(-1, 1, 1) == -2


def test_binding_refuses_on_the_host():
    q, kn = torch.zeros(4, 2, 192, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    kr, cu = torch.zeros(4, 64, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    for args in [(q, kn, kr, kn), (q[..., :128], kn, kr, kn), (q.float(), kn, kr, kn), (q, kn, None, kn)]:
        with pytest.raises(af.AttnError):
            af.attn_fwd_latent(*args, cu, cu, 4, 4)
