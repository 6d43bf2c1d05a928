"""Append to the paged cache of latent attention against its definition in 64
bits, and its refusals."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import latent_ref as L
import ops_ref as R

gpu = pytest.mark.gpu

# b, s_new, page, pages, cached lengths (one for each element), new lengths or None, norm, rotation, adjacent pairs, type
CASES = [
    (1, 1, 16, 2, (0,), None, True, True, False, "bf16"),
    (3, 1, 64, 2, (63, 64, 127), None, True, True, True, "fp16"),
    (2, 33, 16, 5, (15, 47), None, True, True, False, "fp16"),
    (4, 70, 48, 3, (0, 100, 143, 200), (70, 0, 5, 3), True, True, True, "bf16"),  # past the capacity, none, at its end
    (2, 9, 128, 1, (3, -4), (-1, 100), True, False, False, "bf16"),              # lengths outside their range
    (2, 9, 32, 2, (30, 31), None, False, True, False, "bf16"),
    (2, 9, 32, 2, (30, 31), None, False, False, False, "fp16"),                  # a copy
    (1, 257, 256, 2, (250,), None, True, True, True, "bf16"),
]


def make(case, seed=5):
    b, s, page, pages, lens, news, norm, turn, adjacent, dt = case
    t = L.DTYPES[dt]
    g = torch.Generator().manual_seed(seed)
    pool, table = L.cache(b, page, pages, t, seed + 1)
    x = (3 * torch.randn((b, s + 1, L.TOKEN + 24), generator=g)).to(t)[:, 1:, 8:8 + L.TOKEN]  # strided, offset
    w = (torch.rand(L.LATENT, generator=g) + 0.5).to(t) if norm else None
    cos, sin = R.tables(page * pages, L.ROPE) if turn else (None, None)
    lens = torch.tensor(lens, dtype=torch.int32)
    news = None if news is None else torch.tensor(news, dtype=torch.int32)
    return x, pool, table, w, cos, sin, lens, news, adjacent


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_append(case):
    x, pool, table, w, cos, sin, lens, news, adjacent = make(case)
    n = np.full(x.shape[0], x.shape[1]) if news is None else news.numpy()
    opt = lambda t: None if t is None else L.f64(t)  # noqa: E731
    want, written = L.append(L.f64(x), L.f64(pool), opt(w), opt(cos), opt(sin), lens.numpy(), n, table.numpy(), 1e-6, adjacent)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    xs = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
    got = pool.cuda()
    af.attn_latent_append_paged(xs, got, lens.cuda(), table.cuda(), norm_weight=dev(w), cos=dev(cos), sin=dev(sin),
                                interleaved=adjacent, new_seqlens=dev(news))
    assert torch.equal(got.cpu()[~torch.from_numpy(written)], pool[~torch.from_numpy(written)])  # nothing else
    # fp32: eight products and sums and five sums of halves for the mean, its root, two products: 2^-20; of a rotated
    # value three roundings of what is as large as its pair
    pair = np.abs(want).copy()
    pair[..., L.LATENT:] = 3 * 2 ** 0.5 * np.abs(want[..., L.LATENT:]).max(-1, keepdims=True)
    L.check(got, want, R.HALF_STEP[x.dtype] * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -20 * pair + 2.0 ** -25, "pool")
    if w is None and cos is None:
        assert np.array_equal(L.f64(got), want)


@gpu
def test_pages_outside_the_pool_are_not_written():
    x, pool, table, w, cos, sin, lens, _, _ = make((2, 40, 16, 4, (0, 10), None, True, True, False, "bf16"))
    table[0, 1], table[1, 2] = -1, pool.shape[0]
    got = pool.cuda()
    af.attn_latent_append_paged(x.cuda(), got, lens.cuda(), table.cuda(), norm_weight=w.cuda(), cos=cos.cuda(), sin=sin.cuda())
    _, written = L.append(L.f64(x), L.f64(pool), None, None, None, lens.numpy(), [40, 40], table.numpy(), 0.0, False)
    same = (got.cpu() == pool).all(-1).numpy()
    assert np.array_equal(same, ~written) and written.sum() == 80 - 16 - 16


@gpu
def test_a_row_of_zeros_and_one_with_infinities():
    """mean 0 and eps 0: 0 times infinity, as the formula has it; an infinity among the values: they become 0 or NaN."""
    t = torch.bfloat16
    x = torch.randn(1, 3, L.TOKEN).to(t)
    x[0, 0, :L.LATENT] = 0
    x[0, 1, 5] = float("inf")
    pool = torch.zeros(2, 16, L.TOKEN, dtype=t, device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    w = torch.ones(L.LATENT, dtype=t, device="cuda")
    af.attn_latent_append_paged(x.cuda(), pool, none, table, norm_weight=w, eps=1e-6)
    got = pool[1, :3].float().cpu()
    assert (got[0, :L.LATENT] == 0).all() and got[1, 5].isnan() and (got[1, 6:L.LATENT] == 0).all() and got[2].isfinite().all()
    af.attn_latent_append_paged(x.cuda(), pool, none, table, norm_weight=w, eps=0.0)
    assert pool[1, 0, :L.LATENT].isnan().all()


# ------------------------------------------------------------------ refusals, on the CPU (no call here reaches a launch)

S3 = ctypes.c_int64 * 3
NEW, POOL, WEIGHT, REST = (i << 20 for i in range(1, 5))


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


def call(lib, new=NEW, pool=POOL, w=WEIGHT, lens=REST, news=None, table=REST, cos=REST, sin=REST, st=(1152, 0, 576), b=2,
         s=2, pages=4, page=32, per=2, length=64, eps=1e-6, dt=1):
    return lib.attn_latent_append_paged(new, pool, w, lens, news, table, cos, sin, S3(*st), b, s, pages, page, per, length, 0,
                                        eps, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(new=None), -1), (dict(pool=None), -1), (dict(lens=None), -1), (dict(table=None), -1), (dict(cos=None), -1),
    (dict(page=24), -2), (dict(page=0), -2), (dict(b=-1), -2), (dict(s=1 << 31), -2), (dict(length=63), -2),
    (dict(pages=0), -2), (dict(dt=3), -4), (dict(eps=-1.0), -5), (dict(eps=float("nan")), -5), (dict(new=NEW + 8), -6),
    (dict(pool=POOL + 2), -6), (dict(w=WEIGHT + 8), -6), (dict(lens=REST + 2), -6), (dict(st=(1152, 0, 572)), -6),
    (dict(st=(-8, 0, 576)), -6), (dict(new=POOL + 1152), -2), (dict(new=POOL - 1152), -2), (dict(w=POOL + 64), -2),
], ids=str)
def test_refused(lib, kw, code):
    assert call(lib, **kw) == code, lib.attn_last_error()
    assert lib.attn_last_error()


@pytest.mark.parametrize("kw", [dict(b=0), dict(s=0)], ids=str)
def test_nothing_to_do(lib, kw):
    assert call(lib, new=None, pool=None, **kw) == 0


def test_binding_refuses_on_the_host():
    x = torch.zeros(1, 2, L.TOKEN, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, L.TOKEN, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for args in [(x[..., :570], pool, i, i[None]), (x.float(), pool, i, i[None]), (x, pool, i, i[None]),
                 (x, pool[..., :64], i, i[None]), (x, None, i, i[None])]:
        with pytest.raises(af.AttnError):
            af.attn_latent_append_paged(*args)
