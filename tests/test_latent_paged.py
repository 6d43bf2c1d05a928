"""Attention over the paged cache of latent attention (absorbed form) against
its definition in 64 bits, and its refusals."""
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

# b, h, sq, page, pages, cached lengths, mask, type
CASES = [
    (1, 1, 1, 16, 1, (1,), "none", "bf16"),
    (1, 16, 1, 64, 4, (200,), "causal", "bf16"),
    (3, 16, 1, 128, 3, (0, 1, 384), "causal", "fp16"),             # nothing cached, one, all of it
    (2, 5, 1, 16, 30, (127, 129), "none", "fp16"),                 # rows that do not fill a tile, pages inside one
    (4, 16, 1, 256, 12, (3000, 17, 128, 1279), "none", "bf16"),    # shared between CTAs, and not
    (2, 32, 1, 48, 11, (500, 260), "causal", "bf16"),
    (2, 24, 1, 32, 9, (280, 31), "none", "fp16"),
    (1, 128, 1, 64, 20, (1275,), "causal", "bf16"),                # two tiles of rows
    (3, 128, 1, 128, 8, (1024, 3, 700), "causal", "fp16"),
    (2, 48, 3, 64, 10, (600, 1), "causal", "bf16"),                # three tiles; queries that see nothing
    (2, 40, 1, 64, 4, (250, 128), "none", "bf16"),                 # one tile of 64 with rows to spare
    (1, 16, 5, 64, 5, (260,), "causal", "bf16"),
    (2, 3, 37, 16, 16, (250, 20), "causal", "fp16"),               # fewer keys than queries
    (1, 20, 33, 128, 3, (300,), "causal", "bf16"),                 # many tiles
    (1, 128, 20, 128, 4, (509,), "none", "fp16"),
    (2, 8, 7, 64, 6, (380, 7), "tree", "bf16"),
    (3, 16, 13, 128, 3, (300, 13, 129), "tree", "fp16"),
    (2, 4, 70, 32, 10, (300, 70), "tree", "bf16"),                 # three words of bits
    (1, 16, 4, 64, 2, (3,), "tree", "bf16"),                       # fewer keys than drafted
    (1, 128, 3, 64, 5, (300,), "tree", "bf16"),
    (2, 64, 11, 64, 6, (300, 384), "causal", "fp16"),              # a team of eleven
    (1, 64, 13, 128, 3, (384,), "tree", "bf16"),                   # thirteen tiles
    (40, 2, 1, 16, 9, tuple(range(3, 123, 3)), "causal", "bf16"),  # more requests than a warp has lanes
    (70, 1, 1, 16, 20, tuple((91 * i) % 321 for i in range(70)), "none", "fp16"),  # and than two for each lane
]


def make(case, seed=11):
    b, h, sq, page, pages, lens, mask, dt = case
    t = L.DTYPES[dt]
    pool, table = L.cache(b, page, pages, t, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((b, sq, h, L.TOKEN), generator=g).to(t).transpose(1, 2)
    tree = L.random_tree(b, sq, seed + 2) if mask == "tree" else None
    return q, pool, torch.tensor(lens, dtype=torch.int32), table, tree


def on_gpu(t):
    return None if t is None else torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


def compare(o, lse, q, pool, lens, table, causal, tree, scale=SCALE):
    ref = L.paged_attend(L.f64(q), L.f64(pool), lens.numpy(), table.numpy(), scale, causal,
                         None if tree is None else tree.numpy().view(np.uint32))
    want, wlse, absolute, size = ref
    L.check(o, want, L.output_error(want, absolute, size, R.HALF_STEP[q.dtype], L.TOKEN // 16), "O")
    L.check(lse, wlse, L.score_error(size, L.TOKEN // 16) + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(wlse), wlse, 0))), "LSE")


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_matches_the_definition(case):
    q, pool, lens, table, tree = make(case)
    causal = case[6] == "causal"
    o, lse = af.attn_fwd_latent_paged(on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), SCALE, causal=causal, tree=on_gpu(tree))
    assert o.shape == (*q.shape[:3], L.LATENT) and o.dtype == q.dtype
    compare(o, lse, q, pool, lens, table, causal, tree)


@gpu
@pytest.mark.parametrize("h,sq,mask", [(16, 1, "none"), (32, 3, "causal"), (64, 4, "tree"), (3, 9, "tree"), (128, 2, "causal")])
def test_what_is_not_seen_does_not_reach_a_row(h, sq, mask):
    """NaN and infinities behind the length, and at drafted or later tokens for the rows that do not see them; a row that
    sees one has NaN."""
    lens = (200, sq, 128 + sq // 2)
    q, pool, lens, table, tree = make((3, h, sq, 64, 4, lens, mask, "bf16"), seed=31)
    pool = pool.clone()
    bad = [float("nan"), float("inf"), float("-inf")]
    clean = pool.clone()
    for e in range(3):
        n = int(lens[e])
        for j in range(n, 256):
            pool[table[e, j // 64].long(), j % 64, ::7] = bad[j % 3]
        if sq > 1:  # the last token but one: hidden from some rows
            j = n - 1
            pool[table[e, j // 64].long(), j % 64, 3] = bad[0]
    args = (lens.cuda(), table.cuda(), SCALE)
    o, lse = af.attn_fwd_latent_paged(on_gpu(q), pool.cuda(), *args, causal=mask == "causal", tree=on_gpu(tree))
    ref, rlse = af.attn_fwd_latent_paged(on_gpu(q), clean.cuda(), *args, causal=mask == "causal", tree=on_gpu(tree))
    for e in range(3):
        seen = L.visible(sq, int(lens[e]), mask == "causal", None if tree is None else tree[e].numpy().view(np.uint32))
        hit = torch.from_numpy(seen[:, int(lens[e]) - 1]) if sq > 1 else torch.zeros(sq, dtype=torch.bool)
        assert torch.equal(o[e][:, ~hit], ref[e][:, ~hit]) and torch.equal(lse[e][:, ~hit], rlse[e][:, ~hit])
        assert o[e][:, hit].isnan().all()
        assert ref[e].isfinite().all()


@gpu
def test_pages_outside_the_pool_read_as_zeros():
    q, pool, lens, table, _ = make((2, 16, 1, 32, 8, (250, 100), "none", "bf16"), seed=41)
    table[0, 2], table[1, 0] = -1, pool.shape[0]
    o, lse = af.attn_fwd_latent_paged(on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), SCALE)
    compare(o, lse, q, pool, lens, table, False, None)


@gpu
def test_scores_of_every_size():
    """Scores that grow along the cache raise the reference tile after tile; a large negative scale; a scale of zero."""
    q, pool, lens, table, _ = make((2, 16, 2, 64, 16, (1000, 513), "causal", "fp16"), seed=51)
    pool = (pool.float() * 0.05).half()
    for e in range(2):
        for pg in range(16):
            pool[table[e, pg].long()] *= 1.0 + pg
    for scale in (3.0, -2.0, 0.0):
        o, lse = af.attn_fwd_latent_paged(on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), scale, causal=True)
        compare(o, lse, q, pool, lens, table, True, None, scale)


@gpu
def test_empty_rows_of_a_tree():
    q, pool, lens, table, tree = make((1, 4, 3, 16, 1, (3,), "tree", "bf16"), seed=61)
    tree.zero_()
    o, lse = af.attn_fwd_latent_paged(on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), SCALE, tree=on_gpu(tree))
    assert (o == 0).all() and torch.isneginf(lse).all()


@gpu
def test_given_outputs_and_strides():
    q, pool, lens, table, _ = make((2, 16, 3, 64, 4, (200, 129), "causal", "bf16"), seed=71)
    whole = torch.full((2, 3, 16, L.LATENT + 64), 7.0, dtype=q.dtype, device="cuda")
    o = whole[..., :L.LATENT].transpose(1, 2)
    lse = torch.empty(2, 16, 3, device="cuda")
    ws = torch.empty(af.latent_paged_workspace_bytes(2, 16, 3), dtype=torch.uint8, device="cuda")
    wide = torch.zeros(2, 16, 5, L.TOKEN + 64, dtype=q.dtype, device="cuda")
    wide[:, :, 1:4, :L.TOKEN] = on_gpu(q)
    got, got_lse = af.attn_fwd_latent_paged(wide[:, :, 1:4, :L.TOKEN], pool.cuda(), lens.cuda(), table.cuda(), SCALE,
                                            causal=True, o=o, lse=lse, workspace=ws)
    assert got is o and got_lse is lse and (whole[..., L.LATENT:] == 7.0).all()
    compare(o, lse, q, pool, lens, table, True, None)


# ------------------------------------------------------------------ refusals, on the CPU (no call here reaches a launch)

S3 = ctypes.c_int64 * 3
Q, POOL, O, REST = (i << 24 for i in range(1, 5))


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


def call(lib, q=Q, pool=POOL, lens=REST, table=REST, tree=None, o=O, lse=None, qst=(576 * 4, 576, 576), ost=(512 * 4, 512, 512),
         b=2, h=4, sq=1, pages=4, page=32, per=2, causal=0, scale=0.1, dt=1, ws=REST, ws_bytes=1 << 40):
    return lib.attn_fwd_latent_paged(q, pool, lens, table, tree, o, lse, S3(*qst), S3(*ost), b, h, sq, pages, page, per, causal,
                                     scale, dt, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(pool=None), -1), (dict(lens=None), -1), (dict(table=None), -1), (dict(o=None), -1),
    (dict(ws=None), -1), (dict(ws_bytes=100), -2), (dict(ws=REST + 8), -6), (dict(page=40), -2), (dict(b=-1), -2),
    (dict(sq=1 << 30, h=64), -2), (dict(scale=float("inf")), -5), (dict(dt=2), -4), (dict(q=Q + 4), -6), (dict(o=O + 8), -6),
    (dict(lse=REST + 2), -6), (dict(tree=REST + 1), -6), (dict(tree=REST, causal=1), -2), (dict(qst=(576 * 4, 576, 580)), -6),
    (dict(ost=(512 * 4, 504, 512)), -2), (dict(ost=(0, 512, 512)), -2), (dict(o=Q + 64), -2), (dict(o=POOL + 64), -2),
    (dict(o=Q - 512), -2),
], ids=str)
def test_refused(lib, kw, code):
    assert call(lib, **kw) == code, lib.attn_last_error()
    assert lib.attn_last_error()


@pytest.mark.parametrize("kw", [dict(b=0), dict(h=0), dict(sq=0)], ids=str)
def test_nothing_to_do(lib, kw):
    assert call(lib, q=None, o=None, ws=None, **kw) == 0


def test_workspace(lib):
    part = 2 * 160 * (512 * 4 + 16)
    for h, sq, tile in [(1, 1, 16), (16, 1, 16), (17, 1, 32), (8, 4, 32), (33, 1, 64), (128, 500, 64)]:
        assert lib.attn_fwd_latent_paged_workspace_bytes(3, h, sq) == part * tile + 160 * 16
    assert lib.attn_fwd_latent_paged_workspace_bytes(1, -1, 1) == -2


def test_binding_refuses_on_the_host():
    q = torch.zeros(1, 4, 1, L.TOKEN, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, L.TOKEN, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for args in [(q, pool, i, i[None], 0.1), (q[..., :512], pool, i, i[None], 0.1), (q.float(), pool, i, i[None], 0.1)]:
        with pytest.raises(af.AttnError):
            af.attn_fwd_latent_paged(*args)
