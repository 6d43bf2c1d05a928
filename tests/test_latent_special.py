"""Attention over the paged cache of latent attention where values are not
finite: keys that some rows of a tile see and a mask hides from others, and
what the formula makes of them."""
import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
import latent_ref as L
import ops_ref as R
import test_latent_paged as P

gpu = pytest.mark.gpu
SCALE = P.SCALE

# h, sq, mask: tiles of 16, 32 and 64 rows, and several of 64
SHAPES = [(4, 3, "causal"), (3, 5, "tree"), (8, 4, "causal"), (5, 6, "tree"), (16, 4, "causal"), (32, 3, "causal"), (32, 3, "tree"),
          (13, 30, "tree"), (1, 64, "causal")]
# of each pair of panels of the latent, its first panel and its second, and of the key part
COLUMNS = (3, 100, 130, 255, 300, 340, 384, 447, 511, 512, 575)


def planted(shape, dt, columns, value, seed):
    """Lengths with several whole tiles before the last one, and `value` in the columns of a token that some rows see:
    (arguments of a call, the pool without it, which rows see it [b, sq])."""
    h, sq, mask = shape
    lens = (700, 130 + sq, 512 + sq // 2)
    q, pool, lens, table, tree = P.make((3, h, sq, 64, 12, lens, mask, dt), seed)
    clean, hit = pool.clone(), []
    for e in range(3):
        j = int(lens[e]) - 1 - (seed + e) % min(sq, 3)
        pool[table[e, j // 64].long(), j % 64, list(columns)] = value
        seen = L.visible(sq, int(lens[e]), mask == "causal", None if tree is None else tree[e].numpy().view(np.uint32))
        hit.append(torch.from_numpy(seen[:, j]))
    return (q, pool, lens, table, tree), clean, torch.stack(hit)


def run(q, pool, lens, table, tree, mask):
    return af.attn_fwd_latent_paged(P.on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), SCALE, causal=mask == "causal",
                                    tree=P.on_gpu(tree))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_nan_reaches_the_rows_that_see_it_and_no_other(shape, dt):
    """In one column at a time: its rows have NaN, whichever products of the scores come last, the others their bits."""
    for i, col in enumerate(COLUMNS * 3):
        (q, pool, lens, table, tree), clean, hit = planted(shape, dt, (col,), float("nan"), seed=100 + i % 3)
        assert hit.any() and not hit.all()
        o, lse = (t.cpu() for t in run(q, pool, lens, table, tree, shape[2]))
        ref, rlse = (t.cpu() for t in run(q, clean, lens, table, tree, shape[2]))
        rows = hit[:, None].expand(-1, shape[0], -1)
        assert o[rows].isnan().all() and lse[rows].isnan().all(), f"column {col}"
        assert torch.equal(o[~rows], ref[~rows]) and torch.equal(lse[~rows], rlse[~rows]), f"column {col}"
        assert ref.isfinite().all()


def by_definition(q, c, seen):
    """One query: q [576], c [n, 576], seen [n], of which some may not be finite: O, LSE, the sum of P |v| of finite values
    and the largest scale sum |q k|."""
    c = c[seen]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = SCALE * (c * q).sum(1)
        m = s.max(initial=-np.inf)
        if m == -np.inf:  # nothing is seen, or nothing but scores of -infinity
            return np.zeros(L.LATENT), m, np.zeros(L.LATENT), 0.0
        p = np.exp(s - m)
        o, lse = (p[:, None] * c[:, :L.LATENT]).sum(0) / p.sum(), m + np.log(p.sum())
    fin = np.where(np.isfinite(c), np.abs(c), 0.0)
    return o, lse, np.nan_to_num(p) @ fin[:, :L.LATENT] / max(np.nan_to_num(p).sum(), 1e-300), SCALE * (fin @ np.abs(q)).max()


# b, h, sq, lengths, mask, whether the tiles in which the tokens stand are seen whole by all rows
INFINITE = [
    (3, 4, 3, (700, 133, 513), "causal", False),
    (3, 3, 5, (700, 135, 514), "tree", False),
    (2, 8, 4, (300, 260), "causal", False),
    (2, 32, 2, (300, 260), "causal", False),
    (2, 13, 10, (300, 260), "tree", False),
    (3, 16, 2, (700, 384, 513), "none", True),
    (2, 32, 2, (300, 260), "causal", True),
    (200, 2, 3, tuple(3 + (7 * i) % 60 for i in range(200)), "causal", False),  # more items than teams: most are not cut
    (200, 33, 1, tuple(2 + (7 * i) % 60 for i in range(200)), "causal", False),
    (2, 5, 2, (1, 2), "causal", False),
]


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", INFINITE, ids=lambda c: str(c)[:60])
def test_infinities_act_as_the_formula_has_it(case, dt):
    """Infinite values, of either sign, in tokens that some rows see: NaN where the score is +infinity or NaN, and where it
    is -infinity NaN in the values' own places alone, in whole tiles and in those that a mask or the length cuts."""
    b, h, sq, lens, mask, whole = case
    q, pool, lens, table, tree = P.make((b, h, sq, 64, 12 if max(lens) > 64 else 1, lens, mask, dt), seed=211)
    for e in range(b):
        n = int(lens[e])
        for i, columns in enumerate([(3,), (140, 200), (300, 511, 575), (384,)][:1 if n < 100 else 4]):
            j = (5 + 9 * i if whole else max(n - 1 - (e + i) % min(sq, 3), 0))
            if whole or i == e % 4 or n < 100:
                pool[table[e, j // 64].long(), j % 64, list(columns)] = float("inf") * (-1) ** (e + i)
    o, lse = (L.f64(t) for t in run(q, pool, lens, table, tree, mask))
    fq, fp, half = L.f64(q), L.f64(pool), R.HALF_STEP[q.dtype]
    alone = 0
    for e in range(b):
        n = int(lens[e])
        c = np.concatenate([fp[int(p)] for p in table[e]])[:n]
        seen = L.visible(sq, n, mask == "causal", None if tree is None else tree[e].numpy().view(np.uint32))
        for i in range(sq):
            for k in range(h):
                want, wlse, absolute, size = by_definition(fq[e, k, i], c, seen[i])
                assert np.array_equal(np.isnan(o[e, k, i]), np.isnan(want)), f"{e} {k} {i}"
                assert np.isnan(lse[e, k, i]) == np.isnan(wlse)
                if np.isnan(wlse):
                    continue
                alone += np.isnan(want).any()
                fin = ~np.isnan(want)
                bound = L.output_error(want, absolute, np.array(size), half, L.TOKEN // 16)
                L.check(torch.from_numpy(o[e, k, i][fin]), want[fin], bound[fin], f"O {e} {k} {i}")
                assert lse[e, k, i] == wlse or abs(lse[e, k, i] - wlse) <= L.score_error(size, L.TOKEN // 16) + 2.0 ** -20 * (1 + abs(wlse))
    assert alone > 0 or case[3] == (1, 2)  # rows with NaN in some places


@gpu
@pytest.mark.parametrize("h,sq", [(1, 1), (4, 1), (8, 1), (2, 4), (17, 1), (16, 1), (3, 11), (33, 1), (32, 1), (40, 2), (65, 1)])
@pytest.mark.parametrize("mask", ["none", "causal", "tree"])
def test_halves_of_a_tile_past_the_last_row(h, sq, mask):
    """Rows that do not fill the first half of a tile, just fill it, or begin the second."""
    q, pool, lens, table, tree = P.make((3, h, sq, 64, 4, (sq, 131, 250), mask, "bf16"), seed=71)
    o, lse = run(q, pool, lens, table, tree, mask)
    P.compare(o, lse, q, pool, lens, table, mask == "causal", tree)
