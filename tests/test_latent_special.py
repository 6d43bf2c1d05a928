"""Attention over the paged cache of latent attention where values are not
finite: keys that some rows of a tile see and a mask hides from others, and
what the formula makes of them."""
import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
import latent_ref as L
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
