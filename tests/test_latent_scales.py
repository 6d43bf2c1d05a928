"""The expanded form of latent attention, its gradients and the attention over
the cache with scales next to zero, and their signs, against the definitions
in 64 bits."""
import numpy as np
import pytest

import attention_forward_14_gb300 as af
import latent_ref as L
import ops_ref as R
import test_latent_expanded as E
import test_latent_paged as P

gpu = pytest.mark.gpu

# (the products of scores and these scales are far below one: every weight is that of the others)
SCALES = [-1e-31, 1e-31, -5e-31, -1e-36, -1e-30, 1e-30, -0.0]


@gpu
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("causal", [False, True])
def test_expanded(scale, causal):
    case = (2, (200, 1, 130), (200, 70, 300), causal, "fp16")  # tiles with masks, and with a remainder
    q, kn, kr, v, gr, cu = E.make(case, seed=29)
    ins, packed = E.call(q, kn, kr, v, cu, case)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=causal, scale=scale)
    f, c, half = [L.f64(t) for t in (q, kn, kr, v)], [x.numpy() for x in cu], R.HALF_STEP[q.dtype]
    want, wlse, absolute, size = L.expanded(*f, *c, causal, scale)
    bound = L.output_error(want, absolute, size.T, half, 12)
    L.check(o, want, bound, "O")
    L.check(lse, wlse, L.score_error(size, 12) + 2.0 ** -20 * (1 + np.abs(wlse)), "LSE")
    got = af.attn_bwd_latent(*ins, o, E.on_gpu(gr), lse, *packed, causal=causal, scale=scale)
    ref = L.expanded_grads(*f, L.f64(gr), *c, causal, scale, half, bound)
    for name, t in zip(ref, got):
        L.check(t, *ref[name], name)


@gpu
@pytest.mark.parametrize("scale", SCALES)
def test_cached(scale):
    q, pool, lens, table, _ = P.make((2, 16, 3, 64, 4, (200, 129), "causal", "fp16"), seed=51)
    o, lse = af.attn_fwd_latent_paged(P.on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), scale, causal=True)
    P.compare(o, lse, q, pool, lens, table, True, None, scale)
