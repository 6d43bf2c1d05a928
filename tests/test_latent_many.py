"""Latent attention with more heads than are taken together, and with more
requests than the lanes of a warp look after one at a time."""
import pytest
import torch

import attention_forward_14_gb300 as af
import ops_ref as R
import test_latent_expanded as E
import test_latent_paged as P

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("h,lens,causal,dt", [(70, (8200, 77), True, "bf16"), (33, (8193,), False, "fp16"), (40, (5, 8300), True, "fp16")],
                         ids=str)
def test_groups_of_heads(h, lens, causal, dt):
    """Sequences so long that the heads are taken in groups, the last of them smaller: every head's bits are those of a call
    of its own, and the shared key part's gradient is the sum of theirs."""
    q, kn, kr, v, gr, cu = E.make((h, lens, lens, causal, dt), seed=5)
    ins, packed = E.call(q, kn, kr, v, cu, (h, lens, lens, causal, dt))
    g = E.on_gpu(gr)
    o, lse = af.attn_fwd_latent(*ins, *packed, causal=causal)
    dq, dkn, dkr, dv = af.attn_bwd_latent(*ins, o, g, lse, *packed, causal=causal)
    total, size = (torch.zeros(dkr.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(h):
        at = slice(i, i + 1)
        one = (ins[0][:, at], ins[1][:, at], ins[2], ins[3][:, at])
        o1, lse1 = af.attn_fwd_latent(*one, *packed, causal=causal)
        assert torch.equal(o1, o[:, at]) and torch.equal(lse1, lse[at]), f"head {i}"
        d = af.attn_bwd_latent(*one, o1, g[:, at], lse1, *packed, causal=causal)
        assert torch.equal(d[0], dq[:, at]) and torch.equal(d[1], dkn[:, at]) and torch.equal(d[3], dv[:, at]), f"head {i}"
        total += d[2].double()
        size += d[2].double().abs()
    # each head's part is rounded where it stands alone, all of them once where they are summed, by h sums in fp32; fp16's
    # smallest step, 2^-24, for what is below its normal numbers
    half = R.HALF_STEP[q.dtype]
    bound = half * (size + total.abs()) * (1 + 2.0 ** -7) + h * 2.0 ** -23 * size + (h + 1) * 2.0 ** -25
    assert ((dkr.double() - total).abs() <= bound).all()


@gpu
@pytest.mark.parametrize("case", [
    (1100, 1, 2, 16, 9, tuple((37 * i) % 145 for i in range(1100)), "causal", "bf16"),
    (1030, 24, 1, 16, 9, tuple((91 * i) % 141 + 1 for i in range(1030)), "none", "fp16"),
    (2100, 3, 1, 16, 2, tuple((5 * i) % 33 for i in range(2100)), "causal", "fp16"),
], ids=lambda c: str(c)[:30])
def test_more_than_a_thousand_requests(case):
    q, pool, lens, table, tree = P.make(case)
    o, lse = af.attn_fwd_latent_paged(P.on_gpu(q), pool.cuda(), lens.cuda(), table.cuda(), P.SCALE, causal=case[6] == "causal")
    P.compare(o, lse, q, pool, lens, table, case[6] == "causal", None)
