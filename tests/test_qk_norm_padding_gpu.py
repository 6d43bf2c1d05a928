"""The norm of queries and keys of a padded batch, with a rotation and without:
tokens of padding are zeros and take no part in a weight's gradient."""
import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def tokens(t):
    a = R.f64(t)
    return a.transpose(0, 2, 1, 3).reshape(-1, a.shape[1], a.shape[3]) if a.ndim == 4 else a


def close(got, ref, t, rows_of):
    """As for every norm: one rounding to the type, and 2^-19 of the row's
    largest value for a dozen fp32 roundings and rsqrt's two ulp."""
    row = np.abs(rows_of).max(-1, keepdims=True)
    assert (np.abs(tokens(got) - ref) <= R.HALF_STEP[t] * np.abs(ref) + 2.0 ** -25 + 2.0 ** -19 * row).all()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_padding_without_tables(packed, weights, d, dtype):
    b, h, hkv, s = 3, 5, 2, 21
    g = torch.Generator().manual_seed(7)
    shape = lambda n: (b * s, n, d) if packed else (b, n, s, d)  # noqa: E731
    q, k, gq, gk = (torch.randn(shape(n), generator=g).to(dtype) for n in (h, hkv, h, hkv))
    w = (torch.rand(d, generator=g) + 0.5).to(dtype) if weights else None
    pos = torch.arange(s, dtype=torch.int32).repeat(b, 1)
    pos[0, 15:], pos[1, 0], pos[2, 5:9] = -1, -(2 ** 31), -7
    pos[2, 20] = 2 ** 31 - 1   # there are no tables for it to lie past
    there = (pos >= 0).numpy().reshape(-1)
    for t in (q, k, gq, gk):   # padding may hold anything
        rows = t if packed else t.transpose(1, 2).reshape(b * s, -1, d)
        rows[~there] = float("nan")
        if not packed:
            t.copy_(rows.view(b, s, -1, d).transpose(1, 2))
    dpos = (pos.reshape(-1) if packed else pos).to(DEV)
    dev = [t.to(DEV) for t in (gq, gk, q, k)]
    dw = None if w is None else w.to(DEV)
    outs = af.attn_qk_norm_rope(dev[2], dev[3], dw, dw, positions=dpos)
    dq, dk, dwq, dwk = af.attn_qk_norm_rope_bwd(*dev, dw, dw, positions=dpos)
    assert af.status()[0] == 0
    for out, dx, got_w, x, up in ((outs[0], dq, dwq, q, gq), (outs[1], dk, dwk, k, gk)):
        x, up = np.nan_to_num(tokens(x)), np.nan_to_num(tokens(up))
        ref = R.norm_rope(x, R.f64(w), None, None, None, 1e-6, False)
        rx, rw = R.norm_rope_bwd(up, x, R.f64(w), None, None, None, 1e-6, False)
        ref[~there] = rx[~there] = 0.0
        close(out, ref, dtype, ref)
        close(dx, rx, dtype, up)
        assert (tokens(out)[~there] == 0).all() and (tokens(dx)[~there] == 0).all()
        assert (got_w is None) == (w is None)
        if w is not None:
            # each term and each partial sum has some ten fp32 roundings
            n = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
            bound = (np.abs(up * n).sum((0, 1)) + 1e-6) * 2.0 ** -24 * 200
            assert (np.abs(R.f64(got_w) - rw) <= bound).all()
