"""Refusals of the q/k norm (on the CPU; no call here reaches a launch):
outputs whose rows coincide, or that are the other side's memory."""
import ctypes

import pytest

from attention_forward_14_gb300 import binding

S3 = ctypes.c_int64 * 3
Q, K, QO, KO, W, DW, GQ, GK = (i << 24 for i in range(1, 9))
B, H, HKV, S, D = 2, 4, 2, 8, 64
DENSE = {"q": (H * S * D, S * D, D), "k": (HKV * S * D, S * D, D)}


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


def forward(lib, q=Q, k=K, q_out=QO, k_out=KO, os=DENSE["q"], dtype=1, b=B, s=S):
    return lib.attn_qk_norm_rope(q, k, W, W, None, None, None, q_out, k_out, S3(*DENSE["q"]), S3(*DENSE["k"]), S3(*os),
                                 S3(*DENSE["k"]), b, H, HKV, s, D, 0, 0, 0, 0, 1e-6, dtype, None)


@pytest.mark.parametrize("os", [
    (H * S * D, D, D),            # heads and tokens with one stride
    (S * D, S * D, D),            # batch elements and heads
    (H * S * D, 2 * D, D),        # a head's rows run into the next one's
    (D, B * D, D),
    (H * S * D, S * D, D - 8),    # shorter than a row
    (2 * D, H * S * D, D),
    (1 << 46, 1 << 46, 1 << 46),
])
def test_rows_of_an_output_that_coincide(lib, os):
    assert forward(lib, os=os) == -2 and b"overlap" in lib.attn_last_error()


@pytest.mark.parametrize("kw", [dict(q_out=K), dict(k_out=Q), dict(k_out=QO), dict(q_out=KO)], ids=str)
def test_an_output_that_is_the_other_sides_memory(lib, kw):
    assert forward(lib, **kw) == -2 and lib.attn_last_error()


@pytest.mark.parametrize("kw", [dict(dq=K), dict(dk=Q), dict(dk=QO), dict(dq=GK), dict(dk=GQ)], ids=str)
def test_a_gradient_that_is_the_other_sides_memory(lib, kw):
    a = dict(dq=QO, dk=KO)
    a.update(kw)
    st, need = [S3(*DENSE[n]) for n in "qkqkqk"], lib.attn_qk_norm_rope_bwd_workspace_bytes(D)
    rc = lib.attn_qk_norm_rope_bwd(GQ, GK, Q, K, W, W, None, None, None, a["dq"], a["dk"], DW, DW + 1024, *st, B, H, HKV, S, D,
                                   0, 0, 0, 0, 1e-6, 1, W, need, None)
    assert rc == -2 and lib.attn_last_error()
