"""Refusals of the paged append (on the CPU; no call here reaches a launch)."""
import ctypes

import pytest

from attention_forward_14_gb300 import binding

S3 = ctypes.c_int64 * 3
# 4 pages of 32 tokens, one head of 64 values, blocks of 16: pools of 8 KB, scales of 32 bytes, new tokens of 256
K_NEW, V_NEW, K_POOL, V_POOL, K_SCALE, V_SCALE, REST = (i << 20 for i in range(1, 8))
POOL, SCALE, NEW = 4 * 32 * 64, 4 * 2 * 4, 2 * 64 * 2


@pytest.fixture(scope="module")
def lib():
    from attention_forward_14_gb300.build import build
    build()
    return binding.load()


@pytest.mark.parametrize("kw", [
    dict(ks=V_SCALE), dict(ks=V_SCALE + SCALE - 4), dict(vs=K_SCALE - SCALE + 4), dict(ks=K_POOL), dict(vs=K_POOL + POOL - 4),
    dict(ks=V_POOL - SCALE + 4), dict(vs=V_POOL + 64), dict(ks=K_NEW), dict(vs=V_NEW + NEW - 4), dict(ks=V_NEW - SCALE + 4),
], ids=str)
def test_scales_over_one_another_a_pool_or_the_new_tokens(lib, kw):
    a = dict(ks=K_SCALE, vs=V_SCALE)
    a.update(kw)
    st = S3(128, 64, 64)
    rc = lib.attn_kvcache_append_paged(K_NEW, V_NEW, K_POOL, V_POOL, a["ks"], a["vs"], REST, None, REST, None, None, st, st, 1,
                                       1, 2, 4, 32, 2, 16, 64, 0, 0, 0, 1, None)
    assert rc == -2 and b"overlap" in lib.attn_last_error()
