"""A model's step as it is documented, on a padded batch: norm and rotation,
append (of keys that are rotated already), attention with every request's
queries at the end of its rows, in one call."""
import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("s,news", [(7, (7, 3, 0, 1)), (60, (60, 1, 33, 59)), (150, (150, 149, 2, 0))])
def test_one_call_for_requests_of_unequal_counts(s, news):
    b, h, hkv, d, page, pages, block = 4, 4, 2, 64, 32, 8, 16
    g = torch.Generator().manual_seed(s)
    cos, sin = R.tables(page * pages, d)
    w = (torch.rand(d, generator=g) + 0.5).bfloat16()
    x = torch.randn((b, s, h + 2 * hkv, d), generator=g).bfloat16().to(DEV)
    q, k, v = (t.transpose(1, 2) for t in x.split((h, hkv, hkv), 2))
    lens, new = np.array([100, 0, 31, 64], dtype=np.int32), np.array(news, dtype=np.int32)
    table = torch.randperm(b * pages, generator=g).reshape(b, pages).to(torch.int32)
    pools, scales = zip(*(R.random_pool(b * pages, page, hkv, d, block, 40 + i, 0.3) for i in range(2)))
    pools, scales = [t.to(DEV) for t in pools], [t.to(DEV) for t in scales]
    at = np.arange(s)
    pos = np.where(at < new[:, None], lens[:, None] + at, -1).astype(np.int32)
    qn, kn = af.attn_qk_norm_rope(q, k, w.to(DEV), w.to(DEV), cos.to(DEV), sin.to(DEV), torch.tensor(pos, device=DEV))
    af.attn_kvcache_append_paged(kn, v, *pools, torch.tensor(lens, device=DEV), table.to(DEV), k_scale=scales[0],
                                 v_scale=scales[1], new_seqlens=torch.tensor(new, device=DEV))
    # row i holds query i - (s - new); the rows before are left out
    place = torch.tensor((at - (s - new[:, None])) % s, device=DEV)
    moved = qn.gather(2, place[:, None, :, None].expand(b, h, s, d))
    total = lens + new
    o, lse = af.attn_fwd_kvcache_paged_fp8(moved, *pools, *scales, torch.tensor(total, device=DEV), table.to(DEV), causal=True)
    torch.cuda.synchronize()
    assert af.status()[0] == 0
    # keys of the new tokens, from the definition: rotated once
    ref = R.norm_rope(R.f64(k).transpose(0, 2, 1, 3).reshape(b * s, hkv, d), R.f64(w), R.f64(cos), R.f64(sin), pos.reshape(-1),
                      1e-6, False).reshape(b, s, hkv, d)
    held, sc = R.f64(pools[0]), R.f64(scales[0])
    for e in range(b):
        n = int(new[e])
        for t in range(n):
            pg, row = table[e, (lens[e] + t) // page], (lens[e] + t) % page
            got = held[pg, row] * sc[pg, :, row // block][:, None]
            # bf16's and e4m3's roundings, and e4m3's subnormal half step at the block's scale
            assert (np.abs(got - ref[e, t]) <= (2.0 ** -4 + 2.0 ** -7) * np.abs(ref[e, t]) + 2.0 ** -10 * sc[pg, :, row // block][:, None]).all()
        if n == 0:
            continue
        ro, rl = R.attend_paged(R.f64(qn[e:e + 1, :, :n]), R.f64(pools[0]), R.f64(pools[1]), R.f64(scales[0]), R.f64(scales[1]),
                                total[e:e + 1], table[e:e + 1].numpy(), True, d ** -0.5)
        go, gl = R.f64(o[e:e + 1, :, s - n:]), R.f64(lse[e:e + 1, :, s - n:])
        vmax = np.abs(R.f64(pools[1]) * R.f64(scales[1]).transpose(0, 2, 1).repeat(block, 1)[..., None]).max()
        # P's 2^-11 of the largest value, bf16's half step, and scores in fp32
        assert (np.abs(go - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * vmax).all()
        assert np.abs(gl - rl).max() <= 2.0 ** -16
