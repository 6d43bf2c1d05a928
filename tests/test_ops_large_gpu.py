"""The operators around the attention where element and byte offsets pass 2^31
and 2^32: the same call on small tensors of the same values has to give the
same bits."""
import pytest
import torch

import attention_forward_14_gb300 as af
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("rows", [1, 32])
@pytest.mark.parametrize("bits", [8, 16])
def test_pages_far_into_the_pool(bits, rows):
    """Pages around 2^31 and 2^32 bytes and at the end of a pool of more."""
    b, h, hkv, d, page, pages, block = 2, 16, 8, 128, 128, 3, 32
    per_page = page * hkv * d * (bits // 8)
    num = (1 << 32) // per_page + 8
    at = [(1 << 31) // per_page - 1, (1 << 31) // per_page, (1 << 32) // per_page - 1, (1 << 32) // per_page, num - 2, num - 1]
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((b, hkv, 200, d), generator=g).half().to(DEV) for _ in range(2))
    k1, v1 = (torch.randn((b, hkv, rows, d), generator=g).half().to(DEV) for _ in range(2))
    q = torch.randn((b, h, rows, d), generator=g).half().to(DEV)
    cos, sin = (t.to(DEV) for t in R.tables(page * pages, d))
    none, lens = torch.zeros(b, dtype=torch.int32, device=DEV), torch.tensor([200, 131], dtype=torch.int32, device=DEV)

    def run(num_pages, where):
        table = torch.tensor(where, dtype=torch.int32, device=DEV).reshape(b, pages)
        t = torch.float8_e4m3fn if bits == 8 else torch.float16
        kp, vp = (torch.empty((num_pages, page, hkv, d), dtype=t, device=DEV) for _ in range(2))
        sc = [torch.empty((num_pages, hkv, page // block), device=DEV) for _ in range(2)] if bits == 8 else [None, None]
        rest = dict(k_scale=sc[0], v_scale=sc[1])
        af.attn_kvcache_append_paged(k, v, kp, vp, none, table, cos, sin, new_seqlens=lens, **rest)
        af.attn_kvcache_append_paged(k1, v1, kp, vp, lens, table, cos, sin, **rest)
        if bits == 8:
            o, lse = af.attn_fwd_kvcache_paged_fp8(q, kp, vp, *sc, lens + rows, table, causal=True)
        else:
            o, lse = af.attn_fwd_kvcache_paged(q[:, :hkv].contiguous(), kp, vp, lens + rows, table, causal=True)
        pos = torch.arange(page * pages, device=DEV)
        seen = [kp[table[e].long()].reshape(-1, hkv, d)[pos < int(lens[e]) + rows].view(torch.uint8) for e in range(b)]
        return [o, lse] + seen

    small = run(6, [4, 2, 0, 1, 3, 5])
    big = run(num, [at[4], at[2], at[0], at[1], at[3], at[5]])
    assert small[0].float().isfinite().all()
    for a, c in zip(small, big):
        assert torch.equal(a, c)


def test_norm_of_more_than_2_to_the_32_bytes():
    h, s, d = 32, 600_000, 128           # 2.46e9 elements
    w = torch.rand(d, dtype=torch.float32, device=DEV).half()
    cos, sin = (t.to(DEV) for t in R.tables(s, d))
    q, gq = (torch.empty((1, s, h, d), dtype=torch.float16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(i))
             .transpose(1, 2) for i in (1, 2))
    k, gk = q[:, :1], gq[:, :1]
    qo, _ = af.attn_qk_norm_rope(q, k, w, w, cos, sin)
    dq, dk, dwq, dwk = af.attn_qk_norm_rope_bwd(gq, gk, q, k, w, w, cos, sin)
    bound = (1 << 31) // (h * d)
    for a, n in ((0, 64), (bound - 32, 64), (s - 64, 64)):
        sl = slice(a, a + n)
        pos = torch.arange(a, a + n, dtype=torch.int32, device=DEV)
        want, _ = af.attn_qk_norm_rope(q[:, :, sl], k[:, :, sl], w, w, cos, sin, pos)
        assert torch.equal(qo[:, :, sl], want)
        ddq, ddk, _, _ = af.attn_qk_norm_rope_bwd(gq[:, :, sl], gk[:, :, sl], q[:, :, sl], k[:, :, sl], w, w, cos, sin, pos)
        assert torch.equal(dq[:, :, sl], ddq) and torch.equal(dk[:, :, sl], ddk)
    # the keys are the queries' first head: its share of the sum, taken in another order
    x, g = k[0, 0].double(), gk[0, 0].double()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    c, sn = cos.double(), sin.double()
    dy = torch.cat([g[:, :d // 2] * c + g[:, d // 2:] * sn, g[:, d // 2:] * c - g[:, :d // 2] * sn], -1)
    ref, size = (dy * n).sum(0), (dy * n).abs().sum(0)
    # each term has some ten fp32 roundings, and passes through sums of up to 250 terms
    assert ((dwk.double() - ref).abs() <= size * 2.0 ** -24 * 300).all()
    assert dwq.isfinite().all()
