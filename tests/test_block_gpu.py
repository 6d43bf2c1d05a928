"""The operators around the attention together, as a model's block calls them:
a serving loop over an 8-bit and over a 16-bit paged cache, and a training
step, each against the fp64 definition of the whole."""
import math

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
import ops_ref as R
import oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _project(x, h, hkv, d):
    """Queries, keys and values as views of a fused projection's output [b, s, h + 2 h_kv, d]."""
    return x[:, :, :h].transpose(1, 2), x[:, :, h:h + hkv].transpose(1, 2), x[:, :, h + hkv:].transpose(1, 2)


def _tokens(t):
    a = R.f64(t)
    return a.transpose(0, 2, 1, 3).reshape(-1, a.shape[1], a.shape[3])


def _normed(t, w, cos, sin, pos):
    b, h, s, d = t.shape
    y = R.norm_rope(_tokens(t), R.f64(w), cos, sin, pos.reshape(-1), 1e-6, False)
    return y.reshape(b, s, h, d).transpose(0, 2, 1, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_serving_loop_over_the_8bit_cache(dtype):
    """A padded batch of prompts, then decoding steps, one of them of a
    drafted run: norm and rotation, append, attention, step by step against
    attention over the cache as it is held (the cache against the definition)."""
    b, h, hkv, d, page, pages, block, cap = 3, 8, 2, 128, 64, 5, 16, 320
    g = torch.Generator().manual_seed(3)
    cos, sin = R.tables(cap, d)
    dcos, dsin = cos.to(DEV), sin.to(DEV)
    wq, wk = ((torch.rand(d, generator=g) + 0.5).to(dtype) for _ in range(2))
    table = torch.randperm(b * pages + 1, generator=g)[:b * pages].reshape(b, pages).to(torch.int32)
    pools = [torch.full((b * pages + 1, page, hkv, d), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.full((b * pages + 1, hkv, page // block), float("nan"), device=DEV) for _ in range(2)]
    held = [np.zeros((b * pages + 1, page, hkv, d)) for _ in range(2)] + [np.ones((b * pages + 1, hkv, page // block))] * 2
    lens = np.zeros(b, dtype=np.int32)
    steps = [(150, (150, 3, 77)), (1, None), (1, None), (5, None), (1, None), (20, (20, 0, 1))]
    for s, news in steps:
        x = torch.randn((b, s, h + 2 * hkv, d), generator=g).to(dtype)
        q, k, v = _project(x.to(DEV), h, hkv, d)
        new = np.full(b, s, dtype=np.int32) if news is None else np.array(news, dtype=np.int32)
        pos = lens[:, None] + np.arange(s)
        pos = np.where(np.arange(s) < new[:, None], pos, -1).astype(np.int32)  # the batch's padding
        dpos, dlens = torch.tensor(pos, device=DEV), torch.tensor(lens, device=DEV)
        qn, _ = af.attn_qk_norm_rope(q, k, wq.to(DEV), wk.to(DEV), dcos, dsin, dpos)
        _, kn = af.attn_qk_norm_rope(q, k, wq.to(DEV), wk.to(DEV))  # the append rotates the keys
        af.attn_kvcache_append_paged(kn, v, *pools, dlens, table.to(DEV), dcos, dsin, k_scale=scales[0],
                                     v_scale=scales[1], new_seqlens=torch.tensor(new, device=DEV))
        held = list(R.append_paged(R.f64(kn), R.f64(v), *held, lens, new, table.numpy(), R.f64(cos), R.f64(sin), False, block))
        lens = lens + new
        got = [np.nan_to_num(R.f64(t)) for t in (*pools, *scales)]
        for e in range(b):
            for t in range(lens[e]):
                pg, row = table[e, t // page], t % page
                for which in range(2):
                    a, r = got[which][pg, row], held[which][pg, row]
                    sc = held[2 + which][pg, :, row // block]
                    assert np.array_equal(got[2 + which][pg, :, row // block], sc)
                    # the two sides round to e4m3 from values a few fp32 roundings apart
                    assert (np.abs(a - r) <= 2.0 ** -3 * np.abs(r) + 2.0 ** -9).all() and (a != r).mean() < 0.02
        qr = np.where((pos >= 0)[:, None, :, None], _normed(q, wq, R.f64(cos), R.f64(sin), np.maximum(pos, 0)), 0.0)
        # queries sit at the end of what is cached: the requests with fewer new tokens are asked one by one
        for e in range(b):
            n = int(new[e])
            if n == 0:
                continue
            o, lse = af.attn_fwd_kvcache_paged_fp8(qn[e:e + 1, :, :n].contiguous(), *pools, *scales,
                                                   torch.tensor(lens[e:e + 1], device=DEV), table[e:e + 1].to(DEV), causal=True)
            ro, rl = R.attend_paged(qr[e:e + 1, :, :n], *got, lens[e:e + 1], table[e:e + 1].numpy(), True, d ** -0.5)
            # the queries' own rounding moves a score by at most a half step of each value, in sum half a
            # step of |q||k| / sqrt(d), and so a weight by that factor
            step = R.HALF_STEP[dtype]
            kmax = np.linalg.norm(got[0] * got[2].transpose(0, 2, 1).repeat(block, 1)[..., None], axis=-1).max()
            err = step * np.linalg.norm(qr[e, :, :n], axis=-1).max() * kmax * d ** -0.5
            vmax = np.abs(got[1] * got[3].transpose(0, 2, 1).repeat(block, 1)[..., None]).max()
            assert np.abs(R.f64(lse) - rl).max() <= err + 1e-5
            assert np.abs(R.f64(o) - ro).max() <= (step + 2 * err) * vmax
    assert af.status()[0] == 0


def test_decoding_over_the_16bit_cache_equals_the_append_within_the_attention():
    """Rotated keys through the append and attn_fwd_kvcache_paged without new
    rows: the same bits as attn_fwd_kvcache_paged with them."""
    b, h, d, page, pages = 2, 4, 128, 128, 3
    g = torch.Generator().manual_seed(4)
    cos, sin = (t.to(DEV) for t in R.tables(page * pages, d))
    table = torch.randperm(b * pages, generator=g).reshape(b, pages).to(torch.int32).to(DEV)
    kp = torch.randn((b * pages, page, h, d), generator=g).bfloat16().to(DEV)
    vp = torch.randn((b * pages, page, h, d), generator=g).bfloat16().to(DEV)
    kp2, vp2 = kp.clone(), vp.clone()
    lens = torch.tensor([200, 17], dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn((b, h, 3, d), generator=g).bfloat16().to(DEV) for _ in range(3))
    pos = lens[:, None] + torch.arange(3, device=DEV, dtype=torch.int32)
    qr, kr = af.attn_qk_norm_rope(q, k, cos=cos, sin=sin, positions=pos)
    o1, l1 = af.attn_fwd_kvcache_paged(qr, kp, vp, lens, table, kr, v, causal=True)
    af.attn_kvcache_append_paged(k, v, kp2, vp2, lens, table, cos, sin)
    o2, l2 = af.attn_fwd_kvcache_paged(qr, kp2, vp2, lens + 3, table, causal=True)
    torch.cuda.synchronize()
    # the rotation alone is the same arithmetic but for one fused rounding: a half step in a few values
    assert (kp.float() - kp2.float()).abs().max() <= 2.0 ** -7 * kp.float().abs().max()
    assert (kp != kp2).float().mean() < 1e-3 and torch.equal(vp, vp2)
    assert (o1.float() - o2.float()).abs().max() <= 2e-2 and (l1 - l2).abs().max() <= 1e-2


def test_training_step_gradients():
    """norm and rotation -> attention -> its backward -> the norm's backward,
    into the fused projection's gradient, against the chain rule in fp64."""
    b, h, s, d = 2, 3, 130, 64
    g = torch.Generator().manual_seed(6)
    x = torch.randn((b, s, 3 * h, d), generator=g).bfloat16()
    wq, wk = ((torch.rand(d, generator=g) + 0.5).bfloat16() for _ in range(2))
    do = torch.randn((b, h, s, d), generator=g).bfloat16()
    cos, sin = R.tables(s, d)
    xd = x.to(DEV)
    q, k, v = _project(xd, h, h, d)
    tail = (wq.to(DEV), wk.to(DEV), cos.to(DEV), sin.to(DEV))
    qn, kn = af.attn_qk_norm_rope(q, k, *tail)
    vc = v.contiguous()
    o, lse = af.attn_fwd(qn, kn, vc, causal=True)
    dqn, dkn, dv = af.attn_bwd(qn, kn, vc, o, do.to(DEV), lse, causal=True)
    dx = torch.zeros_like(xd)
    dq, dk = _project(dx, h, h, d)[:2]
    _, _, dwq, dwk = af.attn_qk_norm_rope_bwd(dqn, dkn, q, k, *tail, dq=dq, dk=dk)
    dx[:, :, 2 * h:] = dv.transpose(1, 2)
    torch.cuda.synchronize()
    pos = np.tile(np.arange(s), b)
    c, sn = R.f64(cos), R.f64(sin)
    rq, rk = _normed(q, wq, c, sn, pos), _normed(k, wk, c, sn, pos)
    gq, gk, gv = oracle.attn_bwd(rq, rk, R.f64(vc), R.f64(do), True, d ** -0.5)
    for got, up, inp, w, dw in ((dq, gq, q, wq, dwq), (dk, gk, k, wk, dwk)):
        ref, rw = R.norm_rope_bwd(up.transpose(0, 2, 1, 3).reshape(-1, h, d), _tokens(inp), R.f64(w), c, sn, pos, 1e-6, False)
        a = _tokens(got)
        # rounded to bf16 on the way: q and k, P, dS and the gradients that meet here
        assert np.linalg.norm(a - ref) <= 2e-2 * np.linalg.norm(ref)
        assert np.linalg.norm(R.f64(dw) - rw) <= 2e-2 * np.linalg.norm(rw)
    assert np.linalg.norm(R.f64(dv) - gv) <= 2e-2 * np.linalg.norm(gv)


def test_a_captured_step_beside_an_eager_one():
    """Two graphs of a decoding step with workspaces of their own, replayed on
    two streams at a time, and eager calls in between."""
    b, h, hkv, d, page, pages, block = 4, 8, 2, 64, 32, 6, 32
    g = torch.Generator().manual_seed(8)
    cos, sin = (t.to(DEV) for t in R.tables(page * pages, d))

    def state(seed):
        kp, ks = R.random_pool(b * pages, page, hkv, d, block, seed)
        vp, vs = R.random_pool(b * pages, page, hkv, d, block, seed + 1)
        t = torch.randperm(b * pages, generator=g).reshape(b, pages).to(torch.int32)
        x = torch.randn((b, 1, h + 2 * hkv, d), generator=g).half()
        return [u.to(DEV) for u in (kp, vp, ks, vs, t, torch.tensor([3, 64, 100, 191], dtype=torch.int32), x)]

    def step(st):
        kp, vp, ks, vs, t, lens, x = st
        q, k, v = _project(x, h, hkv, d)
        qn, _ = af.attn_qk_norm_rope(q, k, cos=cos, sin=sin, positions=lens[:, None])
        af.attn_kvcache_append_paged(k, v, kp, vp, lens, t, cos, sin, k_scale=ks, v_scale=vs)
        return af.attn_fwd_kvcache_paged_fp8(qn, kp, vp, ks, vs, lens + 1, t, causal=True)

    states = [state(10), state(20)]
    want = [[u.clone() for u in step([w.clone() for w in st])] for st in states]
    graphs, outs = [], []
    for st in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(st))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        step([w.clone() for w in states[0]])
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        assert all(torch.equal(a, r) for a, r in zip(out, ref))


def test_calls_one_after_another_equal_calls_one_at_a_time():
    """Launches overlap the end of what came before them in the stream: each
    result here is the next call's input (or written over by torch between
    two calls), and nothing waits on the host."""
    g = torch.Generator().manual_seed(29)
    b, h, hkv, d, page, pages, block = 3, 8, 2, 128, 64, 8, 16
    w = torch.rand(d, generator=g).to(torch.bfloat16).to(DEV)
    cos, sin = (t.to(DEV) for t in R.tables(pages * page, d))
    table = torch.randperm(b * pages, generator=g).to(torch.int32).reshape(b, pages).to(DEV)
    x0 = torch.randn(b, h, 1, d, generator=g).to(torch.bfloat16).to(DEV)

    def run(wait):
        kp, vp = (torch.zeros(b * pages, page, hkv, d, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
        ks, vs = (torch.ones(b * pages, hkv, page // block, device=DEV) for _ in range(2))
        lens = torch.tensor([0, 17, 200], dtype=torch.int32, device=DEV)
        pos = lens[:, None].clone()
        x, outs = x0.clone(), []
        for _ in range(40):
            k = x[:, :hkv] * 2
            wait()
            q, kk = af.attn_qk_norm_rope(x, k, w, w, cos, sin, pos)
            wait()
            af.attn_kvcache_append_paged(kk, k, kp, vp, lens, table, k_scale=ks, v_scale=vs)
            wait()
            lens += 1
            pos += 1
            o, lse = af.attn_fwd_kvcache_paged_fp8(q, kp, vp, ks, vs, lens, table)
            wait()
            dq, dk, dw, _ = af.attn_qk_norm_rope_bwd(o, o[:, :hkv], x, k, w, w, cos, sin, pos)
            wait()
            x = x0 + 0.5 * o + 0.01 * (dq + dw.to(o.dtype))
            k.zero_()
            outs += [x, lse, dk]
        torch.cuda.synchronize()
        return outs + [kp.view(torch.uint8), vp.view(torch.uint8), ks, vs]

    for a, c in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert a.float().isfinite().all() and torch.equal(a, c)


def test_launches_after_copies_clears_and_other_streams():
    """Eager and captured: each call follows, in its stream, a copy, a memset
    or an event of another stream, and not only a kernel; and is followed by
    copies out of its results."""
    g = torch.Generator().manual_seed(31)
    b, h, hkv, d, page, pages, block = 2, 8, 2, 64, 32, 4, 16
    w = torch.rand(d, generator=g).half().to(DEV)
    cos, sin = (t.to(DEV) for t in R.tables(pages * page, d))
    table = torch.arange(b * pages, dtype=torch.int32, device=DEV).reshape(b, pages)
    lens = torch.tensor([40, 77], dtype=torch.int32, device=DEV)
    pos = torch.zeros((b, 1), dtype=torch.int32, device=DEV)
    src = torch.randn(b, h, 1, d, generator=g).half().to(DEV)
    pool, scale = R.random_pool(b * pages, page, hkv, d, block, 5)
    pool, scale = pool.view(torch.uint8).to(DEV), scale.to(DEV)
    other = torch.cuda.Stream()
    x, grad = torch.empty_like(src), torch.empty_like(src)
    kp, vp = torch.empty_like(pool), torch.empty_like(pool)
    ks, vs = torch.empty_like(scale), torch.empty_like(scale)
    now = torch.empty_like(lens)

    def elsewhere(f):
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            f()
        here.wait_stream(other)

    def step():
        kp.copy_(pool), vp.copy_(pool), ks.copy_(scale), vs.copy_(scale), now.copy_(lens), pos.copy_(lens[:, None])
        x.copy_(src)                                   # a copy, right before
        q, k = af.attn_qk_norm_rope(x, x[:, :hkv], w, w, cos, sin, pos)
        elsewhere(lambda: ks[0].copy_(scale[0]))       # an event of another stream
        e = (kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn))
        af.attn_kvcache_append_paged(k, k, *e, now, table, k_scale=ks, v_scale=vs)
        elsewhere(lambda: now.add_(1))
        o, lse = af.attn_fwd_kvcache_paged_fp8(q, *e, ks, vs, now, table)
        grad.zero_()                                   # a memset
        dq, dk, dw, _ = af.attn_qk_norm_rope_bwd(grad, grad[:, :hkv], x, x[:, :hkv], w, w, cos, sin, pos)
        grad.copy_(o)
        dq2, dk2, dw2, _ = af.attn_qk_norm_rope_bwd(grad, grad[:, :hkv], x, x[:, :hkv], w, w, cos, sin, pos)
        out = [q, k, o, lse, dq, dk, dw, dq2, dk2, dw2]
        return [torch.empty_like(t).copy_(t) for t in out]

    def waited():
        torch.cuda.synchronize()
        r = step()
        torch.cuda.synchronize()
        return [t.clone() for t in r]

    want = waited()
    assert all(t.float().isfinite().all() for t in want) and want[8].abs().sum() > 0 and not want[4].any()
    for _ in range(20):
        got = step()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(got, want))
