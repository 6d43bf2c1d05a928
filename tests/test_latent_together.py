"""The operators of latent attention as they are used: a server's prompt,
steps and drafts over one cache, the expanded and the absorbed form of the
same attention, a training step; on streams, in graphs, by several threads,
and where offsets pass 32 bits."""
import threading

import numpy as np
import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import latent_ref as L
import ops_ref as R
import test_latent_paged as P

gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
SCALE = 192 ** -0.5


# ------------------------------------------------------------------ two forms of one attention

def two_forms(b=2, h=3, n=40, sq=5, seed=1):
    """In 64 bits: queries and latents, and what each form makes of them."""
    g = np.random.default_rng(seed)
    q, c = g.standard_normal((b, h, sq, L.KEY)), g.standard_normal((b, n, L.TOKEN))
    uk, uv = (g.standard_normal((h, 128, L.LATENT)) / 16 for _ in range(2))
    absorbed = np.concatenate([np.einsum("bhsd,hdl->bhsl", q[..., :128], uk), q[..., 128:]], -1)
    kn, v = np.einsum("bnl,hdl->bnhd", c[..., :L.LATENT], uk), np.einsum("bnl,hdl->bnhd", c[..., :L.LATENT], uv)
    return q, c, uv, absorbed, kn, v


def test_the_absorbed_form_is_the_expanded_one():
    """The definitions that the kernels are compared with, against one another."""
    q, c, uv, absorbed, kn, v = two_forms()
    b, h, sq, _ = q.shape
    n = c.shape[1]
    cu = [np.arange(b + 1) * m for m in (sq, n)]
    o, lse, _, _ = L.expanded(q.transpose(0, 2, 1, 3).reshape(-1, h, L.KEY), kn.reshape(-1, h, 128), c[..., L.LATENT:].reshape(-1, 64),
                              v.reshape(-1, h, 128), *cu, True, SCALE)
    table = np.arange(b)[:, None]
    lat, lse2, _, _ = L.paged_attend(absorbed, c, np.full(b, n), table, SCALE, True, None)
    o2 = np.einsum("bhsl,hdl->bshd", lat, uv).reshape(-1, h, 128)
    assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2.transpose(1, 0, 2).reshape(h, -1), atol=1e-12)


# ------------------------------------------------------------------ a server

class Server:
    """Two requests: prompts, in chunks, then steps, then a tree of drafts.  Nothing waits for the device meanwhile."""

    def __init__(self, seed=3, h=16, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.h, self.page, self.pages, self.b = h, 64, 6, 2
        rand = lambda *s: torch.randn(s, generator=g).to(dtype).to(DEV)  # noqa: E731
        self.prompt, self.prompt_q = rand(2, 150, L.TOKEN), rand(2, 150, h, L.TOKEN).transpose(1, 2)
        self.step, self.step_q = rand(4, 2, 1, L.TOKEN), [rand(2, 1, h, L.TOKEN).transpose(1, 2) for _ in range(4)]
        self.draft, self.draft_q = rand(2, 6, L.TOKEN), rand(2, 6, h, L.TOKEN).transpose(1, 2)
        self.tree = L.random_tree(2, 6, seed).to(DEV)
        self.news = torch.tensor([150, 97], dtype=torch.int32, device=DEV)
        self.weight = (torch.rand(L.LATENT, generator=g) + 0.5).to(dtype).to(DEV)
        self.cos, self.sin = (t.to(DEV) for t in R.tables(self.page * self.pages, L.ROPE))
        self.table = torch.randperm(14, generator=g)[:12].reshape(2, 6).to(torch.int32).to(DEV)
        self.pool = torch.zeros(14, self.page, L.TOKEN, dtype=dtype, device=DEV)
        self.lens = torch.zeros(2, dtype=torch.int32, device=DEV)

    def append(self, new, news=None, stream=None):
        af.attn_latent_append_paged(new, self.pool, self.lens, self.table, norm_weight=self.weight, cos=self.cos, sin=self.sin,
                                    new_seqlens=news, stream=stream)

    def attend(self, q, causal=True, tree=None, stream=None):
        return af.attn_fwd_latent_paged(q, self.pool, self.lens, self.table, SCALE, causal=causal, tree=tree, stream=stream)

    def run(self):
        """[(o, lse, queries, pool, lengths, causal, tree)] of every call of the attention."""
        self.pool.zero_()
        self.lens.zero_()
        out = []

        def keep(q, causal=True, tree=None):
            out.append((*self.attend(q, causal, tree), q, self.pool.clone(), self.lens.clone(), causal, tree))

        self.append(self.prompt, self.news)
        self.lens += self.news
        keep(self.prompt_q)                              # (the shorter one's queries stand at its end)
        for i in range(4):
            self.append(self.step[i])
            self.lens += 1
            keep(self.step_q[i])
        self.append(self.draft)
        self.lens += 6
        keep(self.draft_q, False, self.tree)
        self.lens -= torch.tensor([4, 2], dtype=torch.int32, device=DEV)  # what was not accepted
        self.append(self.step[0])
        self.lens += 1
        keep(self.step_q[0])
        return out


@gpu
def test_a_server():
    s = Server()
    for o, lse, q, pool, lens, causal, tree in s.run():
        P.compare(o, lse, q.cpu(), pool.cpu(), lens.cpu(), s.table.cpu(), causal, None if tree is None else tree.cpu())
    # and the cache itself: the prompt's tokens as appended
    none = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros_like(s.pool)
    want, written = L.append(L.f64(s.prompt), L.f64(pool), L.f64(s.weight), L.f64(s.cos), L.f64(s.sin), none.numpy(), s.news.cpu().numpy(),
                             s.table.cpu().numpy(), 1e-6, False)
    got = L.f64(s.pool)[written]
    assert np.abs(got - want[written]).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -18 * np.abs(want).max()


@gpu
def test_both_forms_of_one_prompt():
    """The expanded form on keys and values projected from the cache's own vectors, and the absorbed one on that cache, in
    fp16: each as far from the 64-bit result of its rounded inputs as its own bound, and those of one another as far as the
    inputs were rounded."""
    h, n = 4, 200
    q, c, uv, absorbed, kn, v = two_forms(1, h, n, n, seed=9)
    half = lambda x: torch.from_numpy(x).half()  # noqa: E731
    qx, kx, rx, vx = half(q[0].transpose(1, 0, 2)), half(kn[0]), half(c[0, :, L.LATENT:]), half(v[0])
    cu = torch.tensor([0, n], dtype=torch.int32)
    o, lse = af.attn_fwd_latent(*(t.to(DEV) for t in (qx, kx, rx, vx)), cu.to(DEV), cu.to(DEV), n, n, causal=True, scale=SCALE)
    want, wlse, absolute, size = L.expanded(*(L.f64(t) for t in (qx, kx, rx, vx)), cu.numpy(), cu.numpy(), True, SCALE)
    L.check(o, want, L.output_error(want, absolute, size.T, 2.0 ** -11, 12), "expanded")
    pool = torch.zeros(4, 64, L.TOKEN, dtype=torch.float16)
    pool.view(-1, L.TOKEN)[:n] = half(c[0])
    table, lens = torch.arange(4, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32)
    lat, lse2 = af.attn_fwd_latent_paged(half(absorbed).to(DEV), pool.to(DEV), lens.to(DEV), table.to(DEV), SCALE, causal=True)
    P.compare(lat, lse2, half(absorbed), pool, lens, table, True, None)
    # scores: 192 (or 576) products of inputs off by 2^-11 each, of both; O: by the scores' error (twice, in P and its sum)
    # and the values' (weights as well, and the output) roundings
    e = 2 * 2.0 ** -11 * size.max() + 2 * 2.0 ** -11 * SCALE * (np.abs(absorbed).reshape(-1, L.TOKEN) @ np.abs(c[0]).T).max()
    o2 = np.einsum("hsl,hdl->shd", L.f64(lat)[0], uv)
    assert np.abs(L.f64(lse) - L.f64(lse2)[0]).max() <= e
    bound = (2 * e + 8 * 2.0 ** -11) * (np.abs(v).max() + np.einsum("hdl,nl->nhd", np.abs(uv), np.abs(c[0, :, :L.LATENT])).max())
    assert np.abs(L.f64(o) - o2).max() <= bound


# ------------------------------------------------------------------ streams, graphs, threads

def packed(seed, h=4, lens=(130, 1, 300)):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    rand = lambda *s: torch.randn(s, generator=g).half().to(DEV)  # noqa: E731
    up = rand(t, h, 256)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    return (rand(t, h, L.KEY), up[..., :128], rand(t, 64), up[..., 128:]), rand(t, h, 128), (cu, cu, max(lens), max(lens))


def cached(seed, h=16, sq=1, lens=(700, 30, 500)):
    g = torch.Generator().manual_seed(seed)
    pool, table = L.cache(len(lens), 64, 12, torch.float16, seed)
    q = torch.randn((len(lens), sq, h, L.TOKEN), generator=g).half().transpose(1, 2)
    return [t.to(DEV) for t in (P.on_gpu(q), pool, torch.tensor(lens, dtype=torch.int32), table)]


def step(seed, stream=None):
    """A forward and its gradients, and a step and a chunk over a cache."""
    ins, g, cu = packed(seed) if seed not in step.inputs else step.inputs[seed][0]
    caches = [cached(seed + 10), cached(seed + 20, 128, 3)] if seed not in step.inputs else step.inputs[seed][1]
    step.inputs[seed] = (ins, g, cu), caches
    o, lse = af.attn_fwd_latent(*ins, *cu, causal=True, stream=stream)
    out = [o, lse, *af.attn_bwd_latent(*ins, o, g, lse, *cu, causal=True, stream=stream)]
    for c in caches:
        out += af.attn_fwd_latent_paged(*c, SCALE, causal=True, stream=stream)
    return out


step.inputs = {}


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    """The last tests' gigabytes, too, which later tests that count what is reserved would find."""
    yield
    step.inputs.clear()
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


@gpu
def test_calls_in_turn_on_the_current_and_on_a_given_stream():
    want = [[t.clone() for t in step(i)] for i in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(i, step(i, side if (i + n) % 2 else None)) for n in range(6) for i in range(3)]
    torch.cuda.synchronize()
    assert all(same(r, want[i]) for i, r in got)


@gpu
def test_memory_of_a_call_on_a_given_stream_is_that_streams():
    here, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(here):
        wanted = step(40)
        torch.cuda.synchronize()
        addresses = {t.data_ptr() for t in wanted}
        del wanted
        out = step(40, side)
        torch.cuda.synchronize()
    assert not addresses & {t.data_ptr() for t in out}


@gpu
def test_captured_and_replayed():
    """New inputs and lengths in the captured tensors; eager calls of the same sizes between the replays."""
    want = [t.clone() for t in step(50)]
    (ins, g, cu), caches = step.inputs[50]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(50)
    for n in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        eager = step(51)
        torch.cuda.synchronize()
        assert same(got, want)
        del eager
    ins[0].mul_(0.5)
    caches[0][2].copy_(torch.tensor([1, 768, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, step(50))


@gpu
def test_two_graphs_replayed_at_once():
    """Each has workspaces of its own."""
    want = [[t.clone() for t in step(60 + i)] for i in range(2)]
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            got.append(step(60 + i))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(same(g, w) for g, w in zip(got, want))
    assert binding.status()[0] == 0


@gpu
def test_calls_from_several_threads():
    want = [[t.clone() for t in step(70 + i)] for i in range(4)]
    torch.cuda.synchronize()
    wrong, gate = [], threading.Barrier(4)

    def work(i):
        try:
            stream = torch.cuda.Stream()
            gate.wait(10)
            for _ in range(20):
                with torch.cuda.stream(stream):
                    got = step(70 + i)
                stream.synchronize()
                if not same(got, want[i]):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong


# ------------------------------------------------------------------ offsets past 32 bits

@gpu
@pytest.mark.parametrize("h,sq", [(16, 1), (128, 2)])
def test_pages_far_into_the_pool(h, sq):
    """Pages around 2^31 and 2^32 bytes and at the end of a pool of more: the bits of a small one."""
    page, per_page = 128, 128 * L.TOKEN * 2
    num = (1 << 32) // per_page + 9000
    at = [(1 << 31) // per_page - 1, (1 << 31) // per_page, (1 << 32) // per_page - 1, (1 << 32) // per_page, num - 2, num - 1]
    g = torch.Generator().manual_seed(7)
    new = torch.randn((2, 300, L.TOKEN), generator=g).half().to(DEV)
    q = torch.randn((2, h, sq, L.TOKEN), generator=g).half().to(DEV)
    none, lens = torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor([300, 131], dtype=torch.int32, device=DEV)

    def run(num_pages, where):
        table = torch.tensor(where, dtype=torch.int32, device=DEV).reshape(2, 3)
        pool = torch.empty((num_pages, page, L.TOKEN), dtype=torch.float16, device=DEV)
        af.attn_latent_append_paged(new, pool, none, table)
        return [*af.attn_fwd_latent_paged(q, pool, lens, table, SCALE, causal=True), pool[table.flatten().long()][:2].clone()]

    small = run(6, [4, 2, 0, 1, 3, 5])
    assert small[0].isfinite().all()
    assert same(small, run(num, [at[4], at[2], at[0], at[1], at[3], at[5]]))


@gpu
def test_packed_rows_far_apart():
    """Tokens 2^22 values from one another: the bits of contiguous ones, of outputs written so as well."""
    lens, h, far = (300, 17, 300), 2, 1 << 22
    ins, g, cu = packed(81, h, lens)
    o, lse = af.attn_fwd_latent(*ins, *cu, causal=True)
    grads = af.attn_bwd_latent(*ins, o, g, lse, *cu, causal=True)
    t = sum(lens)

    def wide(x):
        flat = torch.empty((t - 1) * far + x[0].numel(), dtype=x.dtype, device=DEV)
        inner = [1] if x.dim() == 2 else [x.shape[2], 1]
        return flat.as_strided(x.shape, [far] + inner).copy_(x)

    def room(x):
        return wide(torch.zeros_like(x, memory_format=torch.contiguous_format))

    far_ins = [wide(x) for x in ins]
    fo = room(o)
    _, flse = af.attn_fwd_latent(*far_ins, *cu, causal=True, o=fo)
    assert torch.equal(fo, o) and torch.equal(flse, lse)
    out = [room(x) for x in grads]
    got = af.attn_bwd_latent(*far_ins, fo, wide(g), lse, *cu, causal=True, dq=out[0], dk_nope=out[1], dk_rope=out[2], dv=out[3])
    assert same(got, grads) and same(out, grads)
