"""Cases that measure the serving and training operators around the fused attention.

Three operators, which run one after the other in a model's attention block:

* ``norm_rope`` / ``norm_rope_bwd``: RMS norm of every query and key head and the rotary
  position rotation in one pass, from views of the fused projection into the layout
  the attention reads; and its gradients.
* ``append``: new keys (rotated on the way) and values into a paged cache, held in 16 bits
  or in e4m3 with one power-of-two scale for each block of tokens and head.
* ``attn8``: attention of the new queries over that e4m3 paged cache.

``own`` chooses between the plain form (elementary torch operations in 32 bits, rounded
once at the end) and this package's kernels.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -64  # the smallest scale a block of the 8-bit cache gets
THETA = 10000.0


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of a small batch: grouped heads, one token each (latency)
        dict(name="norm_rope_step_b8_h32_kv8_d128_bf16", op="norm_rope", b=8, h=32, hkv=8, s=1, d=128, rot=128,
             interleaved=False, packed=False, dtype="bf16"),
        # a training batch of two 4096-token sequences, as many key heads as query heads
        dict(name="norm_rope_b2_h32_kv32_s4096_d128_bf16", op="norm_rope", b=2, h=32, hkv=32, s=4096, d=128, rot=128,
             interleaved=False, packed=False, dtype="bf16"),
        # packed sequences, an odd number of tokens, d = 64, adjacent pairs, half of the head rotated
        dict(name="norm_rope_packed_30011_h16_kv4_d64_fp16", op="norm_rope", b=16, h=16, hkv=4, s=30011, d=64, rot=32,
             interleaved=True, packed=True, dtype="fp16"),
        # the gradients of the training batch
        dict(name="norm_rope_bwd_b2_h32_kv32_s4096_d128_bf16", op="norm_rope_bwd", b=2, h=32, hkv=32, s=4096, d=128,
             rot=128, interleaved=False, packed=False, dtype="bf16"),
        # the gradients of packed sequences
        dict(name="norm_rope_bwd_packed_8191_h16_kv4_d64_fp16", op="norm_rope_bwd", b=5, h=16, hkv=4, s=8191, d=64,
             rot=64, interleaved=True, packed=True, dtype="fp16"),
        # one decoding step of 64 requests into the 8-bit cache (latency)
        dict(name="append_step_b64_kv8_e4m3_d128", op="append", b=64, hkv=8, s_new=1, d=128, rot=128, interleaved=False,
             pages=16, page=256, block=64, cached=3500, bits=8, padded=False, dtype="bf16"),
        # the prompts of a padded batch into the 8-bit cache, behind what is there
        dict(name="append_prefill_b4_kv8_s4001_e4m3_d128", op="append", b=4, hkv=8, s_new=4001, d=128, rot=128,
             interleaved=False, pages=48, page=128, block=16, cached=1000, bits=8, padded=True, dtype="bf16"),
        # a chunk of a prompt into the 16-bit cache that the 16-bit paged attention reads
        dict(name="append_chunk_b8_h32_s1000_fp16_d64", op="append", b=8, hkv=32, s_new=1000, d=64, rot=64,
             interleaved=True, pages=16, page=256, block=0, cached=2000, bits=16, padded=False, dtype="fp16"),
        # one request, a short context (latency)
        dict(name="attn8_step_b1_h32_kv8_len1001_d128", op="attn8", b=1, h=32, hkv=8, sq=1, d=128, pages=8, page=128,
             block=16, shortest=1001, longest=1001, causal=True, dtype="bf16"),
        # a decoding step of eight requests of very different lengths, grouped heads
        dict(name="attn8_step_b8_h32_kv8_len16383_d128", op="attn8", b=8, h=32, hkv=8, sq=1, d=128, pages=64, page=256,
             block=64, shortest=1, longest=16383, causal=True, dtype="bf16"),
        # the same with a key head for every query head, d = 64 and a drafted run of five tokens
        dict(name="attn8_draft_b16_h32_kv32_len8000_d64", op="attn8", b=16, h=32, hkv=32, sq=5, d=64, pages=64, page=128,
             block=32, shortest=500, longest=8000, causal=True, dtype="fp16"),
        # a chunk of a long prompt over what is cached
        dict(name="attn8_chunk_b1_h32_kv8_s2048_len16384_d128", op="attn8", b=1, h=32, hkv=8, sq=2048, d=128, pages=64,
             page=256, block=64, shortest=16384, longest=16384, causal=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attn8", "attn8"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    dtype = rng.choice(["bf16", "fp16"])
    interleaved = rng.random() < 0.5
    rot = rng.choice([d, d, d // 2])
    if op in ("norm_rope", "norm_rope_bwd"):
        h = hkv * rng.choice([1, 2, 4]) if hkv <= 8 else hkv
        tokens = _log_int(rng, 1, 8192)
        packed = rng.random() < 0.5
        b = rng.randint(1, 8) if packed else rng.choice([1, 2, 3, 4])
        s = tokens if packed else max(1, tokens // b)
        return dict(op=op, b=min(b, s) if packed else b, h=h, hkv=hkv, s=s, d=d, rot=rot, interleaved=interleaved,
                    packed=packed, dtype=dtype)
    if op == "append":
        hkv = min(hkv, 8)
        b = _log_int(rng, 1, 64)
        s_new = _log_int(rng, 1, 16000 // b)
        page = rng.choice([64, 128, 256])
        cached = _log_int(rng, 1, 2000)
        bits = rng.choice([8, 8, 16])
        return dict(op=op, b=b, hkv=hkv, s_new=s_new, d=d, rot=rot, interleaved=interleaved,
                    pages=-(-(cached + s_new) // page), page=page, block=rng.choice([16, 32, 64]) if bits == 8 else 0,
                    cached=cached, bits=bits, padded=rng.random() < 0.5, dtype=dtype)
    page = rng.choice([16, 64, 128, 256])
    group = rng.choice([1, 2, 4, 8]) if hkv <= 8 else 1
    sq = rng.choice([1, 1, 1, 2, 7, _log_int(rng, 16, 1000)])
    longest = _log_int(rng, max(64, sq), 16000)
    b = max(1, min(_log_int(rng, 1, 64), (1 << 20) // (longest * hkv), (1 << 26) // (longest * hkv * group * sq)))
    return dict(op=op, b=b, h=hkv * group, hkv=hkv, sq=sq, d=d, pages=-(-longest // page) + rng.randint(0, 2), page=page,
                block=min(page, rng.choice([16, 32, 64, 128])), shortest=rng.randint(1, longest), longest=longest,
                causal=rng.random() < 0.7, dtype=dtype)


def _lengths(case):
    """The cached tokens of every request: a property of the case, the same for every seed."""
    r = random.Random(case["b"] * 1000003 + case["pages"])
    if case["op"] == "append":
        return [r.randint(case["cached"] // 2, case["cached"]) for _ in range(case["b"])]
    lens = [r.randint(case["shortest"], case["longest"]) for _ in range(case["b"])]
    lens[0] = case["longest"]
    if case["b"] > 1:
        lens[1] = case["shortest"]
    return lens


def _news(case):
    """How many of a padded batch's new tokens are there, for every request."""
    r = random.Random(case["b"] * 7919 + case["s_new"])
    return [r.randint(1, case["s_new"]) if case["padded"] else case["s_new"] for _ in range(case["b"])]


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _table(length, rot, dev):
    """cos and sin of position times frequency: angles in 64 bits, kept in 32."""
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(length, dtype=torch.float64, device=dev)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _scale_of(amax):
    """The smallest power of two, at least MIN_SCALE, that brings amax to at most 448."""
    m, e = torch.frexp(amax.clamp_min(E4M3_MAX * MIN_SCALE) / E4M3_MAX)
    return torch.ldexp(torch.ones_like(amax), torch.where(m == 0.5, e - 1, e))


def _filled_pool(case, gen, dev):
    """A pool as a server has it: every block of every page quantised with its own scale."""
    n, page, hkv, d, block = case["b"] * case["pages"] + 3, case["page"], case["hkv"], case["d"], case["block"]
    x = torch.randn((n, page // block, block, hkv, d), generator=gen, device=dev, dtype=torch.float16).float()
    x *= torch.rand((n, page // block, 1, hkv, 1), generator=gen, device=dev) * 2 + 0.25
    scale = _scale_of(x.abs().amax(dim=(2, 4)))
    pool = (x / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).reshape(n, page, hkv, d)
    return pool, scale.transpose(1, 2).contiguous()  # [pages, heads, blocks of a page]


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    t, d = _dtype(case), case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(t)

    st = dict(case=case)
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        b, h, hkv, s = case["b"], case["h"], case["hkv"], case["s"]
        st["q_weight"] = (torch.rand(d, generator=gen, device=dev) + 0.5).to(t)
        st["k_weight"] = (torch.rand(d, generator=gen, device=dev) + 0.5).to(t)
        if case["packed"]:
            x = randn(s, h + 2 * hkv, d)  # the fused projection's output; q and k are views of it
            st["q"], st["k"] = x[:, :h], x[:, h:h + hkv]
            cuts = sorted(random.Random(s).sample(range(1, s), case["b"] - 1)) if case["b"] > 1 else []
            runs = [e - a for a, e in zip([0] + cuts, cuts + [s])]
            pos = torch.cat([torch.arange(n, device=dev, dtype=torch.int32) for n in runs])
            length = max(runs)
            shapes = (s, h, d), (s, hkv, d)
        else:
            x = randn(b, s, h + 2 * hkv, d)
            st["q"], st["k"] = x[:, :, :h].transpose(1, 2), x[:, :, h:h + hkv].transpose(1, 2)
            first = torch.randint(0, 2000, (b, 1), generator=gen, device=dev) if s == 1 else torch.zeros((b, 1), device=dev)
            pos = (first + torch.arange(s, device=dev)).to(torch.int32)
            length = 2000 if s == 1 else s
            shapes = (b, h, s, d), (b, hkv, s, d)
        st["positions"] = pos
        st["cos"], st["sin"] = _table(length, case["rot"], dev)
        if case["op"] == "norm_rope_bwd":
            st["dq_out"], st["dk_out"] = randn(*shapes[0]), randn(*shapes[1])
        return st
    b, hkv, pages, page = case["b"], case["hkv"], case["pages"], case["page"]
    perm = torch.randperm(b * pages + 3, generator=gen, device=dev)
    st["block_table"] = perm[:b * pages].reshape(b, pages).to(torch.int32).contiguous()
    st["cache_seqlens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    if case["op"] == "append":
        s = case["s_new"]
        x = randn(b, s, 2 * hkv, d)  # keys and values as the projection writes them
        st["k_new"], st["v_new"] = x[:, :, :hkv].transpose(1, 2), x[:, :, hkv:].transpose(1, 2)
        st["cos"], st["sin"] = _table(page * pages, case["rot"], dev)
        st["new_seqlens"] = torch.tensor(_news(case), dtype=torch.int32, device=dev) if case["padded"] else None
        if case["bits"] == 8:
            st["k_pool"], st["k_scale"] = _filled_pool(case, gen, dev)
            st["v_pool"], st["v_scale"] = _filled_pool(case, gen, dev)
        else:
            st["k_pool"], st["v_pool"] = (randn(b * pages + 3, page, hkv, d) for _ in range(2))
            st["k_scale"] = st["v_scale"] = None
        return st
    st["q"] = randn(b, case["h"], case["sq"], d)
    st["k_pool"], st["k_scale"] = _filled_pool(case, gen, dev)
    st["v_pool"], st["v_scale"] = _filled_pool(case, gen, dev)
    st["scale"] = d ** -0.5
    return st


# ------------------------------------------------------------------ plain forms

EPS = 1e-6


def _angles(st, like):
    """cos and sin of every token of a [b, h, s, d] or [tokens, h, d] tensor, with its head axis of one."""
    pos = st["positions"].long()
    axis = 1
    return st["cos"][pos].unsqueeze(axis), st["sin"][pos].unsqueeze(axis)


def _rotate(x, cos, sin, interleaved):
    """The rotation of the first 2 * cos.shape[-1] of every head's values; the others are left."""
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, c = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2), rest], -1)
    a, c = r[..., :half], r[..., half:]
    return torch.cat([a * cos - c * sin, c * cos + a * sin, rest], -1)


def _norm_rope(x, w, cos, sin, interleaved):
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    return _rotate(x32 * r * w.float(), cos, sin, interleaved).to(x.dtype).contiguous()


def _norm_rope_bwd(g, x, w, cos, sin, interleaved):
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    n = x32 * r
    dy = _rotate(g.float(), cos, -sin, interleaved)  # the rotation's transpose turns the other way
    dn = dy * w.float()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dw = (dy * n).sum(tuple(range(x.dim() - 1)))
    return dx.to(x.dtype), dw


def _append_plain(st, new, pool, scale):
    """Rows `new` ([b, heads, s, d], 32 bits) into the pool behind what is cached; returns nothing."""
    case = st["case"]
    b, hkv, s, d = new.shape
    page, pages = case["page"], case["pages"]
    block = case["block"] or 1
    dev = new.device
    start = st["cache_seqlens"].long()
    count = st["new_seqlens"].long() if st["new_seqlens"] is not None else torch.full_like(start, s)
    first = start // block
    nblk = (s + block - 1) // block + 1
    # a window of whole blocks from the block that holds the first new row
    w = torch.arange(nblk * block, device=dev)
    pos = first[:, None] * block + w
    t = pos - start[:, None]
    fits = pos < page * pages
    is_new = (t >= 0) & (t < count[:, None]) & fits
    table = st["block_table"].long().gather(1, (pos // page).clamp_max(pages - 1))
    token = table * page + pos % page
    rows = new.transpose(1, 2).gather(1, t.clamp(0, s - 1)[:, :, None, None].expand(b, nblk * block, hkv, d))
    if scale is None:
        pool.view(-1, hkv, d)[token[is_new]] = rows[is_new].to(pool.dtype)
        return
    flat = pool.view(torch.uint8).view(-1, hkv, d)
    old = flat[token].view(torch.float8_e4m3fn).float()
    is_old = (t < 0) & (is_new.view(b, nblk, block).any(2).repeat_interleave(block, 1))
    at = (table.view(b, nblk, block)[:, :, 0], (pos.view(b, nblk, block)[:, :, 0] % page) // block)
    was = scale[at[0], :, at[1]]  # [b, blocks, heads]
    amax = (rows.abs() * is_new[:, :, None, None]).view(b, nblk, block, hkv, d).amax(dim=(2, 4))
    need = _scale_of(amax)
    keeps = is_old.view(b, nblk, block).any(2)[:, :, None]
    now = torch.where(keeps, torch.maximum(was, need), need)
    to_rows = lambda x: x.repeat_interleave(block, 1)[..., None]  # noqa: E731
    value = torch.where(is_new[:, :, None, None], rows / to_rows(now), old * to_rows(was / now))
    write = is_new | is_old
    flat[token[write]] = value[write].clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    touched = is_new.view(b, nblk, block).any(2)
    scale[at[0][touched], :, at[1][touched]] = now[touched]


def _cached(st, pool, scale):
    """The values that a request's pages hold: [b, heads, pages * page, d] in 32 bits."""
    case = st["case"]
    b, hkv, d, page, block = case["b"], case["hkv"], case["d"], case["page"], case["block"]
    table = st["block_table"].long()
    x = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()  # [b, pages, page, heads, d]
    s = scale[table].transpose(2, 3).repeat_interleave(block, 2)  # [b, pages, page, heads]
    return (x * s[..., None]).flatten(1, 2).transpose(1, 2)


def _attn8_plain(st):
    case = st["case"]
    b, h, hkv, sq, d = case["b"], case["h"], case["hkv"], case["sq"], case["d"]
    q = st["q"].float().view(b, hkv, h // hkv * sq, d)
    k, v = _cached(st, st["k_pool"], st["k_scale"]), _cached(st, st["v_pool"], st["v_scale"])
    length = st["cache_seqlens"].long()
    j = torch.arange(k.shape[2], device=q.device)
    i = torch.arange(sq, device=q.device)
    end = length[:, None] - sq + i + 1 if case["causal"] else length[:, None].expand(b, sq)
    seen = j < torch.minimum(end, length[:, None])[..., None]  # [b, sq, keys]
    x = torch.matmul(q, k.transpose(2, 3)).view(b, hkv, h // hkv, sq, -1) * st["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, h // hkv * sq, -1), v).view(b, hkv, h // hkv, sq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total)).squeeze(-1)
    return o.view(b, h, sq, d).to(st["q"].dtype), lse.view(b, h, sq)


# ------------------------------------------------------------------ one pass

def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if own:
        import attention_forward_14_gb300 as af
        if op == "norm_rope":
            return af.attn_qk_norm_rope(st["q"], st["k"], st["q_weight"], st["k_weight"], st["cos"], st["sin"],
                                        st["positions"], eps=EPS, interleaved=case["interleaved"])
        if op == "norm_rope_bwd":
            return af.attn_qk_norm_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"], st["q_weight"],
                                            st["k_weight"], st["cos"], st["sin"], st["positions"], eps=EPS,
                                            interleaved=case["interleaved"])
        if op == "append":
            af.attn_kvcache_append_paged(st["k_new"], st["v_new"], st["k_pool"], st["v_pool"], st["cache_seqlens"],
                                         st["block_table"], cos=st["cos"], sin=st["sin"],
                                         interleaved=case["interleaved"], k_scale=st["k_scale"],
                                         v_scale=st["v_scale"], new_seqlens=st["new_seqlens"])
            return [x for x in (st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"]) if x is not None]
        return af.attn_fwd_kvcache_paged_fp8(st["q"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"],
                                             st["cache_seqlens"], st["block_table"], causal=case["causal"],
                                             scale=st["scale"])
    if op == "norm_rope":
        cos, sin = _angles(st, st["q"])
        return (_norm_rope(st["q"], st["q_weight"], cos, sin, case["interleaved"]),
                _norm_rope(st["k"], st["k_weight"], cos, sin, case["interleaved"]))
    if op == "norm_rope_bwd":
        cos, sin = _angles(st, st["q"])
        dq, dwq = _norm_rope_bwd(st["dq_out"], st["q"], st["q_weight"], cos, sin, case["interleaved"])
        dk, dwk = _norm_rope_bwd(st["dk_out"], st["k"], st["k_weight"], cos, sin, case["interleaved"])
        return dq, dk, dwq, dwk
    if op == "append":
        pos = (st["cache_seqlens"].long()[:, None] + torch.arange(case["s_new"], device=st["cos"].device))
        pos = pos.clamp_max(st["cos"].shape[0] - 1)  # rows past the capacity are dropped
        cos, sin = st["cos"][pos].unsqueeze(1), st["sin"][pos].unsqueeze(1)
        _append_plain(st, _rotate(st["k_new"].float(), cos, sin, case["interleaved"]), st["k_pool"], st["k_scale"])
        _append_plain(st, st["v_new"].float(), st["v_pool"], st["v_scale"])
        return [x for x in (st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"]) if x is not None]
    return _attn8_plain(st)


# ------------------------------------------------------------------ work

def work(case):
    d, op = case["d"], case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        tokens = case["s"] if case["packed"] else case["b"] * case["s"]
        n = tokens * (case["h"] + case["hkv"]) * d
        angles = case["s"] * case["rot"] * 4  # each position's cos and sin once
        if op == "norm_rope":
            return {"bytes": 2 * n * 2 + angles + tokens * 4 + 4 * d, "flops": 8 * n}
        return {"bytes": 3 * n * 2 + angles + tokens * 4 + 4 * d + 8 * d, "flops": 16 * n}
    lens = _lengths(case)
    if op == "append":
        room = case["page"] * case["pages"]
        rows = sum(min(n, room - c) for n, c in zip(_news(case), lens))
        values = 2 * rows * case["hkv"] * d
        scales = 0
        if case["bits"] == 8:
            blocks = sum((c + n - 1) // case["block"] - c // case["block"] + 1 for n, c in zip(_news(case), lens))
            scales = 2 * 4 * blocks * case["hkv"]
        return {"bytes": values * 2 + values * case["bits"] // 8 + scales + rows * case["rot"] * 4, "flops": 3 * values}
    h, hkv, sq = case["h"], case["hkv"], case["sq"]
    if case["causal"]:
        pairs = sum(max(0, n - sq + i + 1) for n in lens for i in range(sq))
    else:
        pairs = sum(lens) * sq
    tokens = sum(lens)
    scales = 2 * 4 * hkv * sum(-(-n // case["block"]) for n in lens)
    rows = case["b"] * h * sq
    return {"bytes": 2 * tokens * hkv * d + scales + 2 * rows * d * 2 + rows * 4, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3_64(x):
    """The nearest e4m3 value, ties to even, by arithmetic on 64-bit numbers."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _turn_64(x, angle_cos, angle_sin, interleaved):
    """The rotation as a product of complex numbers."""
    rot = 2 * angle_cos.shape[-1]
    turn = torch.complex(angle_cos, angle_sin)
    y = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).reshape(*x.shape[:-1], rot)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_norm_rope(st):
    case = st["case"]
    pos = st["positions"].long()
    c, s = st["cos"].double()[pos].unsqueeze(1), st["sin"].double()[pos].unsqueeze(1)
    out, weights = [], []
    for name in ("q", "k"):
        x, w = st[name].double(), st[name + "_weight"].double()
        rms = (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
        if case["op"] == "norm_rope":
            out.append(_turn_64(x / rms * w, c, s, case["interleaved"]))
            continue
        g = _turn_64(st["d" + name + "_out"].double(), c, -s, case["interleaved"])
        dot = (g * w * x).sum(-1, keepdim=True)
        out.append(g * w / rms - x * dot / (case["d"] * rms.pow(3)))
        weights.append((g * x / rms).flatten(0, -2).sum(0))
    return tuple(out + weights)


def _exact_append(st):
    case = st["case"]
    page, block, d = case["page"], case["block"], case["d"]
    lens, news = _lengths(case), _news(case)
    outs = []
    for name in ("k", "v"):
        pool = st[name + "_pool"]
        pool = (pool.float() if case["bits"] == 8 else pool).double()
        scale = st[name + "_scale"].double() if case["bits"] == 8 else None
        for e in range(case["b"]):
            n = min(news[e], page * case["pages"] - lens[e])
            new = st[name + "_new"][e, :, :n].double()  # [heads, n, d]
            if name == "k":
                at = slice(lens[e], lens[e] + n)
                new = _turn_64(new, st["cos"].double()[at], st["sin"].double()[at], case["interleaved"])
            pos = torch.arange(lens[e], lens[e] + n, device=new.device)
            pg, row = st["block_table"][e].long()[pos // page], pos % page
            if scale is None:
                pool[pg, row] = new.transpose(0, 1)
                continue
            first, last = lens[e] // block, (lens[e] + n - 1) // block
            whole = torch.zeros((new.shape[0], (last - first + 1) * block, d), dtype=torch.float64, device=new.device)
            whole[:, lens[e] - first * block:lens[e] - first * block + n] = new
            amax = whole.abs().view(new.shape[0], -1, block, d).amax((2, 3))
            need = torch.exp2(torch.ceil(torch.log2((amax / E4M3_MAX).clamp_min(MIN_SCALE))))
            at = torch.arange(first, last + 1, device=new.device) * block
            bp, bk = st["block_table"][e].long()[at // page], at % page // block
            old = lens[e] % block
            if old:
                was = scale[bp[0], :, bk[0]]
                need[:, 0] = torch.maximum(need[:, 0], was)
                rows = slice(int(at[0]) % page, int(at[0]) % page + old)
                pool[bp[0], rows] = _e4m3_64(pool[bp[0], rows] * (was / need[:, 0])[:, None])
            scale[bp, :, bk] = need.T
            pool[pg, row] = _e4m3_64(new / need[:, pos // block - first, None]).transpose(0, 1)
        outs.append((pool, scale))
    return [outs[0][0], outs[1][0]] + ([outs[0][1], outs[1][1]] if case["bits"] == 8 else [])


def _exact_attn8(st):
    case = st["case"]
    b, h, hkv, sq, d, page, block = (case[n] for n in ("b", "h", "hkv", "sq", "d", "page", "block"))
    o = torch.zeros((b, h, sq, d), dtype=torch.float64, device=st["q"].device)
    lse = torch.full((b, h, sq), -math.inf, dtype=torch.float64, device=st["q"].device)
    group = h // hkv
    for e, n in enumerate(_lengths(case)):
        pos = torch.arange(n, device=o.device)
        pg, row = st["block_table"][e].long()[pos // page], pos % page
        for g in range(hkv):
            k = st["k_pool"][:, :, g].view(torch.uint8)[pg, row].view(torch.float8_e4m3fn).double()
            v = st["v_pool"][:, :, g].view(torch.uint8)[pg, row].view(torch.float8_e4m3fn).double()
            k = k * st["k_scale"][pg, g, row // block].double()[:, None]
            v = v * st["v_scale"][pg, g, row // block].double()[:, None]
            for i in range(g * group, (g + 1) * group):
                x = st["q"][e, i].double() @ k.T * st["scale"]
                if case["causal"]:
                    x += torch.full((sq, n), -math.inf, dtype=torch.float64, device=o.device).triu(n - sq + 1)
                lse[e, i] = torch.logsumexp(x, -1)
                p = torch.exp(x - lse[e, i][:, None])
                o[e, i] = torch.where(lse[e, i][:, None] == -math.inf, torch.zeros_like(o[e, i]), p @ v)
    return o, lse


def exact(case, seed):
    if case["op"] == "attn8":
        if work(case)["flops"] > 1e12:
            return None
        return _exact_attn8(prepare(case, seed))
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_norm_rope(st)
