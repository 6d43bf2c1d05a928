"""Cases that measure the operators of latent attention: attention whose keys and values
come from one vector a token, shared by all heads.

A token is [latent (512 values) | rotated key part (64)].  Four operators:

* ``append``: the norm of new tokens' latents, the rotation of their key parts, and both
  into a paged cache of 576 values a token.
* ``attend``: the absorbed form over that cache, where queries have been multiplied by the
  keys' projection: scores from all 576 values, outputs from the latent's 512.  One token
  of a request, a drafted tree of them, or a chunk of a prompt.
* ``forward`` / ``backward``: the expanded form over packed sequences, for prompts and
  training: a head's keys are 128 values of its own and the 64 shared ones, its values 128;
  and its gradients.

``own`` chooses between the plain form (elementary torch operations in 32 bits, rounded
once at the end) and this package's kernels.
"""
import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
TOKEN, KDIM = LATENT + ROPE, NOPE + ROPE
SCALE = KDIM ** -0.5  # of the expanded keys' size, in either form
EPS = 1e-6
THETA = 10000.0


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of 64 requests into the cache (latency)
        dict(name="append_step_b64", op="append", b=64, s_new=1, pages=64, page=64, cached=3500, interleaved=True,
             padded=False, dtype="bf16"),
        # the prompts of a padded batch into the cache, behind what is there
        dict(name="append_prefill_b4_s4001", op="append", b=4, s_new=4001, pages=40, page=128, cached=1000,
             interleaved=False, padded=True, dtype="fp16"),
        # one request, a short context, the heads of one of several cards (latency)
        dict(name="attend_step_b1_h16_len1001", op="attend", b=1, h=16, sq=1, pages=16, page=64, shortest=1001, longest=1001,
             mask="causal", dtype="bf16"),
        # a decoding step of requests of very different lengths, the same heads
        dict(name="attend_step_b32_h16_len16383", op="attend", b=32, h=16, sq=1, pages=64, page=256, shortest=1,
             longest=16383, mask="causal", dtype="fp16"),
        # a decoding step of a large batch with all 128 heads on one card
        dict(name="attend_step_b64_h128_len8191", op="attend", b=64, h=128, sq=1, pages=128, page=64, shortest=1000,
             longest=8191, mask="causal", dtype="bf16"),
        # drafted trees of thirteen tokens, checked in one pass
        dict(name="attend_tree_b8_h32_s13_len4000", op="attend", b=8, h=32, sq=13, pages=32, page=128, shortest=300,
             longest=4000, mask="tree", dtype="bf16"),
        # a chunk of a long prompt over what is cached
        dict(name="attend_chunk_b1_h128_s512_len8192", op="attend", b=1, h=128, sq=512, pages=128, page=64, shortest=8192,
             longest=8192, mask="causal", dtype="bf16"),
        # a short prompt, few heads, every key seen (latency)
        dict(name="forward_300_h8_fp16", op="forward", h=8, runs="300", before="0", causal=False, dtype="fp16"),
        # a training batch of two 4096-token sequences
        dict(name="forward_2x4096_h32_bf16", op="forward", h=32, runs="4096 4096", before="0 0", causal=True, dtype="bf16"),
        # prompts of unequal lengths, packed, one of them behind keys that were there before
        dict(name="forward_packed_6001_h16_bf16", op="forward", h=16, runs="1 3107 893 2000", before="0 0 1500 0",
             causal=True, dtype="bf16"),
        # the gradients of the training batch
        dict(name="backward_2x4096_h32_bf16", op="backward", h=32, runs="4096 4096", before="0 0", causal=True,
             dtype="bf16"),
        # the gradients of packed sequences
        dict(name="backward_packed_4001_h16_fp16", op="backward", h=16, runs="1000 17 2107 877", before="0 0 0 0",
             causal=True, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "forward", "backward"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        b = _log_int(rng, 1, 64)
        s_new = _log_int(rng, 1, 16000 // b)
        page = rng.choice([16, 64, 128, 256])
        cached = _log_int(rng, 1, 2000)
        return dict(op=op, b=b, s_new=s_new, pages=-(-(cached + s_new) // page), page=page, cached=cached,
                    interleaved=rng.random() < 0.5, padded=rng.random() < 0.5, dtype=dtype)
    if op == "attend":
        h = rng.choice([4, 8, 16, 16, 24, 32, 64, 128])
        sq = rng.choice([1, 1, 2, 5, 13, _log_int(rng, 16, 500)])
        page = rng.choice([16, 64, 128, 256])
        longest = _log_int(rng, max(64, sq), 16000)
        b = max(1, min(_log_int(rng, 1, 64), (1 << 18) // longest, (1 << 29) // (longest * h * sq), (1 << 16) // (h * sq)))
        mask = rng.choice(["causal", "causal", "none", "tree"]) if sq <= 64 else rng.choice(["causal", "none"])
        return dict(op=op, b=b, h=h, sq=sq, pages=-(-longest // page) + rng.randint(0, 2), page=page,
                    shortest=rng.randint(sq, longest), longest=longest, mask=mask, dtype=dtype)
    h = rng.choice([1, 4, 8, 16, 32])
    n = rng.choice([1, 1, 2, 3, 5])
    total = _log_int(rng, 100, 4096)
    cuts = sorted(rng.sample(range(1, total), n - 1))
    runs = [e - a for a, e in zip([0] + cuts, cuts + [total])]
    before = [rng.choice([0, 0, 0, rng.randint(1, 1000)]) for _ in runs]
    return dict(op=op, h=h, runs=" ".join(map(str, runs)), before=" ".join(map(str, before)),
                causal=rng.random() < 0.75, dtype=dtype)


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


def _parents(case):
    """A drafted tree for every request: the parent of each of its tokens (-1: the first of a branch)."""
    r = random.Random(case["b"] * 31 + case["sq"])
    return [[r.randint(-1, i - 1) if i and r.random() < 0.6 else i - 1 for i in range(case["sq"])] for _ in range(case["b"])]


def _bounds(runs):
    at = [0]
    for n in runs:
        at.append(at[-1] + n)
    return at


def _runs(case):
    """Queries of every packed sequence."""
    return [int(n) for n in case["runs"].split()]


def _key_runs(case):
    """Keys of every packed sequence: those that were there before, and its own."""
    return [n + int(m) for n, m in zip(_runs(case), case["before"].split())]


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _table(length, dev):
    """cos and sin of position times frequency: angles in 64 bits, kept in 32."""
    freq = THETA ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=dev) / ROPE)
    angle = torch.arange(length, dtype=torch.float64, device=dev)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    t = _dtype(case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(t)

    st = dict(case=case)
    if case["op"] in ("forward", "backward"):
        h, tq, tk = case["h"], sum(_runs(case)), sum(_key_runs(case))
        st["q"] = randn(tq, h, KDIM)
        up = randn(tk, h, NOPE + VDIM)  # what the latents' projection writes; keys and values are views of it
        st["k_nope"], st["v"] = up[..., :NOPE], up[..., NOPE:]
        st["k_rope"] = randn(tk, TOKEN)[:, LATENT:]  # and the shared key part a view of the token's vector
        st["cu_q"] = torch.tensor(_bounds(_runs(case)), dtype=torch.int32, device=dev)
        st["cu_k"] = torch.tensor(_bounds(_key_runs(case)), dtype=torch.int32, device=dev)
        if case["op"] == "backward":
            st["dout"] = randn(tq, h, VDIM)
            st["o"], st["lse"] = _forward_plain(st)  # kept from the forward
        return st
    b, pages, page = case["b"], case["pages"], case["page"]
    perm = torch.randperm(b * pages + 3, generator=gen, device=dev)
    st["block_table"] = perm[:b * pages].reshape(b, pages).to(torch.int32).contiguous()
    st["cache_seqlens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    st["pool"] = randn(b * pages + 3, page, TOKEN)
    if case["op"] == "append":
        st["kv_new"] = randn(b, case["s_new"], TOKEN + 128)[..., :TOKEN]  # a view of the projection's output
        st["weight"] = (torch.rand(LATENT, generator=gen, device=dev) + 0.5).to(t)
        st["cos"], st["sin"] = _table(page * pages, dev)
        st["new_seqlens"] = torch.tensor(_news(case), dtype=torch.int32, device=dev) if case["padded"] else None
        return st
    st["q"] = randn(b, case["sq"], case["h"], TOKEN).transpose(1, 2)  # token by token, as the projection writes them
    st["tree"] = None
    if case["mask"] == "tree":
        words = (case["sq"] + 31) // 32
        tree = torch.zeros((b, case["sq"], words), dtype=torch.int64)
        for e, parents in enumerate(_parents(case)):
            for i, up in enumerate(parents):
                if up >= 0:
                    tree[e, i] = tree[e, up]
                tree[e, i, i // 32] |= 1 << (i % 32)
        st["tree"] = torch.where(tree >= 1 << 31, tree - (1 << 32), tree).to(torch.int32).to(dev)
    return st


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, c = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
    a, c = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)


def _append_plain(st):
    case = st["case"]
    b, s, page, pages = case["b"], case["s_new"], case["page"], case["pages"]
    x = st["kv_new"].float()
    start = st["cache_seqlens"].long()
    t = torch.arange(s, device=x.device)
    pos = start[:, None] + t
    count = st["new_seqlens"].long() if st["new_seqlens"] is not None else torch.full_like(start, s)
    there = (t < count[:, None]) & (pos < page * pages)
    pos = pos.clamp_max(page * pages - 1)
    latent = x[..., :LATENT]
    latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
    key = _rotate(x[..., LATENT:], st["cos"][pos], st["sin"][pos], case["interleaved"])
    token = st["block_table"].long().gather(1, pos // page) * page + pos % page
    st["pool"].view(-1, TOKEN)[token[there]] = torch.cat([latent, key], -1)[there].to(st["pool"].dtype)
    return st["pool"]


def _softmax(x):
    """Weights of the last axis and the log of their sum; nothing for a row that sees nothing."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, torch.zeros_like(p)), (m + torch.log(total)).squeeze(-1)


def _seen_plain(st, length, keys):
    """[b, sq, keys]: what the mask leaves."""
    case = st["case"]
    sq = case["sq"]
    j = torch.arange(keys, device=length.device)
    i = torch.arange(sq, device=length.device)
    seen = (j < length[:, None])[:, None].expand(-1, sq, -1)
    if case["mask"] == "causal":
        return seen & (j <= length[:, None, None] - sq + i[:, None])
    if case["mask"] == "tree":
        drafted = j - (length[:, None] - sq)  # [b, keys], which of the drafted tokens
        d = drafted.clamp(0, sq - 1)
        word = st["tree"].long().gather(2, (d // 32)[:, None].expand(-1, sq, -1))
        bit = (word >> (d % 32)[:, None]) & 1
        return seen & ((drafted < 0)[:, None] | (bit == 1))
    return seen


def _attend_plain(st):
    case = st["case"]
    b, h, sq = case["b"], case["h"], case["sq"]
    c = st["pool"][st["block_table"].long()].flatten(1, 2).float()  # [b, pages * page, 576]
    x = torch.matmul(st["q"].float().reshape(b, h * sq, TOKEN), c.transpose(1, 2)).view(b, h, sq, -1) * SCALE
    seen = _seen_plain(st, st["cache_seqlens"].long(), c.shape[1])
    p, lse = _softmax(x.masked_fill(~seen[:, None], -math.inf))
    o = torch.matmul(p.view(b, h * sq, -1), c[..., :LATENT]).view(b, h, sq, LATENT)
    return o.to(st["q"].dtype), lse


def _sequences(st):
    """For each packed sequence its tokens, and which keys each query sees."""
    case = st["case"]
    cq, ck = _bounds(_runs(case)), _bounds(_key_runs(case))
    for i, n in enumerate(_runs(case)):
        m = ck[i + 1] - ck[i]
        seen = torch.ones((n, m), dtype=torch.bool, device=st["q"].device)
        if case["causal"]:
            seen = seen.tril(m - n)
        yield slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1]), seen


def _heads(st, name, at):
    return st[name][at].float().transpose(0, 1)  # [h, tokens, d]


def _keys_plain(st, ks):
    kn = _heads(st, "k_nope", ks)
    return torch.cat([kn, st["k_rope"][ks].float().expand(kn.shape[0], -1, -1)], -1)


def _forward_plain(st):
    o = torch.empty((*st["q"].shape[:2], VDIM), dtype=st["q"].dtype, device=st["q"].device)
    lse = torch.empty((st["q"].shape[1], st["q"].shape[0]), device=o.device)
    for qs, ks, seen in _sequences(st):
        x = torch.matmul(_heads(st, "q", qs), _keys_plain(st, ks).transpose(1, 2)) * SCALE
        p, lse[:, qs] = _softmax(x.masked_fill(~seen, -math.inf))
        o[qs] = torch.matmul(p, _heads(st, "v", ks)).transpose(0, 1).to(o.dtype)
    return o, lse


def _backward_plain(st):
    dq, dkn, dkr, dv = (torch.empty(st[n].shape, dtype=st[n].dtype, device=st[n].device) for n in ("q", "k_nope", "k_rope", "v"))
    for qs, ks, seen in _sequences(st):
        q, k, v, g = _heads(st, "q", qs), _keys_plain(st, ks), _heads(st, "v", ks), _heads(st, "dout", qs)
        p, _ = _softmax((torch.matmul(q, k.transpose(1, 2)) * SCALE).masked_fill(~seen, -math.inf))
        dv[ks] = torch.matmul(p.transpose(1, 2), g).transpose(0, 1).to(dv.dtype)
        dp = torch.matmul(g, v.transpose(1, 2))
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * SCALE
        dq[qs] = torch.matmul(ds, k).transpose(0, 1).to(dq.dtype)
        dk = torch.matmul(ds.transpose(1, 2), q)
        dkn[ks] = dk[..., :NOPE].transpose(0, 1).to(dkn.dtype)
        dkr[ks] = dk[..., NOPE:].sum(0).to(dkr.dtype)
    return dq, dkn, dkr, dv


# ------------------------------------------------------------------ one pass

def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"append": _append_plain, "attend": _attend_plain, "forward": _forward_plain, "backward": _backward_plain}[op](st)
    import attention_forward_14_gb300 as af
    if op == "append":
        af.attn_latent_append_paged(st["kv_new"], st["pool"], st["cache_seqlens"], st["block_table"], norm_weight=st["weight"],
                                    cos=st["cos"], sin=st["sin"], eps=EPS, interleaved=case["interleaved"],
                                    new_seqlens=st["new_seqlens"])
        return st["pool"]
    if op == "attend":
        return af.attn_fwd_latent_paged(st["q"], st["pool"], st["cache_seqlens"], st["block_table"], SCALE,
                                        causal=case["mask"] == "causal", tree=st["tree"])
    packed = (st["cu_q"], st["cu_k"], max(_runs(case)), max(_key_runs(case)))
    if op == "forward":
        return af.attn_fwd_latent(st["q"], st["k_nope"], st["k_rope"], st["v"], *packed, causal=case["causal"], scale=SCALE)
    return af.attn_bwd_latent(st["q"], st["k_nope"], st["k_rope"], st["v"], st["o"], st["dout"], st["lse"], *packed,
                              causal=case["causal"], scale=SCALE)


# ------------------------------------------------------------------ work

def _pairs(n, m, causal):
    """(query, key) pairs of a sequence of n queries and m keys."""
    return sum(max(0, min(m, m - n + i + 1)) for i in range(n)) if causal else n * m


def work(case):
    op = case["op"]
    if op in ("forward", "backward"):
        h, tq, tk = case["h"], sum(_runs(case)), sum(_key_runs(case))
        pairs = h * sum(_pairs(n, m, case["causal"]) for n, m in zip(_runs(case), _key_runs(case)))
        qs, ks = tq * h * KDIM * 2, tk * (h * (NOPE + VDIM) + ROPE) * 2
        outs, lse = tq * h * VDIM * 2, tq * h * 4
        if op == "forward":
            return {"bytes": qs + ks + outs + lse, "flops": 2 * (KDIM + VDIM) * pairs}
        return {"bytes": 2 * qs + 2 * ks + 2 * outs + lse, "flops": 2 * (3 * KDIM + 2 * VDIM) * pairs}
    lens = _lengths(case)
    if op == "append":
        room = case["page"] * case["pages"]
        rows = sum(min(n, room - c) for n, c in zip(_news(case), lens))
        return {"bytes": rows * (2 * TOKEN * 2 + ROPE * 4) + LATENT * 2, "flops": rows * (4 * LATENT + 3 * ROPE)}
    h, sq = case["h"], case["sq"]
    if case["mask"] == "tree":
        drafted = [len(_ancestors(p, i)) for p in _parents(case) for i in range(sq)]
        pairs = sum((n - sq) * sq for n in lens) + sum(drafted)
    else:
        pairs = sum(_pairs(sq, n, case["mask"] == "causal") for n in lens)
    rows = case["b"] * h * sq
    return {"bytes": sum(lens) * TOKEN * 2 + rows * (TOKEN + LATENT) * 2 + rows * 4, "flops": 2 * h * (TOKEN + LATENT) * pairs}


def _ancestors(parents, i):
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_append(st):
    case = st["case"]
    page = case["page"]
    pool = st["pool"].double()
    for e, (n, m) in enumerate(zip(_lengths(case), _news(case))):
        m = min(m, page * case["pages"] - n)
        x = st["kv_new"][e, :m].double()
        pos = torch.arange(n, n + m, device=x.device)
        rms = (x[:, :LATENT].pow(2).sum(-1, keepdim=True) / LATENT + EPS).sqrt()
        turn = torch.complex(st["cos"].double()[pos], st["sin"].double()[pos])
        k = x[:, LATENT:]
        if case["interleaved"]:
            key = torch.view_as_real(torch.view_as_complex(k.reshape(m, ROPE // 2, 2).contiguous()) * turn).reshape(m, ROPE)
        else:
            z = torch.complex(k[:, :ROPE // 2].contiguous(), k[:, ROPE // 2:].contiguous()) * turn
            key = torch.cat([z.real, z.imag], -1)
        pool[st["block_table"][e].long()[pos // page], pos % page] = torch.cat([x[:, :LATENT] / rms * st["weight"].double(), key], -1)
    return pool


def _exact_attend(st):
    case = st["case"]
    b, h, sq, page = case["b"], case["h"], case["sq"], case["page"]
    o = torch.zeros((b, h, sq, LATENT), dtype=torch.float64, device=st["q"].device)
    lse = torch.full((b, h, sq), -math.inf, dtype=torch.float64, device=o.device)
    trees = _parents(case) if case["mask"] == "tree" else None
    for e, n in enumerate(_lengths(case)):
        pos = torch.arange(n, device=o.device)
        c = st["pool"][st["block_table"][e].long()[pos // page], pos % page].double()
        hidden = torch.zeros((sq, n), dtype=torch.bool)
        if case["mask"] == "causal":
            hidden = torch.ones((sq, n), dtype=torch.bool).triu(n - sq + 1)
        if case["mask"] == "tree":
            hidden[:, n - sq:] = True
            for i in range(sq):
                hidden[i, [n - sq + a for a in _ancestors(trees[e], i)]] = False
        hidden = hidden.to(o.device)
        for i in range(h):
            x = (st["q"][e, i].double() @ c.T * SCALE).masked_fill(hidden, -math.inf)
            lse[e, i] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[e, i][:, None])
            o[e, i] = torch.where(lse[e, i][:, None] == -math.inf, torch.zeros_like(o[e, i]), p @ c[:, :LATENT])
    return o, lse


def _exact_expanded(st):
    """Outputs or gradients, head by head; the gradients by differentiating the outputs."""
    case = st["case"]
    back = case["op"] == "backward"
    leaves = {n: st[n].double() for n in ("q", "k_nope", "k_rope", "v")}
    grads = {n: torch.zeros_like(x) for n, x in leaves.items()}
    o = torch.zeros((*st["q"].shape[:2], VDIM), dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros((o.shape[1], o.shape[0]), dtype=torch.float64, device=o.device)
    for qs, ks, seen in _sequences(st):
        for i in range(case["h"]):
            x = {n: leaves[n][(qs if n == "q" else ks)] for n in leaves}
            x = {n: (t if n == "k_rope" else t[:, i]).clone().requires_grad_(back) for n, t in x.items()}
            with torch.set_grad_enabled(back):
                s = x["q"][:, :NOPE] @ x["k_nope"].T + x["q"][:, NOPE:] @ x["k_rope"].T
                s = (s * SCALE).masked_fill(~seen, -math.inf)
                some = seen.any(-1)
                w = torch.softmax(s[some], -1) @ x["v"]
            if back:
                w.backward(st["dout"][qs, i].double()[some])
                for n, t in x.items():
                    if n == "k_rope":
                        grads[n][ks] += t.grad
                    else:
                        grads[n][qs if n == "q" else ks, i] = t.grad
                continue
            lse[i, qs] = torch.logsumexp(s, -1)
            o[qs.start:qs.stop, i] = torch.zeros_like(o[qs, i]).masked_scatter(some[:, None].expand(-1, VDIM), w)
    return tuple(grads.values()) if back else (o, lse)


def exact(case, seed):
    if work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_attend(st) if case["op"] == "attend" else _exact_expanded(st)
