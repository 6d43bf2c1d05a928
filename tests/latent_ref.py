"""Plain fp64 implementations (numpy) of the operators of latent attention,
straight from their definitions, with bounds of what rounding may do to them.

Nothing here shares code with the library or imports it.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import ops_ref as R

LATENT, ROPE, TOKEN = 512, 64, 576
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.detach().cpu().double().numpy()


def append(new, pool, weight, cos, sin, lens, news, table, eps, interleaved):
    """pool [pages, page, 576] with new [b, s, 576] in it, unrounded; and which of its tokens were written."""
    pool = pool.copy()
    pages, page, _ = pool.shape
    cap = table.shape[1] * page
    written = np.zeros((pages, page), dtype=bool)
    for e in range(new.shape[0]):
        start = min(max(int(lens[e]), 0), cap)
        for t in range(min(max(int(news[e]), 0), new.shape[1])):
            pos = start + t
            if pos >= cap or not 0 <= table[e, pos // page] < pages:
                continue
            x = new[e, t].copy()
            if weight is not None:
                x[:LATENT] = x[:LATENT] / math.sqrt((x[:LATENT] ** 2).mean() + eps) * weight
            if cos is not None:
                x[LATENT:] = R.rotate(x[LATENT:], cos[pos], sin[pos], interleaved)
            pool[table[e, pos // page], pos % page] = x
            written[table[e, pos // page], pos % page] = True
    return pool, written


def visible(sq, n, causal, tree):
    """[sq, n]: the keys that each query of a request with n cached tokens sees; tree [sq, words]."""
    j = np.arange(n)
    seen = np.ones((sq, n), dtype=bool)
    for i in range(sq):
        if causal:
            seen[i] = j <= i + n - sq
        if tree is not None:
            for k in range(max(n - sq, 0), n):
                t = k - (n - sq)
                seen[i, k] = int(tree[i, t // 32]) >> (t % 32) & 1
    return seen


def attend(q, k, v, seen, scale):
    """One head: q [sq, dk], k [n, dk], v [n, dv], seen [sq, n].  (O, LSE, sum of P |v|, largest scale sum |q k| of a
    row's seen keys)."""
    s = scale * (q @ k.T)
    s[~seen] = -np.inf
    some = seen.any(1)
    m = np.where(some, s.max(1, initial=-np.inf), 0.0)
    p = np.exp(s - m[:, None])
    total = p.sum(1)
    p = np.divide(p, total[:, None], out=np.zeros_like(p), where=some[:, None])
    with np.errstate(divide="ignore"):
        lse = np.where(some, m + np.log(total), -np.inf)
    size = abs(scale) * np.where(seen, np.abs(q) @ np.abs(k).T, 0.0).max(1, initial=0.0)
    return p @ v, lse, p @ np.abs(v), size


def score_error(size, steps):
    """How far a score may be off: `steps` products of 16 pairs are added up one after another in fp32, each sum off by
    2^-23 of what has been summed, and the 16 pairs of a product as much; the exponential by 2^-22."""
    return (steps + 16) * 2.0 ** -23 * size + 2.0 ** -21


def output_error(o, absolute, size, half, steps):
    """P off by its rounding and by the scores' error, in the product and (as rounded) in the sum that divides it; the
    product's own sums, 2^-23 for each of the keys' steps; the output's rounding."""
    w = 2 * half + 4 * score_error(size, steps) + 2.0 ** -15
    return w[..., None] * (absolute + np.abs(o)) + half * np.abs(o) + 1e-30


def paged_attend(q, pool, lens, table, scale, causal, tree):
    """q [b, h, sq, 576]: (O, LSE, error bound of O, of LSE) for half steps filled in by the caller."""
    b, h, sq, _ = q.shape
    pages, page, _ = pool.shape
    cap = table.shape[1] * page
    o, a = np.zeros((b, h, sq, LATENT)), np.zeros((b, h, sq, LATENT))
    lse, size = np.zeros((b, h, sq)), np.zeros((b, h, sq))
    for e in range(b):
        n = min(max(int(lens[e]), 0), cap)
        c = np.zeros((n, TOKEN))
        for j in range(0, n, page):
            pg = table[e, j // page]
            if 0 <= pg < pages:
                c[j:j + page] = pool[pg, :min(page, n - j)]
        seen = visible(sq, n, causal, None if tree is None else tree[e])
        for i in range(h):
            o[e, i], lse[e, i], a[e, i], size[e, i] = attend(q[e, i], c, c[:, :LATENT], seen, scale)
    return o, lse, a, size


def check(got, want, bound, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= bound)
    bad &= ~(np.isneginf(got) & np.isneginf(want))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]!r} for {want[bad][0]!r} +- {np.broadcast_to(bound, bad.shape)[bad][0]!r}"


def random_tree(b, sq, seed):
    """Ancestor bits [b, sq, words] (int32 tensor) of trees in which a token's parent is an earlier one, or none."""
    g = np.random.default_rng(seed)
    words = (sq + 31) // 32
    t = np.zeros((b, sq, words), dtype=np.uint32)
    for e in range(b):
        for i in range(sq):
            up = int(g.integers(-1, i)) if i else -1
            if up >= 0:
                t[e, i] = t[e, up]
            t[e, i, i // 32] |= np.uint32(1) << np.uint32(i % 32)
    return torch.from_numpy(t.view(np.int32).copy())


def cache(b, page, pages, dtype, seed, spare=2):
    """A pool whose every token is filled, and a table of distinct pages in a random order."""
    g = torch.Generator().manual_seed(seed)
    n = b * pages + spare
    pool = torch.randn((n, page, TOKEN), generator=g).to(dtype)
    table = torch.randperm(n, generator=g)[:b * pages].reshape(b, pages).to(torch.int32)
    return pool, table


# ------------------------------------------------------------------ expanded form

NOPE, KEY, VALUE = 128, 192, 128


def causal_seen(n, m, causal):
    return np.ones((n, m), dtype=bool) if not causal else np.arange(m) <= np.arange(n)[:, None] + m - n


def sequences(cu_q, cu_k):
    for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        yield slice(int(a), int(b)), slice(int(c), int(d))


def expanded(q, kn, kr, v, cu_q, cu_k, causal, scale):
    """(O [t, h, 128], LSE [h, t], sum of P |v|, largest scale sum |q k| [h, t])."""
    o, a = np.zeros((*q.shape[:2], VALUE)), np.zeros((*q.shape[:2], VALUE))
    lse, size = np.full((q.shape[1], q.shape[0]), -np.inf), np.zeros((q.shape[1], q.shape[0]))
    for qs, ks in sequences(cu_q, cu_k):
        seen = causal_seen(qs.stop - qs.start, ks.stop - ks.start, causal)
        if seen.size == 0:
            continue
        for i in range(q.shape[1]):
            k = np.concatenate([kn[ks, i], kr[ks]], 1)
            o[qs, i], lse[i, qs], a[qs, i], size[i, qs] = attend(q[qs, i], k, v[ks, i], seen, scale)
    return o, lse, a, size


def expanded_grads(q, kn, kr, v, g, cu_q, cu_k, causal, scale, half, o_error):
    """The gradients by the formula, each with a bound of its error for o off by o_error: {name: (value, bound)}.

    P is off by twice a score's error (its own and LSE's) and rounded; dP by its sums in fp32; D by what o is off; dS by
    all of these and its rounding; sums over queries or keys by 2^-15 of the sums of magnitudes; then the output's
    rounding."""
    names = dict(dq=q, dk_nope=kn, dk_rope=kr, dv=v)
    val, err = ({n: np.zeros(x.shape) for n, x in names.items()} for _ in range(2))
    for qs, ks in sequences(cu_q, cu_k):
        seen = causal_seen(qs.stop - qs.start, ks.stop - ks.start, causal)
        if seen.size == 0:
            continue
        for i in range(q.shape[1]):
            qi, vi, gi = q[qs, i], v[ks, i], g[qs, i]
            k = np.concatenate([kn[ks, i], kr[ks]], 1)
            s = scale * (qi @ k.T)
            s[~seen] = -np.inf
            some = seen.any(1)
            m = np.where(some, s.max(1, initial=-np.inf), 0.0)
            p = np.exp(s - m[:, None])
            p /= np.where(some, p.sum(1), 1.0)[:, None]
            dp = gi @ vi.T
            d = (p * dp).sum(1, keepdims=True)
            ds = p * (dp - d)
            size = abs(scale) * np.where(seen, np.abs(qi) @ np.abs(k).T, 0.0).max(1, initial=0.0)
            ep = 2 * score_error(size, 12)[:, None]
            edp = 24 * 2.0 ** -23 * (np.abs(gi) @ np.abs(vi).T)
            ed = (np.abs(gi) * o_error[qs, i]).sum(1, keepdims=True) + 2.0 ** -20 * (np.abs(gi) @ np.abs(vi).T * p).sum(1, keepdims=True)
            eds = p * (ep * np.abs(dp - d) + edp + ed) + half * np.abs(ds) + 2.0 ** -15 * np.abs(ds)
            val["dv"][ks, i] = p.T @ gi
            err["dv"][ks, i] = ((half + ep + 2.0 ** -15) * p).T @ np.abs(gi)
            val["dq"][qs, i] = scale * ds @ k
            err["dq"][qs, i] = abs(scale) * eds @ np.abs(k)
            dk, ek = scale * ds.T @ qi, abs(scale) * eds.T @ np.abs(qi)
            val["dk_nope"][ks, i], err["dk_nope"][ks, i] = dk[:, :NOPE], ek[:, :NOPE]
            val["dk_rope"][ks] += dk[:, NOPE:]
            err["dk_rope"][ks] += ek[:, NOPE:]
    # (fp16's smallest step, for a P or dS below its smallest normal: half of 2^-24 for each key or query)
    return {n: (val[n], err[n] + half * np.abs(val[n]) + 2.0 ** -25 * 64) for n in names}
