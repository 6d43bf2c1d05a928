"""Plain fp64 implementations (numpy) of the operators around the attention,
straight from their definitions, and their inputs for the tests.

Nothing here shares code with the library or imports it.
"""
from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -64
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def tables(length, rot, theta=10000.0):
    """cos and sin, fp32 tensors [length, rot / 2]."""
    freq = theta ** (-np.arange(0, rot, 2) / rot)
    angle = np.arange(length)[:, None] * freq
    return torch.tensor(np.cos(angle), dtype=torch.float32), torch.tensor(np.sin(angle), dtype=torch.float32)


def rotate(x, cos, sin, interleaved):
    """x [..., d] turned by angles [..., rot / 2]."""
    half = cos.shape[-1]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = a * cos - b * sin
        y[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half] = a * cos - b * sin
        y[..., half:2 * half] = b * cos + a * sin
    return y


def _angles(cos, sin, positions):
    """Angles of positions [...] with a head axis before the last; positions outside the tables: where."""
    good = (positions >= 0) & (positions < cos.shape[0])
    at = np.where(good, positions, 0)
    return cos[at], sin[at], good


def norm_rope(x, w, cos, sin, positions, eps, interleaved):
    """x [tokens, heads, d], positions [tokens] (or None: no rotation)."""
    y = x.copy()
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if cos is not None:
        c, s, good = _angles(cos, sin, positions)
        y = rotate(y, c[:, None], s[:, None], interleaved) * good[:, None, None]
        y[~good] = 0.0
    return y


def norm_rope_bwd(g, x, w, cos, sin, positions, eps, interleaved):
    """(dx, dw) for the gradient g of norm_rope's output."""
    dy = g.copy()
    if cos is not None:
        c, s, good = _angles(cos, sin, positions)
        dy = rotate(dy, c[:, None], -s[:, None], interleaved)
        dy[~good] = 0.0
    if w is None:
        return dy, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dn = dy * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    return dx, (dy * n).sum((0, 1))


def round_e4m3(x):
    """The nearest e4m3 value (ties to even), saturating; NaN stays."""
    a = np.minimum(np.abs(x), E4M3_MAX)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.sign(x) * np.minimum(np.round(a / step) * step, E4M3_MAX)


def scale_of(amax):
    """The smallest power of two >= MIN_SCALE that brings amax to at most 448."""
    m, e = np.frexp(np.maximum(amax, E4M3_MAX * MIN_SCALE) / E4M3_MAX)
    return np.ldexp(1.0, np.where(m == 0.5, e - 1, e))


def append_paged(k_new, v_new, k_pool, v_pool, k_scale, v_scale, lens, news, table, cos, sin, interleaved, block):
    """Row by row on fp64 copies of the pools (values) and scales; returns them.
    k_new, v_new [b, heads, s, d]; block 0: a 16-bit pool (no rounding here)."""
    pools, scales = [k_pool.copy(), v_pool.copy()], [None if block == 0 else k_scale.copy(),
                                                     None if block == 0 else v_scale.copy()]
    b, h, s, d = k_new.shape
    num_pages, page = k_pool.shape[:2]
    cap = table.shape[1] * page
    for e in range(b):
        start = min(max(int(lens[e]), 0), cap)
        count = s if news is None else min(max(int(news[e]), 0), s)
        end = min(start + count, cap)
        if end <= start:
            continue
        for which, new in enumerate((k_new, v_new)):
            for hh in range(h):
                rows = new[e, hh, :end - start]
                if which == 0 and cos is not None:
                    rows = rotate(rows, cos[start:end], sin[start:end], interleaved)
                if block == 0:
                    for t, pos in enumerate(range(start, end)):
                        pg = table[e, pos // page]
                        if 0 <= pg < num_pages:
                            pools[which][pg, pos % page, hh] = rows[t]
                    continue
                for first in range(start // block * block, end, block):
                    pg = table[e, first // page]
                    if not 0 <= pg < num_pages:
                        continue
                    lo, hi = max(first, start), min(first + block, end)
                    part = rows[lo - start:hi - start]
                    finite = np.abs(part[np.isfinite(part)])
                    need = scale_of(finite.max() if finite.size else 0.0)
                    at, off = first % page // block, first % page
                    old = lo - first
                    was = scales[which][pg, hh, at]
                    now = max(was, need) if old else need
                    if old and now > was:
                        pools[which][pg, off:off + old, hh] = round_e4m3(pools[which][pg, off:off + old, hh] * (was / now))
                    scales[which][pg, hh, at] = now
                    pools[which][pg, off + old:off + hi - first, hh] = round_e4m3(part / now)
    return pools[0], pools[1], scales[0], scales[1]


def attend_paged(q, k_pool, v_pool, k_scale, v_scale, lens, table, causal, scale):
    """O, LSE of q [b, h, sq, d] over pools of values times the scales of their blocks."""
    b, h, sq, d = q.shape
    num_pages, page, hkv, _ = k_pool.shape
    cap = table.shape[1] * page
    o, lse = np.zeros_like(q), np.full((b, h, sq), -np.inf)
    block = page // k_scale.shape[2]
    for e in range(b):
        n = min(max(int(lens[e]), 0), cap)
        pos = np.arange(n)
        pg = table[e][pos // page].astype(np.int64)
        good = (pg >= 0) & (pg < num_pages)
        pg = np.where(good, pg, 0)
        row, at = pos % page, pos % page // block
        for hh in range(h):
            g = hh // (h // hkv)
            k = np.where(good[:, None], k_pool[pg, row, g] * k_scale[pg, g, at][:, None], 0.0)
            v = np.where(good[:, None], v_pool[pg, row, g] * v_scale[pg, g, at][:, None], 0.0)
            for i in range(sq):
                end = n - sq + i + 1 if causal else n
                if end <= 0:
                    continue
                x = (k[:end] @ q[e, hh, i]) * scale
                m = x.max()
                p = np.exp(x - m)
                o[e, hh, i] = p @ v[:end] / p.sum()
                lse[e, hh, i] = m + np.log(p.sum())
    return o, lse


def f64(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def random_pool(num_pages, page, heads, d, block, seed, spread=2.0):
    """An e4m3 pool and its power-of-two scales, as an append leaves them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((num_pages, page // block, block, heads, d), generator=g)
    x *= torch.exp(spread * torch.randn((num_pages, page // block, 1, heads, 1), generator=g))
    scale = torch.tensor(scale_of(x.abs().amax((2, 4)).double().numpy()), dtype=torch.float32)
    pool = (x / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).reshape(num_pages, page, heads, d)
    return pool, scale.transpose(1, 2).contiguous()
