"""Plain 64-bit forms of the paged-cache operators and builders of their
inputs, shared by the host and GPU tests."""
import math

import numpy as np

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative


def frequencies(d, scaling="plain", factor=1.0, base=10000.0, orig_len=0.0, fast=None, slow=1.0):
    """Angles per position of the d / 2 pairs, from the formulas."""
    j = np.arange(d // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (d / (d - 2))
    f = base ** (-2 * j / d)
    if scaling == "linear":
        return f / factor
    if scaling == "ramp":
        pair = [d * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast or 32.0, slow)]
        lo, hi = max(0, math.floor(pair[0])), min(d - 1, math.ceil(pair[1]))
        r = np.clip((j - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - r) + f * r / factor
    if scaling == "band":
        r = np.clip((orig_len * f / (2 * math.pi) - slow) / ((fast or 4.0) - slow), 0, 1)
        return f * r + f * (1 - r) / factor
    return f


def rotate(x, pos, freqs, rot, layout, out_scale=1.0, grad=False):
    """x [rows, heads, D] turned by angle pos * f; pos [rows] (freqs [rot/2])
    or [rows, 3] (freqs a list of three). Angles in extended precision."""
    pos = np.asarray(pos)
    if pos.ndim == 1:
        ang = pos.astype(np.longdouble)[:, None] * np.asarray(freqs, np.longdouble)[None]
    else:
        ang = np.concatenate([pos[:, a].astype(np.longdouble)[:, None] * np.asarray(freqs[a], np.longdouble)[None]
                              for a in range(3)], 1)
    c = np.cos(ang).astype(np.float64)[:, None] * out_scale
    s = np.sin(ang).astype(np.float64)[:, None] * out_scale * (-1 if grad else 1)
    y = np.array(x, dtype=np.float64)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a] = u * c - v * s
    y[..., b] = u * s + v * c
    return y


def rotation_bound(x, rot, layout, u, out_scale=1.0, pos=None, freqs=None):
    """|error| of the kernel against rotate(): u |result| of the output's
    rounding, plus 2^-21 (|a| + |b|) of a pair's f32 arithmetic (cos and sin
    within 2^-23 of their value and 2^-25 of the remainder's rounding, the
    scale's product, two products and a sum of 2^-24 each: below 2^-21), plus
    the angles' difference: the frequencies are f64 evaluations on both
    sides, each a power, a product and a quotient (2 pi is rounded too), at
    most 4 roundings of 2^-53 relative, so two of them differ by at most
    2^-50 f and the angles by |pos| f 2^-50, which moves a pair's result by
    as much times (|a| + |b|); only positions of 2^29 and more show it."""
    x = np.abs(np.asarray(x, np.float64))
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
    t = np.zeros_like(x)
    t[..., a] = t[..., b] = (x[..., a] + x[..., b]) * abs(out_scale)
    far = np.zeros_like(x)
    if pos is not None:
        f = np.abs(np.asarray(pos, np.float64))
        f = f[:, None] * freqs[None] if f.ndim == 1 else np.concatenate([f[:, k:k + 1] * freqs[k][None]
                                                                         for k in range(3)], 1)
        far[..., a] = far[..., b] = f[:, None] * 2.0 ** -50
    return lambda ref: u * np.abs(ref) + (2.0 ** -21 + u * 2.0 ** -20 + far) * t + 2.0 ** -25


class Batch:
    """A ragged batch over a paged cache: pages in a shuffled order, stale
    values everywhere no row was written."""

    def __init__(self, counts, lens, prefix, kv_heads, dim, page, seed=0, spare=2, stale=None, amp=1.0):
        rng = np.random.default_rng(seed)
        self.counts, self.lens, self.prefix = list(counts), list(lens), prefix
        self.hk, self.d, self.page = kv_heads, dim, page
        need = [-(-m // page) for m in lens]
        npre = -(-prefix // page)
        total = npre + sum(need) + spare
        order = rng.permutation(total).astype(np.int32)
        self.prefix_pages = order[:npre].copy()
        self.table = np.full((len(lens), max([1] + need)), -1, np.int32)
        at = npre
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        self.pool = np.full((total, page, 2, kv_heads, dim), np.nan if stale is None else stale, np.float32)
        self.keys = []  # per sequence: [prefix + own, 2, hk, d]
        pre = (amp * rng.standard_normal((prefix, 2, kv_heads, dim))).astype(np.float32)
        self.put(self.prefix_pages, 0, pre)
        for b, m in enumerate(lens):
            own = (amp * rng.standard_normal((m, 2, kv_heads, dim))).astype(np.float32)
            self.put(self.table[b], 0, own)

    def put(self, pages, first, rows):
        for i in range(rows.shape[0]):
            self.pool[pages[(first + i) // self.page], (first + i) % self.page] = rows[i]

    def get(self, pages, n, pool):
        if n == 0:
            return np.zeros((0, 2, self.hk, self.d))
        flat = pool[pages[:-(-n // self.page)]].reshape(-1, 2, self.hk, self.d)
        return flat[:n].astype(np.float64)

    def seen(self, causal, vis=None):
        out = []
        for b, (n, m) in enumerate(zip(self.counts, self.lens)):
            for i in range(n):
                t = self.cu[b] + i
                full = self.prefix + m
                out.append(min(int(vis[t]), full) if vis is not None else
                           (self.prefix + m - n + i + 1 if causal else full))
        return out


def attention(batch, pool, q, seen, scale, u):
    """(result, bound on the kernel's error) in 64 bits. The bound: the
    output's rounding u |out|; each weight rounded to the values' type, u W
    with W = sum p |v| / sum p; each score off by d = 2^-24 (D + 40)
    max|scale q.k| terms, which shifts a weight by a factor 1 +- 2 d and the
    result by 2 d (W + |out|); the f32 sums of n products 2^-23 (n / 8 + 32) W."""
    rows, heads, d = q.shape
    g = heads // batch.hk
    out = np.zeros((rows, heads, d))
    bound = np.zeros((rows, heads, d))
    q = q.astype(np.float64)
    pre = batch.get(batch.prefix_pages, batch.prefix, pool)
    for b, (n, m) in enumerate(zip(batch.counts, batch.lens)):
        if n == 0:
            continue
        kv = np.concatenate([pre, batch.get(batch.table[b], m, pool)])
        t0 = batch.cu[b]
        for i in range(n):
            k = seen[t0 + i]
            if k == 0:
                continue
            for h in range(heads):
                kk, vv = kv[:k, 0, h // g], kv[:k, 1, h // g]
                qv = q[t0 + i, h]
                s = kk @ qv * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t0 + i, h] = p @ vv
                w = p @ np.abs(vv)
                terms = (np.abs(kk) @ np.abs(qv)).max() * scale
                ds = 2.0 ** -24 * ((d + 40) * terms + 40)
                bound[t0 + i, h] = (u + 4 * ds + 2.0 ** -23 * (k / 8 + 32)) * w + u * np.abs(out[t0 + i, h])
    return out, bound + 2.0 ** -25
