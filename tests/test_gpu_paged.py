"""The paged cache's kernels (rotation, append, shared-prefix attention)
against plain 64-bit forms; the bounds are derived in tests/pagedcheck.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import diffusion_transformer_denoiser_qi21_gb300 as q  # noqa: E402
from tests import pagedcheck as P  # noqa: E402

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert q.device_status() == 0, "a kernel raised the status word"


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(dtype) if dtype is not None else t).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ rope ----

ROPES = [(128, 128, "interleaved", "plain"), (128, 128, "half", "ramp"), (64, 64, "half", "band"),
         (128, 64, "interleaved", "base"), (128, 48, "half", "linear"), (64, 20, "half", "plain"),
         (64, 10, "half", "plain"), (64, 20, "interleaved", "linear"), (80, 80, "half", "plain"),
         (250, 6, "interleaved", "plain"), (256, 256, "half", "plain"), (2, 2, "half", "plain")]


def _rope(d, rot, layout, scaling):
    kw = dict(scaling=scaling, factor=1.0 if scaling == "plain" else 8.0)
    if scaling in ("ramp", "band"):
        kw["orig_len"] = 8192.0
    return q.rope(d, rot, layout=layout, **kw), P.frequencies(rot, **kw)


def _check_rope(r, freqs, x, pos, got, layout, dt, grad=False):
    want = P.rotate(x, pos, freqs, r.rot_dim, layout, r.out_scale, grad)
    bound = P.rotation_bound(x, r.rot_dim, layout, P.U[dt], r.out_scale, pos, freqs)(want)
    worst = float((np.abs(got - want) / bound).max())
    assert worst <= 1, worst
    np.testing.assert_array_equal(got[..., r.rot_dim:], x[..., r.rot_dim:])


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,rot,layout,scaling", ROPES)
def test_rope(d, rot, layout, scaling, dt):
    r, freqs = _rope(d, rot, layout, scaling)
    for rows, heads in ((1, 1), (3, 5), (700, 2)):
        rng = np.random.default_rng(rows)
        x = dev(rng.standard_normal((rows, heads, d)), TD[dt])
        pos = rng.integers(-(1 << 40), 1 << 40, rows)
        pos[: rows // 2] = rng.integers(0, 200000, rows // 2)
        keep = x.clone()
        out = torch.full_like(x, 7.0)
        assert q.op_rope(r, x, dev(pos), out=out) is out
        _check_rope(r, freqs, host(keep), pos, host(out), layout, dt)
        assert torch.equal(x, keep)
        back = q.op_rope(r, x, dev(pos), out=torch.empty_like(x), grad=True)
        _check_rope(r, freqs, host(keep), pos, host(back), layout, dt, grad=True)
        q.op_rope(r, x, dev(pos))  # in place: the same bits
        assert torch.equal(x, out)


def test_rope_in_a_panel_and_unaligned():
    # q and k turned at once inside q | k | v rows, v left; then rows that
    # start at an odd element (2-byte aligned)
    r, freqs = _rope(128, 128, "interleaved", "plain")
    rng = np.random.default_rng(0)
    panel = dev(rng.standard_normal((37, 12, 128)), torch.float16)
    before = host(panel)
    pos = np.arange(37) + 5
    q.op_rope(r, panel[:, :8], dev(pos))
    got = host(panel)
    _check_rope(r, freqs, before[:, :8], pos, got[:, :8], "interleaved", "f16")
    np.testing.assert_array_equal(got[:, 8:], before[:, 8:])
    for layout in ("interleaved", "half"):
        r, freqs = _rope(64, 48, layout, "plain")
        flat = dev(rng.standard_normal(9 * 131 + 1), torch.bfloat16)
        x = flat[1:].as_strided((9, 2, 64), (131, 64, 1))
        before, keep = host(x), flat.clone()
        q.op_rope(r, x, dev(np.arange(9)))
        _check_rope(r, freqs, before, np.arange(9), host(x), layout, "bf16")
        m = torch.ones_like(flat, dtype=torch.bool)
        m[1:].as_strided((9, 2, 64), (131, 64, 1)).fill_(False)
        assert torch.equal(flat[m], keep[m])  # between the rows nothing moved


def test_rope_three_axes():
    axes = (16, 56, 56)
    r = q.rope(128, axes=axes)
    rng = np.random.default_rng(1)
    x = dev(rng.standard_normal((300, 3, 128)), torch.bfloat16)
    pos = rng.integers(-70, 70, (300, 3))
    out = q.op_rope(r, x, dev(pos), out=torch.empty_like(x))
    _check_rope(r, [P.frequencies(w) for w in axes], host(x), pos, host(out), "interleaved", "bf16")


def test_rope_gradient_against_differences():
    # <g, R(x + h e) - R(x)> / h = (R^T g) . e: the map is linear, so a step
    # of 1 leaves only rounding (f32: 2^-20 of the terms)
    r, _ = _rope(64, 48, "half", "ramp")
    rng = np.random.default_rng(2)
    x, g = (dev(rng.standard_normal((5, 2, 64)), torch.float32) for _ in range(2))
    pos = dev(rng.integers(0, 10000, 5))
    base = host(q.op_rope(r, x, pos, out=torch.empty_like(x)))
    grad = host(q.op_rope(r, g, pos, out=torch.empty_like(g), grad=True))
    gh = host(g)
    for _ in range(20):
        i = tuple(rng.integers(0, s) for s in x.shape)
        y = x.clone()
        y[i] += 1.0
        diff = (gh * (host(q.op_rope(r, y, pos, out=torch.empty_like(x))) - base)).sum()
        assert abs(diff - grad[i]) <= 2.0 ** -19 * (1 + np.abs(gh).max() * np.abs(base).max() * 4)


def test_rope_far_rows_pass_32_bits():
    # rows whose elements lie past 2^31 of the first
    r, freqs = _rope(64, 64, "half", "plain")
    rows, ld = 3, (1 << 30) + 8
    flat = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((rows, 1, 64), (ld, 64, 1))
    vals = np.random.default_rng(3).standard_normal((rows, 1, 64))
    x.copy_(dev(vals, torch.bfloat16))
    before = host(x)
    q.op_rope(r, x, dev(np.array([1, 2, 3])))
    _check_rope(r, freqs, before, np.array([1, 2, 3]), host(x), "half", "bf16")


# ---------------------------------------------------------------- append ----

def _paged(batch, pool):
    return q.PagedKV(pool, dev(batch.table), dev(np.array(batch.lens, np.int32)), dev(batch.cu),
                     prefix_pages=dev(batch.prefix_pages), prefix_len=batch.prefix)


APPENDS = [([1], [1], 0, 1, 64, 16), ([3, 0, 1, 17], [3, 0, 40, 33], 20, 2, 128, 16),
           ([100, 7], [101, 55], 0, 8, 128, 48), ([5] * 70, [9] * 70, 3, 1, 128, 64)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("counts,lens,prefix,hk,d,page", APPENDS)
@pytest.mark.parametrize("rope", [None, "half", "interleaved"])
def test_append(counts, lens, prefix, hk, d, page, rope, dt):
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=len(counts), stale=3.5)
    pool = dev(b.pool, TD[dt])
    before = host(pool)
    rng = np.random.default_rng(9)
    pad = 5  # rows behind the last sequence
    k = dev(rng.standard_normal((b.rows + pad, hk, d)), TD[dt])
    wide = dev(rng.standard_normal((b.rows + pad, 3 * hk, d)), TD[dt])
    v = wide[:, hk:2 * hk]
    rot = d // 2 if rope == "half" else d
    r, freqs = _rope(d, rot, rope, "plain") if rope else (None, None)
    q.op_kv_append(_paged(b, pool), k, v, rope=r)
    own = np.concatenate([np.arange(m - n, m) for n, m in zip(counts, lens)])
    kh, vh = host(k)[:b.rows], host(v)[:b.rows]
    want_k = P.rotate(kh, own + prefix, freqs, rot, rope, 1.0) if rope else kh
    bound = P.rotation_bound(kh, rot, rope, P.U[dt])(want_k) if rope else np.zeros_like(kh)
    got = host(pool)
    seq = np.repeat(np.arange(len(counts)), counts)
    for t in range(b.rows):
        at = (b.table[seq[t], own[t] // page], own[t] % page)
        assert np.all(np.abs(got[at][0] - want_k[t]) <= bound[t])
        np.testing.assert_array_equal(got[at][1], vh[t])
        got[at] = before[at] = 0
    np.testing.assert_array_equal(got, before)  # no other row moved


def test_append_given_positions_three_axes_and_unaligned():
    b = P.Batch([20, 13], [25, 13], 0, 2, 128, 16, stale=0.0)
    pool = dev(b.pool, torch.float16)
    rng = np.random.default_rng(4)
    flat = dev(rng.standard_normal(33 * 300 + 1), torch.float16)
    k = flat[1:].as_strided((33, 2, 128), (299, 128, 1))
    v = dev(rng.standard_normal((33, 2, 128)), torch.float16)
    pos = rng.integers(-40, 40, (33, 3))
    axes = (16, 56, 56)
    q.op_kv_append(_paged(b, pool), k, v, rope=q.rope(128, axes=axes), pos=dev(pos))
    want = P.rotate(host(k), pos, [P.frequencies(w) for w in axes], 128, "interleaved")
    bound = P.rotation_bound(host(k), 128, "interleaved", P.U["f16"])(want)
    got = host(pool)
    for t in range(33):
        s, i = (0, 5 + t) if t < 20 else (1, t - 20)
        at = (b.table[s, i // 16], i % 16)
        assert np.all(np.abs(got[at][0] - want[t]) <= bound[t])
        np.testing.assert_array_equal(got[at][1], host(v)[t])


def test_append_many_sequences():
    # more sequences than one round of the search narrows
    n = 5000
    counts = np.random.default_rng(5).integers(0, 3, n)
    lens = counts + 1
    table = np.arange(n, dtype=np.int32)[:, None]
    pool = torch.zeros(n, 16, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    kv = q.PagedKV(pool, dev(table), dev(lens.astype(np.int32)), dev(cu))
    k = dev(np.random.default_rng(6).standard_normal((cu[-1], 1, 64)), torch.bfloat16)
    q.op_kv_append(kv, k, k)
    want = torch.zeros_like(pool)
    seq = np.repeat(np.arange(n), counts)
    row = np.concatenate([np.arange(m - c, m) for c, m in zip(counts, lens)])
    want[dev(seq), dev(row)] = k[:, None].expand(-1, 2, -1, -1)
    assert torch.equal(pool, want)


def test_append_skips_rows_without_a_place():
    b = P.Batch([2, 2, 2, 2], [2, 2, 40, 2], 0, 1, 64, 16, stale=1.0)
    pool = dev(b.pool, torch.float16)
    before = pool.clone()
    table = b.table.copy()
    table[0, 0] = pool.shape[0]   # past the pool
    table[1, 0] = -1              # none
    lens = np.array([2, 2, 1000, 1], np.int32)  # past the table; fewer own rows than new ones
    kv = q.PagedKV(pool, dev(table), dev(lens), dev(b.cu))
    k = torch.full((8, 1, 64), 9.0, dtype=torch.float16, device="cuda")
    q.op_kv_append(kv, k, k)
    assert q.device_status() == 2
    want = before.clone()
    want[table[3, 0], 0] = 9.0    # the last sequence's second row has a place
    assert torch.equal(pool, want)


# ------------------------------------------------------------- attention ----

def _attend(b, dt, heads, causal=True, vis=None, seed=0, scale=None, pad=0, amp=1.0, kv=None, pool=None):
    rng = np.random.default_rng(seed + 100)
    if pool is None:
        pool = dev(b.pool, TD[dt])
    if kv is None:
        kv = _paged(b, pool)
    qx = dev(amp * rng.standard_normal((b.rows + pad, heads, b.d)), TD[dt])
    out = torch.full_like(qx, 5.0)
    ws = torch.full((q.attention_paged_bytes(kv, b.rows + pad, heads),), 255, dtype=torch.uint8, device="cuda")
    vt = None
    if vis is not None:
        vt = dev(np.concatenate([vis, np.full(pad, 9)]).astype(np.int32))
    q.op_attention_paged(kv, qx, out, ws, causal=causal, vis=vt, scale=scale)
    got = host(out)
    assert np.all(got[b.rows:] == 5.0)  # rows behind the last sequence
    want, bound = P.attention(b, host(pool), host(qx)[:b.rows], b.seen(causal, vis), scale or b.d ** -0.5, P.U[dt])
    err = np.abs(got[:b.rows] - want)
    assert np.all(err <= bound), f"worst {np.nanmax(err / bound)}, {np.isnan(got).sum()} NaN"
    return qx, out, got


# counts, lens, prefix, heads, kv_heads, dim, page
ATTNS = [
    ([1], [1], 0, 1, 1, 128, 16),
    ([1], [1], 1, 4, 1, 64, 16),
    ([1, 1], [9, 40], 200, 8, 2, 128, 16),
    ([1] * 5, [1, 17, 16, 15, 300], 130, 14, 2, 64, 48),
    ([3, 0, 5, 1], [3, 7, 64, 1], 0, 6, 2, 128, 32),
    ([2, 4, 1], [70, 4, 129], 1000, 16, 1, 128, 64),
    ([1] * 40, list(range(1, 41)), 77, 8, 2, 64, 16),
    ([1] * 9, [30] * 9, 700, 40, 2, 128, 128),
    ([60, 1, 33], [60, 200, 90], 50, 4, 4, 128, 64),
    ([140], [150], 0, 8, 2, 64, 16),
    ([65, 200], [300, 200], 333, 3, 1, 128, 16),
    ([300], [300], 129, 2, 2, 128, 256),
    ([129, 128, 127], [129, 256, 127], 128, 2, 1, 64, 64),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", ATTNS, ids=[str(i) for i in range(len(ATTNS))])
def test_attention_causal(case, dt):
    counts, lens, prefix, heads, hk, d, page = case
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=7)  # stale rows are NaN
    _attend(b, dt, heads, pad=3)


@pytest.mark.parametrize("case", ATTNS[::2], ids=[str(i) for i in range(0, len(ATTNS), 2)])
def test_attention_all_keys(case):
    counts, lens, prefix, heads, hk, d, page = case
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=8)
    _attend(b, "bf16", heads, causal=False)


@pytest.mark.parametrize("case", ATTNS, ids=[str(i) for i in range(len(ATTNS))])
def test_attention_runs(case):
    counts, lens, prefix, heads, hk, d, page = case
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=9)
    rng = np.random.default_rng(10)
    full = np.repeat([prefix + m for m in lens], counts)
    vis = (rng.random(b.rows) * (full + 20)).astype(np.int64)
    vis[::4] = 0
    _attend(b, "f16", heads, vis=vis, pad=2)
    _attend(b, "f16", heads, vis=np.minimum(vis, prefix // 2))  # no own key at all
    _attend(b, "f16", heads, vis=np.zeros(b.rows, np.int64))    # nothing at all


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("case", [([5], [20], 30, 8, 2, 128, 16), ([3, 6], [3, 90], 0, 4, 1, 64, 16),
                                  ([150, 70], [170, 70], 100, 4, 2, 128, 16), ([140], [140], 0, 2, 1, 64, 64),
                                  ([2] * 40, [9] * 40, 6000, 8, 2, 128, 64)],
                         ids=["few", "few64", "many", "many64", "prefix"])
def test_attention_odd_values_behind_the_mask(case, bad):
    # K and V rows that are not finite, at keys that only a sequence's later
    # rows see: the rows before them must not notice
    counts, lens, prefix, heads, hk, d, page = case
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=21)
    last = [m - 1 for m in lens]                      # seen by the last row alone
    spots = [(s, m - (3 if n > 60 else 1)) for s, (n, m) in enumerate(zip(counts, lens))]
    for s, i in spots:
        b.pool[b.table[s, i // page], i % page, 1, :, 5] = bad
    for s, m in enumerate(last):
        b.pool[b.table[s, m // page], m % page, :, :, 7] = bad
    pool = dev(b.pool, torch.bfloat16)
    rng = np.random.default_rng(5)
    qx = dev(rng.standard_normal((b.rows, heads, d)), torch.bfloat16)
    out = torch.empty_like(qx)
    kv = _paged(b, pool)
    ws = torch.empty(q.attention_paged_bytes(kv, b.rows, heads), dtype=torch.uint8, device="cuda")
    q.op_attention_paged(kv, qx, out, ws)
    with np.errstate(invalid="ignore", over="ignore"):
        want, bound = P.attention(b, host(pool), host(qx), b.seen(True), d ** -0.5, P.U["bf16"])
    got = host(out)
    ok = np.isfinite(want)
    assert ok.any() and not ok.all()
    assert np.all(np.abs(got[ok] - want[ok]) <= bound[ok])
    assert not np.isfinite(got[~ok]).any()


def test_attention_odd_values_behind_runs():
    # leading runs of their own lengths over a prefix with such rows
    b = P.Batch([40, 90], [40, 95], 300, 2, 128, 16, seed=22, stale=0.0)
    for i in (77, 150):
        b.pool[b.prefix_pages[i // 16], i % 16, 1, :, i % 128] = np.nan
    pool = dev(b.pool, torch.float16)
    kv = _paged(b, pool)
    rng = np.random.default_rng(6)
    qx = dev(rng.standard_normal((130, 8, 128)), torch.float16)
    vis = rng.integers(0, 250, 130)
    out = torch.empty_like(qx)
    ws = torch.empty(q.attention_paged_bytes(kv, 130, 8), dtype=torch.uint8, device="cuda")
    q.op_attention_paged(kv, qx, out, ws, vis=dev(vis.astype(np.int32)))
    want, bound = P.attention(b, host(pool), host(qx), b.seen(False, vis), 128 ** -0.5, P.U["f16"])
    got = host(out)
    ok = np.isfinite(want)
    assert np.all(np.abs(got[ok] - want[ok]) <= bound[ok])
    assert not np.isfinite(got[~ok]).any()


def test_attention_wide_scores_and_scale():
    # scores of +-100 and more: one key takes all the weight
    b = P.Batch([1, 50], [60, 70], 300, 2, 128, 16, amp=4.0, seed=11)
    _attend(b, "bf16", 4, amp=6.0)
    _attend(b, "bf16", 4, amp=1.0, scale=0.01)
    b = P.Batch([130, 50], [160, 70], 300, 2, 128, 16, amp=4.0, seed=11)
    _attend(b, "f16", 4, amp=6.0)


def test_attention_long_prefix_few_rows():
    b = P.Batch([1, 1], [5, 33], 20011, 2, 128, 64, seed=12)
    _attend(b, "bf16", 8)
    b = P.Batch([1] * 30, [5] * 30, 9000, 1, 64, 64, seed=13)
    _attend(b, "f16", 8)


@pytest.mark.parametrize("case", [
    ([1] * 10, [40] * 10, 3000, 8, 2, 128, 64),         # few-row tiles of the prefix
    ([1] * 20, [40] * 20, 5000, 8, 2, 128, 64),         # prefix tiles of one CTA, 128-wide heads
    ([2] * 24, [40] * 24, 9000, 8, 4, 64, 48),          # and 64-wide ones
    ([1] * 90, [3] * 90, 2500, 4, 1, 128, 16),          # pairs of CTAs
    ([9] * 60, [20] * 60, 1500, 16, 8, 128, 16),        # few-row tiles of 32 rows, behind a prefix
    ([5] * 60, [33] * 60, 0, 32, 8, 64, 16),            # and without one
    ([1, 0, 2], [5, 9, 40], 100, 160, 1, 64, 16),       # more heads to a key head than a tile has rows
    ([100], [130], 40, 80, 1, 128, 32),                 # one token to a tile
    ([1] * 33, [700] * 33, 0, 2, 1, 128, 16),           # parts of own keys
    ([0, 1, 2] * 100, [3, 1, 40] * 100, 20, 2, 1, 64, 16),   # more sequences than one round finds
    ([0, 30, 0, 0, 90] * 60, [1, 30, 0, 9, 95] * 60, 0, 1, 1, 64, 16),
], ids=["few", "one", "one64", "pair", "two", "two64", "wide_group", "group80", "own_parts", "rounds", "rounds_many"])
def test_attention_paths(case):
    counts, lens, prefix, heads, hk, d, page = case
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=18)
    _attend(b, "bf16", heads, pad=1)
    rng = np.random.default_rng(19)
    vis = rng.integers(0, prefix + max(lens) + 1, b.rows)
    _attend(b, "f16", heads, vis=vis)


def test_attention_in_a_table_far_larger_than_its_sequences():
    b = P.Batch([1, 3, 1], [700, 40, 3], 500, 2, 64, 16, seed=23)
    wide = np.full((3, 3000), -1, np.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    _attend(b, "bf16", 4)
    b = P.Batch([100], [120], 500, 2, 128, 16, seed=24)
    wide = np.full((1, 3000), -1, np.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    _attend(b, "f16", 4)


def test_attention_reads_pages_past_32_bits():
    # a pool of more than 2^31 values, the used pages at its end
    page, hk, d = 256, 8, 128
    n = (1 << 31) // (page * 2 * hk * d) + 3
    pool = torch.zeros(n, page, 2, hk, d, dtype=torch.bfloat16, device="cuda")
    b = P.Batch([2], [300], 100, hk, d, page, seed=14, stale=0.0)
    last = n - b.pool.shape[0]
    pool[last:] = dev(b.pool, torch.bfloat16)
    b.table = np.where(b.table >= 0, b.table + last, -1).astype(np.int32)
    small = b.prefix_pages
    b.prefix_pages = (b.prefix_pages + last).astype(np.int32)
    kv = _paged(b, pool)
    tail = pool[last:]
    b2 = P.Batch([2], [300], 100, hk, d, page, seed=14, stale=0.0)
    assert np.array_equal(b2.prefix_pages, small)
    _attend(b2, "bf16", 16, kv=kv, pool=tail)
    k = dev(np.random.default_rng(0).standard_normal((2, hk, d)), torch.bfloat16)
    q.op_kv_append(kv, k, k)
    for i, t in ((298, 0), (299, 1)):
        assert torch.equal(pool[b.table[0, i // page], i % page], k[t][None].expand(2, -1, -1))


def test_attention_bad_pages_read_as_zeros():
    b = P.Batch([1, 1], [40, 40], 64, 2, 128, 16, seed=15, stale=0.0)
    pool = dev(b.pool, torch.float16)
    b.table[1, 1], b.prefix_pages[2] = pool.shape[0] + 5, -7
    kv = _paged(b, pool)
    qx = dev(np.random.default_rng(1).standard_normal((2, 4, 128)), torch.float16)
    out = torch.empty_like(qx)
    ws = torch.empty(q.attention_paged_bytes(kv, 2, 4), dtype=torch.uint8, device="cuda")
    q.op_attention_paged(kv, qx, out, ws)
    assert q.device_status() == 2
    zero = pool.clone()
    free = [i for i in range(pool.shape[0]) if i not in set(b.table.ravel()) | set(b.prefix_pages)][0]
    zero[free] = 0
    b.table[1, 1] = b.prefix_pages[2] = free
    want, bound = P.attention(b, host(zero), host(qx), b.seen(True), 128 ** -0.5, P.U["f16"])
    assert np.all(np.abs(host(out) - want) <= bound)


def test_attention_strided_rows_and_streams():
    # q out of a q | k | v panel, out into wider rows, on a side stream
    b = P.Batch([5, 90], [20, 90], 100, 2, 128, 16, seed=16)
    pool = dev(b.pool, torch.bfloat16)
    kv = _paged(b, pool)
    rng = np.random.default_rng(3)
    panel = dev(rng.standard_normal((95, 12, 128)), torch.bfloat16)
    wide = torch.full((95, 10, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(q.attention_paged_bytes(kv, 95, 8), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q.op_attention_paged(kv, panel[:, :8], wide[:, :8], ws, stream=s)
    s.synchronize()
    want, bound = P.attention(b, host(pool), host(panel)[:, :8], b.seen(True), 128 ** -0.5, P.U["bf16"])
    got = host(wide)
    assert np.all(np.abs(got[:, :8] - want) <= bound)
    assert np.all(got[:, 8:] == 2.0)


def test_attention_repeats_bit_for_bit():
    b = P.Batch([1] * 20 + [150], [50] * 20 + [170], 3000, 2, 128, 16, seed=17)
    outs = [_attend(b, "bf16", 8)[1] for _ in range(2)]
    assert torch.equal(outs[0], outs[1])


_FIRST = """
import sys; sys.path.insert(0, {root!r})
import torch
import diffusion_transformer_denoiser_qi21_gb300 as q
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
for n, prefix in ((1, 100), (1, 4000), (200, 100)):
    pool = torch.randn(400, 16, 2, 2, 128, device="cuda").half()
    kv = q.PagedKV(pool, i([[300 + k for k in range(20)]] * 30), i([n] * 30), i([n * k for k in range(31)]),
                   prefix_pages=i(list(range(256))), prefix_len=prefix)
    x, k = (torch.randn(30 * n, h, 128, device="cuda").half() for h in (8, 2))
    out, pos = torch.empty_like(x), torch.arange(30 * n, device="cuda")
    ws = torch.empty(q.attention_paged_bytes(kv, 30 * n, 8), dtype=torch.uint8, device="cuda")
    r = q.rope(128)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # nothing of the library has run before
        q.op_rope(r, x, pos)
        q.op_kv_append(kv, k[:0], k[:0], rope=r)
        q.op_attention_paged(kv, x, out, ws)
    out.fill_(9)
    y = x.clone()
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    q.op_rope(r, y, pos)
    q.op_attention_paged(kv, y, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(got, out) and q.device_status() == 0
print("captured")
"""


def test_first_calls_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("case", [([1] * 4, [9] * 4, 100), ([1] * 40, [50] * 40, 6000), ([90, 20], [90, 70], 100)],
                         ids=["small", "parts", "many"])
def test_captures_that_fork_and_that_start_with_a_call(case):
    # the call alone in a graph; in two branches of one; behind a copy
    counts, lens, prefix = case
    b = P.Batch(counts, lens, prefix, 2, 128, 16, seed=33)
    pool = dev(b.pool, torch.bfloat16)
    kv = _paged(b, pool)
    x = dev(np.random.default_rng(34).standard_normal((b.rows, 8, 128)), torch.bfloat16)
    new = lambda: (torch.zeros_like(x),  # noqa: E731
                   torch.empty(q.attention_paged_bytes(kv, b.rows, 8), dtype=torch.uint8, device="cuda"))
    (want, w0), (o1, w1), (o2, w2), (o3, w3) = new(), new(), new(), new()
    q.op_attention_paged(kv, x, want, w0)
    torch.cuda.synchronize()
    alone, forked = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(alone):
        q.op_attention_paged(kv, x, o1, w1)
    y = torch.zeros_like(x)
    with torch.cuda.graph(forked):
        main, side = torch.cuda.current_stream(), torch.cuda.Stream()
        side.wait_stream(main)
        q.op_attention_paged(kv, x, o2, w2, stream=side)
        y.copy_(x)
        q.op_attention_paged(kv, y, o3, w3)
        main.wait_stream(side)
        o3.add_(o2)
    for _ in range(3):
        alone.replay()
        forked.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, want) and torch.equal(o2, want) and torch.equal(o3, want + want)


@pytest.mark.parametrize("case", [([1] * 6, [30] * 6, 100), ([300, 700, 90], [300, 800, 90], 400), ([2] * 40, [60] * 40, 6000)],
                         ids=["small", "many", "parts"])
def test_chains_of_calls_that_start_early(case):
    # kernels that may start before the one ahead of them has ended: a chain
    # in which each call reads what the one before wrote, against the same
    # with the host waiting in between; eager, captured, and in two branches
    counts, lens, prefix = case
    b = P.Batch(counts, lens, prefix, 2, 128, 16, seed=50)
    rng = np.random.default_rng(51)
    x0 = dev(rng.standard_normal((b.rows, 12, 128)), torch.bfloat16)
    pos = torch.arange(b.rows, device="cuda")
    r = q.rope(128, layout="half")

    class State:
        def __init__(self):
            self.pool = dev(b.pool, torch.bfloat16)
            self.kv = _paged(b, self.pool)
            self.x, self.out = x0.clone(), torch.zeros(b.rows, 8, 128, dtype=torch.bfloat16, device="cuda")
            self.ws = torch.empty(q.attention_paged_bytes(self.kv, b.rows, 8), dtype=torch.uint8, device="cuda")

        def run(self, wait=lambda: None, stream=None):
            for i in range(3):
                q.op_rope(r, self.x, pos, stream=stream)
                wait()
                q.op_kv_append(self.kv, self.x[:, 8:10], self.x[:, 10:], rope=r, stream=stream)
                wait()
                q.op_attention_paged(self.kv, self.x[:, :8], self.out, self.ws, stream=stream)
                wait()
                q.op_rope(r, self.out, pos, out=self.x[:, :8], grad=bool(i & 1), stream=stream)
                wait()

        def same(self, o):
            return torch.equal(self.x, o.x) and torch.equal(self.out, o.out) and torch.equal(
                self.pool.view(torch.int16), o.pool.view(torch.int16))

    want = State()
    want.run(torch.cuda.synchronize)
    for _ in range(5):
        got = State()
        torch.cuda.synchronize()
        got.run()
        torch.cuda.synchronize()
        assert got.same(want)
    a, c = State(), State()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main, side = torch.cuda.current_stream(), torch.cuda.Stream()
        side.wait_stream(main)
        c.run(stream=side)
        a.run()
        main.wait_stream(side)
        both = a.out + c.out
    g.replay()
    torch.cuda.synchronize()
    assert a.same(want) and c.same(want) and torch.equal(both, want.out + want.out)


def test_calls_of_two_streams_at_once():
    # two batches over one pool, each with its workspace, on streams that run
    # side by side
    b = [P.Batch([1] * 30 + [40], [60] * 30 + [90], 4000, 2, 128, 16, seed=30 + i) for i in range(2)]
    pools = [dev(x.pool, torch.bfloat16) for x in b]
    kvs = [_paged(x, p) for x, p in zip(b, pools)]
    xs = [dev(np.random.default_rng(40 + i).standard_normal((70, 8, 128)), torch.bfloat16) for i in range(2)]
    ws = [torch.empty(q.attention_paged_bytes(k, 70, 8), dtype=torch.uint8, device="cuda") for k in kvs]
    alone = []
    for k, x, w in zip(kvs, xs, ws):
        alone.append(torch.empty_like(x))
        q.op_attention_paged(k, x, alone[-1], w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(x) for x in xs]
    for _ in range(20):
        for s, k, x, o, w in zip(streams, kvs, xs, outs, ws):
            q.op_attention_paged(k, x, o, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(alone, outs))


# Tiles of many rows with more items than there are CTAs (a CTA then takes
# several of them): as pairs of CTAs, as single ones for 64-wide heads and for
# one tile a sequence; ragged, with an empty sequence and one of a single row.
STAYS = [
    ([300, 0, 140, 1, 77], [300, 9, 333, 1, 90], 300, 64, 16, 128, 16),
    ([200, 317], [211, 317], 70, 64, 32, 64, 48),
    ([30] * 39 + [31], list(range(40, 80)), 130, 16, 4, 128, 64),
]
STAY_IDS = ["pair", "single64", "single128"]


@pytest.mark.parametrize("case", STAYS, ids=STAY_IDS)
def test_attention_several_items_a_cta(case):
    counts, lens, prefix, heads, hk, d, page = case
    b = P.Batch(counts, lens, prefix, hk, d, page, seed=41)
    _attend(b, "bf16", heads, pad=3)
    rng = np.random.default_rng(42)
    vis = rng.integers(0, prefix + max(lens) + 1, b.rows)
    vis[: b.rows // 3] = 0  # items without keys among the others
    _attend(b, "f16", heads, vis=vis, pad=1)
    # the same batch in a table of many more rows: an item to a CTA
    wide = np.full((len(counts), 40000 // page), -1, np.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    _attend(b, "bf16", heads)


@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
@pytest.mark.parametrize("case", [([150, 90] * 10, [170, 90] * 10, 100, 16, 4, 128, 16),
                                  ([130] * 13, [150] * 13, 0, 12, 12, 64, 64)], ids=["pair", "single64"])
def test_attention_several_items_a_cta_odd_values(case, bad):
    test_attention_odd_values_behind_the_mask(case, bad)


@pytest.mark.parametrize("copies", [1, 20], ids=["item", "items"])
def test_attention_many_rows_bad_pages_read_as_zeros(copies):
    # whole pages and the one that the end cuts (rows 144 .. 149)
    b = P.Batch([140] * copies, [150] * copies, 64, 4, 128, 16, seed=43, stale=0.0)
    pool = dev(b.pool, torch.float16)
    b.table[0, 1], b.table[0, 9], b.table[copies - 1, 3], b.prefix_pages[2] = pool.shape[0] + 5, -1, -7, pool.shape[0]
    bad = [(0, 1), (0, 9), (copies - 1, 3)]
    kv = _paged(b, pool)
    qx = dev(np.random.default_rng(1).standard_normal((b.rows, 8, 128)), torch.float16)
    out = torch.empty_like(qx)
    ws = torch.empty(q.attention_paged_bytes(kv, b.rows, 8), dtype=torch.uint8, device="cuda")
    q.op_attention_paged(kv, qx, out, ws)
    assert q.device_status() == 2
    zero = torch.cat([pool, torch.zeros_like(pool[:1])])
    for at in bad:
        b.table[at] = pool.shape[0]
    b.prefix_pages[2] = pool.shape[0]
    want, bound = P.attention(b, host(zero), host(qx), b.seen(True), 128 ** -0.5, P.U["f16"])
    assert np.all(np.abs(host(out) - want) <= bound)


def test_attention_many_rows_past_32_bits():
    # a pool of more than 2^31 values, the used pages at its end
    page, hk, d = 256, 8, 128
    n = (1 << 31) // (page * 2 * hk * d) + 6
    pool = torch.zeros(n, page, 2, hk, d, dtype=torch.bfloat16, device="cuda")
    b = P.Batch([200, 30], [299, 30], 100, hk, d, page, seed=44)
    last = n - b.pool.shape[0]
    pool[last:] = dev(b.pool, torch.bfloat16)
    tail = pool[last:]
    small = b.table.copy(), b.prefix_pages.copy()
    b.table = np.where(b.table >= 0, b.table + last, -1).astype(np.int32)
    b.prefix_pages = (b.prefix_pages + last).astype(np.int32)
    kv = _paged(b, pool)
    b.table, b.prefix_pages = small
    _attend(b, "bf16", 16, kv=kv, pool=tail)


def test_captures_of_several_items_a_cta():
    test_captures_that_fork_and_that_start_with_a_call(([90] * 20, [95] * 20, 100))


def test_several_items_a_cta_on_two_streams():
    b = P.Batch([90] * 20, [95] * 20, 500, 4, 128, 16, seed=45)
    pool = dev(b.pool, torch.bfloat16)
    kv = _paged(b, pool)
    xs = [dev(np.random.default_rng(46 + i).standard_normal((b.rows, 8, 128)), torch.bfloat16) for i in range(2)]
    ws = [torch.empty(q.attention_paged_bytes(kv, b.rows, 8), dtype=torch.uint8, device="cuda") for _ in xs]
    alone = [torch.empty_like(x) for x in xs]
    for x, w, o in zip(xs, ws, alone):
        q.op_attention_paged(kv, x, o, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [torch.empty_like(x) for x in xs]
    for _ in range(20):
        for s, x, o, w in zip(streams, xs, outs, ws):
            q.op_attention_paged(kv, x, o, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(alone, outs))


def test_python_refusals():
    b = P.Batch([2], [4], 10, 2, 64, 16, seed=1)
    pool = dev(b.pool, torch.float16)
    kv = _paged(b, pool)
    x = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    ws = torch.empty(q.attention_paged_bytes(kv, 2, 4), dtype=torch.uint8, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    r = q.rope(64)
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (lambda: q.op_attention_paged(kv, x.cpu(), x, ws), lambda: q.op_attention_paged(kv, x.float(), x, ws),
                lambda: q.op_attention_paged(kv, x, x.bfloat16(), ws), lambda: q.op_kv_append(kv, k.float(), k),
                lambda: q.op_rope(r, x.double(), pos), lambda: q.op_rope(r, x, pos.int()),
                lambda: q.op_attention_paged(kv, x, x.clone(), ws, vis=pos)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: q.op_attention_paged(kv, x, x[:1], ws), lambda: q.op_attention_paged(kv, x[..., :32], x, ws),
                lambda: q.op_attention_paged(kv, x.transpose(0, 1), x, ws), lambda: q.op_kv_append(kv, x, x),
                lambda: q.op_kv_append(kv, k, k[:1]), lambda: q.op_rope(r, x, pos[:1]),
                lambda: q.op_rope(r, x[:1].expand(2, 4, 64), pos), lambda: q.op_rope(r, x, pos, out=x[:, :2]),
                lambda: q.PagedKV(pool[0], dev(b.table), kv._keep[2], kv._keep[3]),
                lambda: q.PagedKV(pool, dev(b.table), kv._keep[2][:0], kv._keep[3]),
                lambda: q.PagedKV(pool, dev(b.table), kv._keep[2], kv._keep[3], prefix_len=5),
                lambda: q.PagedKV(pool, dev(b.table), kv._keep[2], kv._keep[3], prefix_pages=kv._keep[4], prefix_len=99)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.Qi21Error) as e:
        q.op_attention_paged(kv, x, x.clone(), ws[:256])
    assert e.value.code == -8
    with pytest.raises(q.Qi21Error):
        q.attention_paged_bytes(kv, 2, 3)


def test_python_refusals_of_lengths_and_positions():
    b = P.Batch([2], [4], 10, 2, 64, 16, seed=1)
    pool = dev(b.pool, torch.float16)
    for n in (-1, 1 << 30, (1 << 32) + 5):
        with pytest.raises(ValueError):
            q.PagedKV(pool, dev(b.table), dev(np.array([4], np.int32)), dev(b.cu),
                      prefix_pages=dev(b.prefix_pages), prefix_len=n)
    r = q.rope(64, axes=(16, 24, 24))
    x = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    pos = torch.zeros(3, 2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        q.op_rope(r, x, pos)
    with pytest.raises(ValueError):
        q.op_kv_append(_paged(b, pool), x, x, rope=r, pos=pos)
    many = torch.zeros(1, 1, 64, dtype=torch.float16, device="cuda").expand((1 << 32) + 1, 1, 64)
    with pytest.raises(ValueError):
        q.op_rope(q.rope(64), many, pos)


# --------------------------------------------------------------- together ----

def test_generation_over_a_shared_prefix():
    """A prompt appended once, then decode steps of five sequences that share
    it: rotate q, append k and v, attend, step after step, captured in one
    graph whose lengths move between the replays; against 64 bits."""
    dt, u = torch.bfloat16, P.U["bf16"]
    d, hk, heads, page, nseq, steps, lp = 64, 2, 6, 16, 5, 20, 37
    rng = np.random.default_rng(20)
    r, freqs = q.rope(d, 48, layout="half", scaling="linear", factor=2.0), P.frequencies(48, "linear", 2.0)
    npre, per = -(-lp // page), -(-steps // page)
    order = rng.permutation(npre + nseq * per).astype(np.int32)
    pool = torch.full((len(order), page, 2, hk, d), float("nan"), dtype=dt, device="cuda")
    pre = dev(order[:npre])
    table = dev(order[npre:].reshape(nseq, per))

    kp, vp = (dev(rng.standard_normal((lp, hk, d)), dt) for _ in range(2))
    prompt = q.PagedKV(pool, pre[None], dev(np.array([lp], np.int32)), dev(np.array([0, lp], np.int32)))
    q.op_kv_append(prompt, kp, vp, rope=r)

    lens = torch.zeros(nseq, dtype=torch.int32, device="cuda")
    kv = q.PagedKV(pool, table, lens, dev(np.arange(nseq + 1, dtype=np.int32)), prefix_pages=pre, prefix_len=lp)
    x, k, v, out = (torch.zeros(nseq, h, d, dtype=dt, device="cuda") for h in (heads, hk, hk, heads))
    pos = torch.zeros(nseq, dtype=torch.int64, device="cuda")
    ws = torch.empty(q.attention_paged_bytes(kv, nseq, heads), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        pos.copy_(lens)
        pos.add_(lp - 1)
        q.op_rope(r, x, pos)
        q.op_kv_append(kv, k, v, rope=r)
        q.op_attention_paged(kv, x, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    lens.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def rotated(t, where):  # as the cache holds it
        y = P.rotate(host(t), where, freqs, 48, "half")
        return torch.from_numpy(y).to(dt).double().numpy()

    keys = [np.repeat(rotated(kp, np.arange(lp))[None], nseq, 0)]
    vals = [np.repeat(host(vp)[None], nseq, 0)]
    for i in range(steps):
        qs, ks, vs = (rng.standard_normal((nseq, h, d)) for h in (heads, hk, hk))
        x.copy_(dev(qs, dt)), k.copy_(dev(ks, dt)), v.copy_(dev(vs, dt))
        at = np.full(nseq, lp + i)
        qr = rotated(x, at)
        keys.append(rotated(k, at)[:, None])
        vals.append(host(v)[:, None])
        graph.replay()
        got = host(out)
        kk, vv = np.concatenate(keys, 1), np.concatenate(vals, 1)
        s = np.einsum("bhgd,bkhd->bhgk", qr.reshape(nseq, hk, 3, d), kk) / 8
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want = np.einsum("bhgk,bkhd->bhgd", p, vv).reshape(nseq, heads, d)
        w = np.einsum("bhgk,bkhd->bhgd", p, np.abs(vv)).reshape(nseq, heads, d)
        # P and out rounded (u each); q and k were rounded from f32 rotations
        # here and from f64 ones in the oracle, so a few may differ by a step
        # (2 u of a value): of the scores that is 4 u sum |q k| / 8 at most
        tq = np.einsum("bhgd,bkhd->bhgk", np.abs(qr).reshape(nseq, hk, 3, d), np.abs(kk)).max() / 8
        assert np.all(np.abs(got - want) <= (u + 8 * u * tq) * w + u * np.abs(want))
        assert np.median(np.abs(got - want)) <= u * np.median(w)
