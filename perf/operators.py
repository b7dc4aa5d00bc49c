"""Cases and plain forms of the serving operators around the paged K/V cache:

  rope       rotary positions of [rows, heads, dim] vectors (forward and gradient)
  append     new keys (rotated on the way) and values into a paged cache
  attention  a batch's queries over [a prefix that all sequences share, own
             pages], the prefix's part computed once for the batch

A cache page holds `page` rows of [2, kv_heads, dim] (K, then V). Lengths of a
ragged batch follow from the case alone (`_spread`), values from the seed.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_AXES = (16, 56, 56)  # frame, height, width: the image layout's split of a 128-wide head


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one new token for each of 8 sequences: queries of a decode step
        dict(name="rope_decode", op="rope", rows=8, heads=32, dim=128, rot=128, layout="interleaved", image=False,
             scaling="plain", factor=1.0, far=20000, dtype="bf16", grad=False, panel=False),
        # a long prompt whose context was stretched: half layout, frequencies scaled by parts, far positions
        dict(name="rope_long", op="rope", rows=32768, heads=32, dim=128, rot=128, layout="half", image=False,
             scaling="ramp", factor=8.0, far=262144, dtype="bf16", grad=False, panel=False),
        # gradient through the rotation of part of the head, read out of the q|k|v panel, odd row count
        dict(name="rope_grad_part", op="rope", rows=4099, heads=16, dim=128, rot=64, layout="interleaved", image=False,
             scaling="linear", factor=4.0, far=16384, dtype="f32", grad=True, panel=True),
        # one token for each of 64 sequences goes to its page
        dict(name="append_decode", op="append", nseq=64, n_min=1, n_max=1, before=900, kv_heads=8, dim=128, rot=128,
             layout="half", image=False, scaling="plain", factor=1.0, page=64, dtype="bf16", panel=False),
        # prompts of 8 requests, ragged, starting inside a page
        dict(name="append_prompts", op="append", nseq=8, n_min=1500, n_max=6500, before=37, kv_heads=8, dim=128,
             rot=128, layout="half", image=False, scaling="band", factor=8.0, page=64, dtype="bf16", panel=False),
        # rows of four 32 x 32 images with their three-axis positions, out of the q|k|v panel
        dict(name="append_images", op="append", nseq=4, n_min=1024, n_max=1024, before=0, kv_heads=32, dim=128,
             rot=128, layout="interleaved", image=True, scaling="plain", factor=1.0, page=16, dtype="f16", panel=True),
        # two short chats behind a short prompt: latency
        dict(name="attn_small", op="attention", nseq=2, n_min=1, n_max=1, own_min=9, own_max=40, prefix=200, heads=32,
             kv_heads=8, dim=128, page=16, mask="causal", dtype="bf16"),
        # a decode step of 48 sequences behind one prompt
        dict(name="attn_decode", op="attention", nseq=48, n_min=1, n_max=1, own_min=1, own_max=700, prefix=8197,
             heads=32, kv_heads=8, dim=128, page=64, mask="causal", dtype="bf16"),
        # a decode step of 128 samples of one very long prompt
        dict(name="attn_decode_long", op="attention", nseq=128, n_min=1, n_max=1, own_min=100, own_max=1000,
             prefix=65536, heads=32, kv_heads=8, dim=128, page=64, mask="causal", dtype="bf16"),
        # several drafted tokens each, 64-wide heads, 7 query heads to a key head
        dict(name="attn_draft", op="attention", nseq=16, n_min=3, n_max=6, own_min=50, own_max=400, prefix=3001,
             heads=28, kv_heads=4, dim=64, page=48, mask="causal", dtype="f16"),
        # prompts' own parts behind a shared system prompt
        dict(name="attn_prompts", op="attention", nseq=3, n_min=700, n_max=1800, own_min=700, own_max=2100,
             prefix=2048, heads=32, kv_heads=8, dim=128, page=64, mask="causal", dtype="bf16"),
        # four 32 x 32 images of one prompt with a condition image (18 + 64 * 64 rows), every key visible
        dict(name="attn_images", op="attention", nseq=4, n_min=1024, n_max=1024, own_min=1024, own_max=1024,
             prefix=4114, heads=32, kv_heads=32, dim=128, page=64, mask="none", dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotation(rng):
    image = rng.random() < 0.2
    dim = 128 if image else rng.choice([64, 128])
    rot = dim if image or rng.random() < 0.6 else rng.choice([dim // 2, dim // 4, dim - 16, 20])
    return dict(dim=dim, rot=rot, image=image,
                layout="interleaved" if image else rng.choice(["interleaved", "half"]),
                scaling="plain" if image else rng.choice(["plain", "linear", "base", "ramp", "band"]),
                factor=rng.choice([2.0, 4.0, 8.0, 32.0]))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    if op == "rope":
        c = dict(op=op, **_draw_rotation(rng))
        c["heads"] = rng.choice([1, 2, 8, 16, 28, 32])
        c["rows"] = _log(rng, 1, 32768 * 32 * 64 // (c["heads"] * c["dim"]) if c["heads"] > 8 else 60000)
        c.update(far=_log(rng, 100, 1 << 20), dtype=rng.choice(["f16", "bf16", "bf16", "f32"]),
                 grad=rng.random() < 0.3, panel=rng.random() < 0.4)
        return c
    if op == "append":
        c = dict(op=op, **_draw_rotation(rng))
        c["kv_heads"] = rng.choice([1, 2, 4, 8, 32])
        c["nseq"] = _log(rng, 1, 100)
        top = max(1, min(6500, 8 * 6500 * 8 * 64 // (c["nseq"] * c["kv_heads"] * c["dim"])))
        n = _log(rng, 1, top)
        c.update(n_min=max(0, n // 3), n_max=n, before=rng.randrange(0, 1000), page=rng.choice([16, 48, 64, 128]),
                 dtype=rng.choice(["f16", "bf16"]), panel=rng.random() < 0.4)
        return c
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), dim=rng.choice([64, 128, 128]),
             page=rng.choice([16, 48, 64, 128, 256]))
    if rng.random() < 0.65:  # decode steps
        c["heads"], c["kv_heads"] = rng.choice([(32, 8), (32, 8), (28, 4), (8, 8), (16, 1), (64, 8), (20, 4), (5, 5)])
        c["nseq"] = _log(rng, 1, 128)
        n = rng.choice([1, 1, 1, 2, 5])
        own_max = _log(rng, n, 1000)
        c.update(n_min=1, n_max=n, own_min=max(1, own_max // 5), own_max=own_max, mask="causal",
                 prefix=rng.choice([0, _log(rng, 30, 40000), _log(rng, 1000, 40000)]))
    else:  # rows of prompts or of images
        c["heads"], c["kv_heads"] = rng.choice([(32, 8), (28, 4), (8, 8), (16, 1), (32, 32)])
        c["nseq"] = rng.randint(1, 4)
        n = _log(rng, 20, 1024)
        c.update(n_min=max(1, n // 2), n_max=n, own_min=n // 2, own_max=n + rng.randrange(0, 500),
                 mask=rng.choice(["causal", "none", "runs"]), prefix=rng.choice([0, _log(rng, 30, 4000)]))
    while work(c)["flops"] > (130e9 if c["n_max"] < 20 else 340e9):  # no dearer than the listed ones
        c["prefix"] //= 2
    return c


def _spread(n, lo, hi, salt):
    """n whole numbers of [lo, hi] that follow from their place alone."""
    return [lo + (((i + 1) * 2654435761 + salt * 40503) >> 7) % (hi - lo + 1) for i in range(n)]


def _counts(case):
    """New rows of each sequence (the first has the most)."""
    return [case["n_max"]] + _spread(case["nseq"], case["n_min"], case["n_max"], 1)[1:]


def _lengths(case, counts):
    """Own rows of each sequence, the new ones among them."""
    if case["op"] == "append":
        before = _spread(case["nseq"], 0, case["before"], 2)
        return [b + n for b, n in zip(before, counts)]
    return [max(n, m) for n, m in zip(counts, _spread(case["nseq"], case["own_min"], case["own_max"], 2))]


def _seen(case, counts, lengths):
    """Keys that each new row sees: a leading run of [prefix, own rows]."""
    p = case["prefix"]
    out = []
    for b, (n, m) in enumerate(zip(counts, lengths)):
        if case["mask"] == "none":
            out += [p + m] * n
        elif case["mask"] == "causal":
            out += [p + m - n + i + 1 for i in range(n)]
        else:  # runs of their own, some of them empty
            out += [0 if (i + b) % 50 == 7 else r for i, r in enumerate(_spread(n, 1, p + m, 3 + b))]
    return out


def work(case):
    if case["op"] == "rope":
        e = 4 if case["dtype"] == "f32" else 2
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * e * n * case["dim"] + 8 * case["rows"] * (3 if case["image"] else 1),
                "flops": 3 * n * case["rot"]}
    counts = _counts(case)
    lengths = _lengths(case, counts)
    rows = sum(counts)
    if case["op"] == "append":
        n = rows * case["kv_heads"]
        return {"bytes": 2 * 2 * 2 * n * case["dim"] + 8 * rows * (3 if case["image"] else 1),
                "flops": 3 * n * case["rot"]}
    keys = case["prefix"] + sum(lengths)
    return {"bytes": 2 * case["dim"] * (2 * rows * case["heads"] + 2 * keys * case["kv_heads"]),
            "flops": 4 * case["dim"] * case["heads"] * sum(_seen(case, counts, lengths))}


# ----------------------------------------------------------------- inputs ----

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(case, rows, heads, g, dtype):
    """[rows, heads, dim] values; with `panel` the columns of wider rows."""
    wide = 3 * heads if case.get("panel") else heads
    x = torch.randn(rows, wide, case["dim"], device="cuda", generator=g, dtype=torch.float32).to(dtype)
    return x[:, wide - heads:] if case.get("panel") else x


def _image_positions(rows):
    """(frame, h, w) of `rows` rows of 32-wide images at frame 18, centred."""
    i = torch.arange(rows, device="cuda")
    return torch.stack([torch.full_like(i, 18), (i // 32) % 32 - 16, i % 32 - 16], 1)


def _pages(lengths, page, first, order):
    """Page table of the sequences: pages order[first ...], spare entries -1."""
    need = [(m + page - 1) // page for m in lengths]
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32)
    at = first
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, at


def prepare(case, seed):
    g = _generator(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}
    if case["op"] == "rope":
        rows = case["rows"]
        st["x"] = _rows(case, rows, case["heads"], g, dt)
        if case["image"]:
            st["pos"] = _image_positions(rows)
        else:
            first = torch.randint(0, case["far"], (1,), device="cuda", generator=g)
            st["pos"] = (torch.arange(rows, device="cuda") + first) % case["far"]
        st["out"] = torch.empty(rows, case["heads"], case["dim"], device="cuda", dtype=dt)
        if own:
            st["plan"] = _own_plan(st)
        return st
    counts = _counts(case)
    lengths = _lengths(case, counts)
    page = case["page"]
    prefix = case.get("prefix", 0)
    n_prefix = (prefix + page - 1) // page
    total = n_prefix + sum((m + page - 1) // page for m in lengths)
    # pages of a long-lived pool: in no order, stale values behind each sequence's end
    order = torch.randperm(total + 3, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, _ = _pages(lengths, page, n_prefix, order)
    st["pool"] = torch.randn(total + 3, page, 2, case["kv_heads"], case["dim"], device="cuda", generator=g,
                             dtype=torch.float32).to(dt)
    st["table"] = table.cuda()
    st["prefix_pages"] = order[:n_prefix].cuda()
    st["lens"] = torch.tensor(lengths, dtype=torch.int32).cuda()
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    rows = cu[-1]
    if case["op"] == "append":
        st["k"] = _rows(case, rows, case["kv_heads"], g, dt)
        st["v"] = _rows(case, rows, case["kv_heads"], g, dt)
        if case["image"]:
            st["pos"] = _image_positions(rows)
        else:
            st["pos"] = torch.tensor([m - n + i for n, m in zip(counts, lengths) for i in range(n)],
                                     dtype=torch.int64).cuda()
    else:
        # queries of a trained model look for some keys: scores wider than those of unit vectors
        st["q"] = (1.5 * torch.randn(rows, case["heads"], case["dim"], device="cuda", generator=g)).to(dt)
        st["out"] = torch.empty_like(st["q"])
        st["vis"] = torch.tensor(_seen(case, counts, lengths), dtype=torch.int32).cuda()
    if own:
        st["plan"] = _own_plan(st)
    return st


# ----------------------------------------------------- the framework's calls ----

def _own_rope(case):
    import diffusion_transformer_denoiser_qi21_gb300 as q
    return q.rope(case["dim"], case["rot"], layout=case["layout"], axes=_AXES if case["image"] else None,
                  base=10000.0, scaling=case["scaling"], factor=case["factor"], orig_len=8192)


def _own_plan(st):
    """What a program keeps between calls: the rotation, the cache's
    description and a workspace."""
    import diffusion_transformer_denoiser_qi21_gb300 as q
    case = st["case"]
    if case["op"] == "rope":
        return {"rope": _own_rope(case)}
    kv = q.PagedKV(st["pool"], st["table"], st["lens"], st["cu"], prefix_pages=st["prefix_pages"],
                   prefix_len=case.get("prefix", 0))
    if case["op"] == "append":
        return {"kv": kv, "rope": _own_rope(case)}
    nbytes = q.attention_paged_bytes(kv, st["q"].shape[0], case["heads"])
    return {"kv": kv, "ws": torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")}


def _run_own(st):
    import diffusion_transformer_denoiser_qi21_gb300 as q
    case = st["case"]
    if "plan" not in st:
        st["plan"] = _own_plan(st)
    plan = st["plan"]
    if case["op"] == "rope":
        q.op_rope(plan["rope"], st["x"], st["pos"], out=st["out"], grad=case["grad"])
        return st["out"]
    if case["op"] == "append":
        q.op_kv_append(plan["kv"], st["k"], st["v"], rope=plan["rope"], pos=st["pos"])
        return st["pool"]
    q.op_attention_paged(plan["kv"], st["q"], st["out"], plan["ws"], causal=case["mask"] == "causal",
                         vis=st["vis"] if case["mask"] == "runs" else None)
    return st["out"]


# ------------------------------------------------------------ plain forms ----

def _frequencies(width, scaling, factor, base=10000.0, orig_len=8192):
    """Angles per position of the width / 2 pairs, in 64 bits."""
    i = torch.arange(width // 2, dtype=torch.float64)
    if scaling == "base":  # the base stretched so that the slowest pair is slowed by the factor
        base = base * factor ** (width / (width - 2))
    f = base ** (-2 * i / width)
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":  # by parts: pairs that turn often keep their speed, slow ones are slowed
        def pair_of(turns):
            return width * math.log(orig_len / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(pair_of(32))), min(width - 1, math.ceil(pair_of(1)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    elif scaling == "band":  # between two wavelengths, mixed by how often the pair turns
        turns = orig_len * f / (2 * math.pi)
        mix = ((turns - 1) / (4 - 1)).clamp(0, 1)
        f = f * mix + f / factor * (1 - mix)
    return f


def _angles(case, pos):
    """[rows, rot / 2] angles in 64 bits."""
    if case["image"]:
        f = [_frequencies(w, "plain", 1.0).to(pos.device) for w in _AXES]
        return torch.cat([pos[:, a:a + 1].double() * f[a] for a in range(3)], 1)
    f = _frequencies(case["rot"], case["scaling"], case["factor"]).to(pos.device)
    return pos.double()[:, None] * f


def _out_scale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


def _rotate(case, x, pos, grad=False):
    a = _angles(case, pos)
    s = _out_scale(case)
    c = (a.cos() * s).float()[:, None]
    sn = (a.sin() * s).float()[:, None]
    if grad:
        sn = -sn
    r = case["rot"]
    out = x.float()
    h = out[..., :r]
    if case["layout"] == "half":
        u, v = h[..., :r // 2], h[..., r // 2:]
        h = torch.cat([u * c - v * sn, u * sn + v * c], -1)
    else:
        u, v = h[..., 0::2], h[..., 1::2]
        h = torch.stack([u * c - v * sn, u * sn + v * c], -1).flatten(-2)
    return torch.cat([h, out[..., r:]], -1)


def _slots(st):
    """Row of the flattened pool for each new row."""
    cu, lens, table = st["cu"].long(), st["lens"].long(), st["table"].long()
    page = st["case"]["page"]
    rows = torch.arange(st["k"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, rows, right=True) - 1
    at = lens[b] - (cu[b + 1] - rows)
    return table[b, at // page] * page + at % page


def _run_attention(st):
    case = st["case"]
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["heads"] // hk
    cu, lens = st["cu"].long(), st["lens"].long()
    counts = _counts(case)
    nseq, n_max, m_max = case["nseq"], max(counts), max(_lengths(case, counts))
    rows = st["q"].shape[0]
    dev = cu.device
    t = torch.arange(rows, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    q = st["q"].float().view(rows, hk, g, d) * (1.0 / math.sqrt(d))
    pool = st["pool"].view(-1, 2, hk, d)

    def keys(pages, n):
        at = torch.arange(n, device=dev)
        return pool[pages.long()[..., at // page].clamp_min(0) * page + at % page].float()

    shared = keys(st["prefix_pages"], case["prefix"]) if case["prefix"] else pool[:0].float()
    mine = keys(st["table"], m_max)                                     # [nseq, m_max, 2, hk, d]
    qp = torch.zeros(nseq, n_max, hk, g, d, device=dev)
    qp[b, i] = q
    s1 = torch.einsum("thgd,khd->thgk", q, shared[:, 0])
    s2 = torch.einsum("bihgd,bkhd->bihgk", qp, mine[:, :, 0])[b, i]
    seen = st["vis"].long()
    at = torch.arange(case["prefix"], device=dev)
    ok1 = at[None] < seen[:, None]
    at = torch.arange(m_max, device=dev)
    ok2 = (at[None] + case["prefix"] < seen[:, None]) & (at[None] < lens[b][:, None])
    s = torch.cat([s1.masked_fill(~ok1[:, None, None], -math.inf), s2.masked_fill(~ok2[:, None, None], -math.inf)], -1)
    m = s.amax(-1, keepdim=True)
    p = (s - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp()
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    p1, p2 = p[..., :case["prefix"]], p[..., case["prefix"]:]
    o = torch.einsum("thgk,khd->thgd", p1, shared[:, 1])
    pp = torch.zeros(nseq, n_max, hk, g, m_max, device=dev)
    pp[b, i] = p2
    # a row behind a sequence's end holds what the page held before
    v = mine[:, :, 1] * (at[None] < lens[:, None])[:, :, None, None]
    o = o + torch.einsum("bihgk,bkhd->bihgd", pp, v)[b, i]
    return o.reshape(rows, case["heads"], d).to(st["q"].dtype)


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "rope":
        return _rotate(case, st["x"], st["pos"], case["grad"]).to(st["x"].dtype)
    if case["op"] == "append":
        rows = torch.stack([_rotate(case, st["k"], st["pos"]), st["v"].float()], 1).to(st["pool"].dtype)
        st["pool"].view(-1, 2, case["kv_heads"], case["dim"])[_slots(st)] = rows
        return st["pool"]
    return _run_attention(st)


# ------------------------------------------------------------------ exact ----

def _exact_rotation(case, pos):
    """Complex factors [rows, rot / 2] of the pairs, from the definition."""
    widths = _AXES if case["image"] else (case["rot"],)
    cols = []
    for a, w in enumerate(widths):
        where = (pos[:, a] if case["image"] else pos).to(torch.float64)
        for j in range(w // 2):
            base, k = 10000.0, case["factor"]
            if case["scaling"] == "base":
                base *= math.pow(k, w / (w - 2.0))
            f = math.pow(base, -2.0 * j / w)
            if case["scaling"] == "linear":
                f /= k
            if case["scaling"] == "ramp":
                edge = [w * math.log(8192 / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32, 1)]
                lo, hi = max(0.0, math.floor(edge[0])), min(w - 1.0, math.ceil(edge[1]))
                y = min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3)))
                f = (1 - y) * f + y * f / k
            if case["scaling"] == "band":
                y = min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 3.0))
                f = y * f + (1 - y) * f / k
            cols.append(torch.polar(torch.ones_like(where), where * f))
    z = torch.stack(cols, 1)
    return z * (1.0 + 0.1 * math.log(case["factor"])) if case["scaling"] == "ramp" else z


def _exact_rotate(case, x, pos, grad=False):
    z = _exact_rotation(case, pos)[:, None]
    if grad:
        z = z.conj()
    r = case["rot"]
    y = x.to(torch.float64).clone()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half" else (slice(0, r, 2),
                                                                                            slice(1, r, 2))
    w = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
    y[..., first] = w.real
    y[..., second] = w.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotate(case, st["x"], st["pos"], case["grad"])
    counts = _counts(case)
    lengths = _lengths(case, counts)
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    table = st["table"].tolist()
    if case["op"] == "append":
        pool = st["pool"].to(torch.float64)
        k = _exact_rotate(case, st["k"], st["pos"])
        row = 0
        for b, (n, m) in enumerate(zip(counts, lengths)):
            at = m - n
            while at < m:  # page by page
                take = min(m - at, page - at % page)
                dst = pool[table[b][at // page], at % page:at % page + take]
                dst[:, 0] = k[row:row + take]
                dst[:, 1] = st["v"][row:row + take].to(torch.float64)
                at += take
                row += take
        return pool
    out = torch.zeros(sum(counts), case["heads"], d, dtype=torch.float64, device="cuda")
    seen = _seen(case, counts, lengths)
    shared = [int(p) for p in st["prefix_pages"].tolist()]
    group = case["heads"] // hk
    head = st["pool"][shared].flatten(0, 1)[:case["prefix"]]
    row = 0
    for b, (n, m) in enumerate(zip(counts, lengths)):
        if n == 0:
            continue
        tail = st["pool"][[p for p in table[b] if p >= 0]].flatten(0, 1)[:m]
        runs = torch.tensor(seen[row:row + n], device="cuda")
        mask = torch.arange(case["prefix"] + m, device="cuda")[None] < runs[:, None]
        for h in range(hk):
            kv = torch.cat([head[:, :, h], tail[:, :, h]]).to(torch.float64)
            qh = st["q"][row:row + n, h * group:(h + 1) * group].to(torch.float64)
            w = torch.exp(torch.matmul(qh.transpose(0, 1), kv[:, 0].T) / math.sqrt(d)) * mask
            z = w.sum(-1, keepdim=True)
            out[row:row + n, h * group:(h + 1) * group] = \
                (torch.matmul(w, kv[:, 1]) / torch.where(z == 0, torch.ones_like(z), z)).transpose(0, 1)
        row += n
    return out
