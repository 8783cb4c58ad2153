"""Cases of the operators around the compressed rows: rotary positions (``rope``), the 8-bit paged
cache's writer (``append``), the attention that reads it (``attend``) and the handling of its pages
(``pages``). Each has a plain form of elementary torch operations in 32 bits (64 for angles) and,
where ``own`` is true, the calls a user makes of the package."""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one decoding step's queries: 16 tokens x 64 heads, the last 64 columns of each head turned
        {"name": "rope step", "op": "rope", "tokens": 16, "heads": 64, "head_dim": 512, "rope_dim": 64, "offset": 448,
         "layout": "interleaved", "dtype": "bf16", "train": False, "rows": False, "far": False, "scaling": "none"},
        # training: the headline pack's compressed rows (ratio 4) turned at their block's first token, and the gradient
        {"name": "rope rows train", "op": "rope", "tokens": 66533, "heads": 1, "head_dim": 512, "rope_dim": 64, "offset": 448,
         "layout": "interleaved", "dtype": "bf16", "train": True, "rows": True, "far": False, "scaling": "none"},
        # a long prompt's keys, whole heads in the half layout, frequencies stretched for long contexts
        {"name": "rope long half", "op": "rope", "tokens": 32768, "heads": 8, "head_dim": 128, "rope_dim": 128, "offset": 0,
         "layout": "half", "dtype": "fp16", "train": False, "rows": False, "far": True, "scaling": "yarn"},
        # one new compressed row for each of 64 sequences
        {"name": "append step", "op": "append", "batch": 64, "new": 1, "held": 4000, "heads": 1, "head_dim": 512, "page": 64, "block": 16,
         "dtype": "bf16", "ragged": False},
        # the headline pack's rows (64 ragged sequences) after the compressor has run over a prompt
        {"name": "append pack", "op": "append", "batch": 64, "new": 2046, "held": 0, "heads": 1, "head_dim": 512, "page": 64, "block": 64,
         "dtype": "bf16", "ragged": True},
        # one short sequence: latency
        {"name": "attend one", "op": "attend", "batch": 1, "queries": 1, "heads": 16, "kv_heads": 1, "head_dim": 512, "shared": True, "held": 300,
         "page": 64, "block": 16, "dtype": "bf16", "ragged": False},
        # a decoding batch, a row is key and value of all heads
        {"name": "attend latent", "op": "attend", "batch": 64, "queries": 1, "heads": 64, "kv_heads": 1, "head_dim": 512, "shared": True,
         "held": 16384, "page": 64, "block": 64, "dtype": "bf16", "ragged": True},
        # a decoding batch, grouped heads with keys and values of their own
        {"name": "attend groups", "op": "attend", "batch": 32, "queries": 1, "heads": 64, "kv_heads": 8, "head_dim": 128, "shared": False,
         "held": 8192, "page": 64, "block": 32, "dtype": "bf16", "ragged": True},
        # one sequence of 262144 tokens (65536 rows at ratio 4)
        {"name": "attend long", "op": "attend", "batch": 1, "queries": 1, "heads": 64, "kv_heads": 1, "head_dim": 512, "shared": True,
         "held": 65536, "page": 64, "block": 64, "dtype": "bf16", "ragged": False},
        # a prompt's chunks: each query sees the rows that end at or before it; one sequence has no rows yet
        {"name": "attend chunk", "op": "attend", "batch": 4, "queries": 255, "heads": 16, "kv_heads": 2, "head_dim": 128, "shared": False,
         "held": 4099, "page": 32, "block": 32, "dtype": "fp16", "ragged": True},
        # 32 sequences forked into 8 branches each, and room for the branches' next rows (shared last pages copied)
        {"name": "pages fork", "op": "pages", "do": "fork", "batch": 32, "branches": 8, "held": 2000, "new": 3, "heads": 1, "head_dim": 512,
         "page": 64, "block": 64, "spare": 600},
        # a third of 192 sequences ends; the others' pages move to the front of the pool
        {"name": "pages compact", "op": "pages", "do": "compact", "batch": 192, "branches": 0, "held": 2000, "new": 0, "heads": 1, "head_dim": 512,
         "page": 64, "block": 64, "spare": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "attend", "attend", "attend", "pages"])
    if op == "rope":
        d = rng.choice([64, 128, 256, 512])
        part = rng.choice([32, 64, d])
        part = min(part, d)
        heads = rng.choice([1, 2, 5, 8, 16])
        return {"op": "rope", "tokens": _log(rng, 1, 30_000_000 // (heads * d)), "heads": heads, "head_dim": d, "rope_dim": part,
                "offset": rng.choice([0, d - part]), "layout": rng.choice(["interleaved", "half"]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "train": rng.random() < 0.4, "rows": rng.random() < 0.4, "far": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "yarn"])}
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (1, 8, 16, 32, 64, 128) if b <= page])
    if op == "append":
        d, heads = rng.choice([(512, 1), (256, 2), (128, 8), (64, 3)])
        batch = _log(rng, 1, 128)
        return {"op": "append", "batch": batch, "new": _log(rng, 1, 2000), "held": _log(rng, 1, 6000) - 1, "heads": heads, "head_dim": d,
                "page": page, "block": block, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "ragged": rng.random() < 0.6}
    if op == "attend":
        d = rng.choice([64, 128, 256, 512])
        shared = rng.random() < 0.5
        kv = 1 if d == 512 else rng.choice([1, 2, 8])
        group = rng.choice([1, 3, 4, 8, 16]) if kv > 1 else rng.choice([1, 8, 16, 40, 64, 128])
        queries = rng.choice([1, 1, 1, 2, 4, 70, 300])
        most = 1.5e11 / (4.0 * d * kv * group * queries)          # rows over all sequences, by operations
        most = min(most, 4e8 / (kv * d * (1 if shared else 2)))    # and by bytes
        most_batch = max(1, min(int(most // 64), 80_000_000 // (queries * kv * group * d)))
        batch = min(_log(rng, 1, 96), most_batch)
        return {"op": "attend", "batch": batch, "queries": queries, "heads": kv * group, "kv_heads": kv, "head_dim": d, "shared": shared,
                "held": _log(rng, 17, max(32, min(65536, int(most // batch)))), "page": page, "block": block,
                "dtype": rng.choice(["bf16", "bf16", "fp16"]), "ragged": rng.random() < 0.7}
    d, heads = rng.choice([(512, 1), (128, 8), (64, 2)])
    batch = _log(rng, 2, 128)
    fork = rng.random() < 0.5
    return {"op": "pages", "do": "fork" if fork else "compact", "batch": batch, "branches": rng.choice([1, 2, 5]) if fork else 0,
            "held": _log(rng, 1, 100_000 // batch + 1), "new": rng.choice([1, 3, 70]) if fork else 0, "heads": heads, "head_dim": d, "page": page,
            "block": block, "spare": batch * 16 + rng.randrange(500)}


def _lens(case, key, n, least=0):
    """Lengths of the sequences: `case[key]`, or spread over [least, case[key]] with the ends among them."""
    top = case[key]
    if not case.get("ragged", True):
        return [top] * n
    r = random.Random("%s %d %d" % (key, top, n))
    v = [r.randint(max(least, top // 4), top) for _ in range(n)]
    if n > 2:
        v[n // 2], v[0] = least, top
    return v


def _counts(case):
    """(rows held, queries) of each sequence of an attend case."""
    n = case["batch"]
    return _lens(case, "held", n), _lens(case, "queries", n, least=1)


def _sums(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _visible(case):
    """Rows that each query sees: a row stands for four tokens, and the queries are the last tokens of their sequence."""
    out = []
    for rows, n in zip(*_counts(case)):
        end = 4 * rows + rows % 4
        out += [min(rows, max(0, (end - n + i + 1) // 4)) for i in range(n)]
    return out


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["head_dim"] * SIZES[case["dtype"]]
        pairs = case["tokens"] * case["heads"] * case["rope_dim"] // 2
        times = 2 if case["train"] else 1
        return {"bytes": times * (2 * n + (0 if case["rows"] else 8 * case["tokens"])), "flops": times * 6 * pairs}
    row = case["heads"] * case["head_dim"] if op != "attend" else case["kv_heads"] * case["head_dim"]
    if op == "append":
        n = sum(_lens(case, "new", case["batch"], 0 if case["new"] > 1 else 1))
        return {"bytes": n * row * (SIZES[case["dtype"]] + 1) + 4 * n * case["heads"] // case["block"], "flops": 2 * n * row}
    if op == "attend":
        rows, n = _counts(case)
        seen, at, pairs = 0, 0, 0
        v = _visible(case)
        for q in n:
            seen += max(v[at: at + q], default=0)
            pairs += sum(v[at: at + q])
            at += q
        size = 2 if case["dtype"] != "fp32" else 4
        cache = seen * row * (1 if case["shared"] else 2)
        return {"bytes": cache + sum(n) * case["heads"] * (2 * case["head_dim"] * size + 4), "flops": 4 * case["head_dim"] * case["heads"] * pairs}
    p = _pool(case)
    page = case["heads"] * (case["page"] * case["head_dim"] + 4 * case["page"] // case["block"])
    return {"bytes": 2 * p["moved"] * page + 4 * (2 * p["table"] + 2 * p["pages"]), "flops": 0}


# ------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _freqs(case):
    """Frequencies (radians a position) and amplitude: powers of a base; a linear stretch; or, part by part, a
    stretch of the slow frequencies with the amplitude 0.1 ln(factor) + 1."""
    n = case["rope_dim"]
    f = [10000.0 ** (-2.0 * i / n) for i in range(n // 2)]
    factor, first = 16.0, 4096.0
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "yarn":
        def dim(turns):
            return n * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), n - 1)
        keep = [1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n // 2)]
        return [x / factor * (1 - k) + x * k for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _prepare_rope(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    t, h, d = case["tokens"], case["heads"], case["head_dim"]
    f, amplitude = _freqs(case)
    s = {"case": case, "x": _normal(g, (t, h, d), dt), "freqs": torch.tensor(f, dtype=torch.float64, device=DEV), "amplitude": amplitude}
    if case["rows"]:
        r = random.Random(seed)
        cuts = sorted(r.randint(0, t) for _ in range(min(63, t // 2)))
        s["cu_rows"] = _int([0] + cuts + [max(cuts[-1] if cuts else 0, t - t // 64)])
    else:
        most = 1_000_000 if case["far"] else 8192
        s["positions"] = torch.randint(0, most, (t,), generator=g, device=DEV)
    if case["train"]:
        s["x"].requires_grad_()
        s["grad"] = _normal(g, (t, h, d), dt)
    return s


def _tables(lens, page, width, order):
    """A page table whose held pages are taken from `order`, -1 elsewhere."""
    at, rows = 0, []
    for n in lens:
        k = -(-n // page)
        rows.append(order[at: at + k] + [-1] * (width - k))
        at += k
    return _int(rows)


def _prepare_append(case, seed):
    g, n, page, block = _gen(seed), case["batch"], case["page"], case["block"]
    h, d = case["heads"], case["head_dim"]
    held = [case["held"]] * n if not case["ragged"] else [max(0, case["held"] - i) for i in range(n)]
    new = _lens(case, "new", n, 0 if case["new"] > 1 else 1)
    ends = [a + b for a, b in zip(held, new)]
    pages = sum(-(-e // page) for e in ends)
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    width = max(-(-e // page) for e in ends) + 1
    bits = torch.randint(0, 127, (pages, h, page, d), generator=g, device=DEV, dtype=torch.uint8)
    return {"case": case, "cache": bits.view(E4M3), "scales": torch.full((pages, h, page // block), 2.0 ** -8, device=DEV),
            "table": _tables(ends, page, width, order), "lens": _int(held), "cu": _int(_sums(new)),
            # a row now and then is far larger than the others
            "rows": (torch.randn((sum(new), h, d), generator=g, device=DEV)
                     * torch.exp2(torch.randint(0, 8, (sum(new), 1, 1), generator=g, device=DEV).float() - 3)).to(DTYPES[case["dtype"]])}


def _prepare_attend(case, seed):
    g, page, block, d = _gen(seed), case["page"], case["block"], case["head_dim"]
    rows, n = _counts(case)
    pages = sum(-(-x // page) for x in rows) + 3
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    h = case["kv_heads"] * (1 if case["shared"] else 2)
    cache = torch.empty((pages, h, page, d), dtype=E4M3, device=DEV)
    scales = torch.empty((pages, h, page // block), device=DEV)
    step = max(1, 2 ** 27 // (h * page * d))
    for a in range(0, pages, step):  # rows ~ N(0, 1) times a power of two, quantised block by block
        b = min(pages, a + step)
        x = torch.randn((b - a, h, page // block, block, d), generator=g, device=DEV)
        x = x * torch.exp2(torch.randint(-2, 2, (b - a, h, page // block, 1, 1), generator=g, device=DEV).float())
        k = torch.frexp(x.abs().amax((3, 4)) / 448)[1].float()
        scales[a:b] = torch.exp2(k)
        cache[a:b] = (x * torch.exp2(-k)[..., None, None]).to(E4M3).view(b - a, h, page, d)
    s = {"case": case, "cache": cache, "scales": scales, "table": _tables(rows, page, max(1, max(-(-x // page) for x in rows)), order),
         "lens": _int(rows), "cu": _int(_sums(n)), "visible": _int(_visible(case)), "most": max(n), "scale": d ** -0.5,
         "q": _normal(g, (sum(n), case["heads"], d), DTYPES[case["dtype"]])}
    if case["queries"] == 1:
        s["visible"] = None  # a single token sees all rows
    return s


def _pool(case):
    """The pool of a pages case: sequences, pages that move, table size."""
    page, n = case["page"], case["batch"]
    r = random.Random("pool %d %d %d" % (n, case["held"], case["spare"]))
    lens = [r.randint(max(1, case["held"] // 2), case["held"]) for _ in range(n)]
    held = sum(-(-x // page) for x in lens)
    pages = held + case["spare"] + n * case["branches"] * (2 + case["new"] // page)
    seqs = n * (1 + case["branches"])
    width = -(-(max(lens) + case["new"]) // page)
    if case["do"] == "fork":
        moved = sum(case["branches"] for x in lens if x % page)
    else:
        moved = None
    order = list(range(pages))
    r.shuffle(order)
    order = order[:held]
    if moved is None:  # pages of the sequences that stay, above the number of them
        at, live = 0, []
        for i, x in enumerate(lens):
            k = -(-x // page)
            live += order[at: at + k] if i % 3 else []
            at += k
        moved = sum(p >= len(live) for p in live)
    return {"lens": lens, "pages": pages, "seqs": seqs, "width": width, "moved": moved, "order": order, "table": seqs * width}


def _prepare_pages(case, seed):
    g, p, n = _gen(seed), _pool(case), case["batch"]
    h, d, page, seqs, width = case["heads"], case["head_dim"], case["page"], p["seqs"], p["width"]
    order = list(p["order"])
    random.Random(seed).shuffle(order) if case["do"] == "fork" else None
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
    table[:n] = _tables(p["lens"], page, width, order)
    refs = torch.zeros(p["pages"], dtype=torch.int32, device=DEV)
    refs[torch.tensor(order, device=DEV)] = 1
    first = torch.cat([table.view(-1), _int(p["lens"] + [0] * (seqs - n)), refs])
    now = first.clone()
    a, b = seqs * width, seqs * width + seqs
    s = {"case": case, "first": first, "now": now, "table": now[:a].view(seqs, width), "lens": now[a:b], "refs": now[b:],
         "cache": torch.randint(0, 127, (p["pages"], h, page, d), generator=g, device=DEV, dtype=torch.uint8).view(E4M3),
         "scales": torch.rand((p["pages"], h, page // case["block"]), generator=g, device=DEV)}
    if case["do"] == "fork":
        k = case["branches"]
        s["parents"] = _int([i for i in range(n) for _ in range(k)])
        s["children"] = _int([n + i for i in range(n * k)])
        s["new"] = _int([case["new"]] * (n * k))
    else:
        s["ended"] = _int(list(range(0, n, 3)))
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "attend": _prepare_attend, "pages": _prepare_pages}[case["op"]](case, seed)


# ------------------------------------------------------------- plain forms


def _turn(x, cos, sin, case):
    o, n = case["offset"], case["rope_dim"]
    part = x[..., o: o + n].float()
    if case["layout"] == "half":
        a, b = part[..., : n // 2], part[..., n // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :o], turned.to(x.dtype), x[..., o + n:]], -1)


def _plain_rope(s):
    case, x = s["case"], s["x"].detach()
    if case["rows"]:
        cu = s["cu_rows"].long()
        i = torch.arange(case["tokens"], device=x.device)
        seq = torch.searchsorted(cu[1:], i, right=True)
        inside = seq < cu.numel() - 1
        p = torch.where(inside, (i - cu[seq.clamp(max=cu.numel() - 2)]) * 4, 0)
    else:
        p = s["positions"]
    angle = p.double()[:, None] * s["freqs"]
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    y = _turn(x, cos, sin, case)
    return [y, _turn(s["grad"], cos, -sin, case)] if case["train"] else y


def _per_row(scales, block):
    return scales.repeat_interleave(block, -1)


def _plain_append(s):
    case, rows, cu, lens = s["case"], s["rows"], s["cu"].long(), s["lens"].long()
    page, block, h, d = case["page"], case["block"], case["heads"], case["head_dim"]
    cache, scales, table = s["cache"].view(torch.uint8), s["scales"], s["table"].long()
    n = rows.shape[0]
    i = torch.arange(n, device=rows.device)
    seq = torch.searchsorted(cu[1:], i, right=True)
    at = lens[seq] + i - cu[seq]
    where, slot = table[seq, at // page], at % page
    blk = where * (page // block) + slot // block
    # what the new rows need, and what the rows before them in their block had
    need = torch.zeros((scales.shape[0] * (page // block), h), device=rows.device)
    need.scatter_reduce_(0, blk[:, None].expand(n, h), rows.float().abs().amax(-1), "amax")
    m, e = torch.frexp(need)
    k = torch.where(need > 0, e - 9 + (m > 0.875).int(), -120).clamp(-120, 120)
    begun = torch.zeros(need.shape[0], dtype=torch.bool, device=rows.device)
    b0 = table[torch.arange(lens.numel(), device=lens.device), (lens // page).clamp(max=table.shape[1] - 1)] * (page // block) + lens % page // block
    part = (lens % block > 0) & (cu[1:] > cu[:-1])
    begun[b0[part]] = True
    touched = torch.zeros_like(begun)
    touched[blk] = True
    old = scales.permute(0, 2, 1).reshape(-1, h)
    new = torch.where(touched[:, None], torch.maximum(torch.exp2(k.float()), torch.where(begun[:, None], old, 0.0)), old)
    b0, upto = b0[part], (lens % block)[part]
    flat = cache.view(-1, h, page // block, block, d).permute(0, 2, 1, 3, 4)
    pg, pb = b0 // (page // block), b0 % (page // block)
    was = flat[pg, pb].view(E4M3).float() * (old[b0] / new[b0])[:, :, None, None]
    keep = (torch.arange(block, device=rows.device) < upto[:, None])[:, None, :, None]
    flat[pg, pb] = torch.where(keep, was.to(E4M3).view(torch.uint8), flat[pg, pb])
    scales.copy_(new.view(-1, page // block, h).permute(0, 2, 1))
    cache.permute(0, 2, 1, 3)[where, slot] = (rows.float() / new[blk][..., None]).to(E4M3).view(torch.uint8)
    return [s["cache"], scales]


def _plain_attend(s):
    case, q, table = s["case"], s["q"], s["table"].long()
    kv, d, page, block = case["kv_heads"], case["head_dim"], case["page"], case["block"]
    b, m = table.shape
    at = table.clamp(min=0)
    sc = _per_row(s["scales"][at], block)  # [b, m, heads, page]

    def side(first):
        x = s["cache"].view(torch.uint8)[at, first: first + kv].view(E4M3).float() * sc[:, :, first: first + kv, :, None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, kv, m * page, d)

    k = side(0)
    v = k if case["shared"] else side(kv)
    cu, t = s["cu"].long(), q.shape[0]
    group = case["heads"] // kv
    i = torch.arange(t, device=q.device)
    seq = torch.searchsorted(cu[1:], i, right=True)
    visible = s["lens"][seq] if s["visible"] is None else torch.minimum(s["visible"], s["lens"][seq])
    qp = torch.zeros((b, s["most"], kv, group, d), device=q.device)
    vp = torch.zeros((b, s["most"]), dtype=visible.dtype, device=q.device)
    qp[seq, i - cu[seq]] = q.float().view(t, kv, group, d)
    vp[seq, i - cu[seq]] = visible
    qp = qp.permute(0, 2, 1, 3, 4).reshape(b, kv, -1, d)
    z = torch.matmul(qp, k.transpose(-1, -2)).mul_(s["scale"])
    seen = torch.arange(m * page, device=q.device) < vp[:, None, :, None]
    z = z.view(b, kv, s["most"], group, -1).masked_fill_(~seen[:, :, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, kv, -1, m * page), v).view(b, kv, s["most"], group, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (total.log() + top).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4)[seq, i - cu[seq]].reshape(t, -1, d).to(q.dtype)
    return [out, lse.permute(0, 2, 1, 3)[seq, i - cu[seq]].reshape(t, -1)]


def _copy_pages(s, src, dst):
    s["cache"].view(torch.uint8)[dst] = s["cache"].view(torch.uint8)[src]
    s["scales"][dst] = s["scales"][src]


def _plain_fork(s):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    parents, children, new = s["parents"].long(), s["children"].long(), s["new"].long()
    one = torch.ones((), dtype=refs.dtype, device=refs.device)
    e = torch.arange(table.shape[1], device=table.device)
    rows = torch.where(e < ((lens[parents] + page - 1) // page)[:, None], table[parents], -1)
    table[children] = rows
    lens[children] = lens[parents]
    held = rows[rows >= 0].long()
    refs.index_put_((held,), one.expand(held.numel()), accumulate=True)
    # room for the children's next rows: the lowest free pages in the children's order; a shared page that will be written is copied
    n = lens[children].long()
    inside = (e >= (n // page)[:, None]) & (e < ((n + new + page - 1) // page)[:, None])
    had = table[children].long()
    shared = inside & (had >= 0) & (refs[had.clamp(min=0)] > 1)
    want = shared | (inside & (had < 0))
    free = (refs == 0).nonzero().flatten()
    got = free[: int(want.sum())]
    old = had[want & shared]
    fresh = had.masked_scatter(want, got)
    refs.index_put_((old,), -one.expand(old.numel()), accumulate=True)
    refs[got] = 1
    table[children] = fresh.int()
    copied = shared & (e * page < n[:, None])
    _copy_pages(s, had[copied], fresh[copied])


def _plain_compact(s):
    table, lens, refs, ended = s["table"], s["lens"], s["refs"], s["ended"].long()
    held = table[ended]
    held = held[held >= 0].long()
    refs.index_put_((held,), -torch.ones((), dtype=refs.dtype, device=refs.device).expand(held.numel()), accumulate=True)
    table[ended] = -1
    lens[ended] = 0
    live = refs > 0
    n = int(live.sum())
    src = live[n:].nonzero().flatten() + n
    dst = (~live[:n]).nonzero().flatten()
    to = torch.arange(refs.numel(), device=refs.device, dtype=torch.int32)
    to[src] = dst.int()
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    refs[dst] = refs[src]
    refs[src] = 0
    _copy_pages(s, src, dst)


# ---------------------------------------------------------------------- run


def _own_run(s):
    import gated_softmax_kv_gb300 as gsk
    from gated_softmax_kv_gb300 import autograd
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        where = {"cu_seqlens_comp": s["cu_rows"], "ratio": 4} if case["rows"] else {"positions": s["positions"]}
        call = autograd.rope if case["train"] else gsk.csa_rope
        y = call(s["x"], s["freqs"], offset=case["offset"], layout=case["layout"], amplitude=s["amplitude"], **where)
        return [y, torch.autograd.grad(y, s["x"], s["grad"])[0]] if case["train"] else y
    if op == "append":
        gsk.csa_cache_append(s["rows"], s["cache"], s["scales"], s["table"], s["lens"], s["cu"])
        return [s["cache"], s["scales"]]
    if op == "attend":
        return list(gsk.csa_cache_attend(s["q"], s["cache"], s["scales"], s["table"], s["lens"], s["cu"], case["kv_heads"], s["scale"],
                                         shared=case["shared"], visible=s["visible"]))
    if case["do"] == "fork":
        gsk.csa_cache_fork(s["table"], s["lens"], s["refs"], s["parents"], s["children"], case["page"], s["status"])
        gsk.csa_cache_reserve(s["cache"], s["scales"], s["table"], s["lens"], s["refs"], s["children"], s["new"], s["status"])
    else:
        gsk.csa_cache_free(s["table"], s["lens"], s["refs"], s["ended"])
        gsk.csa_cache_compact(s["cache"], s["scales"], s["table"], s["refs"])


def run(state):
    op = state["case"]["op"]
    if op == "pages":
        state["now"].copy_(state["first"])  # each pass begins with the same tables
    if own:
        out = _own_run(state)
    elif op == "pages":
        out = _plain_fork(state) if state["case"]["do"] == "fork" else _plain_compact(state)
    else:
        out = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[op](state)
    return [state["table"], state["lens"], state["refs"], state["cache"], state["scales"]] if op == "pages" else out


# -------------------------------------------------------------------- exact


def _exact_rope(s):
    case, x = s["case"], s["x"].detach().double()
    t = case["tokens"]
    if case["rows"]:
        cu, p = s["cu_rows"].tolist(), [0] * t
        for a, b in zip(cu, cu[1:]):
            p[a:b] = range(0, 4 * (b - a), 4)
        p = torch.tensor(p, dtype=torch.float64, device=DEV)
    else:
        p = s["positions"].double()
    o, n = case["offset"], case["rope_dim"]
    turn = torch.polar(torch.full_like(p, s["amplitude"])[:, None].expand(t, n // 2), p[:, None] * s["freqs"][None])

    def apply(v, w):
        y, part = v.clone(), v[..., o: o + n]
        z = part.unflatten(-1, (2, n // 2)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (n // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w[:, None])
        y[..., o: o + n] = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
        return y

    return [apply(x, turn), apply(s["grad"].double(), turn.conj())] if case["train"] else apply(x, turn)


def _grid(x):
    """The nearest value with three bits after the leading one and exponents from -6, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    case, page, block = s["case"], s["case"]["page"], s["case"]["block"]
    cache, scales = s["cache"].double(), s["scales"].double()
    rows, cu, lens, table = s["rows"].double(), s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for i, held in enumerate(lens):
        at, end = held, held + cu[i + 1] - cu[i]
        while at < end:
            upto = min(end, (at // block + 1) * block)
            pg, a, b = table[i][at // page], at % page, at % page + upto - at
            blk, begin = a // block, a // block * block
            x = rows[cu[i] + at - held: cu[i] + upto - held].transpose(0, 1)
            top = x.abs().amax((1, 2))
            new = torch.exp2(torch.floor(torch.log2(top / 448).clamp(min=-120)))
            new = torch.where(448 * new < top, 2 * new, new)
            if a > begin:
                new = torch.maximum(new, scales[pg, :, blk])
                cache[pg, :, begin:a] = _grid(cache[pg, :, begin:a] * (scales[pg, :, blk] / new)[:, None, None])
            scales[pg, :, blk] = new
            cache[pg, :, a:b] = _grid(x / new[:, None, None])
            at = upto
    return [cache, scales]


def _exact_attend(s):
    case, page, block, kv = s["case"], s["case"]["page"], s["case"]["block"], s["case"]["kv_heads"]
    cu, lens, d, group = s["cu"].tolist(), s["lens"].tolist(), case["head_dim"], case["heads"] // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(lens):
        if not n or cu[i] == cu[i + 1]:
            continue
        held = s["table"][i, : -(-n // page)].long()
        x = s["cache"].view(torch.uint8)[held].view(E4M3).double() * _per_row(s["scales"][held].double(), block)[..., None]
        x = x.transpose(0, 1).flatten(1, 2)[:, :n]
        q = s["q"][cu[i]: cu[i + 1]].double().unflatten(1, (kv, group))
        for h in range(kv):
            z = torch.einsum("tgd,jd->tgj", q[:, h], x[h]) * s["scale"]
            if s["visible"] is not None:
                z[(torch.arange(n, device=DEV) >= s["visible"][cu[i]: cu[i + 1], None])[:, None].expand_as(z)] = -math.inf
            total = torch.logsumexp(z, -1)
            p = torch.where(total[..., None] > -math.inf, torch.exp(z - total[..., None]), 0.0)
            out[cu[i]: cu[i + 1], h * group: (h + 1) * group] = p @ x[h if case["shared"] else kv + h]
            lse[cu[i]: cu[i + 1], h * group: (h + 1) * group] = total
    return [out, lse]


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
