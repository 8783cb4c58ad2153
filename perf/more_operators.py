"""Cases of the operators on the uncompressed side of a layer: the norms of queries and keys of each head
with the position rotation in the same pass (``norm``), and causal attention over packed prompts with
grouped heads (``prompt``), both with their gradients. Each has a plain form of elementary torch operations
in 32 bits (64 for angles) and, where ``own`` is true, the calls a user makes of the package."""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one decoding step: the queries and keys of 16 tokens, each at its own position
        {"name": "norm step", "op": "norm", "tokens": 16, "heads": 64, "kv_heads": 8, "head_dim": 128, "rope_dim": 128, "offset": 0,
         "layout": "half", "dtype": "bf16", "weights": "same", "packed": 0, "fused": True, "train": False},
        # a batch of prompts, queries and keys as they lie in the projection's output
        {"name": "norm prompt", "op": "norm", "tokens": 32768, "heads": 32, "kv_heads": 8, "head_dim": 128, "rope_dim": 64, "offset": 64,
         "layout": "interleaved", "dtype": "bf16", "weights": "same", "packed": 16, "fused": True, "train": False},
        # training: the same with gradients of inputs and weights
        {"name": "norm train", "op": "norm", "tokens": 16384, "heads": 32, "kv_heads": 8, "head_dim": 128, "rope_dim": 128, "offset": 0,
         "layout": "half", "dtype": "bf16", "weights": "fp32", "packed": 8, "fused": True, "train": True},
        # training: the headline pack's compressed rows (one head of 512, the last 64 columns turned) before they are keys
        {"name": "norm rows train", "op": "norm", "tokens": 66533, "heads": 1, "kv_heads": 0, "head_dim": 512, "rope_dim": 64, "offset": 448,
         "layout": "interleaved", "dtype": "bf16", "weights": "fp32", "packed": 64, "fused": False, "train": True},
        # one short prompt: latency
        {"name": "prompt one", "op": "prompt", "batch": 1, "tokens": 300, "held": 0, "heads": 16, "kv_heads": 2, "head_dim": 128,
         "window": 0, "dtype": "bf16", "ragged": False, "spare": 0, "train": False},
        # a batch of ragged prompts, with a static capacity's rows behind the last
        {"name": "prompt pack", "op": "prompt", "batch": 12, "tokens": 2047, "held": 0, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "window": 0, "dtype": "bf16", "ragged": True, "spare": 100, "train": False},
        # one long prompt
        {"name": "prompt long", "op": "prompt", "batch": 1, "tokens": 16384, "held": 0, "heads": 16, "kv_heads": 2, "head_dim": 128,
         "window": 0, "dtype": "bf16", "ragged": False, "spare": 0, "train": False},
        # the local window beside compressed rows: each query sees the last 128 tokens
        {"name": "prompt window", "op": "prompt", "batch": 2, "tokens": 5003, "held": 0, "heads": 64, "kv_heads": 8, "head_dim": 64,
         "window": 128, "dtype": "fp16", "ragged": True, "spare": 0, "train": False},
        # chunks of prompts behind what is held already
        {"name": "prompt chunk", "op": "prompt", "batch": 4, "tokens": 255, "held": 4099, "heads": 16, "kv_heads": 2, "head_dim": 128,
         "window": 0, "dtype": "fp16", "ragged": True, "spare": 0, "train": False},
        # one new token for each of 32 sequences over the keys that they hold
        {"name": "prompt step", "op": "prompt", "batch": 32, "tokens": 1, "held": 8191, "heads": 64, "kv_heads": 8, "head_dim": 128,
         "window": 0, "dtype": "bf16", "ragged": True, "spare": 0, "train": False},
        # training on a ragged pack, three query heads share a key head of 64 columns
        {"name": "prompt train pack", "op": "prompt", "batch": 8, "tokens": 1500, "held": 0, "heads": 24, "kv_heads": 8, "head_dim": 64,
         "window": 0, "dtype": "fp16", "ragged": True, "spare": 77, "train": True},
        # training on one long sequence
        {"name": "prompt train long", "op": "prompt", "batch": 1, "tokens": 8192, "held": 0, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "window": 0, "dtype": "bf16", "ragged": False, "spare": 0, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        d = rng.choice([64, 96, 128, 256, 512])
        part = min(d, rng.choice([32, 64, d]))
        heads, kv = rng.choice([(1, 0), (5, 1), (16, 2), (32, 8), (64, 8), (12, 12)])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        train = rng.random() < 0.5
        most = 220_000_000 // ((heads + kv) * d * SIZES[dtype] * (2 if train else 1))
        return {"op": "norm", "tokens": _log(rng, 1, most), "heads": heads, "kv_heads": kv, "head_dim": d, "rope_dim": part,
                "offset": rng.choice([0, d - part]), "layout": rng.choice(["interleaved", "half"]), "dtype": dtype,
                "weights": rng.choice(["same", "fp32"]), "packed": rng.choice([0, 1, 7, 100]), "fused": rng.random() < 0.6, "train": train}
    kv, group = rng.choice([(1, 1), (1, 8), (1, 64), (2, 4), (2, 8), (8, 1), (8, 3), (8, 4), (8, 8), (5, 5), (12, 1)])
    heads, d = kv * group, rng.choice([64, 64, 128, 128, 128, 96, 80])
    train = rng.random() < 0.45
    held = 0 if train and rng.random() < 0.7 or rng.random() < 0.5 else _log(rng, 1, 8192)
    tokens = _log(rng, 1, 300 if held else 4096)
    pairs = tokens * (held + tokens)  # of one sequence, in the plain form
    most = min(4e9 / (4 * heads * pairs), 5e11 / (14 * d * heads * pairs), 2e8 / (kv * d * (held + tokens)))
    return {"op": "prompt", "batch": _log(rng, 1, max(1, min(48, int(most)))), "tokens": tokens, "held": held, "heads": heads, "kv_heads": kv,
            "head_dim": d, "window": _log(rng, 1, 2048) if rng.random() < 0.3 else 0, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
            "ragged": rng.random() < 0.7, "spare": rng.choice([0, 0, 9, 300]), "train": train}


def _lens(case, key, n, least):
    """Lengths of the sequences: `case[key]`, or spread over [least, case[key]] with the ends among them."""
    top = case[key]
    if not case["ragged"]:
        return [top] * n
    r = random.Random("%s %d %d" % (key, top, n))
    v = [r.randint(max(least, top // 4), top) for _ in range(n)]
    v[0] = top
    if n > 2:
        v[n // 2] = least
    return v


def _counts(case):
    """(queries, keys) of each sequence of a prompt case; one sequence of a ragged pack has no queries."""
    n = case["batch"]
    q = _lens(case, "tokens", n, 0 if case["tokens"] > 1 else 1)
    return q, [a + b for a, b in zip(q, _lens(case, "held", n, 0))]


def _sums(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def work(case):
    size, d = SIZES[case["dtype"]], case["head_dim"]
    if case["op"] == "norm":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * d
        turned = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["rope_dim"]
        w = 2 * d * (4 if case["weights"] == "fp32" else size)
        # forward: x in, y out; backward: x and the gradient in, the gradient out
        return {"bytes": n * size * (5 if case["train"] else 2) + w, "flops": (4 * n + 3 * turned) * (4 if case["train"] else 1)}
    q, k = _counts(case)
    pairs = keys = 0
    for a, b in zip(q, k):
        w = case["window"] or b
        first = b - a  # query i sees keys max(0, first + i + 1 - w) .. first + i
        full = max(0, a - max(0, w - first))  # queries that see w of them
        part = a - full
        pairs += full * w + part * first + part * (part + 1) // 2
        keys += min(b, a + w - 1) if a else 0
    rows, cells = sum(q) * case["heads"], keys * case["kv_heads"]
    nbytes = rows * (2 * d * size + 4) + 2 * cells * d * size
    if case["train"]:  # q, k, v, the result and its gradient in, three gradients out
        nbytes += rows * (4 * d * size + 4) + 4 * cells * d * size
    return {"bytes": nbytes, "flops": pairs * case["heads"] * d * (14 if case["train"] else 4)}


# ------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prepare_norm(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    t, h, kv, d, n = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], case["rope_dim"]
    wt = torch.float32 if case["weights"] == "fp32" else dt
    # tokens differ in size, as the projections of a residual stream do
    size = torch.exp2(torch.randint(-3, 4, (t, 1, 1), generator=g, device=DEV).float())
    if case["fused"]:  # queries, keys and values side by side
        x = (torch.randn((t, h + 2 * kv, d), generator=g, device=DEV) * size).to(dt)
        q, k = x[:, :h], x[:, h: h + kv]
    else:
        q = (torch.randn((t, h, d), generator=g, device=DEV) * size).to(dt)
        k = (torch.randn((t, kv, d), generator=g, device=DEV) * size).to(dt)
    s = {"case": case, "q": q, "k": k if kv else None, "freqs": torch.tensor([10000.0 ** (-2.0 * i / n) for i in range(n // 2)], dtype=torch.float64, device=DEV),
         "wq": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(wt), "wk": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(wt) if kv else None}
    if case["packed"]:
        r = random.Random(seed)
        cuts = sorted(r.randint(0, t) for _ in range(min(case["packed"] - 1, t // 2)))
        s["cu"] = _int([0] + cuts + [max(cuts[-1] if cuts else 0, t - t // 64)])
        s["ratio"] = 1 if kv else 4
    else:
        s["positions"] = torch.randint(0, 1_000_000, (t,), generator=g, device=DEV)
    if case["train"]:
        for name in ("q", "k", "wq", "wk"):
            if s[name] is not None:
                s[name] = s[name].detach().requires_grad_()
        s["gq"] = _normal(g, (t, h, d), dt)
        s["gk"] = _normal(g, (t, kv, d), dt) if kv else None
    return s


def _prepare_prompt(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    q, k = _counts(case)
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    t, n = sum(q) + case["spare"], sum(k) + case["spare"]
    if case["held"]:
        qs, ks, vs = _normal(g, (t, h, d), dt, 1.5), _normal(g, (n, kv, d), dt), _normal(g, (n, kv, d), dt)
    else:  # as they lie in the projection's output
        x = torch.randn((t, h + 2 * kv, d), generator=g, device=DEV)
        x[:, :h] *= 1.5
        x = x.to(dt)
        qs, ks, vs = x[:, :h], x[:, h: h + kv], x[:, h + kv:]
    s = {"case": case, "q": qs, "k": ks, "v": vs, "cu_q": _int(_sums(q)), "cu_k": _int(_sums(k)), "most_q": max(q), "most_k": max(k), "scale": d ** -0.5}
    if case["train"]:
        for name in ("q", "k", "v"):
            s[name] = s[name].detach().requires_grad_()
        s["grad"] = _normal(g, (t, h, d), dt)
    return s


def prepare(case, seed):
    return _prepare_norm(case, seed) if case["op"] == "norm" else _prepare_prompt(case, seed)


# ------------------------------------------------------------- plain forms


def _turn(x, cos, sin, case):
    o, n = case["offset"], case["rope_dim"]
    part = x[..., o: o + n]
    if case["layout"] == "half":
        a, b = part[..., : n // 2], part[..., n // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :o], turned, x[..., o + n:]], -1)


def _plain_positions(s):
    if "positions" in s:
        return s["positions"]
    cu, t = s["cu"].long(), s["q"].shape[0]
    i = torch.arange(t, device=cu.device)
    seq = torch.searchsorted(cu[1:], i, right=True)
    inside = seq < cu.numel() - 1
    return torch.where(inside, (i - cu[seq.clamp(max=cu.numel() - 2)]) * s["ratio"], 0)


def _plain_norm(s):
    case = s["case"]
    angle = _plain_positions(s).double()[:, None] * s["freqs"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def side(x, w, g):
        if x is None:
            return [], []
        dt, wt = x.dtype, w.dtype
        x, w = x.detach().float(), w.detach().float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        y = _turn(x * r * w, cos, sin, case).to(dt)
        if g is None:
            return [y], []
        g = _turn(g.float(), cos, -sin, case)
        dw = (g * x * r).sum((0, 1))
        u = g * w
        dx = r * (u - x * r.square() * (u * x).mean(-1, keepdim=True))
        return [y, dx.to(dt)], [dw.to(wt)]

    a, b = side(s["q"], s["wq"], s.get("gq")), side(s["k"], s["wk"], s.get("gk"))
    return a[0] + a[1] + b[0] + b[1]


def _seen(s, i, seq, nq, nk):
    """[first, last) keys that the query i of its sequence sees, within the sequence."""
    last = nk[seq] - nq[seq] + i + 1
    first = (last - s["case"]["window"]).clamp(min=0) if s["case"]["window"] else torch.zeros_like(last)
    return first, last


def _plain_prompt(s):
    case, q = s["case"], s["q"].detach()
    kv, d, b = case["kv_heads"], case["head_dim"], case["batch"]
    group = case["heads"] // kv
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q.diff(), cu_k.diff()

    def places(cu, n):  # (sequence, index in it) of the rows of all sequences
        i = torch.arange(n, device=cu.device)
        seq = torch.searchsorted(cu[1:], i, right=True)
        return seq, i - cu[seq]

    tq, tk = sum(_counts(case)[0]), sum(_counts(case)[1])
    sq, iq = places(cu_q, tq)
    sk, ik = places(cu_k, tk)

    def rows(x):  # [b, kv, most_q * group, d], zeros where there is no row
        out = torch.zeros((b, s["most_q"], kv, group, x.shape[-1]), device=x.device)
        out[sq, iq] = x[:tq].float().view(tq, kv, group, -1)
        return out.permute(0, 2, 1, 3, 4).reshape(b, kv, -1, x.shape[-1])

    def back(x, like):
        out = torch.zeros(like.shape, dtype=like.dtype, device=like.device)
        out[:tq] = x.view(b, kv, s["most_q"], group, d).permute(0, 2, 1, 3, 4)[sq, iq].reshape(tq, -1, d).to(like.dtype)
        return out

    def keys(x):
        out = torch.zeros((b, s["most_k"], kv, d), device=x.device)
        out[sk, ik] = x.detach()[:tk].float()
        return out.transpose(1, 2)

    def keys_back(x, like):
        out = torch.zeros(like.shape, dtype=like.dtype, device=like.device)
        out[:tk] = x.transpose(1, 2)[sk, ik].to(like.dtype)
        return out

    first, last = (torch.zeros((b, s["most_q"]), dtype=torch.long, device=q.device) for _ in range(2))
    first[sq, iq], last[sq, iq] = _seen(s, iq, sq, nq, nk)
    j = torch.arange(s["most_k"], device=q.device)
    seen = ((j >= first[..., None]) & (j < last[..., None]))[:, None, :, None]
    qp, kp, vp = rows(q), keys(s["k"]), keys(s["v"])
    z = torch.matmul(qp, kp.transpose(-1, -2)).mul_(s["scale"])
    z.view(b, kv, s["most_q"], group, -1).masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, 1.0))
    out = back(torch.matmul(p, vp), q)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device)
    lse[:tq] = (total.log() + top).view(b, kv, -1, group).transpose(1, 2)[sq, iq].reshape(tq, -1)
    if not case["train"]:
        return [out, lse]
    g = rows(s["grad"])
    dv = torch.matmul(p.transpose(-1, -2), g)
    dp = torch.matmul(g, vp.transpose(-1, -2))
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    return [out, lse, back(torch.matmul(ds, kp), q), keys_back(torch.matmul(ds.transpose(-1, -2), qp), s["k"]), keys_back(dv, s["v"])]


# ---------------------------------------------------------------------- run


def _own_run(s):
    import gated_softmax_kv_gb300 as gsk
    from gated_softmax_kv_gb300 import autograd
    case = s["case"]
    if case["op"] == "norm":
        where = {"cu_seqlens_comp": s["cu"], "ratio": s["ratio"]} if case["packed"] else {"positions": s["positions"]}
        call = autograd.norm_rope if case["train"] else gsk.csa_norm_rope
        y, z = call(s["q"], s["wq"], s["freqs"], k=s["k"], k_weight=s["wk"], offset=case["offset"], layout=case["layout"], eps=1e-6, **where)
        if not case["train"]:
            return [y] if z is None else [y, z]
        if z is None:
            d = torch.autograd.grad(y, [s["q"], s["wq"]], s["gq"])
            return [y, d[0], d[1]]
        d = torch.autograd.grad([y, z], [s["q"], s["wq"], s["k"], s["wk"]], [s["gq"], s["gk"]])
        return [y, d[0], d[1], z, d[2], d[3]]
    call = autograd.prompt_attend if case["train"] else gsk.csa_prompt_attend
    out, lse = call(s["q"], s["k"], s["v"], s["cu_q"], s["scale"], cu_k=s["cu_k"] if case["held"] else None, window=case["window"] or None)
    if not case["train"]:
        return [out, lse]
    return [out, lse, *torch.autograd.grad(out, [s["q"], s["k"], s["v"]], s["grad"])]


def run(state):
    if own:
        return _own_run(state)
    return _plain_norm(state) if state["case"]["op"] == "norm" else _plain_prompt(state)


# -------------------------------------------------------------------- exact


def _exact_norm(s):
    case, o, n = s["case"], s["case"]["offset"], s["case"]["rope_dim"]
    t = case["tokens"]
    if case["packed"]:
        cu, p = s["cu"].tolist(), [0] * t
        for a, b in zip(cu, cu[1:]):
            p[a:b] = range(0, s["ratio"] * (b - a), s["ratio"])
        p = torch.tensor(p, dtype=torch.float64, device=DEV)
    else:
        p = s["positions"].double()
    angle = p[:, None] * s["freqs"][None]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def apply(v, w):
        y, part = v.clone(), v[..., o: o + n]
        z = part.unflatten(-1, (2, n // 2)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (n // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w)
        y[..., o: o + n] = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
        return y

    out = []
    for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        if x is None:
            continue
        x, w = x.detach().double(), w.detach().double()
        size = ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()
        unit = x / size
        out.append(apply(unit * w, turn))
        if g is not None:
            h = apply(g.double(), turn.conj())
            along = (h * w * unit).sum(-1, keepdim=True) / x.shape[-1]
            out += [(h * w - unit * along) / size, torch.einsum("thd,thd->d", h, unit)]
    return out


def _exact_prompt(s):
    case, q = s["case"], s["q"].detach()
    kv, d = case["kv_heads"], case["head_dim"]
    group, scale = case["heads"] // kv, s["scale"]
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    grads = [torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k", "v")] if case["train"] else None
    for i in range(case["batch"]):
        a, b, e, f = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
        if a == b:
            continue
        row = torch.arange(f - e - (b - a), f - e, device=DEV)[:, None]  # the query's own place among the keys
        col = torch.arange(f - e, device=DEV)[None]
        hidden = col > row
        if case["window"]:
            hidden |= col <= row - case["window"]
        for h in range(case["heads"]):
            x, k, v = q[a:b, h].double(), s["k"].detach()[e:f, h // group].double(), s["v"].detach()[e:f, h // group].double()
            z = (x @ k.T * scale).masked_fill_(hidden, -math.inf)
            lse[a:b, h] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            out[a:b, h] = p @ v
            if grads:
                g = s["grad"][a:b, h].double()
                dz = p * (g @ v.T - (g * out[a:b, h]).sum(-1, keepdim=True)) * scale
                grads[0][a:b, h] = dz @ k
                grads[1][e:f, h // group] += dz.T @ x
                grads[2][e:f, h // group] += p.T @ g
    return [out, lse] + (grads or [])


def exact(case, seed):
    if case["op"] == "prompt" and work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_prompt(s)
