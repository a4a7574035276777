"""The operators of a rollout decoder layer that sit between its FP4 linear
layers, as cases to be measured: the paged key/value cache held in FP4
(``append``: quantize new tokens into it and read them back; ``attention``:
attention over it), the router of the expert layer (``route``: scores, top-k,
expert order, and its gradient) and the combination of the experts' outputs
(``combine``, and its gradient).

Each case runs in two ways: in plain torch operations (``own`` false), or by
the calls that a user of the library makes (``own`` true).  Both read what
``prepare`` made; ``exact`` computes the same outputs from the definitions in
64 bits.

Lengths that vary within a case follow its number ``ragged`` (0: all equal),
so that ``work`` knows them without a tensor.
"""
import math
import random

import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32}
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---- the cases ------------------------------------------------------------

def listed():
    return [
        # One decode step of a serving batch: every sequence stores one token.
        dict(name="append_step", kind="append", fmt="nvfp4", batch=64, new=1, length=4096,
             kv_heads=8, dim=128, page=64, ragged=1),
        # A prompt pass of several sequences at once, stored in MXFP4.
        dict(name="append_prompt", kind="append", fmt="mxfp4", batch=7, new=4096, length=4096,
             kv_heads=8, dim=128, page=64, ragged=2),
        # One user, a short past: the latency of a single token.
        dict(name="attend_one", kind="attention", fmt="nvfp4", batch=1, new=1, length=777,
             heads=32, kv_heads=8, dim=128, page=16, window=0, ragged=0),
        # A rollout batch in mid-generation, every sequence of another length.
        dict(name="attend_batch", kind="attention", fmt="nvfp4", batch=64, new=1, length=8192,
             heads=64, kv_heads=8, dim=128, page=64, window=0, ragged=3),
        # Few sequences with a very long past: one token over many pages.
        dict(name="attend_long", kind="attention", fmt="mxfp4", batch=3, new=1, length=131072,
             heads=32, kv_heads=8, dim=128, page=128, window=0, ragged=4),
        # Prompts of a rollout batch, each attending to itself (causal).
        dict(name="attend_prompt", kind="attention", fmt="nvfp4", batch=4, new=4096, length=4096,
             heads=32, kv_heads=4, dim=128, page=64, window=0, ragged=5),
        # A chunk of a long prompt over what is stored already, sliding window.
        dict(name="attend_chunk", kind="attention", fmt="mxfp4", batch=2, new=512, length=16001,
             heads=24, kv_heads=8, dim=64, page=32, window=4096, ragged=6),
        # The router at one token: latency.
        dict(name="route_one", kind="route", tokens=1, experts=128, k=8, score="softmax",
             groups=1, top_groups=1, bias=False, renorm=True, dtype="bf16", train=False),
        # The router of a batch: sigmoid scores, balance bias, limited groups.
        dict(name="route_groups", kind="route", tokens=4096, experts=256, k=8, score="sigmoid",
             groups=8, top_groups=4, bias=True, renorm=True, dtype="f32", train=False),
        # A training step's router: forward and gradient of the logits.
        dict(name="route_train", kind="route", tokens=16384, experts=128, k=8, score="softmax",
             groups=1, top_groups=1, bias=False, renorm=True, dtype="f32", train=True),
        # Experts' outputs back to the tokens in a decode step.
        dict(name="combine_step", kind="combine", tokens=64, k=8, cols=2048, dtype="bf16",
             train=False),
        # The same in a training step over a batch of tokens, with its gradient.
        dict(name="combine_train", kind="combine", tokens=4096, k=8, cols=2048, dtype="bf16",
             train=True),
    ]


def _log_between(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """A case of the same ranges, brought below the largest listed one's cost."""
    case = _drawn(rng)
    most = [work(c) for c in listed()]
    cap = {x: max(w[x] for w in most) for x in ("bytes", "flops")}
    while any(work(case)[x] > cap[x] for x in cap):
        size = "tokens" if "tokens" in case else "batch" if case["batch"] > 1 else "length"
        case[size] = -(-case[size] // 2)
        if "new" in case:
            case["new"] = min(case["new"], case["length"])
    return case


def _drawn(rng):
    kind = rng.choice(["append", "attention", "attention", "attention", "route", "combine"])
    if kind == "route":
        experts = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(10, experts // groups * top_groups))
        return dict(kind=kind, tokens=_log_between(rng, 1, 16384), experts=experts, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups,
                    top_groups=top_groups, bias=rng.random() < 0.5, renorm=rng.random() < 0.7,
                    dtype=rng.choice(["bf16", "f32"]), train=rng.random() < 0.4)
    if kind == "combine":
        return dict(kind=kind, tokens=_log_between(rng, 1, 4096), k=rng.randint(1, 8),
                    cols=8 * _log_between(rng, 16, 512), dtype=rng.choice(["bf16", "f32"]),
                    train=rng.random() < 0.5)
    fmt = rng.choice(["nvfp4", "mxfp4"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    ragged = rng.randint(1, 1 << 20)
    if kind == "append":
        new = _log_between(rng, 1, 2048)
        return dict(kind=kind, fmt=fmt, batch=_log_between(rng, 1, max(1, min(64, 8192 // new))),
                    new=new, length=new + rng.randint(0, 2048), kv_heads=kv_heads, dim=dim,
                    page=page, ragged=ragged)
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if rng.random() < 0.55:      # decode: one token, or the few of a speculative step
        length = _log_between(rng, 1, 65536)
        batch = _log_between(rng, 1, max(1, min(64, 262144 // length)))
        new = min(length, rng.choice([1, 1, 1, 2, 3, 4]))
    else:                        # prompts and chunks
        new = _log_between(rng, 5, 2048)
        length = new + rng.choice([0, _log_between(rng, 1, 4096)])
        batch = _log_between(rng, 1, max(1, min(8, 4096 // new)))
    return dict(kind=kind, fmt=fmt, batch=batch, new=new, length=length, heads=group * kv_heads,
                kv_heads=kv_heads, dim=dim, page=page,
                window=rng.choice([0, 0, 0, _log_between(rng, 1, 4096)]), ragged=ragged)


def lengths(case):
    """New tokens and total length of each sequence of an append or attention case."""
    B, new, length = case["batch"], case["new"], case["length"]
    if not case["ragged"]:
        return [new] * B, [length] * B
    rng = random.Random(case["ragged"])
    n, t = [new], [length]       # the first sequence has the largest size
    for _ in range(B - 1):
        total = _log_between(rng, max(1, length // 16), length)
        t.append(total)
        n.append(min(total, new if new <= 4 else rng.randint(1, new)))
    return n, t


def work(case):
    if case["kind"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        el = 2 if case["dtype"] == "bf16" else 4
        b = T * E * el + (4 * E if case["bias"] else 0) + T * k * 16 + 4 * (E + 1)
        f = T * E * 8
        if case["train"]:        # read the weights' gradient, write the logits'
            b += T * k * 4 + T * E * el
            f += T * E * 4
        return {"bytes": b, "flops": f}
    if case["kind"] == "combine":
        T, k, N = case["tokens"], case["k"], case["cols"]
        el = 2 if case["dtype"] == "bf16" else 4
        b = T * k * N * el + T * N * el + T * k * 8
        f = 2 * T * k * N
        if case["train"]:        # read the output's gradient, write the rows' and the weights'
            b += T * N * el + T * k * N * el + 4 * T * k
            f += 3 * T * k * N
        return {"bytes": b, "flops": f}
    n, t = lengths(case)
    H, D = case["kv_heads"], case["dim"]
    token = 2 * H * (D // 2 + D // BLOCK[case["fmt"]])   # packed bytes of one token, K and V
    if case["kind"] == "append":
        rows = sum(n)
        # read K and V, write them packed, read that back, write the values
        return {"bytes": rows * (2 * H * D * 2 + token + token + 2 * H * D * 2),
                "flops": rows * H * D * 8}
    heads, w = case["heads"], case["window"]
    pairs = keys = 0
    for nb, tb in zip(n, t):
        first, last = tb - nb + 1, tb                    # keys seen by the first and last query
        if w:
            pairs += sum(min(c, w) for c in range(first, last + 1))
            keys += tb - max(0, first - w)
        else:
            pairs += (first + last) * nb // 2
            keys += tb
    return {"bytes": sum(n) * heads * D * 4 + keys * token + 4 * keys // case["page"],
            "flops": 4 * D * heads * pairs}


# ---- inputs ---------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    if case["kind"] == "route":
        T, E = case["tokens"], case["experts"]
        # some experts are liked more than others, as a trained router has it
        logits = 1.5 * _normal(g, T, E) + _normal(g, E)
        s = {"case": case,
             "logits": logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32),
             "bias": 0.1 * _normal(g, E) if case["bias"] else None}
        if case["train"]:
            s["d_weights"] = _normal(g, T, case["k"])
        return s
    if case["kind"] == "combine":
        T, k, N = case["tokens"], case["k"], case["cols"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s = {"case": case, "y": _normal(g, T * k, N).to(dt),
             "row_of": torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k),
             "weights": torch.softmax(_normal(g, T, k), 1)}
        if case["train"]:
            s["d_out"] = _normal(g, T, N).to(dt)
        return s
    n, t = lengths(case)
    B, H, D, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    need = [-(-x // page) for x in t]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    rows = ids.cpu()
    at = 0
    for b in range(B):
        table[b, :need[b]] = rows[at:at + need[b]]
        at += need[b]
    off = [0]
    for x in n:
        off.append(off[-1] + x)
    s = {"case": case, "table": table.to(DEV), "lens": _ints(t), "offsets": _ints(off)}
    if case["fmt"] == "nvfp4":   # calibrated tensor scales, one for each head
        s["k_scale"] = (6.0 + 4.0 * torch.rand(H, generator=g, device=DEV)) / 2688.0
        s["v_scale"] = (6.0 + 4.0 * torch.rand(H, generator=g, device=DEV)) / 2688.0
    else:
        s["k_scale"] = s["v_scale"] = None
    # where row r of the new tokens stands: its sequence and its place among the new ones
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(n, device=DEV))
    s["seq"], s["place"] = seq, torch.arange(off[-1], device=DEV) - s["offsets"][seq].long()
    s["max_new"], s["max_len"], s["rows"] = max(n), max(t), off[-1]
    row_bytes = D // 2 + D // BLOCK[case["fmt"]]
    if case["kind"] == "append":
        # keys have a few strong channels, values have none
        strong = 1.0 + 4.0 * (torch.rand(H, D, generator=g, device=DEV) < 0.03)
        s["k"] = (_normal(g, off[-1], H, D) * strong).to(torch.bfloat16)
        s["v"] = _normal(g, off[-1], H, D).to(torch.bfloat16)
        s["cache"] = torch.randint(0, 256, (pages, H, 2 * page * row_bytes), generator=g,
                                   dtype=torch.uint8, device=DEV)
        return s
    s["q"] = (2.0 * _normal(g, off[-1], case["heads"], D)).to(torch.bfloat16)
    kc, ks, _ = quantize(case["fmt"], _normal(g, pages, page, H, D).to(torch.bfloat16),
                         s["k_scale"])
    vc, vs, _ = quantize(case["fmt"], _normal(g, pages, page, H, D).to(torch.bfloat16),
                         s["v_scale"])
    s["cache"] = pack(kc, ks, vc, vs)
    return s


# ---- the plain forms ------------------------------------------------------

def quantize(fmt, x, tscale):
    """x [..., heads, D] bf16 -> codes [..., D], block scale codes [..., D/blk]
    and the values they stand for; tscale one f32 for each head (NVFP4)."""
    blk = BLOCK[fmt]
    b = x.float().unflatten(-1, (-1, blk))
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        t = tscale[:, None]
        # (a division by a tensor: by a number it may become a product with 1/6)
        sb = torch.clamp(amax / torch.full_like(amax, 6.0) / t, max=448.0).to(torch.float8_e4m3fn)
        code, d = sb.view(torch.uint8), (sb.float() * t)[..., None]
        q = torch.where(d > 0, b / torch.where(d > 0, d, torch.ones_like(d)), 0.0 * b)
    else:
        m, e = torch.frexp(amax)                         # amax = m 2^e, m in [0.5, 1)
        e = torch.clamp(torch.where(m <= 0.75, e - 3, e - 2), -127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        code = (e + 127).to(torch.uint8)
        d = torch.exp2(e.double())[..., None]
        q = (b.double() / d).float()
    a = q.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
           + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    neg = torch.signbit(b)
    val = _grid(x.device)[(mag + 8 * neg).to(torch.uint8).int()]
    if fmt == "nvfp4":
        val = (val * sb.float()[..., None]) * t[..., None]
    else:
        val = (val.double() * d).float()
    return (mag + 8 * neg).to(torch.uint8).flatten(-2), code, val.flatten(-2)


def _grid(dev):
    m = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(m + [-x for x in m], device=dev)


def pack(kc, ks, vc, vs):
    """Codes [pages, page, H, D] and scale codes -> the cache [pages, H, bytes]:
    for each page and head the K codes, V codes, K scales and V scales.  K
    rows lie one after another, two neighbouring elements to a byte; V rows
    interleave by four tokens, and a byte holds two elements 16 apart."""
    kc, ks, vc, vs = (x.transpose(1, 2) for x in (kc, ks, vc, vs))
    P, H, page, D = kc.shape
    k = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(P, H, -1)
    v = vc.reshape(P, H, page // 4, 4, D // 16, 16).permute(0, 1, 2, 5, 3, 4)
    v = (v[..., 0::2] | (v[..., 1::2] << 4)).reshape(P, H, -1)
    return torch.cat([k, v, ks.reshape(P, H, -1), vs.reshape(P, H, -1)], -1).contiguous()


def unpack(fmt, cache, page, D):
    """The cache's K and V values [..., page, D] in f32, tensor scales left out."""
    lead, blk = cache.shape[:-1], BLOCK[fmt]
    kc, vc, ks, vs = cache.split([page * D // 2] * 2 + [page * D // blk] * 2, -1)
    kc = kc.reshape(*lead, page, D // 2)
    kc = torch.stack([kc & 15, kc >> 4], -1).reshape(*lead, page, D)
    vc = vc.reshape(*lead, page // 4, 16, 4, D // 32)
    vc = torch.stack([vc & 15, vc >> 4], -1).reshape(*lead, page // 4, 16, 4, D // 16)
    vc = vc.movedim(-3, -1).reshape(*lead, page, D)
    grid, out = _grid(cache.device), []
    for c, s in ((kc, ks), (vc, vs)):
        s = s.reshape(*lead, page, D // blk, 1)
        s = s.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(s.float() - 127)
        out.append((grid[c.int()].unflatten(-1, (-1, blk)) * s).flatten(-2))
    return out


def _plain_attention(s):
    case = s["case"]
    H, D, heads, page = case["kv_heads"], case["dim"], case["heads"], case["page"]
    B, L, n = case["batch"], s["table"].shape[1] * page, s["max_new"]
    k, v = unpack(case["fmt"], s["cache"][s["table"].long().clamp(min=0)], page, D)
    k = k.transpose(1, 2).reshape(B, H, L, D)            # pages and heads change places
    v = v.transpose(1, 2).reshape(B, H, L, D)
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    q = torch.zeros(B, n, heads, D, device=DEV)
    q[s["seq"], s["place"]] = s["q"].float()
    # the heads of a group one after another, all their queries with them
    q = q.transpose(1, 2).reshape(B, H, heads // H * n, D)
    lens = s["lens"].long()
    at = (lens - (s["offsets"][1:] - s["offsets"][:-1]).long())[:, None] + torch.arange(n, device=DEV)
    key = torch.arange(L, device=DEV)
    see = (key <= at[..., None]) & (key < lens[:, None, None])         # [B, n, L]
    if case["window"]:
        see &= key > at[..., None] - case["window"]
    x = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5
    x = x.view(B, H, heads // H, n, L).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    z = p.sum(-1, keepdim=True)
    v = torch.where((key < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p.view(B, H, -1, L), v).view(B, H, heads // H, n, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    o = o.reshape(B, heads, n, D).transpose(1, 2)
    return o[s["seq"], s["place"]].to(torch.bfloat16)


def _plain_route(s):
    case, x = s["case"], s["logits"].double()
    T, E, k, G = case["tokens"], case["experts"], case["k"], case["groups"]
    if case["score"] == "softmax":
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    ranked = score + s["bias"].double() if case["bias"] else score
    order = ranked if case["bias"] else x    # without a bias the logits have the scores' order
    if G > 1:                                # the best groups by the sum of their two best
        best = ranked.view(T, G, E // G).sort(dim=2, descending=True).values[..., :2].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        out = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter_(1, keep, False)
        order = order.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    idx = order.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    # expert order: the rows of an expert by their token
    flat = idx.reshape(-1)
    row = flat.sort(stable=True).indices
    row_of = torch.empty_like(row)
    row_of[row] = torch.arange(T * k, device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = (flat[:, None] == torch.arange(E, device=DEV)).sum(0).cumsum(0)
    got = {"experts": idx.int(), "weights": w.float(), "offsets": offsets.int(),
           "row_src": (row // k).int(), "row_of": row_of.view(T, k).int()}
    if case["train"]:
        dw = s["d_weights"].double()
        p = score.gather(1, idx)
        if case["renorm"]:                   # through w = p / sum(p)
            dw = (dw - (dw * w).sum(1, keepdim=True)) / p.sum(1, keepdim=True)
        ds = torch.zeros_like(score).scatter_(1, idx, dw)
        if case["score"] == "softmax":
            dx = score * (ds - (ds * score).sum(1, keepdim=True))
        else:
            dx = ds * score * (1.0 - score)
        got["d_logits"] = dx.to(s["logits"].dtype)
    return got


def _plain_combine(s):
    y = s["y"].float()[s["row_of"].long()]               # [T, k, N]
    w = s["weights"]
    got = {"out": (y * w[..., None]).sum(1).to(s["y"].dtype)}
    if s["case"]["train"]:
        do = s["d_out"].float()[:, None]
        dy = torch.empty_like(s["y"])
        dy[s["row_of"].long()] = (w[..., None] * do).to(dy.dtype)
        got["d_y"], got["d_weights"] = dy, (y * do).sum(-1)
    return got


# ---- one pass -------------------------------------------------------------

def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import fp4_w4a4_quantized_amd as fq
        if kind == "route":
            how = dict(score=fq.SIGMOID if case["score"] == "sigmoid" else fq.SOFTMAX,
                       renorm=case["renorm"])
            r = fq.route(s["logits"], case["k"], bias=s["bias"], n_groups=case["groups"],
                         top_groups=case["top_groups"], **how)
            if case["train"]:
                r["d_logits"] = fq.route_backward(s["logits"], r["experts"], s["d_weights"], **how)
            return r
        if kind == "combine":
            got = {"out": fq.combine(s["y"], s["row_of"], s["weights"])}
            if case["train"]:
                got["d_y"], got["d_weights"] = fq.combine_backward(s["y"], s["row_of"],
                                                                   s["weights"], s["d_out"])
            return got
        fmt = fq.NVFP4 if case["fmt"] == "nvfp4" else fq.MXFP4
        where = (s["cache"], case["page"], s["offsets"], s["table"], s["lens"])
        if kind == "append":
            fq.kv_append(fmt, *where, s["k"], s["v"], s["k_scale"], s["v_scale"])
            k, v = fq.kv_read(fmt, *where, s["rows"], case["dim"], s["k_scale"], s["v_scale"])
            return {"k": k, "v": v}
        return fq.kv_attention(fmt, *where, s["q"], s["max_new"], s["max_len"], s["k_scale"],
                               s["v_scale"], window=case["window"])
    if kind == "route":
        return _plain_route(s)
    if kind == "combine":
        return _plain_combine(s)
    if kind == "append":
        return {x: quantize(case["fmt"], s[x], s[x + "_scale"])[2].to(torch.bfloat16)
                for x in ("k", "v")}
    return _plain_attention(s)


# ---- from the definitions, in 64 bits -------------------------------------

def _exact_quantized(fmt, x, tscale):
    """What stands in the cache for x [rows, heads, D]: by the format's rule,
    whose steps are single f32 operations (each rounded here from 64 bits)."""
    rows, H, D = x.shape
    blk = BLOCK[fmt]
    v = x.double().reshape(rows, H, D // blk, blk)
    amax = v.abs().amax(-1, keepdim=True)

    def f32(z):
        return z.float().double()

    if fmt == "nvfp4":
        t = tscale.double().view(1, H, 1, 1)
        z = f32(f32(amax / 6.0) / t).clamp(max=448.0)
        # nearest of 8 steps to a power of two, never finer than 2^-9, ties to even
        step = torch.exp2(torch.floor(torch.log2(z.clamp(min=2.0 ** -6))) - 3)
        sb = torch.round(z / step) * step
        d = f32(sb * t)
        r = torch.where(d > 0, f32(v / d.clamp(min=1e-300)), torch.zeros_like(v))
    else:
        e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 6.0))
        e = torch.where(6.0 * torch.exp2(e - 1) >= amax, e - 1, e)     # log2 next to a whole number
        e = torch.where(6.0 * torch.exp2(e) < amax, e + 1, e).clamp(-127, 127)
        sb, t = torch.exp2(e), 1.0
        r = v / sb
    a = r.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    a = torch.round(a / step) * step                     # ties to even, also at the step's changes
    return (f32(a * sb) * t * torch.where(torch.signbit(v), -1.0, 1.0)).reshape(rows, H, D)


def _exact_attention(s, case):
    n, t = lengths(case)
    H, D, heads, page, blk = (case["kv_heads"], case["dim"], case["heads"], case["page"],
                              BLOCK[case["fmt"]])
    G, rb = heads // H, D // 2
    d = torch.arange(D, device=DEV)
    out = torch.empty(sum(n), heads, D, dtype=torch.float64, device=DEV)
    r0 = 0
    for b, (nb, tb) in enumerate(zip(n, t)):
        pos = torch.arange(tb, device=DEV)
        pid, p = s["table"][b].long()[pos // page], pos % page
        qpos = torch.arange(tb - nb, tb, device=DEV)
        lo = max(0, tb - nb + 1 - case["window"]) if case["window"] else 0
        pid, p, pos = pid[lo:], p[lo:], pos[lo:]
        see = pos[None, :] <= qpos[:, None]
        if case["window"]:
            see &= pos[None, :] > qpos[:, None] - case["window"]
        for h in range(H):
            kv = []
            for part in range(2):
                if part == 0:
                    byte = p[:, None] * rb + (d // 2)[None]
                    high = (d % 2).expand(len(p), D)
                else:
                    byte = (page * rb + (p // 4)[:, None] * 4 * rb
                            + ((d % 16)[None] * 4 + (p % 4)[:, None]) * (D // 32) + (d // 32)[None])
                    high = (d // 16 % 2).expand(len(p), D)
                c = s["cache"][pid[:, None], h, byte].long()
                c = torch.where(high > 0, c >> 4, c & 15)
                ex, man = (c >> 1) & 3, c & 1
                val = torch.where(ex > 0, (2.0 + man) * torch.exp2(ex.double() - 2), 0.5 * man)
                val = torch.where(c >= 8, -val, val)
                at = 2 * page * rb + part * page * (D // blk) + p[:, None] * (D // blk) + (d // blk)[None]
                sc = s["cache"][pid[:, None], h, at].long()
                if blk == 16:
                    ex, man = sc >> 3, (sc & 7).double()
                    f = torch.where(ex > 0, (8.0 + man) * torch.exp2(ex.double() - 10), man * 2.0 ** -9)
                    f = f * s["k_scale" if part == 0 else "v_scale"][h].double()
                else:
                    f = torch.exp2(sc.double() - 127)
                kv.append(val * f)
            for j in range(h * G, h * G + G):
                x = s["q"][r0:r0 + nb, j].double() @ kv[0].T / math.sqrt(D)
                x = x.masked_fill(~see, -math.inf)
                out[r0:r0 + nb, j] = torch.softmax(x, 1) @ kv[1]
        r0 += nb
    return out


def _exact_route(s, case):
    x = s["logits"].double()
    T, E, k = case["tokens"], case["experts"], case["k"]
    score = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    ranked = score if s["bias"] is None else score + s["bias"].double()
    order = x if s["bias"] is None else ranked
    if case["groups"] > 1:
        per = ranked.view(T, case["groups"], -1)
        top = per.max(2)
        one = torch.zeros_like(per, dtype=torch.bool).scatter_(2, top.indices[..., None], True)
        best = top.values
        if per.shape[2] > 1:
            best = best + per.masked_fill(one, -math.inf).amax(2)
        # how many groups come before each one
        g = torch.arange(case["groups"], device=DEV)
        before = (best[:, None] > best[..., None]) | ((best[:, None] == best[..., None])
                                                      & (g[None, :] < g[:, None]))
        order = torch.where((before.sum(2) < case["top_groups"])[..., None].expand_as(per)
                            .reshape(T, E), order, -math.inf)
    picks = []
    left = order.clone()
    for _ in range(k):
        m = left.amax(1, keepdim=True)
        i = (left == m).to(torch.int8).argmax(1, keepdim=True)         # the first of the best
        # (a row of nothing but excluded experts cannot occur: k fits the kept groups)
        picks.append(i)
        left = left.scatter(1, i, -math.inf)
    idx = torch.cat(picks, 1)
    w = score.gather(1, idx)
    total = w.sum(1, keepdim=True)
    if case["renorm"]:
        w = w / total
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    slot = torch.argsort(idx.reshape(-1) * (T * k) + torch.arange(T * k, device=DEV))
    row_of = torch.argsort(slot)
    got = {"experts": idx.int(), "weights": w, "offsets": offsets.int(),
           "row_src": (slot // k).int(), "row_of": row_of.view(T, k).int()}
    if case["train"]:
        # the sum over the chosen of (dw_j / dx_i), from d score_j / d x_i
        dw = s["d_weights"].double()
        if case["renorm"]:
            dw = (dw - (w * dw).sum(1, keepdim=True)) / total
        p = score.gather(1, idx)
        if case["score"] == "softmax":
            dx = -score * (dw * p).sum(1, keepdim=True)
            dx.scatter_add_(1, idx, dw * p)
        else:
            dx = torch.zeros_like(score).scatter_add_(1, idx, dw * p * (1 - p))
        got["d_logits"] = dx
    return got


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "append":
        return {x: _exact_quantized(case["fmt"], s[x], s[x + "_scale"]) for x in ("k", "v")}
    if kind == "attention":
        return _exact_attention(s, case)
    if kind == "route":
        return _exact_route(s, case)
    T, k, N = case["tokens"], case["k"], case["cols"]
    y, w = s["y"].double(), s["weights"].double()
    row = s["row_of"].long()
    got = {"out": sum(w[:, j, None] * y[row[:, j]] for j in range(k))}
    if case["train"]:
        do = s["d_out"].double()
        dy = torch.empty_like(y)
        dw = torch.empty(T, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            dy[row[:, j]] = w[:, j, None] * do
            dw[:, j] = (y[row[:, j]] * do).sum(1)
        got["d_y"], got["d_weights"] = dy, dw
    return got
