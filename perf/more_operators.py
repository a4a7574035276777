"""What a rollout decoder layer computes beside its FP4 products, as cases to
be measured: the rotation of queries and keys by their positions on the way
into the FP4 cache (``rotate``), attention over that cache with a sliding
window and first tokens that stay visible (``sinks``), the root-mean-square
norm with the residual's addition, into the quantized operand of the next
product (``norm``) or with its gradient (``train``), and low-rank adapters of
many requests beside a shared projection (``lora``).

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

BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---- the cases ------------------------------------------------------------

def listed():
    return [
        # One decode step of a serving batch, each sequence at another position.
        dict(name="rotate_step", kind="rotate", fmt="nvfp4", batch=64, new=1, length=8192, heads=32,
             kv_heads=8, dim=128, rot=128, pairs="halves", page=64, ragged=1),
        # Prompts of several sequences at once, far into their contexts; half of
        # each head is rotated, in neighbouring pairs.
        dict(name="rotate_prompt", kind="rotate", fmt="mxfp4", batch=7, new=4096, length=131072,
             heads=32, kv_heads=8, dim=128, rot=64, pairs="neighbours", page=64, ragged=2),
        # One user, one token: latency.
        dict(name="sinks_one", kind="sinks", fmt="nvfp4", batch=1, new=1, length=2777, heads=32,
             kv_heads=8, dim=128, page=16, window=1024, sinks=4, ragged=0),
        # A rollout batch in mid-generation, long contexts cut by the window.
        dict(name="sinks_batch", kind="sinks", fmt="nvfp4", batch=64, new=1, length=65536, heads=64,
             kv_heads=8, dim=128, page=64, window=4096, sinks=4, ragged=3),
        # Chunks of long prompts over what is stored already.
        dict(name="sinks_chunk", kind="sinks", fmt="mxfp4", batch=3, new=2048, length=32768, heads=24,
             kv_heads=8, dim=64, page=32, window=2048, sinks=68, ragged=4),
        # The norm before a decode step's projections: FP4 operand with the tensor's own scale.
        dict(name="norm_step", kind="norm", fmt="nvfp4", rows=64, cols=2048, dtype="bf16",
             residual=True, given_scale=False, chans=64, tiled=False),
        # A prompt pass, into the FP4 operand of the large product.
        dict(name="norm_prompt", kind="norm", fmt="nvfp4", rows=8192, cols=4096, dtype="bf16",
             residual=True, given_scale=False, chans=128, tiled=True),
        # The same pass where the layer behind it is kept in 8 bits.
        dict(name="norm_mxfp8", kind="norm", fmt="mxfp8", rows=8192, cols=4096, dtype="bf16",
             residual=True, given_scale=False, chans=0, tiled=False),
        # A training step's norm over a batch of tokens: forward and gradients.
        dict(name="norm_train", kind="train", rows=4099, cols=4096, dtype="bf16", residual=True),
        # One request with its adapter: latency.
        dict(name="lora_one", kind="lora", rows=1, requests=1, adapters=4, rank=16, k=2048, n=11008,
             dtype="f32", ragged=0),
        # A decode step: 64 requests of one token, many with an adapter of their own.
        dict(name="lora_step", kind="lora", rows=64, requests=64, adapters=48, rank=16, k=4096, n=14336,
             dtype="bf16", ragged=5),
        # Prompts of several requests with different adapters.
        dict(name="lora_prompt", kind="lora", rows=8192, requests=11, adapters=6, rank=32, k=4096,
             n=14336, dtype="bf16", ragged=6),
    ]


def _log_between(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """A case of the same ranges, brought below the largest listed one's cost."""
    case = _drawn(rng)
    most = [work(c) for c in listed()]
    cap = {x: max(w[x] for w in most) for x in ("bytes", "flops")}
    while any(work(case)[x] > cap[x] for x in cap):
        size = ("rows" if "rows" in case else "batch" if case["batch"] > 1
                else "window" if case["kind"] == "sinks" and case["window"] > case["new"] else "new")
        case[size] = -(-case[size] // 2)
        if "requests" in case:
            case["requests"] = min(case["requests"], case["rows"])
    return case


def _drawn(rng):
    kind = rng.choice(["rotate", "sinks", "sinks", "norm", "norm", "train", "lora", "lora"])
    if kind == "norm":
        fmt = rng.choice(["nvfp4", "mxfp4", "mxfp8"])
        tiled = fmt != "mxfp8" and rng.random() < 0.4
        unit = 128 if tiled else 32
        cols = unit * _log_between(rng, 256 // unit, 12288 // unit)
        return dict(kind=kind, fmt=fmt, rows=_log_between(rng, 1, 8192), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.7,
                    given_scale=fmt == "nvfp4" and rng.random() < 0.4,
                    chans=0 if fmt == "mxfp8" else rng.choice([0, 8 * rng.randint(1, 16)]), tiled=tiled)
    if kind == "train":
        return dict(kind=kind, rows=_log_between(rng, 1, 8192), cols=_log_between(rng, 64, 12288),
                    dtype=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.7)
    if kind == "lora":
        rows = _log_between(rng, 1, 8192)
        return dict(kind=kind, rows=rows, requests=_log_between(rng, 1, min(rows, 64)),
                    adapters=_log_between(rng, 1, 32), rank=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                    k=8 * _log_between(rng, 64, 1024), n=_log_between(rng, 500, 14336),
                    dtype=rng.choice(["bf16", "f32"]), ragged=rng.randint(1, 1 << 20))
    fmt = rng.choice(["nvfp4", "mxfp4"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    ragged = rng.randint(1, 1 << 20)
    if kind == "rotate":
        new = _log_between(rng, 1, 2048)
        return dict(kind=kind, fmt=fmt, batch=_log_between(rng, 1, max(1, min(64, 8192 // new))),
                    new=new, length=new + _log_between(rng, 1, 131072), heads=group * kv_heads,
                    kv_heads=kv_heads, dim=dim, rot=16 * rng.choice([dim // 16, dim // 16, rng.randint(1, dim // 16)]),
                    pairs=rng.choice(["halves", "halves", "neighbours"]), page=page, ragged=ragged)
    if rng.random() < 0.55:      # decode: one token, or the few of a speculative step
        length = _log_between(rng, 1, 65536)
        new = min(length, rng.choice([1, 1, 1, 2, 3, 4]))
        batch = _log_between(rng, 1, 64)
    else:                        # prompts and chunks
        new = _log_between(rng, 5, 2048)
        length = new + rng.choice([0, _log_between(rng, 1, 16384)])
        batch = _log_between(rng, 1, max(1, min(8, 4096 // new)))
    return dict(kind=kind, fmt=fmt, batch=batch, new=new, length=length, heads=group * kv_heads,
                kv_heads=kv_heads, dim=dim, page=page, window=_log_between(rng, 1, 4096),
                sinks=_log_between(rng, 1, 256), ragged=ragged)


def lengths(case):
    """New tokens and total length of each sequence of a rotate or sinks case."""
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


def requests(case):
    """Rows and adapter (-1: none) of each request of a lora case."""
    R, T = case["requests"], case["rows"]
    if not case["ragged"]:
        return [T // R + (i < T % R) for i in range(R)], [i % case["adapters"] for i in range(R)]
    rng = random.Random(case["ragged"])
    cuts = sorted(rng.sample(range(1, T), R - 1))
    n = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    return n, [rng.randrange(case["adapters"]) if rng.random() < 0.9 else -1 for _ in range(R)]


def _seen(case, nb, tb):
    """(pairs of token and key, keys that some token sees) of one sequence."""
    w, s = case["window"], case["sinks"]
    pairs = 0
    for pos in range(tb - nb, tb):
        lo = max(0, pos - w + 1)
        pairs += pos + 1 - lo + min(s, lo)
    lo = max(0, tb - nb - w + 1)
    return pairs, tb - lo + min(s, lo)


def work(case):
    kind = case["kind"]
    if kind in ("norm", "train"):
        M, N = case["rows"], case["cols"]
        el = 2 if case["dtype"] == "bf16" else 4
        b = M * N * el * (3 if case["residual"] else 1) + N * 4
        if kind == "train":      # y, 1/rms; then h, y's and h's gradients in, x's and the weight's out
            return {"bytes": b + M * N * el * (4 + case["residual"]) + M * 8 + N * 8, "flops": M * N * 16}
        blk = BLOCK[case["fmt"]]
        packed = M * (N // (1 if case["fmt"] == "mxfp8" else 2) + N // blk)
        if case["fmt"] != "mxfp8":   # the operand is read back as the values it stands for
            packed = 2 * packed + M * N * 2
        return {"bytes": b + packed + 2 * M * case["chans"], "flops": M * N * 8}
    if kind == "lora":
        n, a = requests(case)
        el = 2 if case["dtype"] == "bf16" else 4
        T, K, N, r = case["rows"], case["k"], case["n"], case["rank"]
        used = len({x for x in a if x >= 0})
        some = sum(x for x, j in zip(n, a) if j >= 0)
        return {"bytes": some * K * 2 + used * r * (K + N) * 2 + 2 * T * N * el,
                "flops": 2 * some * r * (K + N)}
    n, t = lengths(case)
    H, D, heads = case["kv_heads"], case["dim"], case["heads"]
    token = 2 * H * (D // 2 + D // BLOCK[case["fmt"]])   # packed bytes of one token, K and V
    if kind == "rotate":
        rows = sum(n)
        # read Q, K and V, write Q and the packed bytes, read those back, write the values
        return {"bytes": rows * (4 * heads * D + 4 * H * D + 2 * token + 4 * H * D),
                "flops": rows * (6 * (heads + H) * case["rot"] // 2 + H * D * 8)}
    pairs = keys = 0
    for nb, tb in zip(n, t):
        p, k = _seen(case, nb, tb)
        pairs += p
        keys += k
    return {"bytes": sum(n) * heads * D * 4 + keys * token + 4 * keys // case["page"],
            "flops": 4 * D * heads * pairs}


# ---- inputs ---------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(n):
    off = [0]
    for x in n:
        off.append(off[-1] + x)
    return off


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    if kind in ("norm", "train"):
        M, N = case["rows"], case["cols"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a few channels of the residual stream are much stronger than the rest
        strong = 1.0 + 20.0 * (torch.rand(N, generator=g, device=DEV) < 0.01)
        s = {"case": case, "x": _normal(g, M, N).to(dt), "eps": 1e-6,
             "residual": (_normal(g, M, N) * strong).to(dt) if case["residual"] else None,
             "weight": (1.0 + 0.2 * _normal(g, N)).to(dt)}
        if kind == "train":
            s["d_y"] = _normal(g, M, N).to(dt)
            s["d_h"] = _normal(g, M, N).to(dt) if case["residual"] else None
        else:
            s["tscale"] = (10.0 + 5.0 * torch.rand(1, generator=g, device=DEV)) / 2688.0 \
                if case["given_scale"] else None
            s["chan"] = torch.randperm(N, generator=g, device=DEV)[:case["chans"]].sort().values.int() \
                if case["chans"] else None
        return s
    if kind == "lora":
        n, a = requests(case)
        T, K, N, r, A = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        return {"case": case, "x": _normal(g, T, K).to(torch.bfloat16), "y": _normal(g, T, N).to(dt),
                "a": (_normal(g, A, r, K) * K ** -0.5).to(torch.bfloat16),
                "b": (_normal(g, A, N, r) * r ** -0.5).to(torch.bfloat16),
                "scale": 0.5 + torch.rand(A, generator=g, device=DEV),
                "offsets": _ints(_offsets(n)), "adapter": _ints(a),
                # the adapter of each row, as the plain form takes it
                "of_row": torch.repeat_interleave(_ints(a), torch.tensor(n, device=DEV))}
    n, t = lengths(case)
    B, H, D, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    need = [-(-x // page) for x in t]
    pages = sum(need) + 3 if kind == "sinks" else min(sum(need), 4096) + 3
    if kind == "rotate":         # the pages of the new tokens only: the rest of the past is not read
        need = [(x - y) // page for x, y in zip(t, n)], need
        ids = torch.randperm(sum(e - b for b, e in zip(*need)) + 3, generator=g, device=DEV).to(torch.int32)
    else:
        need = [0] * B, need
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    pages = ids.numel()
    table = torch.full((B, max(need[1])), -1, dtype=torch.int32)
    rows = ids.cpu()
    at = 0
    for b in range(B):
        first, end = need[0][b], need[1][b]
        table[b, first:end] = rows[at:at + end - first]
        at += end - first
    off = _offsets(n)
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
    s["q"] = (2.0 * _normal(g, off[-1], case["heads"], D)).to(torch.bfloat16)
    if kind == "rotate":
        # keys have a few strong channels, values have none
        strong = 1.0 + 4.0 * (torch.rand(H, D, generator=g, device=DEV) < 0.03)
        s["k"] = (_normal(g, off[-1], H, D) * strong).to(torch.bfloat16)
        s["v"] = _normal(g, off[-1], H, D).to(torch.bfloat16)
        s["cache"] = torch.randint(0, 256, (pages, H, 2 * page * row_bytes), generator=g,
                                   dtype=torch.uint8, device=DEV)
        base = 10000.0 * (1.0 + 49.0 * torch.rand(1, generator=g, device=DEV))
        half = case["rot"] // 2
        s["freqs"] = base ** (-torch.arange(half, device=DEV) / half)
        return s
    kc, ks, _ = quantize(case["fmt"], _normal(g, pages, page, H, D).to(torch.bfloat16),
                         s["k_scale"])
    vc, vs, _ = quantize(case["fmt"], _normal(g, pages, page, H, D).to(torch.bfloat16),
                         s["v_scale"])
    s["cache"] = pack(kc, ks, vc, vs)
    return s


# ---- the plain forms ------------------------------------------------------

def quantize(fmt, x, tscale):
    """x [..., D] bf16 -> codes [..., D], block scale codes [..., D/blk] and the
    values they stand for.  FP4 formats; tscale f32 (NVFP4), one for each of
    the dimension before the last, or a single one."""
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
        code, d = _power(amax, 0.75, 3)
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


def _power(amax, most, down):
    """The code and the value (64 bits, [..., 1]) of the smallest 2^e that brings
    amax = m 2^E, m in [0.5, 1), to the element's largest, `most` 2^down."""
    m, e = torch.frexp(amax)
    e = torch.clamp(torch.where(m <= most, e - down, e - down + 1), -127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    return (e + 127).to(torch.uint8), torch.exp2(e.double())[..., None]


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


def _plain_rotate(s):
    case = s["case"]
    half = case["rot"] // 2
    # (64 bits: a far position's angle has no digits left in 32, and what is
    # quantized afterwards may lie next to a border)
    pos = s["lens"].long()[s["seq"]] - (s["offsets"][1:] - s["offsets"][:-1]).long()[s["seq"]] + s["place"]
    angle = (pos.double()[:, None] * s["freqs"].double())[:, None]       # [rows, 1, half]
    c, sn = torch.cos(angle), torch.sin(angle)

    def turn(x):
        y = x.clone()
        r = x[..., :2 * half].double()
        if case["pairs"] == "halves":
            a, b = r[..., :half], r[..., half:]
            y[..., :half] = (a * c - b * sn).float().to(x.dtype)
            y[..., half:2 * half] = (b * c + a * sn).float().to(x.dtype)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            y[..., 0:2 * half:2] = (a * c - b * sn).float().to(x.dtype)
            y[..., 1:2 * half:2] = (b * c + a * sn).float().to(x.dtype)
        return y

    return {"q": turn(s["q"]),
            "k": quantize(case["fmt"], turn(s["k"]), s["k_scale"])[2].to(torch.bfloat16),
            "v": quantize(case["fmt"], s["v"], s["v_scale"])[2].to(torch.bfloat16)}


def _plain_sinks(s):
    case = s["case"]
    H, D, heads, page = case["kv_heads"], case["dim"], case["heads"], case["page"]
    B, n, W, S = case["batch"], s["max_new"], case["window"], case["sinks"]
    # the pages of the first tokens, and as many more as any sequence's window spans
    lens = s["lens"].long()
    new = (s["offsets"][1:] - s["offsets"][:-1]).long()
    cols = s["table"].shape[1]
    first = min(-(-S // page), cols)
    more = min(-(-(W + n) // page) + 1, cols)
    start = (torch.clamp(lens - new - W + 1, min=0) // page)[:, None]    # the window's first page
    pg = torch.cat([torch.arange(first, device=DEV).expand(B, first),
                    start + torch.arange(more, device=DEV)], 1)
    there = pg < cols
    there[:, :first] &= pg[:, :first] < start                            # (each page once)
    ids = s["table"].long().gather(1, pg.clamp(max=cols - 1)).clamp(min=0)
    key = (pg[..., None] * page + torch.arange(page, device=DEV)).flatten(1)
    key = torch.where(there.repeat_interleave(page, 1), key, torch.full_like(key, 1 << 40))
    L = key.shape[1]
    k, v = unpack(case["fmt"], s["cache"][ids], page, D)
    k = k.transpose(1, 2).reshape(B, H, L, D)            # pages and heads change places
    v = v.transpose(1, 2).reshape(B, H, L, D)
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    q = torch.zeros(B, n, heads, D, device=DEV)
    q[s["seq"], s["place"]] = s["q"].float()
    # the heads of a group one after another, all their queries with them
    q = q.transpose(1, 2).reshape(B, H, heads // H * n, D)
    at = (lens - new)[:, None] + torch.arange(n, device=DEV)
    key = key[:, None]
    see = (key <= at[..., None]) & (key < lens[:, None, None])
    see &= (key > at[..., None] - W) | (key < S)                         # [B, n, L]
    x = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5
    x = x.view(B, H, heads // H, n, L).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    z = p.sum(-1, keepdim=True)
    v = torch.where((key < lens[:, None, None]).transpose(1, 2)[:, None], v, torch.zeros_like(v))
    o = torch.matmul(p.view(B, H, -1, L), v).view(B, H, heads // H, n, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    o = o.reshape(B, heads, n, D).transpose(1, 2)
    return o[s["seq"], s["place"]].to(torch.bfloat16)


def _plain_norm(s):
    case, x = s["case"], s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    # (64 bits: what is quantized afterwards may lie next to a border)
    r = torch.rsqrt(h.double().square().mean(1, keepdim=True) + s["eps"])
    y = (h.double() * r * s["weight"].double()).float().to(torch.bfloat16)
    got = {} if s["residual"] is None else {"h": h}
    if case["fmt"] == "mxfp8":
        b = y.float().unflatten(-1, (-1, 32))
        code, d = _power(b.abs().amax(-1), 0.875, 9)
        got["q"] = (b.double() / d).float().to(torch.float8_e4m3fn).flatten(-2)
        got["scales"] = code.view(torch.float8_e8m0fnu)
        return got
    t = s["tscale"]
    if case["fmt"] == "nvfp4" and t is None:
        amax = y.float().abs().amax()
        t = (amax / torch.full_like(amax, 2688.0)).view(1)
        t = torch.where(t > 0, t, torch.ones_like(t))
    val = quantize(case["fmt"], y, t)[2]
    got["values"] = val.to(torch.bfloat16)
    if s["chan"] is not None:
        c = s["chan"].long()
        got["resid"] = (y.float()[:, c] - val[:, c]).to(torch.bfloat16)
    return got


def _plain_train(s):
    x, dt = s["x"].float(), s["x"].dtype
    h = s["x"] if s["residual"] is None else (x + s["residual"].float()).to(dt)
    hf, w, dy = h.float(), s["weight"].float(), s["d_y"].float()
    r = torch.rsqrt(hf.square().mean(1, keepdim=True) + s["eps"])
    g = w * dy
    dx = r * g - hf * r ** 3 * ((g * hf).sum(1, keepdim=True) / hf.shape[1])
    got = {"y": (hf * r * w).to(dt)}
    if s["residual"] is not None:
        got["h"] = h
        dx = dx + s["d_h"].float()
    got["d_x"], got["d_weight"] = dx.to(dt), (dy * hf * r).sum(0)
    return got


def _plain_lora(s):
    case = s["case"]
    A, r = case["adapters"], case["rank"]
    u = torch.matmul(s["x"].float(), s["a"].float().reshape(A * r, -1).T).view(-1, A, r)
    on = s["of_row"][:, None] == torch.arange(A, device=DEV)
    u = torch.where(on[..., None], u * s["scale"][:, None], torch.zeros_like(u))
    b = s["b"].float().transpose(1, 2).reshape(A * r, -1)
    return (s["y"].float() + torch.matmul(u.view(-1, A * r), b)).to(s["y"].dtype)


# ---- one pass -------------------------------------------------------------

def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import fp4_w4a4_quantized_amd as fq
        if kind == "lora":
            return fq.lora(s["x"], s["a"], s["b"], s["offsets"], s["adapter"], s["scale"], y=s["y"])
        if kind == "train":
            f = fq.rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"])
            dx, dw = fq.rms_norm_backward(f["h"], s["weight"], f["rstd"], s["d_y"], d_h=s["d_h"])
            got = {"y": f["y"], "d_x": dx, "d_weight": dw}
            if s["residual"] is not None:
                got["h"] = f["h"]
            return got
        if kind == "norm":
            fmt = {"nvfp4": fq.NVFP4, "mxfp4": fq.MXFP4, "mxfp8": fq.MXFP8}[case["fmt"]]
            a = fq.rms_norm_quantize(fmt, s["x"], s["weight"], s["eps"], residual=s["residual"],
                                     tscale=s["tscale"], chan_idx=s["chan"],
                                     layout=fq.TILED if case["tiled"] else fq.ROWMAJOR)
            got = {} if s["residual"] is None else {"h": a["h"]}
            if fmt == fq.MXFP8:
                got["q"] = a["q"].view(torch.float8_e4m3fn)
                got["scales"] = a["scales"].view(torch.float8_e8m0fnu)
                return got
            got["values"] = fq.dequantize(fmt, a)
            if s["chan"] is not None:
                got["resid"] = a["resid"].view(torch.bfloat16)
            return got
        fmt = fq.NVFP4 if case["fmt"] == "nvfp4" else fq.MXFP4
        where = (s["cache"], case["page"], s["offsets"], s["table"], s["lens"])
        if kind == "rotate":
            q = fq.kv_append_rotated(fmt, *where, s["q"], s["k"], s["v"], s["freqs"], s["k_scale"],
                                     s["v_scale"], interleaved=case["pairs"] == "neighbours")
            k, v = fq.kv_read(fmt, *where, s["rows"], case["dim"], s["k_scale"], s["v_scale"])
            return {"q": q, "k": k, "v": v}
        return fq.kv_attention(fmt, *where, s["q"], s["max_new"], s["max_len"], s["k_scale"],
                               s["v_scale"], window=case["window"], sinks=case["sinks"])
    return {"rotate": _plain_rotate, "sinks": _plain_sinks, "norm": _plain_norm,
            "train": _plain_train, "lora": _plain_lora}[kind](s)


# ---- from the definitions, in 64 bits -------------------------------------

def _f32(z):
    return z.float().double()


def _bf16(z):
    return z.float().to(torch.bfloat16).double()


def _least_power(amax, largest):
    """The smallest e in -127 .. 127 with largest 2^e >= amax."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / largest))
    e = torch.where(largest * torch.exp2(e - 1) >= amax, e - 1, e)   # log2 next to a whole number
    return torch.where(largest * torch.exp2(e) < amax, e + 1, e).clamp(-127, 127)


def _exact_quantized(fmt, v, t):
    """What v [..., blocks, blk] (64 bits) stands for after quantization, by the
    format's rule, whose steps are single f32 operations (each rounded here from
    64 bits); t: NVFP4's tensor scale, as v's leading dimensions have it."""
    amax = v.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        z = _f32(_f32(amax / 6.0) / t).clamp(max=448.0)
        # nearest of 8 steps to a power of two, never finer than 2^-9, ties to even
        step = torch.exp2(torch.floor(torch.log2(z.clamp(min=2.0 ** -6))) - 3)
        sb = torch.round(z / step) * step
        d = _f32(sb * t)
        r = torch.where(d > 0, _f32(v / d.clamp(min=1e-300)), torch.zeros_like(v))
    else:
        sb, t = torch.exp2(_least_power(amax, 6.0)), 1.0
        r = v / sb
    a = r.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    a = torch.round(a / step) * step                     # ties to even, also at the step's changes
    return _f32(_f32(a * sb) * t) * torch.where(torch.signbit(v), -1.0, 1.0)


def _exact_rotate(s, case):
    n, t = lengths(case)
    half, blk = case["rot"] // 2, BLOCK[case["fmt"]]
    pos = torch.cat([torch.arange(tb - nb, tb, device=DEV) for nb, tb in zip(n, t)]).double()
    i = torch.arange(half, device=DEV)
    e1, e2 = (i, i + half) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
    # as a complex number turned by its angle
    w = torch.polar(torch.ones_like(pos)[:, None].expand(-1, half).contiguous(),
                    pos[:, None] * s["freqs"].double())
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        z = torch.complex(x[..., e1], x[..., e2]) * w[:, None]
        x[..., e1], x[..., e2] = z.real, z.imag
        got[name] = x
    for name in ("k", "v"):
        x = _bf16(got["k"]) if name == "k" else s["v"].double()
        ts = s[name + "_scale"]
        x = x.unflatten(-1, (-1, blk))
        got[name] = _exact_quantized(case["fmt"], x, None if ts is None else ts.double()[:, None, None]).flatten(-2)
    return got


def _exact_sinks(s, case):
    n, t = lengths(case)
    H, D, heads, page, blk = (case["kv_heads"], case["dim"], case["heads"], case["page"],
                              BLOCK[case["fmt"]])
    G, rb, W, S = heads // H, D // 2, case["window"], case["sinks"]
    d = torch.arange(D, device=DEV)
    out = torch.empty(sum(n), heads, D, dtype=torch.float64, device=DEV)
    r0 = 0
    for b, (nb, tb) in enumerate(zip(n, t)):
        qpos = torch.arange(tb - nb, tb, device=DEV)
        lo = max(0, tb - nb + 1 - W)
        pos = torch.cat([torch.arange(min(S, lo), device=DEV), torch.arange(lo, tb, device=DEV)])
        pid, p = s["table"][b].long()[pos // page], pos % page
        see = (pos[None, :] <= qpos[:, None]) & ((pos[None, :] > qpos[:, None] - W) | (pos < S)[None])
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


def _exact_norm(s, case):
    h = s["x"].double()
    got = {}
    if s["residual"] is not None:
        got["h"] = h + s["residual"].double()
        h = _f32(got["h"]) if case["dtype"] == "f32" else _bf16(got["h"])
    y = h * s["weight"].double() / torch.sqrt(torch.mean(h * h, 1, keepdim=True) + s["eps"])
    y = _bf16(y)
    b = y.unflatten(-1, (-1, BLOCK[case["fmt"]]))
    if case["fmt"] == "mxfp8":
        sc = torch.exp2(_least_power(b.abs().amax(-1, keepdim=True), 448.0))
        a = b.abs() / sc
        step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        got["q"] = (torch.round(a / step) * step * torch.sign(b)).flatten(-2)
        got["scales"] = sc[..., 0]
        return got
    t = s["tscale"]
    if case["fmt"] == "nvfp4":
        t = _f32(y.abs().max() / 2688.0) if t is None else t.double()
        t = torch.where(t > 0, t, torch.ones_like(t))
    val = _exact_quantized(case["fmt"], b, t).flatten(-2)
    got["values"] = val
    if s["chan"] is not None:
        got["resid"] = (y - val)[:, s["chan"].long()]
    return got


def _exact_train(s, case):
    x, w, dy = s["x"].double(), s["weight"].double(), s["d_y"].double()
    got, h = {}, x
    if s["residual"] is not None:
        got["h"] = x + s["residual"].double()
        h = _f32(got["h"]) if case["dtype"] == "f32" else _bf16(got["h"])
    n = h.shape[1]
    rms = torch.sqrt((h * h).sum(1, keepdim=True) / n + s["eps"])
    u = h / rms
    got["y"] = u * w
    # through u = h / rms(h): the part along u is taken out
    dx = (dy * w - u * ((dy * w * u).sum(1, keepdim=True) / n)) / rms
    got["d_x"] = dx if s["residual"] is None else dx + s["d_h"].double()
    got["d_weight"] = (dy * u).sum(0)
    return got


def _exact_lora(s, case):
    n, a = requests(case)
    out, r0 = s["y"].double(), 0
    for rows, j in zip(n, a):
        if j >= 0:
            x = s["x"][r0:r0 + rows].double()
            out[r0:r0 + rows] += s["scale"][j].double() * (x @ s["a"][j].double().T) @ s["b"][j].double().T
        r0 += rows
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "sinks": _exact_sinks, "norm": _exact_norm,
            "train": _exact_train, "lora": _exact_lora}[case["kind"]](s, case)
