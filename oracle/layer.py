"""Plain 64-bit forms of the operators between the FP4 linear layers: the
paged FP4 key/value cache (with the position rotation), attention over it, the
norm, low-rank adapters, the router and the combination of the experts' outputs.
numpy only, written from the definitions that include/fp4q.h states:
nearest-value searches over the enumerated grids for the formats, loops over
sequences, heads and tokens for the rest.
"""
from __future__ import annotations

import math

import numpy as np

NVFP4, MXFP4 = 0, 1
BLOCK = {NVFP4: 16, MXFP4: 32}
SOFTMAX, SIGMOID = 0, 1

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite E4M3 magnitudes by code
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def bf16_round(x):
    """f64 -> f32 -> bf16 (nearest, ties to even), as float64."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def _nearest(grid, a):
    """Index of the nearest grid value, ties to the even index."""
    i = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo, hi = a - grid[i - 1], grid[i] - a
    up = (hi < lo) | ((hi == lo) & (i % 2 == 0))
    return np.where(up, i, i - 1)


def kv_quantize(fmt, x, t=None):
    """x float [..., D] (bf16 values), t f32 broadcastable to x's leading
    dimensions (NVFP4) -> (codes u8 [..., D], scale codes u8 [..., D/blk],
    the values they stand for: NVFP4 after the f32 product, as float64)."""
    blk = BLOCK[fmt]
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, blk)
    amax = np.abs(b).max(-1)
    if fmt == NVFP4:
        t = np.broadcast_to(np.asarray(t, np.float32)[..., None], amax.shape)
        v = (amax / np.float32(6)) / t                          # two f32 divisions
        sc = _nearest(E4M3, np.minimum(v.astype(np.float64), 448.0))
        sb = E4M3[sc].astype(np.float32)
        d = (sb * t)[..., None]
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(d > 0, b / d, np.float32(0))           # one f32 division
    else:
        e = np.full(amax.shape, -127)
        for k in range(-127, 128):                              # the smallest e with 6 2^e >= amax
            e = np.where(6.0 * 2.0 ** (k - 1) < amax.astype(np.float64), k, e)
        sc = e + 127
        sb, t = 2.0 ** e.astype(np.float64), np.ones_like(amax)
        q = b.astype(np.float64) / sb[..., None]
    mag = _nearest(E2M1, np.minimum(np.abs(q).astype(np.float64), 6.0))
    neg = np.signbit(b)
    val = np.where(neg, -1.0, 1.0) * E2M1[mag] * sb[..., None].astype(np.float64)
    if fmt == NVFP4:
        val = (val.astype(np.float32) * t[..., None]).astype(np.float64)
    codes = (mag + 8 * neg).astype(np.uint8).reshape(x.shape)
    return codes, sc.astype(np.uint8), val.reshape(x.shape)


def kv_places(fmt, page, dim):
    """Where a page's tokens stand: (K byte, K shift, V byte, V shift) for each
    [token, element] and (K, V) scale bytes for each [token, block]."""
    s, d = np.arange(page)[:, None], np.arange(dim)[None, :]
    blk = BLOCK[fmt]
    kb = s * (dim // 2) + d // 2
    vb = page * dim // 2 + (s // 4) * 2 * dim + ((d % 16) * 4 + s % 4) * (dim // 32) + d // 32
    g = np.arange(dim // blk)[None, :]
    ks = page * dim + s * (dim // blk) + g
    vs = ks + page * (dim // blk)
    return kb, 4 * (d % 2) + 0 * s, vb, 4 * (d % 32 // 16) + 0 * s, ks, vs


def kv_page_bytes(fmt, page, dim):
    return page * (dim + 2 * (dim // BLOCK[fmt]))


def kv_append(fmt, cache, page, offsets, table, lens, k, v, kt=None, vt=None):
    """Stores k, v [rows, H, D] into cache [pages, H, bytes] in place."""
    pages, H, _ = cache.shape
    D = k.shape[-1]
    kb, kh, vb, vh, ks, vs = kv_places(fmt, page, D)
    kc, ksc, _ = kv_quantize(fmt, k, kt)
    vc, vsc, _ = kv_quantize(fmt, v, vt)
    for r, pid, slot in kv_positions(page, offsets, table, lens, pages):
        if pid < 0:
            continue
        for h in range(H):
            row = cache[pid, h]
            for bytes_, shift, codes in ((kb[slot], kh[slot], kc[r, h]), (vb[slot], vh[slot], vc[r, h])):
                for sh in (0, 4):
                    m = shift == sh
                    row[bytes_[m]] = (row[bytes_[m]] & (0xF0 if sh == 0 else 0x0F)) | (codes[m] << sh)
            row[ks[slot]] = ksc[r, h]
            row[vs[slot]] = vsc[r, h]


def kv_positions(page, offsets, table, lens, pages):
    """(row, page id or -1, slot) of each new token."""
    for b in range(len(lens)):
        n = offsets[b + 1] - offsets[b]
        for i in range(n):
            pos = int(lens[b]) - int(n) + i
            pid = -1
            if 0 <= pos < table.shape[1] * page:
                pid = int(table[b, pos // page])
                pid = pid if 0 <= pid < pages else -1
            yield int(offsets[b]) + i, pid, pos % page


def kv_values(fmt, cache, page, dim, pid, slot, h, kt=None, vt=None):
    """K and V values [n, D] (float64, exact: tensor scale in full) of tokens
    (pid[n], slot[n]) of head h."""
    kb, kh, vb, vh, ks, vs = kv_places(fmt, page, dim)
    out = []
    for by, sh, sc, t in ((kb, kh, ks, kt), (vb, vh, vs, vt)):
        c = (cache[pid[:, None], h, by[slot]] >> sh[slot]) & 15
        val = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
        s = cache[pid[:, None], h, sc[slot]]
        if fmt == NVFP4:
            f = np.append(E4M3, np.nan)[s & 127] * float(t[h])
        else:
            f = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
        out.append(val * np.repeat(f, BLOCK[fmt], 1))
    return out


def kv_read(fmt, cache, page, offsets, table, lens, rows, dim, kt=None, vt=None):
    """(k, v) as fp4q_kv_read gives them, as float64."""
    pages, H, _ = cache.shape
    k, v = np.zeros((2, rows, H, dim))
    for r, pid, slot in kv_positions(page, offsets, table, lens, pages):
        if pid < 0:
            continue
        for h in range(H):
            one = (np.array([pid]), np.array([slot]))
            kk, vv = kv_values(fmt, cache, page, dim, *one, h, np.ones(H), np.ones(H))
            for out, val, t in ((k, kk, kt), (v, vv, vt)):
                f = val[0].astype(np.float32) * (np.float32(t[h]) if t is not None else np.float32(1))
                out[r, h] = bf16_round(f)
    return k, v


def attention(fmt, cache, page, offsets, table, lens, q, kt=None, vt=None, window=0, scale=None,
              sinks=0):
    """(o, bound): the outputs [rows, heads, D] in 64 bits and, beside them,
    what an implementation may be off by, short of the rounding of its result:
    `weights` = sum p |v| / z and `scores` = the largest sum |q k| scale of a
    row, for the tolerances."""
    pages, H, _ = cache.shape
    rows, heads, D = q.shape
    G = heads // H
    scale = D ** -0.5 if scale is None else scale
    o = np.zeros((rows, heads, D))
    weights, scores = np.zeros((rows, heads, D)), np.zeros((rows, heads, 1))
    for b in range(len(lens)):
        n = int(offsets[b + 1] - offsets[b])
        if n == 0:
            continue
        r0, first = int(offsets[b]), int(lens[b]) - n
        pos = np.arange(max(0, min(int(lens[b]), table.shape[1] * page)))
        pid = table[b][pos // page].astype(np.int64)
        ok = (pid >= 0) & (pid < pages)
        pos, pid = pos[ok], pid[ok]
        if pos.size == 0:
            continue
        at = first + np.arange(n)[:, None]
        see = pos[None, :] <= at
        if window > 0:
            see &= (pos[None, :] > at - window) | (pos[None, :] < sinks)
        any_ = see.any(0)                        # keys that no row sees may hold anything
        pos, pid, see = pos[any_], pid[any_], see[:, any_]
        if pos.size == 0:
            continue
        for h in range(H):
            k, v = kv_values(fmt, cache, page, D, pid, pos % page, h, kt, vt)
            for j in range(h * G, h * G + G):
                x = q[r0:r0 + n, j] @ k.T * scale
                m = np.where(see, x, -np.inf).max(1, keepdims=True)
                p = np.where(see, np.exp(x - np.where(np.isfinite(m), m, 0)), 0.0)
                z = p.sum(1, keepdims=True)
                z = np.where(z > 0, z, 1.0)
                o[r0:r0 + n, j] = p @ v / z
                weights[r0:r0 + n, j] = p @ np.abs(v) / z
                a = np.abs(q[r0:r0 + n, j]) @ np.abs(k).T * scale
                scores[r0:r0 + n, j, 0] = np.where(see, a, 0).max(1)
    return o, weights, scores


def route(logits, k, score=SOFTMAX, bias=None, n_groups=1, top_groups=1, renorm=True):
    """dict as fp4q_route's outputs (weights float64), row by row."""
    logits = logits_of(logits)
    T, E = logits.shape
    ex, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        s = scores_of(logits[t], score)
        r = s if bias is None else s + np.asarray(bias, np.float64)
        key = logits[t] if bias is None else r
        allowed = np.ones(E, bool)
        if n_groups > 1:
            gs = E // n_groups
            best = [sum(sorted(r[g * gs:(g + 1) * gs])[-2:]) for g in range(n_groups)]
            keep = sorted(range(n_groups), key=lambda g: (-best[g], g))[:top_groups]
            allowed = np.repeat([g in keep for g in range(n_groups)], gs)
        order = sorted(np.flatnonzero(allowed), key=lambda e: (-key[e], e))[:k]
        ex[t], w[t] = order, s[order]
        if renorm:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    out = expert_order(ex, E)
    out.update(experts=ex, weights=w)
    return out


def logits_of(x):
    """NaN as -inf, +inf as the largest finite f32 number."""
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), -np.inf, np.minimum(x, float(np.finfo(np.float32).max)))


def scores_of(x, score):
    x = logits_of(x)
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    if not np.isfinite(x).any():
        return np.zeros_like(x)
    e = np.exp(x - x.max())
    return e / e.sum()


def expert_order(experts, E):
    T, k = experts.shape
    rows = sorted(range(T * k), key=lambda i: (experts.reshape(-1)[i], i))
    row_of = np.empty(T * k, np.int32)
    row_of[rows] = np.arange(T * k)
    offsets = np.zeros(E + 1, np.int32)
    np.cumsum(np.bincount(experts.reshape(-1), minlength=E), out=offsets[1:])
    return {"offsets": offsets, "row_src": (np.array(rows, np.int64) // k).astype(np.int32),
            "row_of": row_of.reshape(T, k)}


def route_weights(logits, experts, score=SOFTMAX, renorm=True):
    """The weights as a function of the logits at fixed experts."""
    w = np.stack([scores_of(x, score)[e] for x, e in zip(logits, experts)])
    return w / w.sum(1, keepdims=True) if renorm else w


def route_backward(logits, experts, d_weights, score=SOFTMAX, renorm=True):
    """(d_logits, size of the terms they are made of)."""
    T, E = logits.shape
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = scores_of(logits[t], score)
        p, dw = s[experts[t]], np.asarray(d_weights[t], np.float64)
        if renorm:
            total = p.sum()
            dp = (dw - (dw * p).sum() / total) / total if total > 0 else 0.0 * dw
            mag = (np.abs(dw) + (np.abs(dw) * p).sum() / total) / total if total > 0 else 0.0 * dw
        else:
            dp, mag = dw, np.abs(dw)
        # the Jacobian of the scores, in full
        jac = (np.diag(s) - np.outer(s, s)) if score == SOFTMAX else np.diag(s * (1 - s))
        d[t] = jac[:, experts[t]] @ dp
        size[t] = np.abs(jac[:, experts[t]]) @ mag
    return d, size


def combine(y, row_of, weights):
    """(out, sum of the magnitudes)."""
    out = np.zeros((row_of.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(row_of.shape[0]):
        for j, r in enumerate(row_of[t]):
            if 0 <= r < y.shape[0]:
                out[t] += weights[t, j] * y[r]
                mag[t] += abs(weights[t, j]) * np.abs(y[r])
    return out, mag


def combine_backward(y, row_of, weights, d_out):
    """(d_y, d_weights, sum of d_weights' magnitudes); unnamed rows 0."""
    d_y = np.zeros_like(y)
    d_w, mag = np.zeros(row_of.shape), np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j, r in enumerate(row_of[t]):
            if 0 <= r < y.shape[0]:
                d_y[r] = weights[t, j] * d_out[t]
                d_w[t, j] = math.fsum(y[r] * d_out[t])
                mag[t, j] = np.abs(y[r] * d_out[t]).sum()
    return d_y, d_w, mag


# ---- rotation, norm, operands' values, adapters -----------------------------

def rotate(x, positions, freqs, interleaved=False):
    """x [rows, heads, D] with each head's first 2 len(freqs) elements turned by
    positions [rows] times freqs, 64 bits, rounded as fp4q_kv_append_rotated
    says: to f32, then to bf16."""
    n = len(freqs)
    a = (np.asarray(positions, np.float64)[:, None] * np.asarray(freqs, np.float32).astype(np.float64))[:, None]
    c, s = np.cos(a), np.sin(a)
    one = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    two = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    out = np.array(x, np.float64)
    x1, x2 = out[..., one].copy(), out[..., two].copy()
    out[..., one], out[..., two] = bf16_round(x1 * c - x2 * s), bf16_round(x2 * c + x1 * s)
    return out


def token_positions(offsets, lens, rows):
    """Each new token's place in its sequence (0 for rows of none)."""
    pos = np.zeros(rows, np.int64)
    for b in range(len(lens)):
        n = int(offsets[b + 1]) - int(offsets[b])
        pos[offsets[b]:offsets[b + 1]] = int(lens[b]) - n + np.arange(n)
    return pos


def rms_norm(x, weight, eps, residual=None, bf16=True):
    """(h, r, y) of fp4q_rms_norm: h rounded to bf16 (or f32), r and y not."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + residual
        h = bf16_round(h) if bf16 else h.astype(np.float32).astype(np.float64)
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, r, h * r * weight


def rms_norm_backward(h, weight, r, d_y, d_h=None):
    """(d_x, d_weight), and for the tolerances the sums of absolute terms beside
    them: of a row's mean of g u, and of d_weight."""
    u, g = h * r, weight * d_y
    d_x = r * (g - u * (g * u).mean(1, keepdims=True))
    if d_h is not None:
        d_x = d_x + d_h
    return d_x, (d_y * u).sum(0), np.abs(g * u).mean(1, keepdims=True), np.abs(d_y * u).sum(0)


def mxfp8_quantize(x):
    """x [rows, cols] (bf16 values) -> (codes u8, scale codes u8, values)."""
    b = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    amax = np.abs(b).max(-1)
    e = np.full(amax.shape, -127)
    for k in range(-127, 128):                              # the smallest e with 448 2^e >= amax
        e = np.where(448.0 * 2.0 ** (k - 1) < amax, k, e)
    f = 2.0 ** e.astype(np.float64)[..., None]
    mag = _nearest(E4M3, np.abs(b) / f)
    neg = np.signbit(b)
    val = np.where(neg, -1.0, 1.0) * E4M3[mag] * f
    return ((mag + 128 * neg).astype(np.uint8).reshape(x.shape), (e + 127).astype(np.uint8),
            val.reshape(x.shape))


def lora(x, a, b, offsets, adapters, scale=None, y=None):
    """(out, inner, outer): out as fp4q_lora's, not rounded, and the sums of
    absolute terms that bound its error: |scale| (|x| |A|^T) |B|^T and |scale|
    |x A^T| |B|^T."""
    rows, N = x.shape[0], b.shape[1]
    out = np.zeros((rows, N)) if y is None else np.array(y, np.float64)
    inner, outer = np.zeros((rows, N)), np.zeros((rows, N))
    for g, j in enumerate(adapters):
        if not 0 <= j < len(a):
            continue
        r = slice(int(offsets[g]), int(offsets[g + 1]))
        s = 1.0 if scale is None else float(scale[j])
        u = s * (x[r] @ a[j].T)
        out[r] += u @ b[j].T
        inner[r] = abs(s) * (np.abs(x[r]) @ np.abs(a[j]).T) @ np.abs(b[j]).T
        outer[r] = np.abs(u) @ np.abs(b[j]).T
    return out, inner, outer
