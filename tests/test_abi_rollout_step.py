"""Refusals of the rotated append, the attention with first tokens, the norm, the
operand's values and the adapters (no GPU): in the C ABI, where every check
runs on the host before any HIP call so that the device addresses are never
read, and in the Python calls' checks of their tensors."""
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from test_abi_layer import A, B, BAD_KV, INVALID, ODD, UNSUP_KV, UNSUPPORTED, WORKSPACE, _kv
from test_layer_binding import BF, I32, cache_args, z

GPU = "a tensor on the GPU is needed"


@pytest.fixture(scope="module")
def L():
    from fp4_w4a4_quantized_amd import binding
    return binding.lib()


def test_rotated_append_refusals(L):
    def f(q=A, ldq=512, heads=4, qo=B, ldqo=512, k=A, ldk=256, v=B, ldv=256, fr=A, rot=32, pairs=0,
          pos=None, ks=A, vs=A, **over):
        return L.fp4q_kv_append_rotated(*_kv(over), q, ldq, heads, qo, ldqo, k, ldk, v, ldv, fr, rot, pairs,
                                        pos, ks, vs, None)

    for over in BAD_KV + [dict(k=None), dict(v=None), dict(k=ODD), dict(ldk=248), dict(ldv=260), dict(q=None),
                          dict(qo=None), dict(q=ODD), dict(qo=ODD), dict(ldq=504), dict(ldqo=516), dict(heads=0),
                          dict(rot=-16), dict(rot=144), dict(pairs=2), dict(fr=None), dict(fr=0x10002),
                          dict(pos=0x10001), dict(fmt=2)]:
        assert f(**over) == INVALID, over
    for over in UNSUP_KV + [dict(rot=24), dict(rot=8), dict(rows=1 << 25), dict(heads=1 << 24)]:
        assert f(**over) == UNSUPPORTED, over
    assert f(rows=0, batch=0, cache=None, q=None, qo=None, k=None, v=None, fr=None) == 0


def test_sinks_refusals(L):
    def f(q=A, ldq=512, heads=4, max_new=1, max_len=40, window=0, sinks=4, scale=0.1, ks=A, vs=A, y=B, dt=1,
          ldy=512, ws=A, wsb=1 << 30, **over):
        return L.fp4q_kv_attention_sinks(*_kv(over), q, ldq, heads, max_new, max_len, window, sinks, scale, ks,
                                         vs, y, dt, ldy, ws, wsb, None)

    for over in BAD_KV + [dict(q=None), dict(y=None), dict(ldq=504), dict(heads=3), dict(max_new=0),
                          dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(dt=2)]:
        assert f(**over) == INVALID, over
    for over in UNSUP_KV + [dict(batch=65536), dict(max_len=1 << 31)]:
        assert f(**over) == UNSUPPORTED, over
    assert f(rows=0, q=None, y=None) == 0

    def need(*a):
        return L.fp4q_kv_attention_sinks_workspace_bytes(0, 5, 4, 2, 128, 2, 1, 1 << 17, *a)

    assert need(4096, 0) == L.fp4q_kv_attention_workspace_bytes(0, 5, 4, 2, 128, 2, 1, 1 << 17, 4096) > 0
    # how calls with first tokens are split is a rule of their own
    assert need(4096, 4) > 0 and need(4096, 1 << 30) > 0 and need(2 ** 31 - 1, 2 ** 31 - 1) > 0
    assert need(0, 7) == need(0, 0) and need(4096, -1) == 0
    for window, sinks in ((0, 4), (1, 1), (4096, 4), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert L.fp4q_kv_attention_sinks_workspace_bytes(0, 5, 4, 2, 128, 2, 1, 0, window, sinks) == 0
    long = dict(max_len=1 << 17, cols=1 << 13, ld=1 << 13, window=4096)
    for over in (dict(ws=None), dict(wsb=need(4096, 4) - 1), dict(ws=ODD)):
        assert f(**long, **over) == WORKSPACE, over


def norm(L, dt=1, x=A, ldx=64, res=None, ldr=0, h=None, ldh=0, w=A, wt=0, eps=1e-6, rows=5, cols=64, y=B,
         yt=1, ldy=64, rstd=A):
    return L.fp4q_rms_norm(dt, x, ldx, res, ldr, h, ldh, w, wt, eps, rows, cols, y, yt, ldy, rstd, None)


NORM_BAD = [dict(dt=2), dict(x=None), dict(x=0x10001), dict(ldx=63), dict(res=A), dict(h=A), dict(rows=-1),
            dict(res=A, ldr=63, h=B, ldh=64), dict(res=A, ldr=64, h=B, ldh=63), dict(cols=0), dict(w=None),
            dict(w=0x10002), dict(wt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
            dict(yt=2), dict(ldy=63), dict(y=0x10001), dict(rstd=0x10002), dict(dt=0, x=0x10002)]


def test_norm_refusals(L):
    for over in NORM_BAD + [dict(y=None)]:
        assert norm(L, **over) == INVALID, over
    big = dict(ldx=32769, ldy=32769, cols=32769)
    assert norm(L, **big) == UNSUPPORTED and norm(L, rows=1 << 31) == UNSUPPORTED
    assert norm(L, rows=0, x=None, y=None, rstd=None) == 0


def test_norm_quantize_refusals(L):
    def f(fmt=0, lay=0, dt=1, x=A, ldx=64, res=None, ldr=0, h=None, ldh=0, w=A, wt=0, eps=1e-6, rows=5, cols=64,
          ch=None, nc=0, q=A, s=A, ts=A, given=1, r=None, y=None, yt=1, ldy=64, rstd=None, ws=A, wsb=1 << 20):
        return L.fp4q_rms_norm_quantize(fmt, lay, dt, x, ldx, res, ldr, h, ldh, w, wt, eps, rows, cols, ch, nc,
                                        q, s, ts, given, r, y, yt, ldy, rstd, ws, wsb, None)

    mx8 = dict(fmt=2, ts=None)
    for over in [d for d in NORM_BAD if "y" not in d and "ldy" not in d] + [
            dict(fmt=3), dict(fmt=-1), dict(lay=2), dict(cols=72, ldx=72, ldy=72), dict(lay=1), dict(ch=A),
            dict(nc=4), dict(ch=A, nc=4), dict(r=A), dict(ch=A, nc=65, r=A), dict(ch=A, nc=-1, r=A),
            dict(ts=None), dict(fmt=1), dict(q=None), dict(q=ODD), dict(s=None), dict(s=0x10002),
            dict(y=B, ldy=63), dict(**mx8, lay=1, cols=128, ldx=128), dict(**mx8, ch=A, nc=4, r=A),
            dict(**mx8, cols=48, ldx=48), dict(ts=0x10001)]:
        assert f(**over) == INVALID, over
    assert f(cols=32784, ldx=32784) == UNSUPPORTED
    need = L.fp4q_rms_norm_quantize_workspace_bytes(0, 5, 0)
    assert need > 0 and L.fp4q_rms_norm_quantize_workspace_bytes(0, 5, 1) == 0
    assert L.fp4q_rms_norm_quantize_workspace_bytes(1, 5, 0) == L.fp4q_rms_norm_quantize_workspace_bytes(0, 0, 0) == 0
    for over in (dict(ws=None), dict(wsb=need - 1), dict(ws=0x10004)):
        assert f(given=0, **over) == WORKSPACE, over


def test_norm_backward_refusals(L):
    def f(dt=1, h=A, ldh=64, w=A, wt=0, r=A, dy=A, dyt=1, lddy=64, dh=None, lddh=0, dx=B, lddx=64, dw=A, rows=5,
          cols=64, ws=A, wsb=1 << 20):
        return L.fp4q_rms_norm_backward(dt, h, ldh, w, wt, r, dy, dyt, lddy, dh, lddh, dx, lddx, dw, rows, cols,
                                        ws, wsb, None)

    for over in [dict(dt=2), dict(h=None), dict(ldh=63), dict(w=None), dict(wt=3), dict(r=None), dict(dy=None),
                 dict(dyt=2), dict(lddy=63), dict(dh=A, lddh=63), dict(dh=0x10001, lddh=64), dict(dx=None),
                 dict(lddx=63), dict(dw=None), dict(dw=0x10002), dict(rows=-1), dict(cols=0)]:
        assert f(**over) == INVALID, over
    assert f(cols=40000, ldh=40000, lddy=40000, lddx=40000) == UNSUPPORTED
    need = L.fp4q_rms_norm_backward_workspace_bytes(5, 64)
    assert need > 0 and L.fp4q_rms_norm_backward_workspace_bytes(0, 64) == 0
    for over in (dict(ws=None), dict(wsb=need - 1), dict(ws=0x10002)):
        assert f(**over) == WORKSPACE, over


def test_dequantize_refusals(L):
    def f(fmt=0, lay=0, q=A, s=A, ts=A, rows=5, cols=64, y=B, yt=1, ldy=64):
        return L.fp4q_dequantize(fmt, lay, q, s, ts, rows, cols, y, yt, ldy, None)

    for over in [dict(fmt=3), dict(lay=2), dict(lay=1), dict(fmt=2, ts=None, lay=1, cols=128, ldy=128),
                 dict(cols=40, ldy=40), dict(cols=0), dict(rows=-1), dict(q=None), dict(s=None), dict(q=ODD),
                 dict(s=0x10002), dict(ts=None), dict(fmt=1), dict(y=None), dict(y=0x10001), dict(yt=2),
                 dict(ldy=63)]:
        assert f(**over) == INVALID, over
    assert f(rows=1 << 31) == UNSUPPORTED and f(rows=1 << 28) == UNSUPPORTED
    assert f(rows=0, q=None, s=None, y=None) == 0


def test_adapter_refusals(L):
    def f(x=A, ldx=64, a=A, b=A, sc=None, n=3, rank=16, off=A, ad=A, G=2, rows=5, K=64, N=30, y=A, ldy=30, out=B,
          dt=1, ldo=30, ws=A, wsb=1 << 20):
        return L.fp4q_lora(x, ldx, a, b, sc, n, rank, off, ad, G, rows, K, N, y, ldy, out, dt, ldo, ws, wsb, None)

    for over in [dict(x=None), dict(x=ODD), dict(ldx=56), dict(ldx=68), dict(a=None), dict(b=None), dict(a=ODD),
                 dict(b=ODD), dict(sc=0x10002), dict(n=0), dict(rank=0), dict(off=None), dict(ad=None), dict(G=0),
                 dict(rows=-1), dict(K=0, ldx=0), dict(N=0), dict(ldy=29), dict(out=None), dict(ldo=29),
                 dict(dt=2), dict(dt=0, out=0x10002), dict(out=A, ldo=40), dict(y=0x10001)]:
        assert f(**over) == INVALID, over
    for over in [dict(rank=12), dict(rank=136), dict(K=60), dict(rows=1 << 24), dict(G=65537)]:
        assert f(**over) == UNSUPPORTED, over
    need = L.fp4q_lora_workspace_bytes(5, 2, 16, 64, 30)
    assert need > 0 and L.fp4q_lora_workspace_bytes(5, 2, 12, 64, 30) == 0
    for over in (dict(ws=None), dict(wsb=need - 1), dict(ws=ODD)):
        assert f(**over) == WORKSPACE, over
    assert f(rows=0, x=None, y=None, out=None) == 0


# ---- the Python calls -------------------------------------------------------

def test_rotated_append_tensors():
    q, k, f = z(5, 4, 64, **BF), z(5, 2, 64, **BF), z(32)
    with pytest.raises(ValueError, match=GPU):
        fq.kv_append_rotated(*cache_args(), q, k, k, f)
    for args, kw, why in (((z(5, 4, 64), k, k, f), {}, "q: bf16"), ((z(6, 4, 64, **BF), k, k, f), {}, "k: q's rows"),
                          ((q, k, z(5, 1, 64, **BF), f), {}, "v: k's shape"), ((q, k, k, z(33)), {}, "freqs: more"),
                          ((q, k, k, z(32, **BF)), {}, "freqs: contiguous f32"),
                          ((q, k, k, f), dict(positions=z(4, **I32)), "positions: another"),
                          ((q, k, k, f), dict(positions=z(5)), "positions: contiguous int32")):
        with pytest.raises(ValueError, match=why):
            fq.kv_append_rotated(*cache_args(), *args, **kw)
    with pytest.raises(ValueError, match="q_out: q's shape"):
        fq.kv_append_rotated_into(*cache_args(), q, k, k, f, None, None, k)


def test_norm_tensors():
    x, w = z(5, 64, **BF), z(64)
    for call in (lambda: fq.rms_norm(x, w), lambda: fq.rms_norm(x, w, residual=x),
                 lambda: fq.rms_norm_quantize(fq.MXFP8, x, w), lambda: fq.rms_norm_quantize(fq.NVFP4, x, w, tscale=z(1)),
                 lambda: fq.rms_norm_backward(x, w, z(5), x)):
        with pytest.raises(ValueError, match=GPU):
            call()
    for args, kw, why in (((z(5, 64, dtype=torch.float16), w), {}, "x: f32 or bf16"), ((x.T, z(5)), {}, "x: a matrix"),
                          ((x, z(63)), {}, "weight: one for each"), ((x, z(64, dtype=torch.float64)), {}, "weight: f32"),
                          ((x, w), dict(residual=z(5, 64)), "residual: x's shape and type"),
                          ((x, w), dict(y_dtype=7), "y_dtype: OUT")):
        with pytest.raises(ValueError, match=why):
            fq.rms_norm(*args, **kw)
    for fmt, kw, why in ((3, {}, "fmt: no such"), (0, dict(layout=2), "layout: no such"),
                         (2, dict(layout=1), "layout: MXFP8"), (0, dict(layout=1), "x: its columns"),
                         (1, dict(tscale=z(1)), "tscale: NVFP4"), (0, dict(tscale=z(2)), "tscale: another"),
                         (2, dict(chan_idx=z(4, **I32)), "chan_idx: not for"),
                         (0, dict(chan_idx=z(4)), "chan_idx: contiguous int32"), (0, dict(h=x), "h: a residual"),
                         (0, dict(residual=x, h=z(5, 64)), "h: x's shape and type")):
        with pytest.raises(ValueError, match=why):
            fq.rms_norm_quantize(fmt, x, w, **kw)
    for args, kw, why in (((x, w, z(4), x), {}, "rstd: another"), ((x, w, z(5), z(5, 63)), {}, "d_y: h's shape"),
                          ((x, w, z(5), x), dict(d_h=z(5, 64)), "d_h: h's shape and type")):
        with pytest.raises(ValueError, match=why):
            fq.rms_norm_backward(*args, **kw)


def test_dequantize_tensors():
    u8 = dict(dtype=torch.uint8)
    a = dict(q=z(5, 32, **u8), scales=z(5, 4, **u8), tscale=z(1), rows=5, cols=64, layout=0)
    with pytest.raises(ValueError, match=GPU):
        fq.dequantize(fq.NVFP4, a)
    for over, why in ((dict(tscale=None), "tscale: NVFP4"), (dict(tscale=z(2)), "tscale: another"),
                      (dict(rows=6), "q: contiguous bytes"), (dict(scales=z(5, 2, **u8)), "scales: contiguous bytes"),
                      (dict(cols=40), "cols: not whole"), (dict(rows=-1), "rows: out of"), (dict(layout=1), "cols: not")):
        with pytest.raises(ValueError, match=why):
            fq.dequantize(fq.NVFP4, {**a, **over})


def test_adapter_tensors():
    x, a, b, off, ad = z(5, 64, **BF), z(3, 16, 64, **BF), z(3, 30, 16, **BF), z(3, **I32), z(2, **I32)
    with pytest.raises(ValueError, match=GPU):
        fq.lora(x, a, b, off, ad, z(3), y=z(5, 30))
    for args, kw, why in (((z(5, 64), a, b, off, ad), {}, "x: bf16"), ((x, z(3, 16, 64), b, off, ad), {}, "a: contiguous"),
                          ((x, z(3, 16, 32, **BF), b, off, ad), {}, "a: x's columns"),
                          ((x, a, z(3, 30, 8, **BF), off, ad), {}, "b: a's adapters"),
                          ((x, a, b, z(4, **I32), ad), {}, "offsets: another"), ((x, a, b, off, z(2)), {}, "adapters: contiguous"),
                          ((x, a, b, off, ad, z(2)), {}, "scale: another"), ((x, a, b, off, ad), dict(y=z(5, 29)), "y: .rows, N"),
                          ((x, a, b, off, ad), dict(y=z(5, 30), y_dtype=fq.OUT_BF16), "y_dtype: y's type")):
        with pytest.raises(ValueError, match=why):
            fq.lora(*args, **kw)
    with pytest.raises(ValueError, match="out: .rows, N"):
        fq.lora_into(x, a, b, off, ad, None, z(5, 30), z(5, 30, **BF))
