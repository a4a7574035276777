"""Refusals of the calls between the FP4 linear layers (no GPU): the key/value
cache, attention over it, the router and the combination.  Every check runs
on the host before any HIP call, so the device addresses are never read."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE, HIP_ERR = -1, -2, -3, -4
A, B, ODD = 0x10000, 0x20000, 0x10008


@pytest.fixture(scope="module")
def L():
    from fp4_w4a4_quantized_amd import binding
    return binding.lib()


KV = dict(fmt=0, cache=A, n_pages=4, page=16, H=2, D=128, off=A, batch=2, table=A, ld=3, cols=3,
          lens=A, rows=5)


def _kv(over):
    a = {**KV, **over}
    return [a[x] for x in ("fmt", "cache", "n_pages", "page", "H", "D", "off", "batch", "table",
                           "ld", "cols", "lens", "rows")]


def copy(L, fn, k=A, ldk=256, v=B, ldv=256, ks=A, vs=A, **over):
    return getattr(L, fn)(*_kv(over), k, ldk, v, ldv, ks, vs, None)


def attend(L, q=A, ldq=512, heads=4, max_new=1, max_len=40, window=0, scale=0.1, ks=A, vs=A, y=B,
           dt=1, ldy=512, ws=A, wsb=1 << 30, **over):
    return L.fp4q_kv_attention(*_kv(over), q, ldq, heads, max_new, max_len, window, scale, ks, vs, y,
                               dt, ldy, ws, wsb, None)


BAD_KV = [dict(fmt=7), dict(cache=None), dict(cache=ODD), dict(n_pages=0), dict(n_pages=-1),
          dict(page=0), dict(H=0), dict(D=0), dict(off=None), dict(batch=0), dict(batch=-1),
          dict(table=None), dict(cols=0), dict(ld=2), dict(lens=None), dict(rows=-1),
          dict(ks=None), dict(vs=None), dict(fmt=1)]
UNSUP_KV = [dict(page=8), dict(page=48), dict(page=2048), dict(D=96), dict(D=32),
            dict(cols=1 << 28, ld=1 << 28)]


@pytest.mark.parametrize("fn", ["fp4q_kv_append", "fp4q_kv_read"])
def test_cache_refusals(L, fn):
    for over in BAD_KV + [dict(k=None), dict(v=None), dict(k=ODD), dict(ldk=248), dict(ldv=260)]:
        assert copy(L, fn, **over) == INVALID, over
    for over in UNSUP_KV + [dict(rows=1 << 31)]:
        assert copy(L, fn, **over) == UNSUPPORTED, over
    assert copy(L, fn, rows=0, batch=0, cache=None, k=None, v=None) == 0


def test_attention_refusals(L):
    for over in BAD_KV + [dict(q=None), dict(y=None), dict(q=ODD), dict(y=ODD), dict(ldq=504),
                          dict(ldq=516), dict(ldy=504), dict(heads=3), dict(heads=0),
                          dict(max_new=0), dict(max_new=-1), dict(max_len=-1), dict(window=-1),
                          dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                          dict(scale=float("inf")), dict(dt=2)]:
        assert attend(L, **over) == INVALID, over
    big = dict(ldq=1 << 20, ldy=1 << 20)
    for over in UNSUP_KV + [dict(heads=258, **big), dict(batch=65536), dict(rows=1 << 29),
                            dict(max_len=1 << 31), dict(max_new=1 << 30)]:
        assert attend(L, **over) == UNSUPPORTED, over
    assert attend(L, rows=0, q=None, y=None) == 0
    long = dict(max_len=1 << 17, cols=1 << 13, ld=1 << 13)
    need = L.fp4q_kv_attention_workspace_bytes(0, 5, 4, 2, 128, 2, 1, 1 << 17, 0)
    assert need > 0
    for over in (dict(ws=None), dict(wsb=need - 1), dict(ws=ODD)):
        assert attend(L, **long, **over) == WORKSPACE, over


def test_queries(L):
    assert L.fp4q_kv_page_bytes(0, 16, 128) == 16 * (128 + 16)
    assert L.fp4q_kv_page_bytes(1, 64, 64) == 64 * (64 + 4)
    assert all(L.fp4q_kv_page_bytes(*a) == 0 for a in ((2, 16, 128), (0, 24, 128), (0, 16, 80)))
    assert L.fp4q_kv_attention_workspace_bytes(0, 0, 4, 2, 128, 2, 1, 100, 0) == 0
    assert L.fp4q_kv_attention_workspace_bytes(0, 4, 5, 2, 128, 2, 1, 1 << 20, 0) == 0
    assert L.fp4q_route_workspace_bytes(0, 128) == 0
    assert L.fp4q_route_workspace_bytes(16384, 128) > 0


def route(L, x=A, dt=1, T=100, E=64, ldx=64, k=4, score=0, bias=None, G=1, top=1, renorm=1, ex=A,
          w=A, off=A, src=A, row=A, ws=A, wsb=1 << 20):
    return L.fp4q_route(x, dt, T, E, ldx, k, score, bias, G, top, renorm, ex, w, off, src, row, ws,
                        wsb, None)


def test_route_refusals(L):
    for over in [dict(x=None), dict(dt=2), dict(T=-1), dict(E=0, ldx=0), dict(ldx=63), dict(k=0),
                 dict(k=65), dict(score=2), dict(G=0), dict(G=3), dict(G=4, top=5),
                 dict(G=4, top=0), dict(G=16, top=1, k=5), dict(ex=None), dict(w=None),
                 dict(off=None), dict(src=None), dict(row=None), dict(x=0x10001),
                 dict(dt=0, x=0x10002), dict(ex=0x10002)]:
        assert route(L, **over) == INVALID, over
    for over in [dict(E=513, ldx=513), dict(E=512, ldx=512, G=128, top=128), dict(k=33),
                 dict(T=1 << 30)]:
        assert route(L, **over) == UNSUPPORTED, over
    need = L.fp4q_route_workspace_bytes(100, 64)
    for over in (dict(ws=None), dict(wsb=need - 1), dict(ws=0x10004)):
        assert route(L, **over) == WORKSPACE, over


def test_route_backward_refusals(L):
    def f(x=A, dt=1, T=10, E=64, ldx=64, k=4, score=0, renorm=1, ex=A, dw=A, d=B, ldd=64):
        return L.fp4q_route_backward(x, dt, T, E, ldx, k, score, renorm, ex, dw, d, ldd, None)

    for over in [dict(x=None), dict(dt=2), dict(T=-1), dict(E=0), dict(ldx=63), dict(ldd=63),
                 dict(k=0), dict(k=65), dict(score=2), dict(ex=None), dict(dw=None), dict(d=None),
                 dict(d=0x20001)]:
        assert f(**over) == INVALID, over
    assert f(E=513, ldx=513, ldd=513) == UNSUPPORTED and f(k=33) == UNSUPPORTED
    assert f(T=0, x=None, ex=None, dw=None, d=None) == 0


def test_combine_refusals(L):
    def f(dt=1, y=A, rows=8, cols=64, ldy=64, row=A, w=A, T=2, k=4, out=B, ldo=64):
        return L.fp4q_combine(dt, y, rows, cols, ldy, row, w, T, k, out, ldo, None)

    def g(dt=1, y=A, rows=8, cols=64, ldy=64, row=A, w=A, T=2, k=4, do=B, ldo=64, dy=A, lddy=64,
          dw=A):
        return L.fp4q_combine_backward(dt, y, rows, cols, ldy, row, w, T, k, do, ldo, dy, lddy, dw,
                                       None)

    both = [dict(dt=2), dict(y=None), dict(rows=-1), dict(cols=0), dict(ldy=63), dict(row=None),
            dict(w=None), dict(T=-1), dict(k=0), dict(ldo=63), dict(y=0x10001), dict(w=0x10002)]
    for fn, more in ((f, [dict(out=None)]), (g, [dict(do=None), dict(dy=None), dict(dw=None),
                                                 dict(lddy=63)])):
        for over in both + more:
            assert fn(**over) == INVALID, over
        for over in [dict(k=129), dict(T=1 << 30), dict(cols=1 << 31, ldy=1 << 31, ldo=1 << 31,
                                                        **({"lddy": 1 << 31} if fn is g else {}))]:
            assert fn(**over) == UNSUPPORTED, over
        assert fn(T=0) == 0


def test_injected_failure(L):
    """Each call reports a launch failure that the hook asks for, once."""
    from fp4_w4a4_quantized_amd import binding as b
    for call in (lambda: copy(L, "fp4q_kv_append"), lambda: copy(L, "fp4q_kv_read"),
                 lambda: attend(L), lambda: route(L)):
        b.test_hook(b.HOOK_FAIL_NEXT_LAUNCH, 719)
        try:
            assert call() == HIP_ERR and L.fp4q_last_hip_error() == 719
        finally:
            b.test_hook(b.HOOK_RESET)


def test_binding_refuses_other_tensors():
    """What the C call cannot see is refused by the binding: types, strides and
    shapes of the tensors."""
    import fp4_w4a4_quantized_amd as fq
    z = torch.zeros
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    cache = z(4, 2, fq.kv_page_bytes(1, 16, 64), dtype=torch.uint8)
    ok = [1, cache, 16, z(3, **i32), z(2, 3, **i32), z(2, **i32), z(5, 2, 64, **bf),
          z(5, 2, 64, **bf)]

    def refuse(i, bad):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            fq.kv_append(*args)

    refuse(1, cache[:, :, 1:])
    refuse(1, cache.to(torch.int16))
    refuse(2, 32)
    refuse(3, z(3, dtype=torch.int64))
    refuse(3, z(4, **i32))
    refuse(4, z(2, 3, dtype=torch.int64))
    refuse(4, z(3, 2, **i32).t())
    refuse(5, z(4, **i32)[::2])
    refuse(6, z(5, 2, 64))
    refuse(6, z(5, 64, 2, **bf).transpose(1, 2))
    refuse(6, z(5, 3, 64, **bf))
    refuse(7, z(4, 2, 64, **bf))
    with pytest.raises(ValueError):
        fq.kv_cache(0, 4, 24, 2, 128, "cpu")
    with pytest.raises(ValueError):
        fq.combine(z(8, 4).t(), z(2, 2, **i32), z(2, 2))
    with pytest.raises(ValueError):
        fq.combine(z(8, 4), z(2, 2, dtype=torch.int64), z(2, 2))
    with pytest.raises(ValueError):
        fq.combine(z(8, 4), z(2, 2, **i32), z(2, 2, **bf))
    with pytest.raises(ValueError):
        fq.route(z(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        fq.route(z(4, 8), 2, bias=z(7))
    with pytest.raises(ValueError):
        fq.route_backward(z(4, 8), z(4, 2, dtype=torch.int64), z(4, 2))
