"""Host checks of the calls between the FP4 linear layers at the edges of their
limits (no GPU): what is refused, and what passes the checks (shown by a launch
failure that the test hook asks for)."""
import pytest

INVALID, UNSUPPORTED, WORKSPACE, HIP_ERR = -1, -2, -3, -4
A, B = 0x10000, 0x20000


@pytest.fixture(scope="module")
def L():
    from fp4_w4a4_quantized_amd import binding
    return binding.lib()


def passes(call):
    """Does the call get past all its checks?"""
    from fp4_w4a4_quantized_amd import binding as b
    b.test_hook(b.HOOK_FAIL_NEXT_LAUNCH, 719)
    try:
        return call() == HIP_ERR
    finally:
        b.test_hook(b.HOOK_RESET)


def test_zeroed_combination_gradient(L):
    def f(dt=1, y=A, rows=8, cols=64, ldy=64, row=A, w=A, T=2, k=4, do=B, ldo=64, dy=A, lddy=64, dw=A, ws=A,
          wsb=32):
        return L.fp4q_combine_backward_zeroed(dt, y, rows, cols, ldy, row, w, T, k, do, ldo, dy, lddy, dw, ws,
                                              wsb, None)

    assert L.fp4q_combine_backward_zeroed_workspace_bytes(8) == 32
    assert L.fp4q_combine_backward_zeroed_workspace_bytes(0) == 0
    for over in [dict(dt=2), dict(y=None), dict(rows=-1), dict(cols=0), dict(ldy=63), dict(row=None), dict(w=None),
                 dict(T=-1), dict(k=0), dict(ldo=63), dict(do=None), dict(dy=None), dict(dw=None), dict(lddy=63),
                 dict(T=0, dy=None), dict(dy=0x10001)]:
        assert f(**over) == INVALID, over
    for over in [dict(k=129), dict(T=1 << 30), dict(rows=1 << 31, wsb=1 << 40)]:
        assert f(**over) == UNSUPPORTED, over
    for over in [dict(ws=None), dict(wsb=31), dict(ws=0x10002)]:
        assert f(**over) == WORKSPACE, over
    assert f(T=0, rows=0, dy=None, ws=None, wsb=0) == 0
    assert passes(f) and passes(lambda: f(T=0, y=None, row=None, w=None, do=None, dw=None))


def attention(L, rows=5, heads=4, kv_heads=2, dim=128, batch=2, max_new=1, max_len=40, window=0, page=16, cols=3):
    """The call with enough workspace, and what it asks for."""
    need = L.fp4q_kv_attention_workspace_bytes(0, rows, heads, kv_heads, dim, batch, max_new, max_len, window)
    return need, lambda: L.fp4q_kv_attention(0, A, 4, page, kv_heads, dim, A, batch, A, cols, cols, A, rows, A,
                                             heads * dim, heads, max_new, max_len, window, 0.1, A, A, B, 1,
                                             heads * dim, A, need, None)


def test_lengths_up_to_the_limit(L):
    """Up to 2^31 - 4096 keys; the kernels' 32-bit key numbers go a little past
    the last one.  A larger max_len is taken where the table ends before."""
    long = (1 << 31) - 4096
    whole = dict(page=1024, cols=(1 << 21) - 1)
    for over in (dict(), dict(max_new=40, rows=40), dict(batch=1, kv_heads=1, dim=64)):
        need, call = attention(L, max_len=long, **whole, **over)
        assert need > 0 and passes(call), over
        for more in (1, 4095):
            assert attention(L, max_len=long + more, **whole, **over)[1]() == UNSUPPORTED, (over, more)
            assert passes(attention(L, max_len=long + more, page=1024, cols=(1 << 21) - 4, **over)[1]), (over, more)
            assert passes(attention(L, max_len=long + more, **over)[1]), (over, more)
        need, call = attention(L, max_len=1 << 31, **over)
        assert need == 0 and call() == UNSUPPORTED, over


@pytest.mark.parametrize("over", [dict(max_len=1 << 60), dict(max_new=1 << 60), dict(rows=1 << 60),
                                  dict(batch=65536), dict(batch=1 << 12, kv_heads=1 << 10, heads=1 << 10),
                                  dict(heads=258)])
def test_no_workspace_for_what_is_refused(L, over):
    need, call = attention(L, **over)
    assert need == 0 and call() == UNSUPPORTED


@pytest.mark.parametrize("dim,tile", [(64, 256), (128, 256), (256, 128)])
def test_long_prompts_of_many_heads(L, dim, tile):
    """The row tiles of one kv head are what the grid bounds, not times the kv
    heads: 131072 new tokens of 128 heads on 8, and up to 65535 tiles."""
    for n in (65536, 131072):
        _, call = attention(L, rows=n, heads=128, kv_heads=8, dim=dim, batch=1, max_new=n, max_len=n, page=64,
                            cols=2048)
        assert passes(call), n
    for heads, kv_heads in ((16, 1), (32, 2)):
        last = 65535 * tile // 16
        _, call = attention(L, rows=8, heads=heads, kv_heads=kv_heads, dim=dim, batch=1, max_new=last, max_len=last)
        assert passes(call)
        need, call = attention(L, rows=8, heads=heads, kv_heads=kv_heads, dim=dim, batch=1, max_new=last + 1,
                               max_len=last + 1)
        assert need == 0 and call() == UNSUPPORTED
