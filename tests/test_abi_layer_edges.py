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
