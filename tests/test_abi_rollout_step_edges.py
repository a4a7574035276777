"""Host checks of the rotated append, the norm and the adapters at the edges of
what they take (no GPU): empty batches, whose tensors have no address."""
import pytest

from test_abi_layer_edges import passes

A, B = 0x10000, 0x20000
INVALID = -1


@pytest.fixture(scope="module")
def L():
    from fp4_w4a4_quantized_amd import binding
    return binding.lib()


def adapters(L, x=A, ldx=64, n=3, rank=16, off=A, ad=A, G=2, rows=5, K=64, N=30, y=A, ldy=30, out=B, dt=1,
             ldo=30, ws=A, wsb=1 << 20):
    return L.fp4q_lora(x, ldx, A, A, None, n, rank, off, ad, G, rows, K, N, y, ldy, out, dt, ldo, ws, wsb, None)


def test_adapters_of_no_rows_without_y(L):
    """y NULL has no stride; it is not out, which has no address either."""
    for dt in (0, 1):
        for ldy in (0, 30):
            for out in (None, B):
                assert adapters(L, rows=0, x=None, y=None, ldy=ldy, out=out, dt=dt) == 0
    assert adapters(L, y=B, ldy=31) == INVALID          # out over y of another stride


def test_adapters_of_no_requests(L):
    for y in (None, A):
        assert adapters(L, rows=0, G=0, ad=None, x=None, y=y, out=None) == 0
    assert adapters(L, rows=0, G=-1, ad=None) == INVALID
    assert adapters(L, rows=0, G=1, ad=None) == INVALID
    assert adapters(L, G=0) == INVALID                  # rows, but no request


def quantized_norm(L, fmt=0, lay=0, rows=5, cols=128, x=A, res=None, h=None, ch=A, nc=4, q=A, s=A, ts=A, given=1,
                   r=B, ws=None, wsb=0):
    return L.fp4q_rms_norm_quantize(fmt, lay, 1, x, cols, res, cols, h, cols, A, 0, 1e-6, rows, cols, ch, nc, q, s,
                                    ts if fmt == 0 else None, given, r, None, 1, cols, None, ws, wsb, None)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("lay", [0, 1])
def test_norm_into_an_operand_of_no_rows_with_channels(L, fmt, lay):
    """(Past the checks: a launch failure that the test hook asks for.)"""
    for given in (0, 1):
        for r in (None, B):
            assert passes(lambda: quantized_norm(L, fmt, lay, rows=0, x=None, q=None, s=None, r=r, given=given))
    assert quantized_norm(L, fmt, lay, r=None) == INVALID
    assert quantized_norm(L, fmt, lay, rows=0, ch=None, nc=0) == INVALID     # a residual of no channels


@pytest.mark.parametrize("fmt", [0, 1])
def test_an_empty_batch_with_channels_through_the_layer(L, fmt):
    """The quantizer, the products and the permutation behind such a norm: no rows'
    residual has no address there either."""
    ats = A if fmt == 0 else None

    def quantizer(rows, r):
        return L.fp4q_quantize(fmt, 0, A, rows, 128, 128, None, 1, A, 4, A, A, ats, r, A, 1 << 20, None)

    def product(M, r):
        return L.fp4q_gemm(fmt, 0, M, 64, 128, A, A, ats, A, A, ats, A, 4, r, A, 1, 64, A, 1 << 20, None)

    def prepared(M, r):
        return L.fp4q_gemm_prepared(fmt, 0, M, 64, 128, A, A, ats, A, A, ats, A, 4, r, A, 1 << 20, A, 1, 64, None)

    def grouped(rows, r):
        return L.fp4q_grouped_gemm(fmt, 0, rows, 64, 128, A, 2, A, A, ats, A, A, ats, A, 4, r, A, 1, A, 1 << 20, None)

    def second(M, r):
        return L.fp4q_gemm_residual_fp4(fmt, 0, M, 64, 128, A, A, ats, A, A, ats, A, 32, r, r, ats, A, 1, 64, A,
                                        1 << 20, None)

    for f in (quantizer, product, prepared, grouped, second):
        assert f(5, None) == INVALID, f.__name__
        for r in (None, A):
            assert passes(lambda: f(0, r)) or f(0, r) == 0, f.__name__

    def permuted(rows, r):
        return L.fp4q_permute_quantized(fmt, A, 5, 128, 128, A, A, ats, A, rows, A, 2, A, 4, A, A, ats, r, None)

    assert permuted(5, None) == INVALID
    assert permuted(0, None) == 0 if fmt else passes(lambda: permuted(0, None))


def test_results_over_inputs_of_another_stride_or_type(L):
    """Each is written over rows that are still to be read; of one row the stride
    does not count."""
    def rotated(qo=A, ldqo=512, rows=5):
        return L.fp4q_kv_append_rotated(0, A, 4, 16, 2, 128, A, 2, A, 3, 3, A, rows, A, 512, 4, qo, ldqo, B, 256, B,
                                        256, A, 32, 0, None, A, A, None)

    assert passes(rotated) and passes(lambda: rotated(qo=B, ldqo=520)) and passes(lambda: rotated(ldqo=520, rows=1))
    assert rotated(ldqo=520) == INVALID

    X, R, H, Y = 0x100000, 0x200000, 0x300000, 0x400000

    def norm(ldx=64, res=R, ldr=64, h=H, ldh=64, y=Y, yt=1, ldy=64, rows=5):
        return L.fp4q_rms_norm(1, X, ldx, res, ldr, h, ldh, A, 0, 1e-6, rows, 64, y, yt, ldy, A, None)

    def operand(ldx=64, res=R, ldr=64, h=H, ldh=64, y=Y, yt=1, ldy=64, rows=5):
        return L.fp4q_rms_norm_quantize(0, 0, 1, X, ldx, res, ldr, h, ldh, A, 0, 1e-6, rows, 64, None, 0, A, A, A, 1,
                                        None, y, yt, ldy, A, None, 0, None)

    for f in (norm, operand):
        for over in (dict(h=X), dict(h=R), dict(y=X), dict(h=X, ldx=66, ldh=66), dict(h=X, ldh=66, rows=1),
                     dict(h=R, y=X), dict(ldh=70, ldy=71, ldx=72, ldr=73)):
            assert passes(lambda: f(**over)), (f.__name__, over)
        for over in (dict(h=X, ldh=65), dict(h=X, ldx=65), dict(h=R, ldr=65), dict(y=X, ldy=66), dict(y=X, yt=0),
                     dict(y=X, yt=0, rows=1), dict(res=None, h=None, y=X, ldx=80), dict(y=R, yt=0), dict(y=H, yt=0)):
            assert f(**over) == INVALID, (f.__name__, over)

    def gradient(dyt=1, lddy=64, dh=R, lddh=64, dx=Y, lddx=64, rows=5, dy=H):
        return L.fp4q_rms_norm_backward(1, X, 64, A, 0, A, dy, dyt, lddy, dh, lddh, dx, lddx, A, rows, 64, A, 1 << 20,
                                        None)

    for over in (dict(dx=H), dict(dx=R), dict(dx=H, lddy=70, lddx=70), dict(dx=R, lddx=70, rows=1), dict(dyt=0)):
        assert passes(lambda: gradient(**over)), over
    for over in (dict(dx=H, lddx=70), dict(dx=H, dyt=0), dict(dx=R, lddh=70), dict(dx=X, lddx=70)):
        assert gradient(**over) == INVALID, over
