"""Host checks of the rotated append, the norm and the adapters at the edges of
what they take (no GPU): empty batches, whose tensors have no address."""
import pytest

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
