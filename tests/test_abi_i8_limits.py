"""include/qlora_i8.h: what its contract allows is not refused, and the calls that
it forbids answer before anything is launched (no GPU needed)."""

import ctypes

import pytest

P = ctypes.c_void_p
X, W, S, T, Y, V = (P(0x10000000 * i) for i in range(1, 7))
OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = range(5)


@pytest.fixture(scope="module")
def so(lib):
    from bit_nf4_quantized_dequant_b200 import _norm_i8
    return _norm_i8._library()


def test_the_gradient_sums_over_n_alone(so):
    """K is not summed over by qlora_i8_linear_dx: the forward's limit on it,
    which keeps the int32 sum from overflowing, is not the gradient's."""
    n = ctypes.c_size_t()
    ws = lambda *a: so.qlora_i8_linear_workspace(*a, ctypes.byref(n))
    dx = lambda N, K, M=4: so.qlora_i8_linear_dx(X, M, W, S, N, K, None, None, 0, Y, None, 0, None, None)
    for K in (131056, 131072, 262144, (1 << 31) - 1024):
        assert ws(4, 64, K) == OK and n.value >= 4 * 64 + 16
        assert dx(64, K) == WORKSPACE      # the first refusal of this call is its missing workspace
    assert ws(4, 64, 1 << 31) == dx(64, 1 << 31) == ws(1 << 31, 64, 64) == dx(64, 64, 1 << 31) == SHAPE
    assert ws(4, 65536, 64) == OK and ws(4, 65552, 64) == dx(65552, 64) == SHAPE
    assert so.qlora_i8_linear_fwd(X, S, 4, W, T, 64, 131072, None, None, 0, Y, None, None) == SHAPE


def test_stream_and_norm_in_one_buffer_are_refused(so):
    """H may be X and Y may be X, but not both in one call: one would overwrite
    the other."""
    # a call that gets past its pointers ends at its K, which is too large
    g = lambda x=X, r=V, h=T, y=Y: so.qlora_rmsnorm_fwd(x, r, 0, W, 0, 1e-5, 4, 32769, h, y, None, None, None)
    assert g() == g(h=X) == g(y=X) == g(h=V, y=X) == g(h=None) == SHAPE
    assert g(h=X, y=X) == g(h=T, y=T) == g(h=V, y=V) == INVALID
