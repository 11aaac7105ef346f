"""The RMS norm and the 8-bit linear at the edges of what their header allows."""

import numpy as np
import pytest

from oracle import i8 as oi8

pytestmark = pytest.mark.gpu

EPS = 1e-5
U32, U16 = 2.0 ** -24, 2.0 ** -8


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("M,N,r", [(3, 48, 0), (140, 16, 16), (300, 48, 40)])
def test_gradient_wider_than_the_longest_contraction(lib, M, N, r):
    """K = 131088 features: the gradient sums over N alone. Off by three fp32
    roundings of the scaled sum, r + 1 of the adapter's on the magnitudes, and bf16's."""
    import torch
    K = 131072 + 16
    g = np.random.default_rng(M)
    wq = g.integers(-127, 128, (N, K), dtype=np.int8)
    sw = (0.5 + g.random(N)).astype(np.float32) * 1e-3
    bf = lambda s, *shape: torch.from_numpy((g.standard_normal(shape) * s).astype(np.float32)).bfloat16()
    dy, t, a = bf(1.0, M, N), bf(0.1, M, r), bf(0.05, r, K)
    W = lib.I8Matrix(torch.from_numpy(wq).cuda(), torch.from_numpy(sw).cuda())
    args = dict(sT=t.cuda(), A=a.cuda()) if r else {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dX = lib.i8_linear_dx(W, dy.cuda(), status=status, **args)
    main = oi8.linear_dx(dy.float().numpy(), wq, sw)
    term, mag = (_f64(t) @ _f64(a), np.abs(_f64(t)) @ np.abs(_f64(a))) if r else (0.0, 0.0)
    ref, tol = main + term, (r + 5) * U32 * (np.abs(main) + mag)
    assert status.item() == 0
    assert np.all(np.abs(_f64(dX) - ref) <= tol + U16 * (np.abs(ref) + tol) + 1e-38)


@pytest.mark.parametrize("M,N,K,r", [(256, 128, 4112, 24), (200, 256, 4096, 64), (300, 272, 2064, 40), (129, 400, 1552, 48),
                                     (513, 128, 8208, 32), (260, 1040, 1040, 56)])
def test_wide_adapters_on_deep_narrow_layers(lib, M, N, K, r):
    """Ranks past 16 with few tiles and a long contraction, in both directions:
    the bound is the one of the test above."""
    import torch
    g = np.random.default_rng(M + N + K)
    bf = lambda s, *shape: torch.from_numpy((g.standard_normal(shape) * s).astype(np.float32)).bfloat16()
    wq, xq = g.integers(-127, 128, (N, K), dtype=np.int8), g.integers(-127, 128, (M, K), dtype=np.int8)
    sw, sx = ((0.5 + g.random(n)).astype(np.float32) * 1e-3 for n in (N, M))
    dy, u, b, t, a = bf(1.0, M, N), bf(1.0, M, r), bf(0.1, N, r), bf(0.1, M, r), bf(0.05, r, K)
    W, X = (lib.I8Matrix(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for c, s in ((wq, sw), (xq, sx)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = lib.i8_linear_fwd(W, X, sU=u.cuda(), B=b.cuda(), status=status)
    dX = lib.i8_linear_dx(W, dy.cuda(), sT=t.cuda(), A=a.cuda(), status=status)
    for got, main, p, q in ((Y, oi8.linear_fwd(xq, sx, wq, sw), _f64(u), _f64(b).T),
                            (dX, oi8.linear_dx(dy.float().numpy(), wq, sw), _f64(t), _f64(a))):
        ref, tol = main + p @ q, (r + 5) * U32 * (np.abs(main) + np.abs(p) @ np.abs(q))
        assert np.all(np.abs(_f64(got) - ref) <= tol + U16 * (np.abs(ref) + tol) + 1e-38)
    assert status.item() == 0


@pytest.mark.parametrize("M,K", [(4, 264), (300, 1001), (40, 2048), (3, 16392)])
def test_bf16_copy_without_the_stream_gradient(lib, M, K):
    """want_dH=False: no dH is allocated or written, the other outputs are the same."""
    import torch
    g = torch.Generator().manual_seed(M)
    dy, h = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(M, K, generator=g).cuda()
    w = (1 + 0.1 * torch.randn(K, generator=g)).cuda()
    _, dX, dW = lib.rmsnorm_bwd(dy, h, w, EPS, dX=torch.empty_like(dy))
    none, dX1, dW1 = lib.rmsnorm_bwd(dy, h, w, EPS, dX=torch.empty_like(dy), want_dH=False)
    assert none is None and torch.equal(dX, dX1) and torch.equal(dW, dW1)
    with pytest.raises(lib.QloraError, match="INVALID_ARG"):
        lib.rmsnorm_bwd(dy, h, w, EPS, want_dH=False)
