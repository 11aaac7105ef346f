"""GPU parity of the int8 row codec (bit for bit) and of the 8-bit linear
(forward and input gradient) against oracle.i8.

The integer sum is exact on both sides, so an output is off by: three fp32
roundings of the scaled sum (its conversion and two scales), r + 1 of the
adapter's sum relative to the sum of its magnitudes, and the bf16 rounding."""

import numpy as np
import pytest

from oracle import i8 as oi8, nf4 as onf4

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def _rows(g, M, K):
    return (g.standard_normal((M, K)) * np.exp(g.standard_normal((M, 1)))).astype(np.float32)


CODEC = [(1, 1), (3, 7), (5, 16), (130, 64), (2, 257), (9, 256), (5, 1024), (3, 1032), (1, 4096), (700, 264), (2, 5127),
         (3, 8192), (2, 8191), (1, 8193), (2, 16384), (2, 16392), (1, 32768), (1, 32761), (2, 32776), (1, 65535),
         (1, 65536)]


@pytest.mark.parametrize("cols", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,K", CODEC)
def test_codec_bit_exact(lib, M, K, f32, cols):
    import torch
    g = np.random.default_rng(M * 70000 + K)
    x = torch.from_numpy(_rows(g, M, K)).to(torch.float32 if f32 else torch.bfloat16)
    cs = (np.abs(g.standard_normal(K)) * 1e-3).astype(np.float32) if cols else None
    q = lib.i8_quantize(x.cuda(), None if cs is None else torch.from_numpy(cs).cuda())
    out = lib.i8_dequantize(q)
    codes, scale = oi8.quantize(x.float().numpy(), cs)
    assert np.array_equal(q.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    want = torch.from_numpy(oi8.dequantize_f32(codes, scale)).bfloat16()
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


def _crafted():
    t = np.zeros((9, 264), np.float32)
    t[0, :255] = np.arange(-127, 128)              # every code
    t[1, 0], t[1, 1:254] = 127, np.arange(-126, 127) + 0.5   # every tie
    t[2, 0] = np.nan
    t[3, 5] = -np.inf
    t[4, :2] = 1e-45, -1e-45                       # scale rounds to zero
    t[5, :3] = 1e-42, -7e-43, 3e-44                # subnormal scale
    t[6, :3] = 1.2e-36, 3e-37, -6e-37              # reciprocal of the scale overflows a float's comfort
    t[7, :3] = 3.4e38, -1.7e38, 1e38
    return t                                       # row 8: zeros


def test_codec_on_crafted_rows(lib):
    import torch
    x = _crafted()
    q = lib.i8_quantize(torch.from_numpy(x).cuda())
    codes, scale = oi8.quantize(x)
    np.testing.assert_array_equal(q.scale.cpu().numpy(), scale)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)


def test_codec_near_ties(lib):
    """Values a few units in the last place around every tie of rows whose scale
    is no power of two: the quick rounding and the division agree there."""
    import torch
    rows = []
    for c in (1.0, 0.3, 7.77, 123.456, 1e-20, 3.3e25):
        s = np.float32(np.float32(c) * (np.float32(1) / np.float32(127)))
        tie = (np.arange(-127, 127) + 0.5).astype(np.float32) * s
        for ulps in (-3, -2, -1, 0, 1, 2, 3):
            v = (tie.view(np.int32) + ulps).view(np.float32)
            rows.append(np.concatenate([[np.float32(c)], np.clip(v, -np.float32(c), np.float32(c)), [0]]))
    x = np.stack(rows).astype(np.float32)
    q = lib.i8_quantize(torch.from_numpy(x).cuda())
    codes, _ = oi8.quantize(x)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


# M: one token, both sides of the token tiles' edges, ragged; N, K: the smallest
# layer, one below and above a tile, odd multiples of 16, deep and wide
LINEAR = [
    # M, N, K, r
    (1, 16, 16, 0), (1, 128, 128, 8), (3, 144, 272, 16), (8, 1040, 2064, 24), (15, 112, 4096, 0), (16, 4096, 1024, 16),
    (17, 256, 256, 64), (33, 272, 144, 32), (64, 1024, 1024, 8), (100, 384, 640, 40), (128, 128, 2048, 48),
    (129, 528, 1040, 16), (200, 1008, 512, 56), (255, 256, 384, 0), (256, 256, 256, 16), (257, 272, 400, 8),
    (300, 4112, 80, 16), (513, 640, 768, 64), (700, 1040, 1296, 24), (1025, 384, 528, 16), (2047, 528, 272, 8),
    # enough tiles for the SM pairs, each rank's template; then several tiles a pair
    (2500, 1296, 1552, 0), (2305, 1552, 1296, 16), (3000, 1280, 1280, 8), (2400, 1360, 1424, 32), (2561, 1296, 1296, 40),
    (2400, 1328, 1536, 64), (5000, 2064, 2320, 24), (4999, 2832, 144, 16), (4990, 144, 2576, 48), (13000, 272, 784, 8),
]


def _linear(torch, M, N, K, r, seed):
    g = np.random.default_rng(seed)
    xq, sx = oi8.quantize(_rows(g, M, K))
    wq, sw = oi8.quantize((g.standard_normal((N, K)) * 0.02).astype(np.float32))
    wq[g.integers(N), g.integers(K)] = -128          # any code is allowed
    xq[0, 0] = -128
    bf = lambda s, *shape: torch.from_numpy((g.standard_normal(shape) * s).astype(np.float32)).bfloat16()
    return xq, sx, wq, sw, bf(2.0, M, r), bf(0.05, N, r), bf(1.0, M, N), bf(0.1, M, r), bf(1.0 / max(r, 1), r, K)


def _i8(lib, torch, codes, scale):
    return lib.I8Matrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda())


def _f64(t):
    return t.double().cpu().numpy()


def _check(got, main, u, b, what):
    ref = main if u is None else main + u @ b
    mag = np.abs(main) if u is None else np.abs(main) + np.abs(u) @ np.abs(b)
    r = 0 if u is None else u.shape[1]
    tol = (r + 5) * U32 * mag
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= tol + U16 * (np.abs(ref) + tol) + 1e-38), (what, err.max(), np.abs(ref).max())


@pytest.mark.parametrize("M,N,K,r", LINEAR)
def test_linear_forward(lib, M, N, K, r):
    import torch
    xq, sx, wq, sw, u, b, *_ = _linear(torch, M, N, K, r, M + 3 * N + 7 * K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(sU=u.cuda(), B=b.cuda()) if r else {}
    lib.i8_linear_fwd(_i8(lib, torch, wq, sw), _i8(lib, torch, xq, sx), Y=Y[1:-1], status=status, **args)
    _check(Y[1:-1], oi8.linear_fwd(xq, sx, wq, sw), _f64(u) if r else None, _f64(b).T, "Y")
    assert status.item() == 0 and (Y[0] == 7).all() and (Y[-1] == 7).all()


@pytest.mark.parametrize("M,N,K,r", LINEAR)
def test_linear_input_gradient(lib, M, N, K, r):
    import torch
    _, _, wq, sw, _, _, dy, t, a = _linear(torch, M, N, K, r, M + 5 * N + 11 * K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dX = torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(sT=t.cuda(), A=a.cuda()) if r else {}
    lib.i8_linear_dx(_i8(lib, torch, wq, sw), dy.cuda(), dX=dX[1:-1], status=status, **args)
    _check(dX[1:-1], oi8.linear_dx(dy.float().numpy(), wq, sw), _f64(t) if r else None, _f64(a), "dX")
    assert status.item() == 0 and (dX[0] == 7).all() and (dX[-1] == 7).all()


@pytest.mark.parametrize("M", [1, 20, 300, 1100])
def test_longest_contraction_does_not_overflow(lib, M):
    """K = 131056 codes of -128 on both sides: the largest sum, 2147221504."""
    import torch
    K, N = 131056, 16
    x = lib.I8Matrix(torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"))
    w = lib.I8Matrix(torch.full((N, K), -128, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"))
    Y = lib.i8_linear_fwd(w, x)
    assert (Y == torch.tensor(float(K * 16384)).bfloat16().cuda()).all()


def test_rows_that_are_empty_or_not_finite(lib):
    """A zero row of activations gives the adapter's term alone; a row that is not
    finite gives NaN, and only in its own row."""
    import torch
    M, N, K, r = 5, 144, 256, 8
    g = np.random.default_rng(4)
    x = _rows(g, M, K)
    x[1] = 0
    x[3, 9] = np.nan
    q = lib.i8_quantize(torch.from_numpy(x).cuda())
    w = lib.i8_quantize(torch.from_numpy(_rows(g, N, K)).cuda())
    u = torch.from_numpy(_rows(g, M, r)).bfloat16().cuda()
    b = torch.from_numpy(_rows(g, N, r)).bfloat16().cuda()
    Y = lib.i8_linear_fwd(w, q, sU=u, B=b)
    assert Y[3].isnan().all() and Y[[0, 1, 2, 4]].isfinite().all()
    term = u[1].double() @ b.double().T
    mag = u[1].double().abs() @ b.double().abs().T
    assert ((Y[1].double() - term).abs() <= U16 * term.abs() + (r + 4) * U32 * mag).all()
    dy = torch.from_numpy(_rows(g, M, N)).bfloat16().cuda()
    dy[2] = 0
    dy[4, 0] = float("inf")
    dX = lib.i8_linear_dx(w, dy)
    assert not dX[2].any() and dX[4].isnan().all() and dX[:4].isfinite().all()


def test_results_do_not_depend_on_the_token_count(lib):
    """Without an adapter the same token gives the same row, bit for bit,
    whatever stands beside it (token tiles, splits and kernels differ): the
    integer sum is exact and the scales come in one order."""
    import torch
    N, K = 1296, 1328
    xq, sx, wq, sw, _, _, dy, _, _ = _linear(torch, 3000, N, K, 0, 77)
    w, X, dy = _i8(lib, torch, wq, sw), _i8(lib, torch, xq, sx), dy.cuda()
    full, fullx = lib.i8_linear_fwd(w, X), lib.i8_linear_dx(w, dy)
    for M in (1, 9, 40, 260, 1200):
        one = lib.i8_linear_fwd(w, lib.I8Matrix(X.codes[:M], X.scale[:M]))
        assert torch.equal(one, full[:M]) and torch.equal(lib.i8_linear_dx(w, dy[:M]), fullx[:M]), M


def test_streams_and_graph_replay(lib):
    import torch
    M, N, K, r = 40, 528, 1040, 16
    xq, sx, wq, sw, u, b, dy, t, a = _linear(torch, M, N, K, r, 5)
    w, X = _i8(lib, torch, wq, sw), _i8(lib, torch, xq, sx)
    u, b, dy, t, a = (z.cuda() for z in (u, b, dy, t, a))
    Y, dX = lib.i8_linear_fwd(w, X, sU=u, B=b), lib.i8_linear_dx(w, dy, sT=t, A=a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y1, dX1 = lib.i8_linear_fwd(w, X, sU=u, B=b, stream=s), lib.i8_linear_dx(w, dy, sT=t, A=a, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(Y, Y1) and torch.equal(dX, dX1)
    codes, dys = torch.zeros_like(X.codes), torch.zeros_like(dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Yg = lib.i8_linear_fwd(w, lib.I8Matrix(codes, X.scale), sU=u, B=b)
        dXg = lib.i8_linear_dx(w, dys, sT=t, A=a)
    for _ in range(2):
        codes.copy_(X.codes)
        dys.copy_(dy)
        g.replay()
        assert torch.equal(Yg, Y) and torch.equal(dXg, dX)
        codes.zero_()
    del g


def test_binding_refusals(lib):
    """Tensors that do not fit are refused by name before the library is called."""
    import torch
    c = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    w, x = lib.I8Matrix.empty(64, 32), lib.I8Matrix.empty(4, 32)
    ok = lib.I8Matrix(torch.zeros_like(w.codes), torch.ones_like(w.scale))
    for match, call in (
            ("W.codes: shape", lambda: lib.i8_linear_fwd(lib.I8Matrix.empty(64, 48), x)),
            ("W.scale: shape", lambda: lib.i8_linear_fwd(lib.I8Matrix(w.codes, x.scale), x)),
            ("X.codes: torch.uint8", lambda: lib.i8_linear_fwd(w, lib.I8Matrix(x.codes.view(torch.uint8), x.scale))),
            ("go together", lambda: lib.i8_linear_fwd(w, x, sU=c(4, 8))),
            ("B: shape", lambda: lib.i8_linear_fwd(w, x, sU=c(4, 8), B=c(64, 16))),
            ("Y: shape", lambda: lib.i8_linear_fwd(w, x, Y=c(4, 32))),
            ("status: torch.int64", lambda: lib.i8_linear_fwd(w, x, status=c(1, dtype=torch.int64))),
            ("not contiguous", lambda: lib.i8_quantize(c(32, 4).T)),
            ("X: torch.float16", lambda: lib.i8_quantize(c(4, 32, dtype=torch.float16))),
            ("col_scale: shape", lambda: lib.i8_quantize(c(4, 32), c(4, dtype=torch.float32))),
            ("col_scale: on cpu", lambda: lib.i8_quantize(c(4, 32), torch.zeros(32))),
            ("weight: shape", lambda: lib.rmsnorm_fwd(c(4, 32), c(4), 1e-5)),
            ("X: shape", lambda: lib.rmsnorm_fwd(c(4, 16), c(32), 1e-5, residual=c(4, 32))),
            ("H: torch.bfloat16", lambda: lib.rmsnorm_fwd(c(4, 32), c(32), 1e-5, residual=c(4, 32, dtype=torch.float32),
                                                          H=c(4, 32))),
            ("dres: torch.float32", lambda: lib.rmsnorm_bwd(c(4, 32), c(4, 32), c(32), 1e-5,
                                                            dres=c(4, 32, dtype=torch.float32)))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(lib.QloraError, match="UNSUPPORTED_SHAPE"):
        lib.i8_linear_fwd(w, x, sU=c(4, 12), B=c(64, 12))
    with pytest.raises(lib.QloraError, match="MISALIGNED"):
        lib.i8_linear_fwd(ok, lib.I8Matrix(c(4 * 32 + 8, dtype=torch.int8)[8:].view(4, 32), x.scale))
    with pytest.raises(lib.QloraError, match="WORKSPACE"):
        lib.i8_linear_dx(ok, c(4, 64), ws=c(16, dtype=torch.uint8))
    with pytest.raises(lib.QloraError, match="INVALID_ARG"):
        lib.i8_quantize(c(0, 32))
