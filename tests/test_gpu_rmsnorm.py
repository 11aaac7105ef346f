"""GPU parity of the RMS norm (forward: stream, bf16 and int8 outputs; backward:
stream, bf16 copy, weight) against oracle.rmsnorm in float64, element by
element, with bounds from the roundings:

* a row's sum of squares (and of w dy h): a thread adds up to 32 elements, then
  ten shuffle steps: at most 48 roundings of 2^-24, relative to the sum of
  magnitudes; half of that in rstd, plus four roundings of its own;
* y has two more products: 32 * 2^-24 in all covers it; bf16 adds 2^-8 of the value.
"""

import numpy as np
import pytest

from oracle import i8 as oi8, nf4 as onf4, rmsnorm as orms

pytestmark = pytest.mark.gpu

EPS = 1e-5
U32, U16 = 2.0 ** -24, 2.0 ** -8
SUM, Y32 = 48 * U32, 32 * U32

# K: one element, below a warp, odd, the warp kernels' last widths and the next
# ones, block widths, the widest; M: one row, ragged blocks of rows, more rows
# than resident blocks
SHAPES = [(1, 1), (3, 7), (5, 16), (2, 31), (129, 64), (7, 129), (301, 256), (300, 264), (5, 512), (3, 1000), (2, 1024),
          (1, 4096), (301, 4096), (9, 4104), (4, 5127), (700, 2056), (2, 8191), (3, 8192), (2, 8200), (2, 11008),
          (2, 16384), (1, 16392), (2, 32761), (2, 32768), (700, 1001), (2500, 63), (320, 5127), (310, 11001),
          (1300, 517), (600, 2), (300, 16390), (16, 4096), (16, 4095), (17, 1000), (11, 5953), (16, 130), (13, 127)]


def _dt(torch, f32):
    return torch.float32 if f32 else torch.bfloat16


def _inputs(torch, M, K, hf, wf, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (0.5 * r(M, K)).bfloat16()
    res = r(M, K).to(_dt(torch, hf))
    w = (1 + 0.1 * r(K)).to(_dt(torch, wf))
    return x, res, w, r(M, K).bfloat16(), r(M, K).to(_dt(torch, hf))


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check_bf16(got, ref, rel, what):
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= (U16 + rel) * np.abs(ref) + 1e-38), (what, (err / (np.abs(ref) + 1e-30)).max())


@pytest.mark.parametrize("hf,wf", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(lib, M, K, hf, wf):
    import torch
    x, res, w, _, _ = _inputs(torch, M, K, hf, wf, M * 40000 + K)
    h = (x.float() + res.float()).to(res.dtype)
    q = lib.I8Matrix.empty(M, K)
    Y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    Y, H, q = lib.rmsnorm_fwd(x.cuda(), w.cuda(), EPS, residual=res.cuda(), Y=Y, q=q)
    torch.cuda.synchronize()
    assert torch.equal(H.cpu(), h)
    y = orms.fwd(_f64(h), _f64(w), EPS)
    _check_bf16(Y, y, Y32, "Y")
    s = q.scale.cpu().numpy()
    c = np.abs(y).max(axis=1)
    assert np.all(np.abs(s - c / 127) <= (Y32 + 2 * U32) * c / 127)
    # half a step from the exact y, up to the roundings of y, the scale and the quotient
    codes = q.codes.cpu().numpy().astype(np.float64)
    assert np.abs(codes).max(axis=1).min() == 127
    step = s[:, None].astype(np.float64)
    assert np.all(np.abs(codes * step - y) <= 0.5 * step + (Y32 + 3 * U32) * 127.5 * step)


def test_codes_alone_and_each_input_alone(lib):
    """The codes do not depend on what else is asked for; with one of X and the
    residual missing, h is the other."""
    import torch
    M, K = 37, 1032
    x, res, w, _, _ = _inputs(torch, M, K, False, True, 3)
    x, res, w = x.cuda(), res.cuda(), w.cuda()
    Y, H, _ = lib.rmsnorm_fwd(x, w, EPS, residual=res)
    both = lib.I8Matrix.empty(M, K)
    Y2, H2, _ = lib.rmsnorm_fwd(x, w, EPS, residual=res, Y=torch.empty_like(x), q=both)
    only = lib.I8Matrix.empty(M, K)
    none, H3, _ = lib.rmsnorm_fwd(x, w, EPS, residual=res, q=only)
    assert none is None and torch.equal(Y, Y2) and torch.equal(H, H2) and torch.equal(H, H3)
    assert torch.equal(both.codes, only.codes) and torch.equal(both.scale, only.scale)
    Ya, Ha, _ = lib.rmsnorm_fwd(H, w, EPS)
    Yb, Hb, _ = lib.rmsnorm_fwd(None, w, EPS, residual=H)
    assert Ha is None and Hb is None and torch.equal(Ya, Y) and torch.equal(Yb, Y)
    Yc, Hc, _ = lib.rmsnorm_fwd(None, w, EPS, residual=H.float())
    assert Hc is None and torch.equal(Yc, Y)
    Yd, Hd, _ = lib.rmsnorm_fwd(x, w, EPS, residual=res, want_H=False)
    assert Hd is None and torch.equal(Yd, Y)


@pytest.mark.parametrize("K", [64, 520, 4096, 5127, 16392])
def test_outputs_in_place(lib, K):
    import torch
    M = 5
    x, res, w, dy, dr = (t.cuda() for t in _inputs(torch, M, K, False, False, K))
    Y, H, _ = lib.rmsnorm_fwd(x, w, EPS, residual=res)
    x1, r1 = x.clone(), res.clone()
    Y1, H1, _ = lib.rmsnorm_fwd(x1, w, EPS, residual=r1, H=r1, Y=x1)
    assert torch.equal(x1, Y) and torch.equal(r1, H)
    x1 = x.clone()
    lib.rmsnorm_fwd(x1, w, EPS, residual=res, H=x1)
    assert torch.equal(x1, H)
    dH, _, dW = lib.rmsnorm_bwd(dy, H, w, EPS, dres=dr)
    for alias in ("dres", "dY"):
        a, b = dy.clone(), dr.clone()
        out, _, dW1 = lib.rmsnorm_bwd(a, H, w, EPS, dres=b, dH=b if alias == "dres" else a)
        assert torch.equal(out, dH) and torch.equal(dW1, dW)
    h32, r32, a = H.float(), dr.float(), dy.clone()
    want, wantX, _ = lib.rmsnorm_bwd(dy, h32, w, EPS, dres=r32, dX=torch.empty_like(dy))
    out, outX, _ = lib.rmsnorm_bwd(a, h32, w, EPS, dres=r32, dH=r32, dX=a)
    assert torch.equal(out, want) and torch.equal(outX, wantX)


@pytest.mark.parametrize("hf,wf", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("M,K", SHAPES)
def test_backward(lib, M, K, hf, wf):
    import torch
    _, h, w, dy, dr = _inputs(torch, M, K, hf, wf, M * 50000 + K)
    for with_dr in (True, False):
        dX = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        dH, dX, dW = lib.rmsnorm_bwd(dy.cuda(), h.cuda(), w.cuda(), EPS, dres=dr.cuda() if with_dr else None, dX=dX)
        torch.cuda.synchronize()
        H, W, D = _f64(h), _f64(w), _f64(dy)
        dh, dw = orms.bwd(D, H, W, EPS, _f64(dr) if with_dr else None)
        rs = orms.rstd(H, EPS)
        g = W * D
        along = rs * rs * np.abs(g * H).mean(axis=1, keepdims=True)
        # rstd, the sum w dy h and four products and sums, on the magnitudes of both terms; the residual's addition
        tol = (SUM + 8 * U32) * 2 * rs * (np.abs(g) + np.abs(H) * along) + 2 * U32 * np.abs(dh)
        err = np.abs(_f64(dH) - dh)
        assert np.all(err <= tol + (0 if hf else U16 * (np.abs(dh) + tol)) + 1e-38), (err / (tol + 1e-38)).max()
        err = np.abs(_f64(dX) - dh)
        assert np.all(err <= tol + U16 * (np.abs(dh) + tol) + 1e-38)
        if not hf:
            assert torch.equal(dH, dX)
        # dw: rows of a block one after the other, then the blocks' partials, and rstd's and two products' roundings
        tol = (M + 40 + 32) * U32 * np.abs(D * H * rs).sum(axis=0)
        assert np.all(np.abs(_f64(dW) - dw) <= tol + 1e-38)


def test_frozen_weight_and_bf16_copy_alone(lib):
    import torch
    M, K = 33, 2048
    _, h, w, dy, dr = (t.cuda() for t in _inputs(torch, M, K, True, True, 11))
    dH, dX, dW = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr, dX=torch.empty_like(dy))
    a, none, no_w = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr, want_dW=False)
    assert none is None and no_w is None and torch.equal(a, dH)
    # the C call without dH, as a first block's norm has no stream below it to go on to
    so = __import__("bit_nf4_quantized_dequant_b200")._norm_i8._library()
    only = torch.empty_like(dy)
    assert so.qlora_rmsnorm_bwd(dy.data_ptr(), h.data_ptr(), 1, w.data_ptr(), 1, EPS, dr.data_ptr(), M, K, None,
                                only.data_ptr(), None, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(only, dX)


def test_rows_that_are_zero_or_not_finite(lib):
    """A zero row gives zeros (scale 0, codes 0); a NaN or an infinity stays in
    its own row."""
    import torch
    M, K = 6, 264
    h = torch.randn(M, K, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    w = torch.ones(K, device="cuda")
    clean = lib.rmsnorm_fwd(h, w, EPS)[0]
    h[1] = 0
    h[2, 7] = float("nan")
    h[3, 260] = float("inf")
    q = lib.I8Matrix.empty(M, K)
    Y, _, _ = lib.rmsnorm_fwd(h, w, EPS, Y=torch.empty_like(h), q=q)
    assert torch.equal(Y[[0, 4, 5]], clean[[0, 4, 5]])
    assert not Y[1].any() and not q.codes[1].any() and q.scale[1] == 0
    assert Y[2].isnan().all() and q.scale[2].isnan() and not q.codes[2].any()
    assert Y[3, 260].isnan() and q.scale[3].isnan() and not q.codes[3].any()   # inf * 0
    dy = torch.ones_like(h)
    dH, _, _ = lib.rmsnorm_bwd(dy, h, w, EPS)
    assert dH[[0, 1, 4, 5]].isfinite().all() and dH[2].isnan().all()
    z = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
    Y, _, _ = lib.rmsnorm_fwd(z, w, 0.0)       # eps 0 and a zero row: 0 * inf
    assert Y.isnan().all()


def test_tiny_and_huge_rows(lib):
    """Rows whose int8 scale is subnormal or near it, and near fp32's top: the
    codes still reach +-127 and stay within their half step."""
    import torch
    K = 512
    h = torch.randn(5, K, generator=torch.Generator().manual_seed(6)).cuda()
    w = torch.ones(K, device="cuda")
    for scale in (1e-41, 1e-37, 1e-31, 1e-30, 1e30, 1e37):
        q = lib.I8Matrix.empty(5, K)
        lib.rmsnorm_fwd(None, w * scale, EPS, residual=h, q=q)
        y = (lib.rmsnorm_fwd(None, w, EPS, residual=h)[0].float() * 0).double()   # shape only
        y = torch.from_numpy(orms.fwd(_f64(h), _f64(w * scale), EPS)).cuda()
        step = q.scale.double()[:, None]
        err = (q.codes.double() * step - y).abs()
        # fp32 subnormals are 2^-149 apart: y and the scale are rounded to that
        tiny = 127.5 * 2.0 ** -149
        assert (err <= 0.5 * step + 40 * U32 * 127.5 * step + tiny).all(), scale
        assert q.codes.abs().max() == 127


def test_streams_and_graph_replay(lib):
    """The calls on another stream than the tensors' own, and captured with their
    workspace and replayed on new data."""
    import torch
    M, K = 300, 4096
    _, h, w, dy, dr = (t.cuda() for t in _inputs(torch, M, K, False, False, 21))
    Y, _, _ = lib.rmsnorm_fwd(h, w, EPS)
    dH, _, dW = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y1, _, _ = lib.rmsnorm_fwd(h, w, EPS, stream=s)
    dH1, _, dW1 = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(Y, Y1) and torch.equal(dH, dH1) and torch.equal(dW, dW1)
    hs, dys = torch.zeros_like(h), torch.zeros_like(dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Yg, _, _ = lib.rmsnorm_fwd(hs, w, EPS)
        dHg, _, dWg = lib.rmsnorm_bwd(dys, hs, w, EPS, dres=dr)
    for _ in range(2):
        hs.copy_(h)
        dys.copy_(dy)
        g.replay()
        assert torch.equal(Yg, Y) and torch.equal(dHg, dH) and torch.equal(dWg, dW)
        hs.zero_()
    del g


def test_rows_past_31_bits(lib):
    """Element offsets beyond 2^31: the last rows of a large stream are those of
    a small one."""
    import torch
    K = 8192
    M = (1 << 31) // K + 5
    h = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    tail = torch.randn(7, K, generator=g).bfloat16().cuda()
    h[-7:] = tail
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    Y, _, _ = lib.rmsnorm_fwd(h, w, EPS)
    want, _, _ = lib.rmsnorm_fwd(tail, w, EPS)
    assert torch.equal(Y[-7:], want) and not Y[:-7].any()
    dH, _, dW = lib.rmsnorm_bwd(h, h, w, EPS, dH=Y)
    want, _, _ = lib.rmsnorm_bwd(tail, tail, w, EPS)
    assert torch.equal(dH[-7:], want)
    q = lib.i8_quantize(h)
    want = lib.i8_quantize(tail)
    assert torch.equal(q.codes[-7:], want.codes) and torch.equal(q.scale[-7:], want.scale) and not q.codes[:-7].any()
    lib.i8_dequantize(q, out=Y)
    assert torch.equal(Y[-7:], lib.i8_dequantize(want))
