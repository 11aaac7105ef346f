"""The RMS norm and the 8-bit linear together with the library's other calls, as
a model uses them: serving the merged weight in 8 bits, training adapters on a
frozen 8-bit base, and the norm around the NF4 linear. Results are compared with
float64, within bounds from the quantisation steps (half a step each) and the
roundings; a captured run replays to the same bits."""

import numpy as np
import pytest

from oracle import i8 as oi8, linear as olin, merge as omerge, nf4 as onf4, rmsnorm as orms
from bit_nf4_quantized_dequant_b200 import inputs

from helpers import assert_close_fp, bf16_dev_to_f64, to_dev_bf16

pytestmark = pytest.mark.gpu

U16, HALF, EPS = 2.0 ** -8, 0.5001, 1e-5


def _f64(t):
    return t.double().cpu().numpy()


def _bits64(b):
    return inputs.bf16_bits_to_f32(b).astype(np.float64)


@pytest.mark.parametrize("M", [1, 8, 300])
def test_serving_the_merged_weight(lib, M):
    """NF4 base + adapter -> merge -> int8 rows; norm -> int8 rows -> product."""
    import torch
    N, K, r, s = 528, 1024, 16, 2.0
    c = inputs.linear_case(N, K, M, r, index=3)
    q = lib.nf4_quantize(torch.from_numpy(c["W"]).cuda())
    W = lib.i8_quantize(lib.nf4_merge(q, to_dev_bf16(c["A"]), to_dev_bf16(c["B"]), s, f32=True))
    x, res = to_dev_bf16(c["X"]), torch.randn(M, K, generator=torch.Generator().manual_seed(M)).cuda()
    w = (1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(9))).cuda()
    X = lib.I8Matrix.empty(M, K)
    _, H, X = lib.rmsnorm_fwd(x, w, EPS, residual=res, q=X)
    Y = lib.i8_linear_fwd(W, X)

    Wd = onf4.dequantize(*onf4.quantize(c["W"]), N, K)
    Wm = omerge.merge(Wd, _bits64(c["A"]), _bits64(c["B"]), s)
    y = orms.fwd(_f64(H), _f64(w), EPS)
    ref = y @ Wm.T
    sx, sw = _f64(X.scale)[:, None], _f64(W.scale)[None, :]
    # an element of y or W' is off by half its row's step
    tol = HALF * sx * np.abs(Wm).sum(1)[None, :] + HALF * sw * np.abs(y).sum(1)[:, None] + K * HALF ** 2 * sx * sw
    err = np.abs(_f64(Y) - ref)
    assert np.all(err <= tol + U16 * (np.abs(ref) + tol))
    # the bound is a worst case; roundings that are independent add up to far less
    assert np.linalg.norm(err) <= 0.02 * np.linalg.norm(ref)


@pytest.mark.parametrize("M", [24, 700])
def test_training_adapters_on_an_8_bit_base(lib, M):
    """Forward and backward of norm + adapted 8-bit linear, against the float64
    gradients of the layer whose weight is the dequantised int8 matrix."""
    import torch
    N, K, r, s = 400, 512, 16, 2.0
    g = torch.Generator().manual_seed(M)
    rn = lambda *sh: torch.randn(*sh, generator=g)
    W = lib.i8_quantize((0.02 * rn(N, K)).cuda())
    A, B = (rn(r, K) / r).bfloat16().cuda(), (0.01 * rn(N, r)).bfloat16().cuda()
    x, res, w = rn(M, K).bfloat16().cuda(), rn(M, K).bfloat16().cuda(), (1 + 0.1 * rn(K)).bfloat16().cuda()
    dY, dres = rn(M, N).bfloat16().cuda(), rn(M, K).bfloat16().cuda()
    ws = torch.zeros(lib.linear_workspace(M, N, K, r), dtype=torch.uint8, device="cuda")

    Xq, X16 = lib.I8Matrix.empty(M, K), torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    X16, H, Xq = lib.rmsnorm_fwd(x, w, EPS, residual=res, Y=X16, q=Xq)
    sU = lib.lora_xa(X16, A, s, torch.empty(M, r, dtype=torch.bfloat16, device="cuda"), ws)
    Y = lib.i8_linear_fwd(W, Xq, sU=sU, B=B)
    sT = lib.lora_dyb(dY, B, s, torch.empty(M, r, dtype=torch.bfloat16, device="cuda"), ws)
    dX = lib.i8_linear_dx(W, dY, sT=sT, A=A)
    dA, dB = torch.empty(r, K, device="cuda"), torch.empty(N, r, device="cuda")
    lib.lora_grads(X16, dY, sU, sT, dA, dB, ws)
    dH, _, dW = lib.rmsnorm_bwd(dX, H, w, EPS, dres=dres)

    Wd = _f64(W.codes) * _f64(W.scale)[:, None]
    y = orms.fwd(_f64(H), _f64(w), EPS)
    term, dterm = _f64(sU) @ _f64(B).T, _f64(sT) @ _f64(A)
    ref = y @ Wd.T + term
    tol = HALF * _f64(Xq.scale)[:, None] * np.abs(Wd).sum(1)[None, :]
    assert np.all(np.abs(_f64(Y) - ref) <= tol + U16 * (np.abs(ref) + tol))
    dref = _f64(dY) @ Wd + dterm
    _, sg = oi8.quantize(dY.float().cpu().numpy(), W.scale.cpu().numpy())
    tol = HALF * sg[:, None] * np.abs(_f64(W.codes)).sum(0)[None, :]
    assert np.all(np.abs(_f64(dX) - dref) <= tol + U16 * (np.abs(dref) + tol))
    assert np.linalg.norm(_f64(dX) - dref) <= 0.02 * np.linalg.norm(dref)
    # the adapter's gradients are those of the layer's bf16 input
    f = [_f64(t) for t in (X16, A, B, dY)]
    _, rA, rB = olin.linear_bwd(Wd, f[0], f[1], f[2], s, f[3])
    assert_close_fp(dA.cpu().numpy(), rA, "dA")
    assert_close_fp(dB.cpu().numpy(), rB, "dB")
    dh, dw = orms.bwd(_f64(dX), _f64(H), _f64(w), EPS, _f64(dres))
    assert_close_fp(bf16_dev_to_f64(dH), dh, "dH")
    assert_close_fp(dW.cpu().numpy(), dw, "dW")


def test_norm_around_the_nf4_linear(lib):
    """Forward and backward of norm + NF4 QLoRA linear with an fp32 stream."""
    import torch
    M, N, K, r, s = 200, 256, 512, 16, 2.0
    c = inputs.linear_case(N, K, M, r, index=5)
    q = lib.nf4_quantize(torch.from_numpy(c["W"]).cuda())
    A, B, dY, x = (to_dev_bf16(c[n]) for n in ("A", "B", "dY", "X"))
    g = torch.Generator().manual_seed(3)
    res, w = torch.randn(M, K, generator=g).cuda(), (1 + 0.1 * torch.randn(K, generator=g)).cuda()
    X16, H, _ = lib.rmsnorm_fwd(x, w, EPS, residual=res)
    Y, sU = lib.linear_fwd(q, X16, A, B, s)
    dX, dA, dB = lib.linear_bwd(q, X16, A, B, s, dY, sU=sU)
    dH, dX16, dW = lib.rmsnorm_bwd(dX, H, w, EPS, dX=torch.empty_like(dX))
    h = _f64(x) + _f64(res)
    assert np.all(np.abs(_f64(H) - h) <= 2.0 ** -24 * np.abs(h))
    Wd = onf4.dequantize(*onf4.quantize(c["W"]), N, K)
    y = orms.fwd(h, _f64(w), EPS)
    ref, _ = olin.linear_fwd(Wd, y, _f64(A), _f64(B), s)
    assert_close_fp(bf16_dev_to_f64(Y), ref, "Y")
    dy, rA, rB = olin.linear_bwd(Wd, y, _f64(A), _f64(B), s, _f64(dY))
    assert_close_fp(dA.cpu().numpy(), rA, "dA")
    assert_close_fp(dB.cpu().numpy(), rB, "dB")
    dh, dw = orms.bwd(dy, h, _f64(w), EPS)
    assert_close_fp(dH.cpu().numpy(), dh, "dH")
    assert torch.equal(dX16, dH.bfloat16())
    assert_close_fp(dW.cpu().numpy(), dw, "dW")


def test_decoding_step_captured_and_replayed(lib):
    """Norm, three 8-bit projections and a grouped NF4 forward in one graph,
    between kernels of another kind that write their inputs: replays on new
    tokens give what the calls give one by one."""
    import torch
    M, K, r, s = 8, 512, 16, 2.0
    g = torch.Generator().manual_seed(8)
    rn = lambda *sh: torch.randn(*sh, generator=g)
    w = torch.ones(K, device="cuda")
    Ws = [lib.i8_quantize((0.02 * rn(n, K)).cuda()) for n in (512, 128, 128)]
    base = lib.nf4_quantize((0.02 * rn(256, 512)).cuda())
    A, B = (rn(r, K) / r).bfloat16().cuda(), (0.01 * rn(256, r)).bfloat16().cuda()
    tok, stream = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, K, device="cuda")
    X = lib.I8Matrix.empty(M, K)
    out = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")

    def step():
        x = tok * 2
        _, h, q = lib.rmsnorm_fwd(x, w, EPS, residual=stream, q=X)
        ys = [lib.i8_linear_fwd(W, q) for W in Ws]
        prob = lib.LinearProblem(base, ys[0], A, B, s, out)
        ws = torch.zeros(lib.linear_fwd_group_workspace([prob], M), dtype=torch.uint8, device="cuda")
        lib.linear_fwd_group([prob], ws=ws, flags=lib.FWD_OVERLAP_PREVIOUS)
        return [h, *ys, out + 0]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        tok.copy_(rn(M, K))
        stream.copy_(rn(M, K))
        graph.replay()
        replayed = [t.clone() for t in got]
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b)
    del graph


def test_calls_on_two_streams_at_once(lib):
    """Independent calls that run at the same time, each with its own workspace,
    and a matrix that is both operands."""
    import torch
    M, N, K = 300, 528, 1040
    g = torch.Generator().manual_seed(12)
    rn = lambda *sh: torch.randn(*sh, generator=g)
    W, dY = lib.i8_quantize((0.02 * rn(N, K)).cuda()), [rn(M, N).bfloat16().cuda() for _ in range(2)]
    h, w = rn(M, K).bfloat16().cuda(), torch.ones(K, device="cuda")
    want = [lib.i8_linear_dx(W, d) for d in dY]
    wantg = lib.rmsnorm_bwd(want[0], h, w, EPS)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for d, s in zip(dY, streams):
            with torch.cuda.stream(s):
                dx = lib.i8_linear_dx(W, d)
                got.append((dx, lib.rmsnorm_bwd(dx, h, w, EPS)))
        torch.cuda.synchronize()
        assert torch.equal(got[0][0], want[0]) and torch.equal(got[1][0], want[1])
        assert torch.equal(got[0][1][0], wantg[0]) and torch.equal(got[0][1][2], wantg[2])
    sq = lib.i8_linear_fwd(W, W)
    ref = oi8.linear_fwd(*(t.cpu().numpy() for t in (W.codes, W.scale, W.codes, W.scale)))
    assert np.all(np.abs(_f64(sq) - ref) <= (U16 + 2.0 ** -21) * np.abs(ref) + 1e-38)


def test_column_scales_off_the_32_byte_grid(lib):
    """Pointers are promised to be 16-byte aligned, no more: fp32 vectors that are
    not 32-byte aligned."""
    import torch
    g = torch.Generator().manual_seed(2)
    M, K = 40, 4096
    room = torch.empty(K + 4, device="cuda")
    off = room[4:]
    assert off.data_ptr() % 32 == 16
    off.copy_(1e-3 + torch.rand(K, generator=g))
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    a, b = lib.i8_quantize(x, off), lib.i8_quantize(x, off.clone())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)
    assert torch.equal(lib.rmsnorm_fwd(x, off, EPS)[0], lib.rmsnorm_fwd(x, off.clone(), EPS)[0])
    for t, u in zip(lib.rmsnorm_bwd(x, x, off, EPS), lib.rmsnorm_bwd(x, x, off.clone(), EPS)):
        assert t is u is None or torch.equal(t, u)
