"""The norm's gradient in its persistent kernel (outputs over inputs, rows that
are not finite, the same bits as the kernel for a few rows), odd widths beside
rows that are not finite, replays on changing data, and launches that read what
the launch ahead of them writes. Results are compared bit for bit unless said."""

import numpy as np
import pytest

from oracle import rmsnorm as orms

pytestmark = pytest.mark.gpu

EPS = 1e-5
U32 = 2.0 ** -24


def _inputs(torch, M, K, f32, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.float32 if f32 else torch.bfloat16
    h, dr = (torch.randn(M, K, generator=g).to(t).cuda() for _ in range(2))
    return h, torch.randn(M, K, generator=g).bfloat16().cuda(), dr, (1 + 0.1 * torch.randn(K, generator=g)).to(t).cuda()


# more rows than resident blocks, whole and odd widths, one and two vectors a
# thread, and rows past the persistent kernel
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,K", [(17, 264), (3000, 263), (700, 1001), (700, 4096), (320, 5127), (400, 9000), (160, 20001)])
def test_gradient_over_its_inputs(lib, M, K, f32):
    import torch
    h, dy, dr, w = _inputs(torch, M, K, f32, M + K)
    want, wantX, wantW = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr, dX=torch.empty_like(dy))
    b = dr.clone()
    dH, _, dW = lib.rmsnorm_bwd(dy, h, w, EPS, dres=b, dH=b)
    assert torch.equal(dH, want) and torch.equal(dW, wantW)
    for over_dr in (False, True):
        a, b = dy.clone(), dr.clone()
        dH, dX, dW = lib.rmsnorm_bwd(a, h, w, EPS, dres=b, dH=b if over_dr else None, dX=a)
        assert torch.equal(dX, wantX) and torch.equal(dH, want) and torch.equal(dW, wantW)
    if not f32:
        a = dy.clone()
        dH, _, dW = lib.rmsnorm_bwd(a, h, w, EPS, dres=dr, dH=a)
        assert torch.equal(dH, want) and torch.equal(dW, wantW)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("K", [7, 63, 264, 1001, 1025, 4103, 9001, 20001])
def test_rows_beside_rows_that_are_not_finite(lib, K, f32):
    """A NaN or an infinity at a row's ends, where a vector of the next or the last
    row begins or ends off phase: every other row keeps its bits."""
    import torch
    for M in (9, 700):
        h, dy, dr, w = _inputs(torch, M, K, f32, K)
        bad = torch.zeros(M, dtype=torch.bool)
        bad[1::4] = bad[-2] = True
        sick, sick_dy = h.clone(), dy.clone()
        rows = bad.nonzero()[:, 0].tolist()
        for i, m in enumerate(rows):
            value = (float("nan"), float("inf"), -float("inf"))[i % 3]
            sick[m, -1 if i % 2 else 0] = value
            sick_dy[m, 0 if i % 2 else -1] = value
        good = (~bad).cuda()
        bad = bad.cuda()

        def all_of(h, dy):
            q = lib.I8Matrix.empty(M, K)
            Y, _, q = lib.rmsnorm_fwd(None, w, EPS, residual=h, Y=torch.empty_like(dy), q=q)
            dH, dX, _ = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr, dX=torch.empty_like(dy))
            dH1, _, _ = lib.rmsnorm_bwd(dy, h, w, EPS, want_dW=False)
            c = lib.i8_quantize(h)
            d = lib.i8_quantize(dy, w.float())
            return [Y, q.codes, q.scale, dH, dX, dH1, c.codes, c.scale, d.codes, d.scale, lib.i8_dequantize(d)]

        for a, b in zip(all_of(h, dy), all_of(sick, sick_dy)):
            assert torch.equal(a[good], b[good])
        out = all_of(sick, sick_dy)
        for scale, codes in ((out[2], out[1]), (out[7], out[6]), (out[9], out[8])):
            assert scale[bad].isnan().all() and not codes[bad].any()
        assert out[3][bad].isnan().any(dim=1).all() and out[10][bad].isnan().all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (16, 31), (2, 264), (16, 2048), (8, 4096), (7, 4095), (5, 5953), (4, 8192),
                                 (3, 8191)])
def test_a_rows_gradient_does_not_depend_on_the_kernel(lib, M, K, f32):
    """A few short rows with the weight's gradient, without it (the persistent
    kernel), and at the head of a larger batch."""
    import torch
    h, dy, dr, w = _inputs(torch, M + 300, K, f32, M * K)
    full, _, _ = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr)
    few, _, _ = lib.rmsnorm_bwd(dy[:M], h[:M], w, EPS, dres=dr[:M])
    assert lib.rmsnorm_workspace(M, K) == 0 and lib.rmsnorm_workspace(M + 300, K) > 0
    alone, _, _ = lib.rmsnorm_bwd(dy[:M], h[:M], w, EPS, dres=dr[:M], want_dW=False)
    assert torch.equal(few, alone) and torch.equal(few, full[:M])


def test_weight_gradient_of_rows_past_31_bits(lib):
    """Only the last rows of a large stream are not zero: its weight gradient is
    theirs, up to the fp32 sums (a block adds its rows in turn, then the blocks'
    partials: fewer than 72 roundings for seven terms, as zeros add none)."""
    import torch
    K = 8192
    M = (1 << 31) // K + 5
    h = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(7, K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    h[-7:] = tail
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    _, _, dW = lib.rmsnorm_bwd(h, h, w, EPS, dH=torch.empty_like(h))
    t = tail.double().cpu().numpy()
    _, dw = orms.bwd(t, t, np.ones(K), EPS)
    tol = 72 * U32 * np.abs(t * t * orms.rstd(t, EPS)).sum(axis=0)
    assert np.all(np.abs(dW.double().cpu().numpy() - dw) <= tol)


@pytest.mark.parametrize("M,K", [(5, 264), (300, 1001), (300, 4096), (20, 20000)])
def test_norm_replayed_on_changing_data(lib, M, K):
    import torch
    h, dy, dr, w = _inputs(torch, M, K, False, 3)
    g = torch.cuda.CUDAGraph()
    q = lib.I8Matrix.empty(M, K)
    lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr)
    with torch.cuda.graph(g):
        Yg, _, _ = lib.rmsnorm_fwd(h, w, EPS, Y=torch.empty_like(h), q=q)
        dHg, _, dWg = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr)
    for seed in range(3):
        for t in (Yg, dHg, dWg, q.codes, q.scale):
            t.fill_(7)
        for old, new in zip((h, dy, dr, w), _inputs(torch, M, K, False, 10 + seed)):
            old.copy_(new)
        g.replay()
        p = lib.I8Matrix.empty(M, K)
        Y, _, _ = lib.rmsnorm_fwd(h, w, EPS, Y=torch.empty_like(h), q=p)
        dH, _, dW = lib.rmsnorm_bwd(dy, h, w, EPS, dres=dr)
        assert torch.equal(Yg, Y) and torch.equal(q.codes, p.codes) and torch.equal(q.scale, p.scale)
        assert torch.equal(dHg, dH) and torch.equal(dWg, dW)
    del g


@pytest.mark.parametrize("M,N,K,r", [(3, 528, 1040, 16), (300, 528, 1040, 64), (1500, 1040, 528, 8)])
def test_linear_replayed_on_changing_data(lib, M, N, K, r):
    import torch

    def data(seed):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g).cuda()
        X, W = lib.i8_quantize(rn(M, K)), lib.i8_quantize(rn(N, K))
        return [X.codes, X.scale, W.codes, W.scale] + [rn(*s).bfloat16() for s in ((M, r), (N, r), (M, N), (M, r), (r, K))]

    def calls(xc, xs, wc, ws, u, b, dy, t, a):
        W = lib.I8Matrix(wc, ws)
        return lib.i8_linear_fwd(W, lib.I8Matrix(xc, xs), sU=u, B=b), lib.i8_linear_dx(W, dy, sT=t, A=a)

    held = data(0)
    calls(*held)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = calls(*held)
    for seed in range(1, 4):
        for t in out:
            t.fill_(7)
        for old, new in zip(held, data(seed)):
            old.copy_(new)
        g.replay()
        for a, b in zip(out, calls(*held)):
            assert torch.equal(a, b)
    del g


def test_gradients_on_two_streams_at_once(lib):
    import torch
    M, N, K = 300, 528, 1040
    g = torch.Generator().manual_seed(12)
    rn = lambda *sh: torch.randn(*sh, generator=g)
    W, dY = lib.i8_quantize((0.02 * rn(N, K)).cuda()), [rn(M, N).bfloat16().cuda() for _ in range(2)]
    h, w = rn(M, K).bfloat16().cuda(), torch.ones(K, device="cuda")
    want = [lib.rmsnorm_bwd(lib.i8_linear_dx(W, d), h, w, EPS) for d in dY]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for d, s in zip(dY, streams):
            with torch.cuda.stream(s):
                got.append(lib.rmsnorm_bwd(lib.i8_linear_dx(W, d), h, w, EPS))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("M,K", [(4, 512), (64, 1024), (1, 4096), (300, 2048)])
def test_launches_read_what_the_launch_ahead_writes(lib, M, K):
    """Each call takes a weight, column scales, activations or an adapter from the
    one before it; the same calls with a synchronisation after each give the same
    bits, with one set of buffers that every pass overwrites."""
    import torch
    r = 16
    g = torch.Generator().manual_seed(K)
    x, dy = (torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(2))
    wide = torch.randn(K, K, generator=g).cuda()
    W, X, G = lib.I8Matrix.empty(K, K), lib.I8Matrix.empty(M, K), lib.I8Matrix.empty(M, K)
    dH, Y, Z, D = (torch.empty_like(x) for _ in range(4))
    dW, U = torch.empty(K, device="cuda"), lib.I8Matrix.empty(M, r)
    sU, B = torch.empty(M, r, dtype=torch.bfloat16, device="cuda"), torch.randn(K, r, generator=g).bfloat16().cuda()

    def chain(x, dy, after):
        steps = [lambda: lib.rmsnorm_bwd(dy, x, dW0, EPS, dH=dH, dW=dW),                # dW: the next norm's weight
                 lambda: lib.rmsnorm_fwd(x, dW, EPS, residual=dH, want_H=False, q=X),
                 lambda: lib.i8_linear_fwd(W, X, Y=Y),                                  # scales of the launch ahead
                 lambda: lib.i8_quantize(Y, dW, out=G),
                 lambda: lib.i8_quantize(Y[:, :r].contiguous(), out=U),
                 lambda: lib.i8_dequantize(U, out=sU),
                 lambda: lib.i8_linear_fwd(W, G, sU=sU, B=B, Y=Z),                      # its adapter's activations
                 lambda: lib.i8_linear_dx(W, Z, dX=D),
                 lambda: lib.i8_quantize(wide, dW, out=W),                              # the next pass's weight
                 lambda: lib.i8_dequantize(G, out=Y)]
        for s in steps:
            s()
            if after:
                torch.cuda.synchronize()
        return [t.clone() for t in (dH, dW, X.codes, X.scale, G.codes, G.scale, sU, Z, D, W.codes, W.scale, Y)]

    dW0 = torch.ones(K, device="cuda")
    start = lib.i8_quantize(wide)
    data = [(x * (1 + i), dy * (1 - 0.3 * i)) for i in range(6)]
    results = []
    for after in (True, False):
        W.codes.copy_(start.codes)
        W.scale.copy_(start.scale)
        torch.cuda.synchronize()
        results.append([chain(a, b, after) for a, b in data])
    torch.cuda.synchronize()
    for one, two in zip(*results):
        for a, b in zip(one, two):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_captured_fork_and_join(lib):
    """Two branches of a captured graph that meet in one call."""
    import torch
    M, N, K = 40, 400, 528
    g = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()
    x, wide, w = rn(M, K).bfloat16(), rn(N, K), torch.ones(K, device="cuda")
    X, W = lib.I8Matrix.empty(M, K), lib.I8Matrix.empty(N, K)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            lib.i8_quantize(wide, out=W)
        lib.rmsnorm_fwd(x, w, EPS, q=X)
        here.wait_stream(side)
        lib.i8_linear_fwd(W, X, Y=Y)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(rn(M, K))
        wide.copy_(rn(N, K))
        Y.fill_(7)
        graph.replay()
        got = Y.clone()
        want = lib.i8_linear_fwd(lib.i8_quantize(wide), lib.rmsnorm_fwd(x, w, EPS, q=lib.I8Matrix.empty(M, K))[2])
        assert torch.equal(got, want)
    del graph


@pytest.mark.parametrize("M", [1, 8, 16])
def test_few_token_launches_between_8_bit_products(lib, M):
    """Few-token NF4 launches that start early (one workspace for all) in a chain
    with norms and 8-bit products, each reading the one before: eager and replayed,
    the bits of the same calls with a synchronisation after each."""
    import torch
    K, r, s = 512, 16, 2.0
    g = torch.Generator().manual_seed(M)
    rn = lambda *sh: torch.randn(*sh, generator=g).cuda()
    base, W = lib.nf4_quantize(0.04 * rn(K, K)), lib.i8_quantize(0.04 * rn(K, K))
    A, B, w = (rn(r, K) / r).bfloat16(), (0.01 * rn(K, r)).bfloat16(), 1 + 0.1 * rn(K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    bufs = [torch.empty_like(x) for _ in range(8)]
    X, Z = lib.I8Matrix.empty(M, K), lib.I8Matrix.empty(M, K)
    probs = [lib.LinearProblem(base, bufs[i], A, B, s, bufs[i + 1]) for i in (1, 2, 5)]
    ws = torch.zeros(lib.linear_fwd_group_workspace(probs[:1], M), dtype=torch.uint8, device="cuda")

    def nf4(i):
        lib.linear_fwd_group([probs[i]], ws=ws, flags=lib.FWD_OVERLAP_PREVIOUS)

    steps = [lambda: lib.rmsnorm_fwd(x, w, EPS, Y=bufs[0], q=X),
             lambda: lib.i8_linear_fwd(W, X, Y=bufs[1]),
             lambda: nf4(0),
             lambda: nf4(1),
             lambda: lib.rmsnorm_fwd(bufs[3], w, EPS, residual=bufs[0], H=bufs[4], q=Z),
             lambda: lib.i8_linear_fwd(W, Z, Y=bufs[5]),
             lambda: nf4(2),
             lambda: lib.i8_linear_dx(W, bufs[6], dX=bufs[7])]

    def chain(after=False):
        for step in steps:
            step()
            if after:
                torch.cuda.synchronize()

    chain(after=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(20):
        x.copy_(rn(M, K))
        torch.cuda.synchronize()
        chain(after=True)
        want = [b.clone() for b in bufs]
        for run in (chain, graph.replay):
            for b in bufs:
                b.fill_(7)
            for _ in range(3):
                run()
            for a, b in zip(want, bufs):
                assert torch.equal(a, b)
    del graph
