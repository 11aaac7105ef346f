"""The RMS norm and the 8-bit integer linear of libqlora, as they are measured.

Each case is one call of one operator:

* ``quantize``     rows of a matrix to int8 codes with one fp32 scale a row
* ``norm``         RMS norm with the residual's addition; bf16 or int8 output
* ``norm_grad``    its gradient (stream, weight)
* ``linear``       int8 x int8 product with token and channel scales and the adapter's term
* ``linear_grad``  the gradient of its input

``run`` computes them by elementary torch operations in fp32 (``own`` false) or
by the library's calls (``own`` true); ``exact`` computes them in float64 from
their definitions.
"""

import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # the merged fp32 weight of the 8B set's down projection, on its way to the 8-bit base
        dict(name="quantize weight 4096x14336", op="quantize", m=4096, k=14336, f32=True, cols=False),
        # activations of a ragged batch ahead of the 7B MLP's down projection
        dict(name="quantize tokens 777x11008", op="quantize", m=777, k=11008, f32=False, cols=False),
        # one decoding step of 8 sequences: the call's latency counts
        dict(name="norm decode 8x4096 int8", op="norm", m=8, k=4096, f32=False, wf32=False, i8=True),
        # a prompt (or training batch) of the 8B set
        dict(name="norm 4096x4096 bf16", op="norm", m=4096, k=4096, f32=False, wf32=False, i8=False),
        # residual stream and norm weights upcast to fp32, an odd width, int8 output
        dict(name="norm 1001x5127 f32 int8", op="norm", m=1001, k=5127, f32=True, wf32=True, i8=True),
        # backward of the training batch above
        dict(name="norm grad 4096x4096", op="norm_grad", m=4096, k=4096, f32=False, wf32=False),
        # fp32 stream, the 7B MLP's width, a ragged batch
        dict(name="norm grad 515x11008 f32", op="norm_grad", m=515, k=11008, f32=True, wf32=True),
        # serving the merged weight: one token through an attention projection
        dict(name="linear 1 token 4096x4096", op="linear", m=1, n=4096, k=4096, r=0),
        # a chunk of a prompt through the 7B MLP's up projection, with an adapter
        dict(name="linear 200 tokens 11008x4096", op="linear", m=200, n=11008, k=4096, r=16),
        # a training batch through the 8B set's gate projection
        dict(name="linear 4096 tokens 14336x4096", op="linear", m=4096, n=14336, k=4096, r=16),
        # its gradient through the 7B MLP's gate projection
        dict(name="linear grad 4096 tokens 11008x4096", op="linear_grad", m=4096, n=11008, k=4096, r=16),
        # a short ragged batch through a small odd layer
        dict(name="linear grad 301 tokens 1040x2064", op="linear_grad", m=301, n=1040, k=2064, r=8),
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` between lo and hi, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(v) // step * step)


def draw(rng):
    op = rng.choice(("quantize", "norm", "norm_grad", "linear", "linear_grad"))
    c = dict(op=op, m=_log(rng, 1, 8192))
    if op in ("linear", "linear_grad"):
        c["m"] = min(c["m"], 4096)
        n, k = _log(rng, 64, 14336, 16), _log(rng, 64, 14336, 16)
        while c["m"] * n * k > 4096 * 11008 * 4096:
            n, k = max(64, n // 32 * 16), max(64, k // 32 * 16)
        return dict(c, n=n, k=k, r=rng.choice((0, 8, 16, 24, 32, 64)))
    c["k"] = _log(rng, 16, 16384)
    c["m"] = min(c["m"], 4096 * 4096 // c["k"])
    if op == "quantize":
        return dict(c, f32=rng.random() < 0.5, cols=rng.random() < 0.5)
    c.update(f32=rng.random() < 0.5, wf32=rng.random() < 0.5)
    return dict(c, i8=rng.random() < 0.5) if op == "norm" else c


# ---- inputs -------------------------------------------------------------------


def _rows_i8(v):
    """Codes and scales of the rows of v, by the library's definition."""
    c = v.float().abs().amax(1)
    s = c / 127.0
    safe = torch.where(s > 0, s, torch.ones_like(s))
    return (v.float() / safe[:, None]).round().clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, m, k = case["op"], case["m"], case["k"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def stream(dtype):
        # hidden states: unit variance with some louder channels
        x = torch.randn(m, k, generator=g, device="cuda")
        loud = torch.rand(k, generator=g, device="cuda") < 1 / 512
        return (x * torch.where(loud, 6.0, 1.0)).to(dtype)

    st = dict(case)
    if op == "quantize":
        st["x"] = normal(m, k, std=0.02) if case["f32"] else stream(torch.bfloat16)
        st["cols"] = torch.rand(k, generator=g, device="cuda") * 1e-3 + 1e-4 if case["cols"] else None
    elif op in ("norm", "norm_grad"):
        ht = torch.float32 if case["f32"] else torch.bfloat16
        st["w"] = (1 + 0.1 * torch.randn(k, generator=g, device="cuda")).to(
            torch.float32 if case["wf32"] else torch.bfloat16)
        if op == "norm":
            st["x"], st["res"] = normal(m, k, std=0.3, dtype=torch.bfloat16), stream(ht)
        else:
            st["h"], st["dy"], st["dres"] = stream(ht), normal(m, k, dtype=torch.bfloat16), normal(m, k, dtype=ht)
    else:
        n, r = case["n"], case["r"]
        st["wq"], st["ws"] = _rows_i8(normal(n, k, std=0.02))
        if op == "linear":
            st["xq"], st["xs"] = _rows_i8(stream(torch.float32))
            st["u"] = normal(m, r, std=2.0, dtype=torch.bfloat16) if r else None
            st["b"] = normal(n, r, std=0.01, dtype=torch.bfloat16) if r else None
        else:
            st["dy"] = normal(m, n, dtype=torch.bfloat16)
            st["t"] = normal(m, r, std=0.1, dtype=torch.bfloat16) if r else None
            st["a"] = normal(r, k, std=1.0 / r, dtype=torch.bfloat16) if r else None
    # the outputs, which a user's program allocates once
    if op == "quantize":
        st["codes"], st["scale"] = _empty(torch.int8, m, k), _empty(torch.float32, m)
    elif op == "norm":
        st["H"], st["Y"] = torch.empty_like(st["res"]), _empty(torch.bfloat16, m, k)
        st["codes"], st["scale"] = _empty(torch.int8, m, k), _empty(torch.float32, m)
    elif op == "norm_grad":
        st["dH"], st["dW"] = torch.empty_like(st["h"]), _empty(torch.float32, k)
        st["dX"] = _empty(torch.bfloat16, m, k) if case["f32"] else None
    else:
        st["Y"] = _empty(torch.bfloat16, m, case["n"] if op == "linear" else k)
    return st


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


# ---- one pass -----------------------------------------------------------------


def run(st):
    if own:
        return _own(st)
    op = st["op"]
    if op == "quantize":
        v = st["x"].float()
        if st["cols"] is not None:
            v = v * st["cols"]
        codes, scale = _rows_i8(v)
        return dict(codes=codes, scale=scale)
    if op == "norm":
        h = (st["x"].float() + st["res"].float()).to(st["res"].dtype)
        f = h.float()
        y = f * (1.0 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)) * st["w"].float()
        if not st["i8"]:
            return dict(h=h, y=y.to(torch.bfloat16))
        codes, scale = _rows_i8(y)
        return dict(h=h, y=(codes.float() * scale[:, None]).to(torch.bfloat16), scale=scale)
    if op == "norm_grad":
        f, dy, w = st["h"].float(), st["dy"].float(), st["w"].float()
        rstd = 1.0 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)
        xhat, wdy = f * rstd, dy * w
        d = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True)) + st["dres"].float()
        out = dict(dh=d.to(st["h"].dtype), dw=(dy * xhat).sum(0))
        if st["f32"]:
            out["dx"] = d.to(torch.bfloat16)
        return out
    w = st["wq"].float()
    if op == "linear":
        y = (st["xq"].float() @ w.t()) * st["xs"][:, None] * st["ws"]
        if st["r"]:
            y = y + st["u"].float() @ st["b"].float().t()
        return dict(y=y.to(torch.bfloat16))
    codes, scale = _rows_i8(st["dy"].float() * st["ws"])
    d = (codes.float() @ w) * scale[:, None]
    if st["r"]:
        d = d + st["t"].float() @ st["a"].float()
    return dict(dx=d.to(torch.bfloat16))


def _own(st):
    import bit_nf4_quantized_dequant_b200 as q

    op = st["op"]
    if op == "quantize":
        out = q.i8_quantize(st["x"], st["cols"], out=q.I8Matrix(st["codes"], st["scale"]))
        return dict(codes=out.codes, scale=out.scale)
    if op == "norm":
        if not st["i8"]:
            y, h, _ = q.rmsnorm_fwd(st["x"], st["w"], EPS, residual=st["res"], H=st["H"], Y=st["Y"])
            return dict(h=h, y=y)
        _, h, codes = q.rmsnorm_fwd(st["x"], st["w"], EPS, residual=st["res"], H=st["H"],
                                    q=q.I8Matrix(st["codes"], st["scale"]))
        return dict(h=h, y=q.i8_dequantize(codes, out=st["Y"]), scale=codes.scale)
    if op == "norm_grad":
        dh, dx, dw = q.rmsnorm_bwd(st["dy"], st["h"], st["w"], EPS, dres=st["dres"], dH=st["dH"], dX=st["dX"],
                                   dW=st["dW"])
        return dict(dh=dh, dw=dw, dx=dx) if st["f32"] else dict(dh=dh, dw=dw)
    w = q.I8Matrix(st["wq"], st["ws"])
    if op == "linear":
        return dict(y=q.i8_linear_fwd(w, q.I8Matrix(st["xq"], st["xs"]), sU=st["u"], B=st["b"], Y=st["Y"]))
    return dict(dx=q.i8_linear_dx(w, st["dy"], sT=st["t"], A=st["a"], dX=st["Y"]))


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        e = 4 if case["f32"] else 2
        return dict(bytes=m * k * (e + 1) + 4 * m + (4 * k if case["cols"] else 0), flops=3 * m * k)
    if op in ("norm", "norm_grad"):
        e, we = (4 if case["f32"] else 2), (4 if case["wf32"] else 2)
        if op == "norm":
            # x, residual, h, and the values: bf16, or codes and scales
            out = m * k + 4 * m if case["i8"] else 2 * m * k
            return dict(bytes=m * k * (2 + 2 * e) + out + we * k, flops=6 * m * k)
        copy = 2 if case["f32"] else 0
        return dict(bytes=m * k * (2 + 3 * e + copy) + (we + 4) * k, flops=12 * m * k)
    n, r = case["n"], case["r"]
    if op == "linear":
        return dict(bytes=m * k + n * k + 4 * (m + n) + 2 * r * (m + n) + 2 * m * n, flops=2 * m * n * (k + r))
    return dict(bytes=2 * m * n + n * k + 4 * n + 2 * r * (m + k) + 2 * m * k, flops=2 * m * k * (n + r))


# ---- the definitions in 64 bits -------------------------------------------------


def _rows64(v):
    """Codes (as float64) and scales of the rows of a float64 matrix."""
    s = torch.max(torch.abs(v), dim=1).values / 127
    q = torch.zeros_like(v)
    some = s > 0
    q[some] = torch.clamp(torch.round(v[some] / s[some].unsqueeze(1)), -127, 127)
    return q, s


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    d = {name: t.double() for name, t in st.items() if torch.is_tensor(t)}
    if op == "quantize":
        v = d["x"] * d["cols"] if "cols" in d else d["x"]
        return dict(codes=None, scale=_rows64(v)[1])
    if op == "norm":
        h = torch.add(d["x"], d["res"]).to(st["res"].dtype)  # what is stored, and read by the norm
        h64 = h.double()
        power = torch.einsum("mk,mk->m", h64, h64) / case["k"] + EPS
        y = torch.einsum("mk,k,m->mk", h64, d["w"], power.pow(-0.5))
        if not case["i8"]:
            return dict(h=h64, y=y)
        q, s = _rows64(y)
        return dict(h=h64, y=q * s.unsqueeze(1), scale=s)
    if op == "norm_grad":
        h, a = d["h"], d["dy"] * d["w"]
        rstd = (torch.einsum("mk,mk->m", h, h) / case["k"] + EPS).pow(-0.5)
        along = torch.einsum("mk,mk->m", a, h) * rstd.pow(3) / case["k"]
        dh = a * rstd.unsqueeze(1) - h * along.unsqueeze(1) + d["dres"]
        out = dict(dh=dh, dw=torch.einsum("mk,mk,m->k", d["dy"], h, rstd))
        return dict(out, dx=dh) if case["f32"] else out
    if op == "linear":
        y = torch.einsum("mk,m->mk", d["xq"], d["xs"]) @ torch.einsum("nk,n->kn", d["wq"], d["ws"])
        return dict(y=y + d["u"] @ d["b"].mT if case["r"] else y)
    q, s = _rows64(d["dy"] * d["ws"])
    dx = (q * s.unsqueeze(1)) @ d["wq"]
    return dict(dx=dx + d["t"] @ d["a"] if case["r"] else dx)
