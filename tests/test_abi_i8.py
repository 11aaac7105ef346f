"""include/qlora_i8.h: every declared entry point is exported and bound, the
header is plain C, and the argument checks answer before anything is launched
(no GPU needed; a C99 client runs the same checks)."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_i8.h")
P = ctypes.c_void_p
X, W, S, T, Y, V = (P(0x10000 * i) for i in range(1, 7))
ODD = P(0x10008)
INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(qlora_[a-z0-9_]+)\s*\(", text)))


@pytest.fixture(scope="module")
def so(lib):
    from bit_nf4_quantized_dequant_b200 import _norm_i8
    return _norm_i8._library()


def test_every_declared_symbol_is_exported_and_bound(lib, so):
    assert declared() == sorted(lib.SYMBOLS_I8)
    for s in declared():
        assert getattr(so, s).argtypes


def test_codec_refusals(so):
    q = lambda x=X, t=0, m=4, k=64, cs=None, c=Y, s=S: so.qlora_i8_quantize(x, t, m, k, cs, c, s, None)
    assert q(x=None) == q(c=None) == q(s=None) == INVALID
    assert q(t=2) == q(t=-1) == q(m=0) == q(m=-1) == q(k=0) == INVALID
    assert q(k=65537) == q(m=1 << 31) == SHAPE
    assert q(x=ODD) == q(cs=ODD) == q(c=ODD) == q(s=ODD) == MISALIGNED
    d = lambda c=X, s=S, m=4, k=64, o=Y: so.qlora_i8_dequantize(c, s, m, k, o, None)
    assert d(c=None) == d(s=None) == d(o=None) == d(m=0) == d(k=0) == INVALID
    assert d(k=65537) == SHAPE
    assert d(c=ODD) == d(s=ODD) == d(o=ODD) == MISALIGNED


def test_norm_refusals(so):
    nan, inf = float("nan"), float("inf")
    f = lambda x=X, r=V, ht=0, w=W, wt=0, eps=1e-5, m=4, k=64, h=T, y=Y, c=None, s=None: so.qlora_rmsnorm_fwd(
        x, r, ht, w, wt, eps, m, k, h, y, c, s, None)
    assert f(x=None, r=None) == f(w=None) == f(ht=2) == f(wt=-1) == INVALID
    assert f(r=None, ht=1) == INVALID                       # no fp32 stream to take the type from
    assert f(y=None) == f(c=X) == f(s=S) == INVALID         # no output, codes without scales, scales without codes
    assert f(eps=-1e-5) == f(eps=nan) == f(eps=inf) == f(m=0) == f(k=0) == INVALID
    assert f(k=32769) == f(m=1 << 31) == SHAPE
    for name in ("x", "r", "w", "h", "y"):
        assert f(**{name: ODD}) == MISALIGNED
    assert f(c=ODD, s=S) == f(c=X, s=ODD) == MISALIGNED
    n = ctypes.c_size_t()
    assert so.qlora_rmsnorm_workspace(4, 64, None) == INVALID
    assert so.qlora_rmsnorm_workspace(0, 64, ctypes.byref(n)) == INVALID
    assert so.qlora_rmsnorm_workspace(4, 32769, ctypes.byref(n)) == SHAPE
    assert so.qlora_rmsnorm_workspace(4, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert so.qlora_rmsnorm_workspace(40, 64, ctypes.byref(n)) == 0 and n.value > 0
    b = lambda dy=X, h=V, ht=0, w=W, wt=0, eps=1e-5, dr=None, m=40, k=64, dh=T, dx=None, dw=Y, ws=S, nb=n.value: \
        so.qlora_rmsnorm_bwd(dy, h, ht, w, wt, eps, dr, m, k, dh, dx, dw, ws, nb, None)
    assert b(dy=None) == b(h=None) == b(w=None) == b(dh=None) == b(ht=2) == b(wt=2) == b(eps=nan) == INVALID
    assert b(m=0) == b(k=0) == INVALID and b(k=32769) == SHAPE
    for name in ("dy", "h", "w", "dr", "dh", "dx", "dw"):
        assert b(**{name: ODD}) == MISALIGNED
    assert b(ws=None) == b(nb=n.value - 1) == WORKSPACE and b(ws=ODD) == MISALIGNED


def test_linear_refusals(so):
    f = lambda x=X, sx=S, m=4, w=W, sw=T, n=64, k=64, u=None, b=None, r=0, y=Y, st=None: so.qlora_i8_linear_fwd(
        x, sx, m, w, sw, n, k, u, b, r, y, st, None)
    for name in ("x", "sx", "w", "sw", "y"):
        assert f(**{name: None}) == INVALID and f(**{name: ODD}) == MISALIGNED
    assert f(m=0) == f(n=0) == f(k=0) == f(r=16) == f(r=16, u=V) == f(r=16, b=V) == INVALID
    assert f(n=72) == f(k=72) == f(k=131072) == f(m=1 << 31) == f(n=1 << 31) == SHAPE
    assert f(r=12) == f(r=4) == f(r=72) == f(r=-8) == SHAPE
    assert f(r=16, u=ODD, b=V) == f(r=16, u=V, b=ODD) == f(st=P(0x20002)) == MISALIGNED
    n = ctypes.c_size_t()
    ws = lambda *a: so.qlora_i8_linear_workspace(*a, ctypes.byref(n))
    assert so.qlora_i8_linear_workspace(4, 64, 64, None) == ws(0, 64, 64) == INVALID
    assert ws(4, 72, 64) == ws(4, 65552, 64) == SHAPE
    assert ws(4, 64, 64) == 0 and n.value >= 4 * 64 + 16
    d = lambda dy=X, m=4, w=W, sw=T, n=64, k=64, t=None, a=None, r=0, dx=Y, ws=S, nb=n.value, st=None: \
        so.qlora_i8_linear_dx(dy, m, w, sw, n, k, t, a, r, dx, ws, nb, st, None)
    for name in ("dy", "w", "sw", "dx"):
        assert d(**{name: None}) == INVALID and d(**{name: ODD}) == MISALIGNED
    assert d(m=0) == d(r=16) == INVALID and d(n=72) == d(k=72) == d(r=12) == d(n=65552) == SHAPE
    assert d(ws=None) == d(nb=n.value - 1) == WORKSPACE and d(ws=ODD) == MISALIGNED


CLIENT = r"""
#include <stdio.h>
#include "qlora_i8.h"
typedef void (*any_fn)(void);
int main(void) {
  const any_fn entry[] = {%s};
  size_t i, n = 0;
  for (i = 0; i < sizeof(entry) / sizeof(entry[0]); ++i) if (!entry[i]) return 1;
  if (qlora_i8_linear_workspace(4, 64, 64, &n) != QLORA_OK || n < 4 * 64 + 16) return 2;
  if (qlora_rmsnorm_fwd(0, 0, QLORA_TYPE_BF16, 0, QLORA_TYPE_F32, 1e-5f, 1, 1, 0, 0, 0, 0, 0) != QLORA_ERR_INVALID_ARG)
    return 3;
  puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not installed")
def test_header_compiles_as_c99_and_links(lib, tmp_path):
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text(CLIENT % ", ".join(f"(any_fn){s}" for s in declared()))
    res = subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                          os.path.join(ROOT, "include"), str(src), "-o", str(exe), lib.library_path,
                          "-Wl,-rpath," + os.path.dirname(lib.library_path)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", (run.returncode, run.stdout)


def test_binding_refuses_tensors_that_do_not_fit(lib):
    """The binding's own checks come before the library is called: on the CPU
    every call stops at the first tensor's device."""
    import torch
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    q = lib.I8Matrix(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    for call in (lambda: lib.i8_quantize(x), lambda: lib.i8_dequantize(q), lambda: lib.rmsnorm_fwd(x, w, 1e-5),
                 lambda: lib.rmsnorm_bwd(x, x, w, 1e-5), lambda: lib.i8_linear_fwd(q, q),
                 lambda: lib.i8_linear_dx(q, x)):
        with pytest.raises(ValueError, match="expected a CUDA device"):
            call()
    with pytest.raises(ValueError, match="dimensions"):
        lib.i8_quantize(w)
    with pytest.raises(ValueError, match="X or residual"):
        lib.rmsnorm_fwd(None, w, 1e-5)
