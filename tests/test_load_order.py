"""Sources of the kernels that are launched before the work ahead of them has
finished: what they read may still be written while they run, so every load has
to stay behind the wait for that work. The compiler keeps that order only where
the source states it; these tests read the sources (no GPU needed)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_nf4_quantized_dequant_b200", "csrc")
EARLY = ["row_device.cuh", "i8_codec.cu", "rmsnorm.cu", "i8_gemm.cuh", "i8_gemm_split.cu", "i8_gemm_pair.cu"]


def _code(name):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _asm_statements(code):
    """(is volatile, text) of every inline asm statement."""
    for m in re.finditer(r"\basm\b\s*(volatile)?\s*\(", code):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = code[i]
            if c == '"' and code[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield m.group(1) is not None, code[m.end():i - 1]


def test_the_list_names_every_early_kernel():
    """A file that launches its kernels early is in EARLY (norm_i8.h declares the launch)."""
    users = {f for f in os.listdir(CSRC) if f.endswith(".cu") and "launch_dependent(" in _code(f)}
    assert users and users <= set(EARLY)


@pytest.mark.parametrize("name", EARLY + ["qlora_device.cuh"])
def test_inline_loads_from_memory_state_their_order(name):
    """An asm load that is neither volatile nor clobbers memory is a function of
    its operands to the compiler, free to move ahead of the wait unless the
    wait's result is one of them."""
    for volatile, text in _asm_statements(_code(name)):
        if re.search(r'"[^"]*\b(ld|cp)\.', text):
            ordered = volatile and re.search(r':\s*"memory"\s*$', text.strip())
            assert ordered or '"r"(w.order)' in text, text


@pytest.mark.parametrize("name", EARLY)
def test_no_load_by_the_read_only_path(name):
    """That path is for memory that nothing writes while the kernel runs: the
    launch ahead may still be writing a scale, an activation or a partial sum.
    const __restrict__ lets the compiler take it by itself."""
    code = _code(name)
    assert not re.findall(r"__ldg\s*\([^;]*|ld\.global\.nc[^;]*", code)
    assert not re.findall(r"\bconst\s+\w+\s*\*\s*__restrict__\s*\w+", code)


def test_few_token_forward_reads_only_weights_by_the_read_only_path():
    """Its overlap flag promises that the NF4 weights are not written by the work
    ahead; activations and adapters may be."""
    code = _code("nf4_small_m.cu")
    assert "grid_dep_wait" in code
    reads = re.findall(r"__ldg\s*\(([^;]*?)\)", code)
    assert reads and all(re.match(r"q\.(scale8|scale2|codes)\b", r) for r in reads), reads
