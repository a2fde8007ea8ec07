"""Checks on the gfx950 code of the fp8b products (spense_fp8b_linear.hip),
built with the flags of the product (host only)."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "sparse_dense_gemm_amd", "csrc", "spense_fp8b_linear.hip")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
BF16, CODES, WIDE = "Li0", "Li1", "Li2"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Name -> assembly lines of each product kernel."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from sparse_dense_gemm_amd.build import EXTRA, FLAGS

    out = tmp_path_factory.mktemp("isa") / "fp8b.s"
    flags = [f for f in FLAGS if f not in ("-fPIC", "-Wall", "-Wno-unused-function")]
    r = subprocess.run([HIPCC, *flags, *EXTRA["spense_fp8b_linear.hip"], "--cuda-device-only", "-S", SRC, "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = out.read_text()
    labels = [(m.start(), m.group(1)) for m in re.finditer(r"^(_Z\w+):", text, re.M)]
    found = {}
    for i, (pos, name) in enumerate(labels):
        m = re.search(r"fp8b_kernelI(\w+?)EEv", name)
        if m:
            end = labels[i + 1][0] if i + 1 < len(labels) else len(text)
            found[m.group(1)] = text[pos:end].splitlines()
    assert len(found) == 23  # five configurations of the bf16 and codes kinds, four of the widened codes; nine of them streamed too
    return found


def test_operands_take_their_instruction(kernels):
    for name, lines in kernels.items():
        text = "\n".join(lines)
        assert ("v_mfma_f32_16x16x128_f8f6f4" in text) == name.startswith(CODES), name
        assert ("v_mfma_f32_16x16x32_bf16" in text) == (not name.startswith(CODES)), name
        assert ("v_cvt_scalef32_pk_bf16_fp8" in text) == (not name.startswith(CODES)), name
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text), name


def test_nothing_spills(kernels):
    for name, lines in kernels.items():
        assert not any("scratch_" in line for line in lines), name


def test_copies_into_lds_have_landed_before_their_barrier(kernels):
    """The copies are assembly that the compiler does not count.  The wait before
    a barrier leaves at most as many loads in flight as were issued after the
    last copy (the counter retires in order), so every copy has landed; and
    every copy has the wait states that a scalar register written by a vector
    instruction needs before it, which cover the one after a write of m0."""
    for name, lines in kernels.items():
        after, wait, barriers = None, None, 0
        for i, line in enumerate(lines):
            t = line.strip()
            if re.match(r"buffer_load_dword\S*\s.*\blds\b", t):
                after = 0
                assert lines[i - 1].strip() == "s_nop 4", name
            elif re.match(r"(global|buffer)_load", t) and after is not None:
                after += 1
            w = re.search(r"s_waitcnt vmcnt\((\d+)\)", t)
            if w:
                wait = (int(w.group(1)), after)
            if t.startswith("s_barrier"):
                barriers += 1
                assert wait is not None, name
                assert wait[1] is None or wait[0] <= wait[1], (name, wait)
        assert barriers >= 2, name
