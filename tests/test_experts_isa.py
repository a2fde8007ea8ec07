"""Checks on the gfx950 code of the expert products (spense_experts.hip),
built with the flags of the product (host only)."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "sparse_dense_gemm_amd", "csrc", "spense_experts.hip")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Name -> assembly lines of each product kernel."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from sparse_dense_gemm_amd.build import EXTRA, FLAGS

    out = tmp_path_factory.mktemp("isa") / "experts.s"
    flags = [f for f in FLAGS if f not in ("-fPIC", "-Wall", "-Wno-unused-function")]
    r = subprocess.run([HIPCC, *flags, *EXTRA["spense_experts.hip"], "--cuda-device-only", "-S", SRC, "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = out.read_text()
    labels = [(m.start(), m.group(1)) for m in re.finditer(r"^(_Z\w+):", text, re.M)]
    found = {}
    for i, (pos, name) in enumerate(labels):
        if "experts_kernel" in name:
            end = labels[i + 1][0] if i + 1 < len(labels) else len(text)
            found[re.search(r"experts_kernelI(\w+?)EEv", name).group(1)] = text[pos:end].splitlines()
    assert len(found) == 15  # five configurations, three kinds of operands
    return found


def _regs(tok):
    m = re.match(r"([va])\[(\d+):(\d+)\]", tok)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"([va])(\d+)$", tok)
    return {(m.group(1), int(m.group(2)))} if m else set()


def test_matrix_instructions_do_not_overwrite_their_sources(kernels):
    for name, lines in kernels.items():
        seen = 0
        for line in lines:
            m = re.match(r"\s+(v_mfma_\S+)\s+(.*)", line)
            if m:
                ops = [o.strip() for o in m.group(2).split(";")[0].split(",")]
                seen += 1
                assert not _regs(ops[0]) & (_regs(ops[1]) | _regs(ops[2])), (name, line.strip())
        assert seen, name


def test_operands_take_their_instruction(kernels):
    for name, lines in kernels.items():
        text = "\n".join(lines)
        mx = name.startswith("Lb1ELb1")
        assert ("v_mfma_scale_f32_16x16x128_f8f6f4" in text) == mx, name
        assert ("v_mfma_f32_16x16x32_bf16" in text) == (not mx), name
        assert ("v_cvt_scalef32_pk_bf16_fp4" in text) == name.startswith("Lb1ELb0"), name
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
