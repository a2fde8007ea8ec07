"""Wait states before the copies into LDS in the gfx950 code of the LDS-staged
kernels of the sparse layers (host only; the expert products have a test of
their own).

The copies are assembly, before which the compiler inserts no wait states of its
own: a memory instruction needs five between a vector instruction that writes
one of its scalar registers (a resource word that a lane read brings back) and
itself, and one after a write of m0.
"""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_dense_gemm_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    """gfx950 assembly of the LDS-staged kernels of the sparse layers, built with the flags of the product."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from sparse_dense_gemm_amd.build import EXTRA, FLAGS

    flags = [f for f in FLAGS if f not in ("-fPIC", "-Wall", "-Wno-unused-function")]
    out = tmp_path_factory.mktemp("isa") / "tile.s"
    r = subprocess.run([HIPCC, *flags, *EXTRA["spense_tile.hip"], "--cuda-device-only", "-S",
                        os.path.join(CSRC, "spense_tile.hip"), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


def scalars(operand):
    """Scalar registers that an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else {"m0"} if operand == "m0" else set()


def shortfalls(text):
    """Number of copies, and those with too few wait states after a write of what they read, on any path to them."""
    code, labels, sources = [], {}, {}  # (operation, operands); label -> index; label -> indices of its branches
    for line in text.splitlines():
        t = line.split(";")[0].strip()
        if t.endswith(":") and not t.startswith(";"):
            labels[t[:-1]] = len(code)
        elif t and not t.startswith("."):
            op, _, rest = t.partition(" ")
            operands = [x for y in rest.split(",") for x in y.split()]
            if op.startswith(("s_cbranch", "s_branch")):
                sources.setdefault(operands[0], []).append(len(code))
            code.append((op, operands, t))
    entered = {}  # index -> indices of the branches to it
    for name, at in labels.items():
        entered.setdefault(at, []).extend(sources.get(name, []))

    def short(i, reads, passed):
        """Whether an instruction before i, `passed` wait states ago, is too close."""
        before = list(entered.get(i, []))
        if i and code[i - 1][0] not in ("s_branch", "s_endpgm"):
            before.append(i - 1)
        for j in before:
            op, operands, _ = code[j]
            first = scalars(operands[0]) if operands else set()
            if (op.startswith("v_") and first & reads) or ("m0" in first and passed < 1):
                return True
            states = passed + (int(operands[0], 0) + 1 if op == "s_nop" else 1)
            if states < 5 and short(j, reads, states):
                return True
        return False

    copies = [i for i, (op, operands, _) in enumerate(code) if op.startswith("buffer_load") and operands[-1] == "lds"]
    return len(copies), [code[i][2] for i in copies if short(i, set().union(*map(scalars, code[i][1])), 0)]


def test_the_scan_finds_what_it_looks_for():
    lane, copy = "v_readlane_b32 s5, v1, 3", "buffer_load_dwordx4 v0, s[4:7], s8 offen lds"
    for between, n in (("", 1), ("s_nop 3", 1), ("s_nop 4", 0), ("v_add_u32 v2, v3, v4\n" * 4, 1),
                       ("v_add_u32 v2, v3, v4\n" * 5, 0)):
        assert len(shortfalls(f"{lane}\n{between}\n{copy}")[1]) == n, between
    assert len(shortfalls(f"s_mov_b32 m0, s3\n{copy}")[1]) == 1
    assert not shortfalls(f"s_mov_b32 m0, s3\ns_nop 0\n{copy}")[1]
    assert not shortfalls(f"v_readlane_b32 s9, v1, 3\n{copy}")[1]
    loop = "loop:\n{0}{1}\nv_readlane_b32 s5, v1, 3\n{2}s_cbranch_scc1 loop"  # round the end of a loop
    assert len(shortfalls(loop.format("", copy, ""))[1]) == 1
    assert len(shortfalls(loop.format("s_nop 2\n", copy, ""))[1]) == 1
    assert not shortfalls(loop.format("s_nop 3\n", copy, ""))[1]
    assert not shortfalls(loop.format("s_nop 1\n", copy, "s_nop 1\n"))[1]


def test_copies_have_their_wait_states(listing):
    copies, short = shortfalls(listing)
    assert copies > 100 and not short, (copies, short[:3])
