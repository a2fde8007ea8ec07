"""Workspaces of a handle, looked at on the host: the library's host code with a
runtime that only hands out addresses."""

import ctypes

import pytest

import host_library as hl
import sparse_dense_gemm_amd as sdg

P = 1 << 20      # a 16-byte aligned address that nothing dereferences
STREAM = 1 << 12
N, K = 64, 8192  # few row tiles, many columns: small calls split K and need partial sums and counters


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return hl.load(tmp_path_factory.mktemp("host"))


def sparse_layer(lib):
    h = ctypes.c_void_p()
    assert lib.spense_pack(P, sdg.DT_FP8, N, K, K, P, None, 0, 0.25, None, ctypes.byref(h)) == 0
    return h


def mx4_layer(lib):
    h = ctypes.c_void_p()
    assert lib.spense_pack_mx4(P, K // 2, P, K // 32, N, K, None, ctypes.byref(h)) == 0
    return h


def experts(lib):
    h = ctypes.c_void_p()
    assert lib.spense_pack_experts(P, sdg.DT_MX4, P, 4, N, K, K // 2, K // 32, 0, None, ctypes.byref(h)) == 0
    return h


def run_experts(lib, h, M, adtype=sdg.DT_MX4, R=None, rows=None, X=P, ldx=K):
    return lib.spense_experts_linear(h, X, adtype, M, ldx, rows, P, M if R is None else R, P, sdg.DT_F32, N, STREAM)


CALLS = {
    "linear": (sparse_layer, lambda lib, h, M: lib.spense_linear(h, P, sdg.DT_BF16, M, K, P, sdg.DT_F32, N, STREAM)),
    "w8a8": (sparse_layer, lambda lib, h, M: lib.spense_linear_w8a8(h, P, M, K, P, sdg.DT_F32, N, 0, STREAM)),
    "mx4": (mx4_layer, lambda lib, h, M: lib.spense_linear(h, P, sdg.DT_BF16, M, K, P, sdg.DT_F32, N, STREAM)),
    "w4a4": (mx4_layer, lambda lib, h, M: lib.spense_linear_w4a4(h, P, M, K, P, sdg.DT_F32, N, STREAM)),
    "experts": (experts, run_experts),
}


def pointers(lib, h, run, M):
    """Workspaces that the launch of a call at M rows was given."""
    lib.host_forget()
    assert run(lib, h, M) == 0
    return [p for p in (lib.host_seen(f) for f in (hl.X, hl.PARTIALS, hl.COUNTERS)) if p not in (0, P)]


@pytest.mark.parametrize("kind", CALLS)
def test_captured_workspaces_outlive_larger_calls(lib, kind):
    """What a graph has recorded stays allocated when a larger call replaces it, and goes with the handle."""
    pack, run = CALLS[kind]
    before = lib.host_live_bytes()
    h = pack(lib)
    pointers(lib, h, run, 4)                # sizes the workspaces
    lib.host_capturing(1)
    recorded = pointers(lib, h, run, 4)
    lib.host_capturing(0)
    assert recorded and all(lib.host_live(p) for p in recorded)
    moved = set()
    for M in (64, 700, 5000):
        moved |= set(pointers(lib, h, run, M)) - set(recorded)
        assert all(lib.host_live(p) for p in recorded), M
    assert moved                            # the larger calls did replace some
    lib.spense_free(h)
    assert lib.host_live_bytes() == before


@pytest.mark.parametrize("kind", CALLS)
def test_growing_without_a_graph_keeps_nothing_old(lib, kind):
    """A handle that grows a little with every call ends with what it holds if the largest call comes first."""
    pack, run = CALLS[kind]
    held = []
    for steps in (range(4000, 99, -100), range(100, 4001, 100)):
        h = pack(lib)
        for M in steps:
            pointers(lib, h, run, M)
        held.append(lib.host_live_bytes())
        lib.spense_free(h)
    assert held[1] <= held[0]


def test_a_graph_keeps_only_what_it_recorded(lib):
    """Workspaces taken after the capture are freed again when they are outgrown."""
    h = mx4_layer(lib)
    run = CALLS["w4a4"][1]
    run(lib, h, 4)
    lib.host_capturing(1)
    run(lib, h, 4)
    lib.host_capturing(0)
    kept = lib.host_live_bytes()
    for M in range(64, 4001, 64):
        run(lib, h, M)
    grown = lib.host_live_bytes()
    lib.spense_free(h)
    h = mx4_layer(lib)
    run(lib, h, 4000)
    assert grown <= lib.host_live_bytes() + kept
    lib.spense_free(h)


MISALIGNED = P + 2
LAYOUTS = {"mx4": (sdg.DT_MX4, P), "bf16": (sdg.DT_BF16, MISALIGNED)}  # calls that lay X out first


def laid_out(lib, h, M, R, rows, form):
    adtype, X = LAYOUTS[form]
    lib.host_forget()
    assert run_experts(lib, h, M, adtype, R, rows, X) == 0
    return lib.host_seen(hl.LAID_OUT), lib.host_seen(hl.PICKED), lib.host_seen(hl.ALLOCATIONS)


@pytest.mark.parametrize("form", LAYOUTS)
def test_only_the_rows_that_are_read_are_laid_out(lib, form):
    h = experts(lib)
    assert laid_out(lib, h, 1000, 10, None, form)[:2] == (10, 0)       # grouped, the rest of X unused
    assert laid_out(lib, h, 1000, 10, P, form)[:2] == (10, 1)          # a few picked rows
    assert laid_out(lib, h, 10, 10, P, form)[:2] == (10, 0)
    assert laid_out(lib, h, 10, 1000, P, form)[:2] == (10, 0)          # rows that repeat: each row of X once
    assert laid_out(lib, h, 1 << 19, 1 << 20, P, form)[:2] == (1 << 20, 1)  # X past 31 bits
    lib.spense_free(h)


@pytest.mark.parametrize("form", LAYOUTS)
@pytest.mark.parametrize("rows", [None, P], ids=["grouped", "picked"])
@pytest.mark.parametrize("M,R", [(1 << 19, 6), ((1 << 19) + 5, 900), (700, 700), (90, 400), (1 << 19, (1 << 19) + 40)])
def test_a_call_sizes_every_call_with_fewer_rows(lib, M, R, rows, form):
    """After a call with M rows of X and R in Y none with fewer of either allocates (as a capture needs)."""
    if rows is None and M < R:
        pytest.skip("grouped rows of X are at least R")
    h = experts(lib)
    laid_out(lib, h, M, R, rows, form)
    for m in (M - 1, M // 2, 1000, 600, 64, 1):
        for r in (R, R - 1, R // 2, 500, 17, 1):
            if 1 <= m <= M and 1 <= r <= R and (rows or m >= r):
                assert laid_out(lib, h, m, r, rows, form)[2] == 0, (m, r)
    lib.spense_free(h)
