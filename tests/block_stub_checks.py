"""Valid calls of every entry point of include/moe_block.h against the host-only build of the library
(tests/block_host_stubs.cpp), run by tests/test_block_sanitize.py under AddressSanitizer and
UndefinedBehaviorSanitizer: workspace carving and the launches of each call, at sizes up to the largest.

Not collected by the default test run (no test_ prefix): it needs the stub library.
"""

import ctypes

import pytest

import sparse_moe_expert_route_amd as moe
from sparse_moe_expert_route_amd import block

M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    L = block._load()
    assert hasattr(L, "moe_block_stub_calls"), "these checks need the host-only stub build"
    L.moe_block_stub_calls.argtypes = [ctypes.c_char_p]
    L.moe_block_stub_calls.restype = ctypes.c_int
    return L


NAMES = ["norm", "residual", "combine", "few", "few_tail"]


def _delta(lib, fn):
    before = {n: lib.moe_block_stub_calls(n.encode()) for n in NAMES}
    st = fn()
    return st, {n: lib.moe_block_stub_calls(n.encode()) - before[n] for n in NAMES
                if lib.moe_block_stub_calls(n.encode()) != before[n]}


def _tail(step, **over):
    f = dict(r=10 * step, r_out=11 * step, w_post=12 * step, gate=13 * step, w_next=14 * step, n_next=15 * step, scale=1.0,
             eps=1e-6, res_dtype=1, param_dtype=1, post_norm=1, gate_per_token=0)
    f.update(over)
    return block._Tail(*f.values())


@pytest.mark.parametrize("T,H", [(1, 128), (64, 4096), (16384, 6144), (3, 16384)])
def test_norm_calls(lib, T, H):
    step = 1 << 40
    p = moe.Problem.make(T, H, 128, 8, 8)
    assert _delta(lib, lambda: lib.moe_block_norm(p, step, 0, None, 0, 1e-6, 2 * step, None)) == (0, {"norm": 1})
    assert _delta(lib, lambda: lib.moe_block_residual(p, 2 * step, 0, _tail(step), None)) == (0, {"residual": 1})
    in_place = _tail(step, r_out=10 * step, w_post=None, gate=None, w_next=None, n_next=None, post_norm=0)
    assert _delta(lib, lambda: lib.moe_block_residual(p, 2 * step, 1, in_place, None)) == (0, {"residual": 1})
    assert _delta(lib, lambda: lib.moe_combine_residual(p, 2 * step, 3 * step, 4 * step, _tail(step, gate_per_token=1),
                                                        None)) == (0, {"combine": 1})


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 128, 1, 1), (16, 6144, 2048, 384, 8), (1, 65536, 65536, 512, 8),
                                       (7, 16384, 640, 100, 3), (16, 7552, 128, 512, 8)])
def test_few_carves_its_workspace(lib, T, H, I, E, k, fmt):
    p = moe.Problem.make(T, H, I, E, k, 1, fmt)
    n = moe.block_workspace_size(p)
    w = moe._Weights(M, M, M, M, 1)
    st, d = _delta(lib, lambda: lib.moe_forward_few(p, M, M, M, w, M, 0, 64 * M, n, None))
    assert st == 0 and d == {"few": 1}


@pytest.mark.parametrize("T,H,I,expect", [(1, 4096, 2048, {"few": 1, "few_tail": 1}), (16, 6144, 2048, {"few": 1, "few_tail": 1}),
                                          (17, 4096, 2048, {"norm": 1, "combine": 1}), (8, 16384, 128, {"norm": 1, "combine": 1}),
                                          (2, 512, 65536 + 128, {"norm": 1, "combine": 1}),
                                          (8192, 4096, 2048, {"norm": 1, "combine": 1})])
def test_block_forward_launches(lib, T, H, I, expect):
    step = 1 << 42
    p = moe.Problem.make(T, H, I, 256, 8)
    n = moe.block_workspace_size(p)
    w = moe._Weights(M, M, M, M, 0)
    st, d = _delta(lib, lambda: lib.moe_block_forward(p, None, M, None, w, _tail(step), 64 * M, n, None))
    assert st == 0 and d == expect
