"""GPU parity of the norms around the layer, the gate and the residual sum against the float64 oracle.

Tolerances, counted in roundings (u = 2^-24, half an ulp of float32; b = 2^-8, half a step of bf16):
  * a float32 norm: the sum of squares is a chain of at most 64 fused additions (a lane's, its wave's
    and the waves'), 10 more leave room for another split of the row (74 u, halved by the root), the
    quotient by H, the sum with eps, the root, its reciprocal and two products (6 u): NORM_U = 43 u of
    the value;
  * r': the norm's error times scale * gate, 3 more products, and one rounding of the sum;
  * bf16 outputs: b of the value on top; n' is compared with the norm of the stored r'.
"""

import numpy as np
import pytest
import torch

from moe_testutil import log
from oracle import block as OB

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = 2.0 ** -8
NORM_U = 43 * U
TINY = 1e-37   # below float32's normal range: hardware may flush


@pytest.fixture(scope="module")
def moe():
    import sparse_moe_expert_route_amd as m
    m.load()
    return m


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(g, shape, dtype, scale=1.0, offset=0.0):
    return (offset + scale * torch.randn(*shape, generator=g)).to(DT[dtype]).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def guarded(T, H, dtype):
    """An output of T rows inside a larger buffer of sentinels; returns (view, check)."""
    buf = torch.full((T + 2, H), 77.0, dtype=dtype, device="cuda")

    def check():
        assert torch.all(buf[0] == 77.0) and torch.all(buf[T + 1] == 77.0)
    return buf[1:T + 1], check


def close(got, ref, tol, what):
    err = np.abs(got - ref)
    bad = err > tol + TINY
    assert not bad.any(), "%s: %d of %d off, worst %.3e of tolerance" % (what, bad.sum(), bad.size,
                                                                       np.max(err / (tol + TINY)))


SHAPES = [(1, 128), (2, 256), (5, 1920), (17, 2176), (64, 4096), (3, 6144), (2, 8192), (3, 16384), (1, 8320), (300, 512)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res,param", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", None)])
def test_block_norm(moe, T, H, res, param):
    log("block_norm T=%d H=%d %s %s" % (T, H, res, param))
    g = torch.Generator().manual_seed(T * 7 + H)
    r = rnd(g, (T, H), res, 3.0)
    r[0] = 0                                     # a zero row: n is 0, not NaN
    if T > 2:
        r[1] *= 2.0 ** 40                        # far from 1, squares still in range
        r[2] *= 2.0 ** -40                       # eps dominates
    w = None if param is None else rnd(g, (H,), param, 0.2, 1.0)
    p = moe.Problem.make(T, H, 128, 8, 2)
    n, check = guarded(T, H, torch.bfloat16)
    moe.block_norm(p, r, w, n, 1e-5)
    torch.cuda.synchronize()
    check()
    ref = OB.rms_norm(f64(r), None if w is None else f64(w), 1e-5)
    close(f64(n), ref, np.abs(ref) * (B + 2 * NORM_U), "n")
    assert torch.all(n[0] == 0)


def check_tail(tail, y, dy, eps, names="r n"):
    """r_out and n_next against the oracle; dy: bound on the error of y as the kernel holds it."""
    opt = lambda t: None if t is None else f64(t)
    r, ro = f64(tail.r_in), f64(tail.r_out)
    z = OB.rms_norm(y, opt(tail.w_post), eps) if tail.post_norm else y
    g = 1.0 if tail.gate is None else f64(tail.gate)
    ref = r + float(np.float32(tail.scale)) * (g * z)
    # error of z from the error of y: directly, and through the root mean square (Cauchy-Schwarz)
    dz = dy
    if tail.post_norm:
        rms = np.sqrt(np.mean(y * y, 1, keepdims=True) + eps)
        w = 1.0 if tail.w_post is None else np.abs(f64(tail.w_post))[None, :]
        drel = np.sqrt(np.mean(dy * dy, 1, keepdims=True)) / rms
        dz = w * (dy + np.abs(y) * drel) / rms + np.abs(z) * NORM_U
    step = np.abs(float(tail.scale)) * np.abs(g)
    half = U if tail.r_out.dtype == torch.float32 else B + U
    tol = step * (dz + 3 * U * np.abs(z)) + np.abs(ref) * half
    close(ro, ref, tol * (1 + 1e-6), "r_out")
    if tail.n_next is not None:
        n_ref = OB.rms_norm(ro, opt(tail.w_next), eps)
        close(f64(tail.n_next), n_ref, np.abs(n_ref) * (B + 2 * NORM_U), "n_next")


def make_tail(moe, g, T, H, res, param, post, gate, nxt, scale, in_place=False, eps=1e-6):
    r = rnd(g, (T, H), res)
    keep = r.clone()
    checks = []
    if in_place:
        r_out = r
    else:
        r_out, c = guarded(T, H, r.dtype)
        checks.append(c)
    n_next = None
    if nxt:
        n_next, c = guarded(T, H, torch.bfloat16)
        checks.append(c)
    t = moe.BlockTail(r, r_out, post_norm=post, w_post=rnd(g, (H,), param, 0.2, 1.0) if post else None,
                      gate={"none": None, "row": rnd(g, (H,), param), "all": rnd(g, (T, H), param)}[gate],
                      scale=scale, eps=eps, w_next=rnd(g, (H,), param, 0.2, 1.0) if nxt == "w" else None,
                      n_next=n_next)
    t.r_in = keep
    return t, checks


TAILS = [("bf16", "bf16", True, "row", "w", 1.0, False), ("f32", "f32", True, "all", "w", 0.25, False),
         ("bf16", "f32", False, "none", "w", 1.0, True), ("f32", "bf16", False, "all", None, -0.5, True),
         ("bf16", "bf16", True, "none", "ones", 0.22, True), ("f32", "bf16", True, "row", None, 0.0, False)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("case", range(len(TAILS)))
def test_block_residual(moe, T, H, case):
    res, param, post, gate, nxt, scale, in_place = TAILS[case]
    log("block_residual T=%d H=%d %s" % (T, H, TAILS[case]))
    g = torch.Generator().manual_seed(T + H + case)
    y = rnd(g, (T, H), "f32" if case % 2 else "bf16", 0.4)
    y[T // 2] = 0                                 # a row of zeros: nothing is added
    tail, checks = make_tail(moe, g, T, H, res, param, post, gate, nxt, scale, in_place)
    p = moe.Problem.make(T, H, 128, 8, 2)
    moe.block_residual(p, y, tail)
    torch.cuda.synchronize()
    for c in checks:
        c()
    assert torch.equal(tail.r_out[T // 2], tail.r_in[T // 2])
    y64 = f64(y)
    check_tail(tail, y64, np.zeros_like(y64), 1e-6)


@pytest.mark.parametrize("T,H,k", [(1, 128, 1), (1, 4096, 8), (2, 256, 2), (5, 1920, 3), (17, 2176, 8), (64, 4096, 8),
                                   (3, 16384, 7), (300, 512, 8), (9, 6144, 6)])
@pytest.mark.parametrize("case", [0, 1, 2, 5])
def test_combine_residual(moe, T, H, k, case):
    res, param, post, gate, nxt, scale, in_place = TAILS[case]
    log("combine_residual T=%d H=%d k=%d %s" % (T, H, k, TAILS[case]))
    g = torch.Generator().manual_seed(T + H + k + case)
    N = T * k
    y_perm = rnd(g, (N, H), "f32", 0.4)
    rows = torch.randperm(N, generator=g).to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    if T > 1:
        rows[k: 2 * k] = torch.tensor([-1, N, 1 << 30, -(1 << 31)] * 2)[:k].to(torch.int32)   # a token without rows
        rows[0] = -1                                                                          # one slot without a row
    tail, checks = make_tail(moe, g, T, H, res, param, post, gate, nxt, scale, in_place)
    p = moe.Problem.make(T, H, 128, 8, k)
    rd, wd = rows.cuda(), w.cuda()
    moe.combine_residual(p, y_perm, rd, wd, tail)
    torch.cuda.synchronize()
    for c in checks:
        c()
    rn, wn, yp = rows.numpy().reshape(T, k), w.double().numpy(), f64(y_perm)
    y, mag = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        ok = (rn[:, j] >= 0) & (rn[:, j] < N)
        term = wn[ok, j:j + 1] * yp[rn[ok, j]]
        y[ok] += term
        mag[ok] += np.abs(term)
    check_tail(tail, y, k * U * mag, 1e-6)
    if T > 1:
        assert torch.equal(tail.r_out[1], tail.r_in[1])
    # the same sum as the package's combine, when nothing follows it
    plain = moe.BlockTail(torch.zeros(T, H, device="cuda"), torch.empty(T, H, device="cuda"), post_norm=False)
    moe.combine_residual(p, y_perm, rd, wd, plain)
    ref = torch.empty(T, H, device="cuda")
    moe.combine(p, y_perm, rd, wd, ref)
    torch.cuda.synchronize()
    assert torch.equal(plain.r_out, ref)


def test_other_streams_and_graphs(moe):
    """The calls on a side stream, and captured: every replay equals the eager result."""
    T, H, k = 33, 2048, 4
    g = torch.Generator().manual_seed(5)
    p = moe.Problem.make(T, H, 128, 8, k)
    y_perm, rows = rnd(g, (T * k, H), "f32"), torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    w = torch.softmax(torch.randn(T, k, generator=g), 1).cuda()
    tail, _ = make_tail(moe, g, T, H, "bf16", "bf16", True, "row", "w", 0.5)
    n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def step():
        moe.block_norm(p, tail.r, tail.w_post, n)
        moe.combine_residual(p, y_perm, rows, w, tail)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (n, tail.r_out, tail.n_next)]
    side = torch.cuda.Stream()
    for t in (n, tail.r_out, tail.n_next):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    moe.block_norm(p, tail.r, tail.w_post, n, stream=side)
    moe.combine_residual(p, y_perm, rows, w, tail, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (n, tail.r_out, tail.n_next)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t in (n, tail.r_out, tail.n_next):
            t.fill_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (n, tail.r_out, tail.n_next)))


def test_more_rows_than_workgroups(moe):
    """Past 2^20 rows a workgroup takes several: the rows around the border and the last ones."""
    T, H = (1 << 20) + 77, 128
    p = moe.Problem.make(T, H, 128, 8, 1)
    r = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    tail = moe.BlockTail(r, torch.empty_like(r), w_next=torch.ones(H, device="cuda"), n_next=torch.empty_like(r))
    n = torch.empty_like(r)
    moe.block_norm(p, r, None, n)
    moe.block_residual(p, r, tail)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 76, 77, 78, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, T - 1], device="cuda")
    q = moe.Problem.make(len(pick), H, 128, 8, 1)
    rp = r[pick].contiguous()
    few = moe.BlockTail(rp, torch.empty_like(rp), w_next=tail.w_next, n_next=torch.empty_like(rp))
    np_ = torch.empty_like(rp)
    moe.block_norm(q, rp, None, np_)
    moe.block_residual(q, rp, few)
    torch.cuda.synchronize()
    assert torch.equal(n[pick], np_) and torch.equal(tail.r_out[pick], few.r_out) and torch.equal(tail.n_next[pick], few.n_next)
    # every row was written: the norm of any row has a root mean square of 1
    assert float((n.float().square().mean(1) - 1).abs().max()) < 0.05


def test_repeated_calls_give_the_same_bits(moe):
    T, H = 128, 6144
    g = torch.Generator().manual_seed(6)
    p = moe.Problem.make(T, H, 128, 8, 2)
    y = rnd(g, (T, H), "f32")
    tail, _ = make_tail(moe, g, T, H, "f32", "f32", True, "all", "w", 1.0)
    moe.block_residual(p, y, tail)
    a = tail.r_out.clone(), tail.n_next.clone()
    for _ in range(3):
        moe.block_residual(p, y, tail)
    torch.cuda.synchronize()
    assert torch.equal(a[0], tail.r_out) and torch.equal(a[1], tail.n_next)


def test_binding_refuses(moe):
    p = moe.Problem.make(4, 256, 128, 8, 2)
    r = torch.zeros(4, 256, device="cuda")
    n = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.block_norm(p, r, torch.ones(256), n)                       # a host parameter
    with pytest.raises(ValueError):
        moe.block_norm(p, r[:3], None, n)
    with pytest.raises(ValueError):
        moe.block_norm(p, r, None, r)                                  # n must be bf16
    with pytest.raises(moe.MoeError):
        moe.block_norm(p, r, None, n, eps=0.0)
    wide = torch.zeros(4, 512, device="cuda")
    with pytest.raises(ValueError):
        moe.block_norm(p, wide[:, ::2], None, n)                       # strided
    flat = torch.zeros(4 * 256 + 4, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.block_norm(p, flat[2:2 + 1024].view(4, 256), None, n)      # 8-byte aligned only
    with pytest.raises(moe.MoeError):
        moe.block_residual(p, r, moe.BlockTail(r, r, post_norm=False))  # r_out over y
