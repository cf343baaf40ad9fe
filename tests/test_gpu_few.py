"""GPU parity of the layer for few tokens (moe_forward_few) and of the whole block (moe_block_forward)
against the float64 oracle.

Tolerances are those of the layer's other parity tests (moe_testutil): 2e-2 RMS plus, on elements the
oracle flags as ambiguous, one step of an FP8 code of h carried through |W2|.  Tokens whose selection
lies within the float32 uncertainty of their logits of a tie are compared by nothing but finiteness.
"""

import functools

import numpy as np
import pytest
import torch

import synthetic as S
from moe_testutil import (dev, host, log, weights, problem, unambiguous_tokens, key_margin, oracle_with_allowance,
                          check_output, bf16_rne, LOGIT_RTOL)
from oracle import block as OB
from oracle import formats as F
from oracle import layer as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_moe_expert_route_amd as m
    m.load()
    return m


def make(over):
    over = dict(over)
    score = over.pop("score", "softmax")
    same = over.pop("same", False)
    lay = S.make_layer("tiny", seed=over.pop("seed", 0), **over)
    lay["score"] = score
    if same:       # every token to the same experts: a bias far above any score
        E, k = lay["w13"].shape[0], lay["top_k"]
        b = np.zeros(E, np.float32)
        b[np.random.default_rng(3).permutation(E)[:k]] = 100.0
        lay["bias"] = b
    return lay


@pytest.fixture(autouse=True)
def product_scales(monkeypatch):
    """The FP8 block-scaled rule of the layer for few tokens: scale amax * (1 / 448)."""
    monkeypatch.setattr(F, "quantize_fp8_blocks_f32", functools.partial(F.quantize_fp8_blocks_f32, product=True))


def guarded(T, H, dtype):
    buf = torch.full((T + 2, H), 77.0, dtype=dtype, device="cuda")

    def check():
        assert torch.all(buf[0] == 77.0) and torch.all(buf[T + 1] == 77.0)
    return buf[1:T + 1], check


def clear_tokens(lay, L_ref):
    """Tokens whose selected set is beyond the float32 error of the logits (a generous 1e-5 RMS)."""
    L = L_ref + 1e-5 * np.sqrt(np.mean(L_ref ** 2))
    return unambiguous_tokens(L_ref, lay["top_k"], lay["bias"], key_margin(L, L_ref, lay["bias"], lay["score"]),
                              order=False, score=lay["score"])


CASES = [dict(T=1), dict(T=16), dict(T=7, E=32, k=4, bias="zipf"), dict(T=1, H=128, I=128, E=1, k=1),
         dict(T=16, H=128, I=128, E=1, k=1), dict(T=2, E=4, k=4), dict(T=16, E=512, k=8, H=512, I=256),
         dict(T=3, E=130, k=8), dict(T=13, E=65, k=5, H=384, I=384), dict(T=5, H=1024, I=640, E=12, k=3),
         dict(T=16, H=640, I=1152, E=24, k=8), dict(T=4, H=2176, I=128, E=16, k=2), dict(T=9, H=256, I=2048, E=8, k=6),
         dict(T=16, E=64, k=8, H=512, I=512, same=True), dict(T=15, E=16, k=3, same=True),
         dict(T=8, H=4096, I=2048, E=16, k=8), dict(T=2, H=6144, I=512, E=16, k=8), dict(T=1, H=8192, I=256, E=8, k=4),
         dict(T=2, H=16512, I=128, E=4, k=2),
         # x too long for bf16 in LDS, with stages that end K early; K in 8, 4 and 2 parts
         dict(T=16, H=4224, I=128, E=8, k=2), dict(T=3, H=6144, I=128, E=8, k=2), dict(T=2, H=4096, I=256, E=16, k=8),
         dict(T=11, H=5120, I=384, E=24, k=2), dict(T=4, H=512, I=256, E=400, k=8)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp4", "fp8_block"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_few_parity(moe, case, fmt, packed):
    over = dict(CASES[case], format=fmt, score="sigmoid" if case % 3 == 2 else "softmax")
    log("forward_few %s packed=%s" % (over, packed))
    lay = make(over)
    p = problem(lay)
    W = weights(lay, packed)
    T, H = lay["x"].shape
    ws = moe.alloc_block_workspace(p)
    ws.fill_(0xFF)                               # nothing of the workspace has to start at zero
    bias = None if lay["bias"] is None else dev(lay["bias"])
    y, check = guarded(T, H, torch.float32)
    moe.forward_few(p, dev(lay["x"]), dev(lay["w_router"]), bias, W, y, ws)
    torch.cuda.synchronize()
    check()
    ref = oracle_with_allowance(lay)
    err, share = check_output(host(y), ref, rows=clear_tokens(lay, ref["logits"]))
    log("  max err / RMS %.2e, share past the plain bar %.2e" % (err, share))
    assert np.all(np.isfinite(host(y)))
    # bf16 output: the rounding of the same float32 sums, from a second call on the same workspace
    yb, check = guarded(T, H, torch.bfloat16)
    moe.forward_few(p, dev(lay["x"]), dev(lay["w_router"]), bias, W, yb, ws, moe.OUT_BF16)
    torch.cuda.synchronize()
    check()
    assert np.array_equal(host(yb.contiguous()), bf16_rne(host(y)))


@pytest.mark.parametrize("T,over", [(16, dict(E=32, k=4, H=1024, I=512)), (3, dict(E=64, k=2, H=2048, I=256)),
                                    (2, dict(E=16, k=2, H=4096, I=128, format="fp8_block"))])
def test_rows_do_not_depend_on_their_neighbours(moe, T, over):
    """A token's output has the same bits whatever the other tokens of a batch of the same size are, and
    the same values up to float32 sums in another order alone (the gate/up sums may be cut differently)."""
    lay = make(dict(T=T, **over))
    p = problem(lay)
    H = p.hidden
    W = weights(lay, True)
    x, wr = dev(lay["x"]), dev(lay["w_router"])
    ws = moe.alloc_block_workspace(p)
    y = torch.empty(T, H, device="cuda")
    moe.forward_few(p, x, wr, None, W, y, ws)
    for t in (0, T - 1):
        others = x.roll(3, dims=1) * 0.5
        others[t] = x[t]
        y2 = torch.empty(T, H, device="cuda")
        moe.forward_few(p, others.contiguous(), wr, None, W, y2, ws)
        torch.cuda.synchronize()
        assert torch.equal(y2[t], y[t]), t
        p1 = moe.Problem.make(1, H, p.intermediate, p.num_experts, p.top_k, 0, p.expert_format)
        y1 = torch.empty(1, H, device="cuda")
        moe.forward_few(p1, x[t:t + 1], wr, None, W, y1, moe.alloc_block_workspace(p1))
        torch.cuda.synchronize()
        assert float((y1[0] - y[t]).norm()) <= 2e-3 * float(y[t].norm()), t


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8_block"])
@pytest.mark.parametrize("over", [dict(T=1, k=8), dict(T=1, k=3), dict(T=1, k=1), dict(T=2, k=4), dict(T=4, k=2), dict(T=8, k=1),
                                  dict(T=2, k=4, same=True), dict(T=8, k=1, E=2), dict(T=1, k=8, I=2176), dict(T=1, k=8, H=128),
                                  dict(T=2, k=4, I=5120, E=8), dict(T=1, k=8, I=15360, H=256, E=8),
                                  dict(T=8, k=1, H=7680, I=128, E=4)])
def test_eight_slots_at_most(moe, over, fmt):
    """Where a workgroup holds every expert's rows of some features (up to 8 routing slots): one expert to
    eight, several tokens of one expert, K that ends inside a stage, and rows too long for it."""
    over = dict(dict(E=16, H=1024, I=384, format=fmt), **over)
    log("few %s" % over)
    lay = make(over)
    p = problem(lay)
    T, H = lay["x"].shape
    ref = oracle_with_allowance(lay)
    x, wr = dev(lay["x"]), dev(lay["w_router"])
    bias = None if lay["bias"] is None else dev(lay["bias"])
    for packed in (True, False):
        ws = moe.alloc_block_workspace(p)
        ws.fill_(0xFF)
        y, check = guarded(T, H, torch.float32)
        moe.forward_few(p, x, wr, bias, weights(lay, packed), y, ws)
        torch.cuda.synchronize()
        check()
        assert moe.error_words(ws) == (0, 0)
        check_output(host(y), ref, rows=clear_tokens(lay, ref["logits"]))


def test_every_slot_its_own_expert(moe):
    """16 tokens x 8 slots on 128 different experts, the most that can be touched."""
    T, k, E, H = 16, 8, 128, 256
    lay = make(dict(T=T, E=E, k=k, H=H, I=128))
    x = np.zeros((T, H), np.float32)
    w = np.zeros((E, H), np.float32)
    rng = np.random.default_rng(4)
    x[:, 32:] = 0.25 * rng.normal(size=(T, H - 32))
    for t in range(T):
        x[t, t] = 4.0
        w[k * t:k * t + k, t] = 1.0 + np.arange(k) / 8
    lay["x"], lay["w_router"] = bf16_rne(x), bf16_rne(w)
    p = problem(lay)
    y = torch.empty(T, H, device="cuda")
    moe.forward_few(p, dev(lay["x"]), dev(lay["w_router"]), None, weights(lay, True), y, moe.alloc_block_workspace(p))
    torch.cuda.synchronize()
    ref = oracle_with_allowance(lay)
    assert len(np.unique(ref["ids"])) == 128
    check_output(host(y), ref)


@pytest.mark.parametrize("over", [dict(T=16, E=64, k=8, H=1024, I=512), dict(T=2, E=16, k=4, H=4096, I=256),
                                  dict(T=9, E=32, k=4, H=512, I=384, format="fp8_block")])
def test_a_workspace_serves_other_inputs(moe, over):
    """Calls with changing inputs on one workspace, back to back: each has the bits of a call with a
    workspace of its own (nothing of an earlier call is read, from memory or from a cache)."""
    lay = make(over)
    p = problem(lay)
    W, wr = weights(lay, True), dev(lay["w_router"])
    T, H = lay["x"].shape
    xs = [dev(S.bf16_normal(100 + i, 5, (T, H), 1.0)) for i in range(4)]
    want = []
    for x in xs:
        y = torch.empty(T, H, device="cuda")
        moe.forward_few(p, x, wr, None, W, y, moe.alloc_block_workspace(p))
        want.append(y)
    ws = moe.alloc_block_workspace(p)
    got = [torch.empty(T, H, device="cuda") for _ in range(24)]
    for i, y in enumerate(got):
        moe.forward_few(p, xs[i % 4], wr, None, W, y, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 4]) for i, y in enumerate(got))
    assert moe.error_words(ws) == (0, 0)


def test_other_batches_of_the_library_between(moe):
    """The block's workspace also serves moe_forward, and calls of both may alternate on it."""
    lay = make(dict(T=6, E=16, k=4, H=512, I=256))
    p = problem(lay)
    W, x, wr, ws = weights(lay, True), dev(lay["x"]), dev(lay["w_router"]), moe.alloc_block_workspace(p)
    a, b = torch.empty(6, 512, device="cuda"), torch.empty(6, 512, device="cuda")
    moe.forward_few(p, x, wr, None, W, a, ws)
    moe.forward(p, x, wr, None, W, b, ws)
    first = a.clone(), b.clone()
    for _ in range(3):
        moe.forward(p, x, wr, None, W, b, ws)
        moe.forward_few(p, x, wr, None, W, a, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, first[0]) and torch.equal(b, first[1])


def test_selection_ties_go_to_the_lowest_id(moe):
    """Equal router rows give equal logits: the lowest ids win, as moe_route selects."""
    E, k, T, H = 48, 6, 4, 256
    lay = make(dict(T=T, E=E, k=k, H=H, I=128))
    lay["w_router"] = np.repeat(lay["w_router"][:1], E, axis=0)
    p = problem(lay)
    y = torch.empty(T, H, device="cuda")
    moe.forward_few(p, dev(lay["x"]), dev(lay["w_router"]), None, weights(lay, True), y, moe.alloc_block_workspace(p))
    torch.cuda.synchronize()
    ref = oracle_with_allowance(lay)
    assert np.array_equal(ref["ids"], np.tile(np.arange(k), (T, 1)))
    check_output(host(y), ref)


def test_zero_rows_and_repeats(moe):
    """An all-zero token gives zeros; repeated calls give the same bits."""
    lay = make(dict(T=6, E=16, k=4, H=512, I=256))
    lay["x"][2] = 0
    p = problem(lay)
    W, x, wr, ws = weights(lay, True), dev(lay["x"]), dev(lay["w_router"]), moe.alloc_block_workspace(p)
    y = torch.empty(6, 512, device="cuda")
    moe.forward_few(p, x, wr, None, W, y, ws)
    first = y.clone()
    assert torch.all(y[2] == 0)
    for _ in range(5):
        moe.forward_few(p, x, wr, None, W, y, ws)
    torch.cuda.synchronize()
    assert torch.equal(first, y)


def test_two_streams_and_graph_replays(moe):
    """Calls that overlap on two streams (a workspace each), and replays of a captured call between eager work."""
    lays = [make(dict(T=16, E=64, k=8, H=1024, I=512, seed=1)), make(dict(T=5, E=32, k=4, H=2048, I=256, seed=2))]
    ps = [problem(l) for l in lays]
    Ws = [weights(l, True) for l in lays]
    xs, wrs = [dev(l["x"]) for l in lays], [dev(l["w_router"]) for l in lays]
    wss = [moe.alloc_block_workspace(p) for p in ps]
    ys = [torch.empty(*x.shape, device="cuda") for x in xs]
    for i in range(2):
        moe.forward_few(ps[i], xs[i], wrs[i], None, Ws[i], ys[i], wss[i])
    torch.cuda.synchronize()
    want = [y.clone() for y in ys]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for y in ys:
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            moe.forward_few(ps[i], xs[i], wrs[i], None, Ws[i], ys[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.forward_few(ps[0], xs[0], wrs[0], None, Ws[0], ys[0], wss[0])
    for i in range(4):
        ys[0].fill_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[0])
        moe.forward_few(ps[1], xs[1], wrs[1], None, Ws[1], ys[1], wss[1])   # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(ys[1], want[1])


BLOCKS = [dict(T=1, E=32, k=4, H=512, I=256), dict(T=16, E=24, k=8, H=1024, I=512, score="sigmoid", bias="zipf"),
          dict(T=3, E=8, k=2, H=128, I=128, format="fp8_block"), dict(T=40, E=16, k=4, H=512, I=512),
          dict(T=300, E=8, k=4, H=512, I=512), dict(T=12, E=40, k=6, H=640, I=384, format="fp8_block"),
          dict(T=2, E=16, k=8, H=6144, I=512), dict(T=5, E=4, k=1, H=2176, I=128),
          # a down run that is not full (7 experts x 12 items), 16 rows of the tail behind it; long rows of the tail
          dict(T=16, E=7, k=7, H=384, I=256), dict(T=7, E=4, k=2, H=16384, I=128), dict(T=3, E=4, k=2, H=8320, I=256)]


@pytest.mark.parametrize("case", range(len(BLOCKS)))
@pytest.mark.parametrize("res,post,gate,in_place", [("f32", True, "row", False), ("bf16", False, None, True),
                                                    ("bf16", True, "all", False)])
def test_block_forward_parity(moe, case, res, post, gate, in_place):
    """The run of the operators together.  The layer's input is held to the oracle's rounding (an element
    one bf16 step off where float32 meets a border), the output to the layer's bar carried through the tail."""
    over = BLOCKS[case]
    log("block_forward %s %s post=%s gate=%s in_place=%s" % (over, res, post, gate, in_place))
    lay = make(over)
    p = problem(lay)
    T, H = lay["x"].shape
    g = torch.Generator().manual_seed(case)
    dt = torch.bfloat16 if res == "bf16" else torch.float32
    par = torch.float32 if case % 2 else torch.bfloat16
    r = torch.randn(T, H, generator=g).to(dt).cuda()
    r_in = r.double().cpu().numpy()
    rnd = lambda *s: (1 + 0.2 * torch.randn(*s, generator=g)).to(par).cuda()
    w_pre, w_post, w_next = rnd(H), rnd(H) if post else None, rnd(H)
    gt = None if gate is None else rnd(H) if gate == "row" else rnd(T, H)
    n_next = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    r_out, check = (r, lambda: None) if in_place else guarded(T, H, dt)
    tail = moe.BlockTail(r, r_out, post_norm=post, w_post=w_post, gate=gt, scale=0.5, w_next=w_next, n_next=n_next)
    bias = None if lay["bias"] is None else dev(lay["bias"])
    ws = moe.alloc_block_workspace(p)
    ws.fill_(0xFF)
    W = weights(lay, case % 2 == 0)
    # the layer's input as the kernel rounds it, from the same norm alone
    n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.block_norm(p, r, w_pre, n)
    torch.cuda.synchronize()
    moe.block_forward(p, w_pre, dev(lay["w_router"]), bias, W, tail, ws)
    torch.cuda.synchronize()
    check()
    f64 = lambda t: None if t is None else t.double().cpu().numpy()
    n_ref = OB.rms_norm(r_in, f64(w_pre))
    assert np.all(np.abs(f64(n) - n_ref) <= np.abs(n_ref) * (2.0 ** -8 + 1e-5))
    lay["x"] = host(n)
    ref = oracle_with_allowance(lay)
    clear = clear_tokens(lay, ref["logits"])
    y = ref["y"]
    rms = np.sqrt(np.mean(y ** 2))
    dy = 2e-2 * rms + ref["allow"]                                  # the layer's bar, per element
    gg = 1.0 if gt is None else f64(gt)
    want = OB.residual(r_in, y, post, f64(w_post), f64(gt), 0.5)
    dz = dy
    if post:
        row = np.sqrt(np.mean(y * y, 1, keepdims=True))
        dz = np.abs(f64(w_post)) * (dy + np.abs(y) * np.sqrt(np.mean(dy * dy, 1, keepdims=True)) / row) / row
    got = f64(tail.r_out)
    tol = 0.5 * np.abs(gg) * dz + np.abs(want) * (2.0 ** -8 if res == "bf16" else 1e-6) + 1e-6 * rms
    err = np.abs(got - want)
    assert np.all(err[clear] <= tol[clear]), np.max((err - tol)[clear])
    nn = OB.rms_norm(got, f64(w_next))
    assert np.all(np.abs(f64(n_next) - nn) <= np.abs(nn) * (2.0 ** -8 + 1e-5))


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8_block"])
@pytest.mark.parametrize("T", [17, 64, 333])
def test_a_prompts_block_is_its_parts(moe, T, fmt):
    """Past the few tokens: the bits of norm, forward and residual one after the other."""
    lay = make(dict(T=T, E=16, k=4, H=640, I=384, format=fmt))
    p = problem(lay)
    g = torch.Generator().manual_seed(T)
    r = torch.randn(T, 640, generator=g).cuda()
    par = lambda *s: (1 + 0.2 * torch.randn(*s, generator=g)).cuda()
    wn, post, gate, nxt = par(640), par(640), par(T, 640), par(640)
    W, wr, ws = weights(lay, T != 64), dev(lay["w_router"]), moe.alloc_block_workspace(p)
    bf = lambda: torch.empty(T, 640, dtype=torch.bfloat16, device="cuda")
    tails = [moe.BlockTail(r, torch.empty_like(r), post_norm=True, w_post=post, gate=gate, scale=0.7, w_next=nxt,
                           n_next=bf()) for _ in range(2)]
    n, y = bf(), torch.empty(T, 640, device="cuda")
    moe.block_norm(p, r, wn, n)
    moe.forward(p, n, wr, None, W, y, ws)
    moe.block_residual(p, y, tails[0])
    ws.fill_(0xFF)
    moe.block_forward(p, wn, wr, None, W, tails[1], ws)
    torch.cuda.synchronize()
    assert torch.equal(tails[0].r_out, tails[1].r_out) and torch.equal(tails[0].n_next, tails[1].n_next)


@pytest.mark.parametrize("T,over", [(1, dict(E=32, k=4, H=2048, I=256)), (16, dict(E=64, k=8, H=1024, I=512)),
                                    (12, dict(E=16, k=4, H=512, I=256, format="fp8_block")),
                                    (48, dict(E=16, k=4, H=512, I=256))])
def test_block_graph_on_its_own_stream(moe, T, over):
    """Two blocks in a row, captured, replayed with eager work and new inputs between the replays."""
    lay = make(dict(T=T, **over))
    p = problem(lay)
    H = lay["x"].shape[1]
    g = torch.Generator().manual_seed(T)
    ins = [torch.randn(T, H, generator=g).cuda() for _ in range(3)]
    r, ws = torch.empty_like(ins[0]), moe.alloc_block_workspace(p)
    W, wr = weights(lay, True), dev(lay["w_router"])
    nn = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(r)
    first = moe.BlockTail(r, r)
    second = moe.BlockTail(r, out, post_norm=True, w_next=torch.ones(H, device="cuda"), n_next=nn)

    def run():
        for tail in (first, second):
            moe.block_forward(p, None, wr, None, W, tail, ws)

    want = []
    for x in ins:
        r.copy_(x)
        run()
        torch.cuda.synchronize()
        want.append((out.clone(), nn.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        r.copy_(ins[0])
        run()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.synchronize()
    for i in range(9):
        r.copy_(ins[i % 3])
        out.zero_(), nn.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i % 3][0]) and torch.equal(nn, want[i % 3][1])
        if i % 3 == 1:                                       # eager work on the same workspace between replays
            r.copy_(ins[2])
            run()
            torch.cuda.synchronize()
            assert torch.equal(out, want[2][0])
    assert moe.error_words(ws) == (0, 0)


def test_few_equals_forward_closely_on_a_decode_layer(moe):
    """The same layer through moe_forward: equal up to FP8 codes of h that sit on a border."""
    lay = make(dict(T=16, E=64, k=8, H=4096, I=2048))
    p = problem(lay)
    W, x, wr, ws = weights(lay, True), dev(lay["x"]), dev(lay["w_router"]), moe.alloc_block_workspace(p)
    a, b = torch.empty(16, 4096, device="cuda"), torch.empty(16, 4096, device="cuda")
    moe.forward_few(p, x, wr, None, W, a, ws)
    moe.forward(p, x, wr, None, W, b, ws)
    torch.cuda.synchronize()
    rel = float((a - b).norm() / b.norm())
    log("  few against forward: relative difference %.2e" % rel)
    assert rel <= 2e-3
