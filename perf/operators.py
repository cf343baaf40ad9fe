"""Workloads of the layer's operators for few tokens and of the decoder block around the layer.

Operators (names of the package's entry points):

  forward_few       the whole routed layer for 1 to 16 tokens: router, top-k, FP8 activations, SwiGLU
                    experts (MXFP4 or FP8 block-scaled), weighted sum
  block_norm        n = RMSNorm(r) * w_pre, the normalised input of the layer
  block_residual    r' = r + scale * gate * RMSNorm(y) * w_post, and optionally n' = RMSNorm(r') * w_next
  combine_residual  block_residual on y = sum_j w_j y_perm[row_j], without storing y
  block_forward     block_norm, the layer and block_residual in one call

Each case is a dict of plain values.  ``own`` selects the package's calls; otherwise ``run`` computes the
plain form: elementary torch operations in 32 bits (64 for the router's keys, which decide a selection).
"""

import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _layer(op, T, H, I, E, k, fmt="mxfp4", layout="packed", score="softmax", bias=False, **more):
    return dict(op=op, T=T, H=H, I=I, E=E, k=k, fmt=fmt, layout=layout, score=score, bias=bias, **more)


def _tail(op, T, H, res="bf16", y="bf16", param="bf16", post=True, gate="row", nxt=True, scale=1.0, **more):
    return dict(op=op, T=T, H=H, res=res, y=y, param=param, post=post, gate=gate, nxt=nxt, scale=scale, **more)


def listed():
    block = dict(res="bf16", param="bf16", post=True, gate="row", nxt=True, scale=1.0)
    return [
        # one sequence decoding on the Flash layer: 8 experts, latency counts
        dict(_layer("forward_few", 1, 4096, 2048, 256, 8), name="few flash T1"),
        # one sequence's speculative-verify block of 8 positions, sigmoid scores with a selection bias
        dict(_layer("forward_few", 8, 4096, 2048, 256, 8, score="sigmoid", bias=True), name="few flash T8 sigmoid"),
        # 16 sequences decoding on the Pro layer: over a hundred experts
        dict(_layer("forward_few", 16, 6144, 2048, 384, 8), name="few pro T16"),
        # one GPU's share of a four-way split Pro layer, weights as the checkpoint stores them
        dict(_layer("forward_few", 3, 6144, 512, 384, 8, layout="canonical"), name="few pro tp4 T3 canonical"),
        # the normalised input of a decode step
        dict(op="block_norm", T=64, H=4096, res="bf16", param="bf16", name="norm flash decode"),
        # ... and of a long prompt whose residual stream is kept in float32
        dict(op="block_norm", T=16384, H=6144, res="f32", param="f32", name="norm pro prefill f32"),
        # after a tensor-parallel sum of the layer's output: a verify batch
        dict(_tail("block_residual", 256, 6144, gate="all", scale=0.25), name="residual pro verify"),
        # a prompt, no norm after the layer, float32 residual stream, the next layer's input written too
        dict(_tail("block_residual", 8191, 4096, res="f32", param="f32", post=False, gate="none"),
             name="residual flash prompt f32"),
        # a decode step's expert rows straight into the residual stream
        dict(_tail("combine_residual", 64, 4096, k=8), name="combine flash decode"),
        # a prompt's expert rows, gate per token and channel
        dict(_tail("combine_residual", 8192, 4096, k=8, gate="all", nxt=False), name="combine flash prompt"),
        # the block of one sequence decoding
        dict(_layer("block_forward", 1, 4096, 2048, 256, 8, **block), name="block flash T1"),
        # the block of a small batch with the FP8 block-scaled experts
        dict(_layer("block_forward", 12, 4096, 2048, 256, 8, fmt="fp8_block", **dict(block, gate="none", nxt=False)),
             name="block flash fp8 T12"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["forward_few", "forward_few", "block_norm", "block_residual", "combine_residual",
                     "block_forward"])
    H = 128 * rng.randint(1, 48)
    tail = dict(res="bf16", param=rng.choice(["bf16", "f32"]), post=rng.random() < 0.6,
                gate=rng.choice(["none", "row", "all"]), nxt=rng.random() < 0.6,
                scale=rng.choice([1.0, 0.25, 0.125]))
    if op in ("forward_few", "block_forward"):
        E = rng.randint(4, 384)
        case = _layer(op, rng.randint(1, 16), H, 128 * rng.randint(1, 16), E, rng.randint(1, min(8, E)),
                      fmt=rng.choice(["mxfp4", "mxfp4", "fp8_block"]), layout=rng.choice(["packed", "canonical"]),
                      score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5)
        return dict(case, **tail) if op == "block_forward" else case
    T = _log_int(rng, 1, 8192)
    if op == "block_norm":
        return dict(op=op, T=T, H=H, res=rng.choice(["bf16", "f32"]), param=tail["param"])
    tail["res"] = rng.choice(["bf16", "f32"])
    if op == "block_residual":
        return _tail(op, T, H, y=rng.choice(["bf16", "f32"]), **tail)
    k = rng.randint(1, 8)
    return _tail(op, min(T, 8192 * 8 * 4096 // (k * H)), H, k=k, **tail)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_MAG = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]   # magnitudes of e2m1


def _pack(codes, scales, fmt):
    """The packed weight layout: 16-row groups, 128 columns per block, 16-byte pieces of the 16 rows together."""
    E, R, B = codes.shape
    step = 128 if fmt == "fp8_block" else 64
    c = codes.view(E, R // 16, 16, B // step, step // 16, 16).permute(0, 1, 3, 4, 2, 5).contiguous().view(E, R, B)
    if fmt == "fp8_block":
        return c, scales
    S = scales.shape[2]
    return c, scales.view(E, R // 16, 16, S // 4, 4).permute(0, 1, 3, 2, 4).contiguous().view(E, R, S)


def _unpack(codes, scales, fmt):
    E, R, B = codes.shape
    step = 128 if fmt == "fp8_block" else 64
    c = codes.view(E, R // 16, B // step, step // 16, 16, 16).permute(0, 1, 4, 2, 3, 5).reshape(E, R, B)
    if fmt == "fp8_block":
        return c, scales
    S = scales.shape[2]
    return c, scales.view(E, R // 16, S // 4, 16, 4).permute(0, 1, 3, 2, 4).reshape(E, R, S)


def _weights(g, E, R, K, fmt):
    """Weights 0.02 * N(0, 1) in the stored format, made a few experts at a time."""
    n = max(1, (1 << 26) // (R * K))
    codes, scales = [], []
    for e in range(0, E, n):
        m = min(n, E - e)
        v = torch.randn(m, R, K, generator=g, device=DEV).mul_(0.02)
        if fmt == "fp8_block":
            b = v.view(m, R // 128, 128, K // 128, 128)
            s = b.abs().amax((2, 4)) / 448.0
            q = (b / s[:, :, None, :, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
            codes.append(q.view(torch.uint8).reshape(m, R, K))
            scales.append(s)
        else:
            b = v.view(m, R, K // 32, 32)
            ex = torch.frexp(b.abs().amax(3))[1] - 3          # largest magnitude in [4, 8) of the grid
            a = b * torch.exp2(-ex.float())[..., None]
            mag = torch.bucketize(a.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV),
                                  out_int32=True).to(torch.uint8)
            c = (mag | ((a < 0).to(torch.uint8) << 3)).view(m, R, K // 2, 2)
            codes.append(c[..., 0] | (c[..., 1] << 4))
            scales.append((ex + 127).to(torch.uint8))
    return torch.cat(codes), torch.cat(scales)


def _tail_inputs(c, g, s):
    T, H = c["T"], c["H"]
    s["r"] = torch.randn(T, H, generator=g, device=DEV).to(_DT[c["res"]])
    s["r_out"] = torch.empty_like(s["r"])
    param = _DT[c["param"]]
    s["w_post"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(param) if c["post"] else None
    rows = {"none": 0, "row": 1, "all": T}[c["gate"]]
    s["gate"] = torch.rand(rows, H, generator=g, device=DEV).to(param) if rows else None
    if rows == 1 and c["gate"] == "row":
        s["gate"] = s["gate"][0]
    s["w_next"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(param) if c["nxt"] else None
    s["n_next"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if c["nxt"] else None


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": c, "kept": {}}
    T, H, op = c["T"], c["H"], c["op"]
    if op in ("forward_few", "block_forward"):
        E, I = c["E"], c["I"]
        if op == "forward_few":
            s["x"] = torch.randn(T, H, generator=g, device=DEV).bfloat16()
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        else:
            _tail_inputs(c, g, s)
            s["w_pre"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(_DT[c["param"]])
        s["w_router"] = (0.02 * torch.randn(E, H, generator=g, device=DEV)).bfloat16()
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
        w13, w2 = _weights(g, E, 2 * I, H, c["fmt"]), _weights(g, E, H, I, c["fmt"])
        if c["layout"] == "packed":
            w13, w2 = _pack(*w13, c["fmt"]), _pack(*w2, c["fmt"])
        s["w13"], s["w2"] = w13, w2
    elif op == "block_norm":
        s["r"] = torch.randn(T, H, generator=g, device=DEV).to(_DT[c["res"]])
        s["w_pre"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(_DT[c["param"]])
        s["n"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    else:
        _tail_inputs(c, g, s)
        if op == "block_residual":
            s["y"] = (0.4 * torch.randn(T, H, generator=g, device=DEV)).to(_DT[c["y"]])
        else:
            k = c["k"]
            s["y_perm"] = 0.4 * torch.randn(T * k, H, generator=g, device=DEV)
            s["rows"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
            s["w"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------

def _fp8(v, fmt):
    """v rounded to FP8 with one scale per row per 128 channels, as the values the codes stand for."""
    b = v.view(v.shape[0], -1, 128)
    amax = b.abs().amax(2, keepdim=True)
    if fmt == "fp8_block":
        s = amax / 448.0
        q = (b / torch.where(amax > 0, s, torch.ones_like(s))).clamp(-448.0, 448.0)
    else:
        m, x = torch.frexp(amax)
        s = torch.exp2(torch.where(m <= 0.875, x - 9, x - 8).clamp(-126, 127).float())
        q = b / s
    return (q.to(torch.float8_e4m3fn).float() * s).view_as(v)


def _decode(codes, scales, fmt, layout):
    """Stored weights [n, R, ..] as float32 [n, R, K]."""
    if layout == "packed":
        codes, scales = _unpack(codes, scales, fmt)
    if fmt == "fp8_block":
        n, R, K = codes.shape
        v = codes.contiguous().view(torch.float8_e4m3fn).float().view(n, R // 128, 128, K // 128, 128)
        return v.mul_(scales[:, :, None, :, None]).view(n, R, K)
    n, R, B = codes.shape
    lut = torch.tensor(_MAG + [-v for v in _MAG], device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([lut[byte & 15], lut[byte >> 4]], 1)
    v = pair[codes.reshape(-1).int()].view(n, R, B // 16, 32)
    return v.mul_(torch.exp2(scales.float() - 127.0)[..., None]).view(n, R, 2 * B)


def _select(x, s):
    """Selected experts [T, k] and their weights; keys in 64 bits, rounded as the definition rounds them."""
    c = s["case"]
    L = (x.double() @ s["w_router"].double().T).float()
    base = (1.0 / (1.0 + torch.exp(-L.double()))).float() if c["score"] == "sigmoid" else L
    key = base if s["bias"] is None else base + s["bias"]
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    sel = base.gather(1, ids)
    if c["score"] != "sigmoid":
        sel = torch.exp(sel - sel.amax(1, keepdim=True))
    return ids, sel / sel.sum(1, keepdim=True)


def _moe(x, s):
    """The layer on x [T, H] bf16, in float32."""
    c = s["case"]
    T, k, I = c["T"], c["k"], c["I"]
    ids, w = _select(x, s)
    e = ids.reshape(-1)
    a = _fp8(x.float(), c["fmt"]).repeat_interleave(k, 0)
    (w13, s13), (w2, s2) = s["w13"], s["w2"]
    gu = torch.bmm(_decode(w13[e], s13[e], c["fmt"], c["layout"]), a[:, :, None])[:, :, 0]
    gate, up = gu[:, :I], gu[:, I:]
    h = _fp8((gate / (1.0 + torch.exp(-gate))) * up, c["fmt"])
    y = torch.bmm(_decode(w2[e], s2[e], c["fmt"], c["layout"]), h[:, :, None])[:, :, 0]
    return (y.view(T, k, -1) * w[:, :, None]).sum(1)


def _rms(v, w):
    n = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    return n if w is None else n * w.float()


def _residual(y, s):
    c = s["case"]
    z = _rms(y, s["w_post"]) if c["post"] else y
    if s["gate"] is not None:
        z = z * s["gate"].float()
    r = (s["r"].float() + c["scale"] * z).to(s["r"].dtype)
    return {"r": r, "n": _rms(r.float(), s["w_next"]).bfloat16()} if c["nxt"] else {"r": r}


def _plain(s):
    op = s["case"]["op"]
    if op == "forward_few":
        return _moe(s["x"], s).bfloat16()
    if op == "block_norm":
        return _rms(s["r"].float(), s["w_pre"]).bfloat16()
    if op == "block_residual":
        return _residual(s["y"].float(), s)
    if op == "combine_residual":
        T, k = s["w"].shape
        return _residual((s["y_perm"][s["rows"].long()].view(T, k, -1) * s["w"][:, :, None]).sum(1), s)
    # 64 bits: the layer's input is rounded to bf16, and a value next to a border can decide a selection
    return _residual(_moe(_rms(s["r"].double(), s["w_pre"]).bfloat16(), s), s)


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _kept(s):
    """What a program keeps between calls: the problem, the weights' handle and the workspace."""
    import sparse_moe_expert_route_amd as moe
    kept, c = s["kept"], s["case"]
    if not kept:
        layer = "E" in c
        p = moe.Problem.make(c["T"], c["H"], c["I"] if layer else 128, c["E"] if layer else 8, c.get("k", 1),
                             1 if c.get("score") == "sigmoid" else 0,
                             moe.EXPERTS_FP8_BLOCK if c.get("fmt") == "fp8_block" else moe.EXPERTS_MXFP4)
        kept["p"] = p
        if layer:
            kept["W"] = moe.ExpertWeights(*s["w13"], *s["w2"], moe.WEIGHTS_PACKED if c["layout"] == "packed"
                                          else moe.WEIGHTS_CANONICAL)
            kept["ws"] = moe.alloc_block_workspace(p, DEV)
        if "r_out" in s:
            kept["tail"] = moe.BlockTail(s["r"], s["r_out"], post_norm=c["post"], w_post=s["w_post"], gate=s["gate"],
                                         scale=c["scale"], eps=EPS, w_next=s["w_next"], n_next=s["n_next"])
    return moe, kept


def _own(s):
    moe, kept = _kept(s)
    op, p = s["case"]["op"], kept["p"]
    if op == "forward_few":
        moe.forward_few(p, s["x"], s["w_router"], s["bias"], kept["W"], s["y"], kept["ws"], moe.OUT_BF16)
        return s["y"]
    if op == "block_norm":
        moe.block_norm(p, s["r"], s["w_pre"], s["n"], EPS)
        return s["n"]
    if op == "block_residual":
        moe.block_residual(p, s["y"], kept["tail"])
    elif op == "combine_residual":
        moe.combine_residual(p, s["y_perm"], s["rows"], s["w"], kept["tail"])
    else:
        moe.block_forward(p, s["w_pre"], s["w_router"], s["bias"], kept["W"], kept["tail"], kept["ws"])
    return {"r": s["r_out"], "n": s["n_next"]} if s["case"]["nxt"] else {"r": s["r_out"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    T, H, op = c["T"], c["H"], c["op"]
    size = {"bf16": 2, "f32": 4}
    nbytes = flops = 0
    if op in ("forward_few", "block_forward"):
        E, I, k = c["E"], c["I"], c["k"]
        touched = E * (1.0 - (1.0 - k / E) ** T)          # expected distinct experts
        per = 3 * H * I * (17 / 32 if c["fmt"] == "mxfp4" else 1 + 4 / 16384)
        nbytes += touched * per + 2 * E * H + (4 * E if c["bias"] else 0)
        flops += T * k * 6 * H * I + 2 * T * E * H
        if op == "forward_few":
            nbytes += 4 * T * H
    if op == "block_norm":
        nbytes += T * H * (size[c["res"]] + 2) + H * size[c["param"]]
        flops += 4 * T * H
    if op == "combine_residual":
        nbytes += T * c["k"] * (4 * H + 8)
        flops += 2 * T * c["k"] * H
    if op == "block_residual":
        nbytes += T * H * size[c["y"]]
    if op in ("block_residual", "combine_residual", "block_forward"):
        p = size[c["param"]]
        nbytes += 2 * T * H * size[c["res"]] + H * p * (c["post"] + c["nxt"] + (op == "block_forward"))
        nbytes += {"none": 0, "row": 1, "all": T}[c["gate"]] * H * p + (2 * T * H if c["nxt"] else 0)
        flops += 10 * T * H
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _round_e4m3(v):
    """float64 values rounded to the e4m3 grid (half to even), |v| <= 448."""
    a = v.abs().clamp(max=448.0)
    ex = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(ex - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _q64(v, fmt):
    out = torch.empty_like(v)
    for b in range(0, v.shape[1], 128):
        blk = v[:, b:b + 128]
        amax = blk.abs().amax(1, keepdim=True)
        if fmt == "fp8_block":
            sc = (amax.float() / 448.0).double()
        else:
            sc = torch.exp2(torch.ceil(torch.log2(amax.clamp(min=2.0 ** -110) / 448.0)))
        sc = torch.where(amax > 0, sc, torch.ones_like(sc))
        out[:, b:b + 128] = _round_e4m3(blk / sc) * sc
    return out


def _w64(codes, scales, fmt, layout):
    """One expert's stored matrix in float64 [R, K]."""
    if layout == "packed":
        R, B = codes.shape
        step = 128 if fmt == "fp8_block" else 64
        codes = codes.view(R // 16, B // step, step // 16, 16, 16).permute(0, 3, 1, 2, 4).reshape(R, B)
        if fmt != "fp8_block":
            scales = scales.view(R // 16, -1, 16, 4).permute(0, 2, 1, 3).reshape(R, -1)
    if fmt == "fp8_block":
        v = codes.contiguous().view(torch.float8_e4m3fn).double()
        return v * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    mag = torch.tensor(_MAG, dtype=torch.float64, device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).long()
    v = mag[nib & 7] * (1 - 2 * (nib >> 3)).double()
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _moe64(x, s):
    c = s["case"]
    T, k, I = c["T"], c["k"], c["I"]
    L = x @ s["w_router"].double().T
    base = torch.sigmoid(L) if c["score"] == "sigmoid" else L
    key = base.float() if s["bias"] is None else base.float() + s["bias"]
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    w = base.gather(1, order)
    w = w / w.sum(1, keepdim=True) if c["score"] == "sigmoid" else torch.softmax(w, 1)
    a = _q64(x, c["fmt"])
    y = torch.zeros(T, k, c["H"], dtype=torch.float64, device=x.device)
    for e in sorted(set(order.reshape(-1).tolist())):
        t, j = torch.nonzero(order == e, as_tuple=True)
        gu = a[t] @ _w64(s["w13"][0][e], s["w13"][1][e], c["fmt"], c["layout"]).T
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y[t, j] = _q64(h, c["fmt"]) @ _w64(s["w2"][0][e], s["w2"][1][e], c["fmt"], c["layout"]).T
    return (y * w[:, :, None]).sum(1)


def _norm64(v, w):
    n = v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)
    return n if w is None else n * w.double()


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    if op == "forward_few":
        return _moe64(s["x"].double(), s)
    if op == "block_norm":
        return _norm64(s["r"].double(), s["w_pre"])
    r = s["r"].double()
    if op == "block_residual":
        y = s["y"].double()
    elif op == "combine_residual":
        y = torch.zeros_like(r)
        rows = s["rows"].view(s["w"].shape).long()
        for j in range(s["w"].shape[1]):
            y += s["w"][:, j:j + 1].double() * s["y_perm"][rows[:, j]].double()
    else:
        # the layer takes the normalised input in bf16
        y = _moe64(_norm64(r, s["w_pre"]).bfloat16().double(), s)
    z = _norm64(y, s["w_post"]) if c["post"] else y
    if s["gate"] is not None:
        z = z * s["gate"].double()
    r = r + c["scale"] * z
    return {"r": r, "n": _norm64(r, s["w_next"])} if c["nxt"] else {"r": r}
