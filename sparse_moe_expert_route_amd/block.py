"""The decoder block around the routed layer, and the layer's form for few tokens.

Python binding of ``include/moe_block.h``, in the manner of the package's other
calls: tensors are checked, device pointers and a HIP stream are passed to the
library, a status other than MOE_OK raises ``MoeError``.  Names follow the C ABI:
``block_norm``, ``block_residual``, ``combine_residual``, ``forward_few``,
``block_forward``.

Work goes to ``stream`` (a ``torch.cuda.Stream``; by default the current stream
of the tensors' device).  Every tensor of a call lies on one device, which need
not be the current one.
"""

import ctypes

import torch

import sparse_moe_expert_route_amd as _moe

__all__ = ["BlockTail", "FEW_MAX_TOKENS", "BLOCK_MAX_HIDDEN", "DEVERR_STALLED", "block_workspace_size", "alloc_block_workspace",
           "block_norm", "block_residual", "combine_residual", "forward_few", "block_forward",
           "EXPORTED_BLOCK_SYMBOLS"]

FEW_MAX_TOKENS = 16        # MOE_FEW_MAX_TOKENS of moe_block.h
BLOCK_MAX_HIDDEN = 16384   # MOE_BLOCK_MAX_HIDDEN
DEVERR_STALLED = 8         # MOE_DEVERR_STALLED

EXPORTED_BLOCK_SYMBOLS = ["moe_block_workspace_size", "moe_block_norm", "moe_block_residual", "moe_combine_residual",
                          "moe_forward_few", "moe_block_forward"]

_DTYPES = {torch.float32: _moe.OUT_F32, torch.bfloat16: _moe.OUT_BF16}


class _Tail(ctypes.Structure):
    _fields_ = [("r", ctypes.c_void_p), ("r_out", ctypes.c_void_p), ("w_post", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("w_next", ctypes.c_void_p), ("n_next", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("res_dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("gate_per_token", ctypes.c_int32)]


_lib = None
_fns = {}

# the current stream's handle and the current device, without building their Python objects (a call on
# a decode batch is bound by what happens on the host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _load():
    """The library with the signatures of moe_block.h set."""
    global _lib
    L = _moe.load()
    if _lib is L:
        return L
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    P, W, B = ctypes.POINTER(_moe.Problem), ctypes.POINTER(_moe._Weights), ctypes.POINTER(_Tail)
    L.moe_block_workspace_size.restype = sz
    L.moe_block_workspace_size.argtypes = [P]
    L.moe_block_norm.argtypes = [P, vp, i32, vp, i32, f32, vp, vp]
    L.moe_block_residual.argtypes = [P, vp, i32, B, vp]
    L.moe_combine_residual.argtypes = [P, vp, vp, vp, B, vp]
    L.moe_forward_few.argtypes = [P, vp, vp, vp, W, vp, i32, vp, sz, vp]
    L.moe_block_forward.argtypes = [P, vp, vp, vp, W, B, vp, sz, vp]
    for name in EXPORTED_BLOCK_SYMBOLS[1:]:
        getattr(L, name).restype = ctypes.c_int
        _fns[name] = getattr(L, name)
    _lib = L
    return L


def _code(t, name):
    """moe_out_dtype of a float32 or bfloat16 tensor."""
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return code


def _check(t, shape, name, device, dtype=None):
    if dtype is not None and t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.get_device() != device:
        raise ValueError("%s must be on the device of the call's other tensors" % name)


def _device(t, name):
    if t is None:
        raise ValueError("%s is required" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.get_device()


def _p(t):
    return None if t is None else t.data_ptr()


def _call(fn, device, stream, *args):
    """fn(*args, stream) with the tensors' device current; raises MoeError on a status."""
    if _lib is None:
        _load()
    f = _fns[fn]
    if stream is None:
        s = _raw_stream(device)
    elif stream.device_index == device:
        s = stream.cuda_stream
    else:
        raise ValueError("stream must be a stream of the tensors' device")
    if _current_device() == device:
        st = f(*args, s)
    else:
        with torch.cuda.device(device):
            st = f(*args, s)
    if st:
        _moe._raise(fn, st)


class BlockTail:
    """What follows the layer: r_out = r + scale * gate * z with z = RMSNorm(y; w_post)
    (post_norm) or y, and n_next = RMSNorm(r_out; w_next).

    r, r_out [T, H] float32 or bfloat16 (r_out may be r); w_post, w_next [H], gate [H] or
    [T, H], all of one type, float32 or bfloat16, or None (ones); n_next [T, H] bfloat16 or
    None (not computed)."""

    def __init__(self, r, r_out, post_norm=True, w_post=None, gate=None, scale=1.0, eps=1e-6, w_next=None,
                 n_next=None):
        self.r, self.r_out, self.post_norm, self.w_post, self.gate = r, r_out, bool(post_norm), w_post, gate
        self.scale, self.eps, self.w_next, self.n_next = float(scale), float(eps), w_next, n_next

    def struct(self, p, device, param=None):
        """Checked arguments as moe_block_tail; `param`: a further parameter whose type the others share."""
        T, H = p.num_tokens, p.hidden
        res = _code(self.r, "r")
        _check(self.r, (T, H), "r", device)
        _check(self.r_out, (T, H), "r_out", device, self.r.dtype)
        per_token = 0
        dt = None if param is None else param.dtype
        for t, name in ((self.w_post, "w_post"), (self.gate, "gate"), (self.w_next, "w_next")):
            if t is None:
                continue
            if dt is None:
                dt = t.dtype
            shape = (H,)
            if name == "gate" and t.dim() == 2:
                shape, per_token = (T, H), 1
            _check(t, shape, name, device, dt)
        code = _moe.OUT_F32 if dt is None else _DTYPES.get(dt)
        if code is None:
            raise ValueError("w_post, gate and w_next must be float32 or bfloat16, got %s" % dt)
        if self.n_next is not None:
            _check(self.n_next, (T, H), "n_next", device, torch.bfloat16)
        return _Tail(_p(self.r), _p(self.r_out), _p(self.w_post), _p(self.gate), _p(self.w_next), _p(self.n_next),
                     self.scale, self.eps, res, code, int(self.post_norm), per_token)


def block_workspace_size(p):
    """Bytes of workspace for forward_few and block_forward (and for the package's other calls) on problem p."""
    n = _load().moe_block_workspace_size(ctypes.byref(p))
    if n == 0:
        raise _moe.MoeError("moe_block_workspace_size", 1, "invalid problem")
    return n


def alloc_block_workspace(p, device="cuda"):
    return torch.empty(block_workspace_size(p), dtype=torch.uint8, device=device)


def block_norm(p, r, w, n, eps=1e-6, stream=None):
    """n [T, H] bfloat16 = RMSNorm(r; w): r [T, H] and w [H] float32 or bfloat16 each, w None for ones."""
    dev = _device(r, "r")
    shape = (p.num_tokens, p.hidden)
    _check(r, shape, "r", dev)
    _check(n, shape, "n", dev, torch.bfloat16)
    if w is not None:
        _check(w, (p.hidden,), "w", dev)
    _call("moe_block_norm", dev, stream, p, r.data_ptr(), _code(r, "r"), _p(w),
          _moe.OUT_F32 if w is None else _code(w, "w"), eps, n.data_ptr())


def block_residual(p, y, tail, stream=None):
    """The tail on a layer output y [T, H], float32 or bfloat16."""
    dev = _device(y, "y")
    _check(y, (p.num_tokens, p.hidden), "y", dev)
    _call("moe_block_residual", dev, stream, p, y.data_ptr(), _code(y, "y"), tail.struct(p, dev))


def combine_residual(p, y_perm, row_of_slot, topk_w, tail, stream=None):
    """The tail on the weighted sum of ``combine``, which is not stored."""
    dev = _device(y_perm, "y_perm")
    T, k = p.num_tokens, p.top_k
    _check(y_perm, (T * k, p.hidden), "y_perm", dev, torch.float32)
    _check(row_of_slot, (T * k,), "row_of_slot", dev, torch.int32)
    _check(topk_w, (T, k), "topk_w", dev, torch.float32)
    _call("moe_combine_residual", dev, stream, p, y_perm.data_ptr(), row_of_slot.data_ptr(), topk_w.data_ptr(),
          tail.struct(p, dev))


def _layer_args(p, dev, w_router, sel_bias, weights, ws):
    _check(w_router, (p.num_experts, p.hidden), "w_router", dev, torch.bfloat16)
    if sel_bias is not None:
        _check(sel_bias, (p.num_experts,), "sel_bias", dev, torch.float32)
    for t, (dt, shape), name in zip((weights.w13, weights.w13_scale, weights.w2, weights.w2_scale),
                                    _moe._weight_specs(p), ("w13", "w13_scale", "w2", "w2_scale")):
        _check(t, shape, name, dev, dt)
    _check(ws, (ws.numel(),), "workspace", dev, torch.uint8)


def forward_few(p, x, w_router, sel_bias, weights, y, ws, out_dtype=_moe.OUT_F32, stream=None):
    """``forward`` for at most FEW_MAX_TOKENS tokens, in fewer launches; ws from alloc_block_workspace."""
    dev = _device(x, "x")
    shape = (p.num_tokens, p.hidden)
    _check(x, shape, "x", dev, torch.bfloat16)
    _check(y, shape, "y", dev, torch.float32 if out_dtype == _moe.OUT_F32 else torch.bfloat16)
    _layer_args(p, dev, w_router, sel_bias, weights, ws)
    _call("moe_forward_few", dev, stream, p, x.data_ptr(), w_router.data_ptr(), _p(sel_bias), weights.struct(),
          y.data_ptr(), int(out_dtype), ws.data_ptr(), ws.numel())


def block_forward(p, w_pre, w_router, sel_bias, weights, tail, ws, stream=None):
    """The block on the residual stream tail.r: n = RMSNorm(r; w_pre), the layer on n, the tail.
    w_pre [H] of the tail's parameter type, or None (ones); ws from alloc_block_workspace."""
    dev = _device(tail.r, "r")
    if w_pre is not None:
        _check(w_pre, (p.hidden,), "w_pre", dev)
    _layer_args(p, dev, w_router, sel_bias, weights, ws)
    _call("moe_block_forward", dev, stream, p, _p(w_pre), w_router.data_ptr(), _p(sel_bias), weights.struct(),
          tail.struct(p, dev, w_pre), ws.data_ptr(), ws.numel())
