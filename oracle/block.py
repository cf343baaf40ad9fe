"""The decoder block around the routed layer, step by step in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

  n  = RMSNorm(r; w_pre)                  the layer's input, rounded to bf16
  y  = the layer on n (``layer.forward``)
  z  = RMSNorm(y; w_post), or y
  r' = r + scale * gate * z
  n' = RMSNorm(r'; w_next)
  RMSNorm(v; w) = v * w / sqrt(mean(v^2) + eps), w = 1 where it is None
"""

import numpy as np

from . import layer as L

__all__ = ["rms_norm", "residual", "round_bf16", "block_forward"]


def rms_norm(v, w=None, eps=1e-6):
    v = np.asarray(v, dtype=np.float64)
    n = v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + float(np.float32(eps)))
    return n if w is None else n * np.asarray(w, dtype=np.float64)[None, :]


def residual(r, y, post_norm=True, w_post=None, gate=None, scale=1.0, eps=1e-6):
    """r' in float64 (not rounded)."""
    z = rms_norm(y, w_post, eps) if post_norm else np.asarray(y, dtype=np.float64)
    if gate is not None:
        g = np.asarray(gate, dtype=np.float64)
        z = z * (g if g.ndim == 2 else g[None, :])
    return np.asarray(r, dtype=np.float64) + float(np.float32(scale)) * z


def round_bf16(v):
    """float64 -> bf16 bits, to nearest, ties to even, in one rounding (normal range and below)."""
    v = np.asarray(v, dtype=np.float64)
    _, ex = np.frexp(v)
    step = np.exp2(np.maximum(ex, -125) - 8.0)         # spacing of bf16 around v (8 significant bits)
    q = (np.round(v / step) * step).astype(np.float32)  # exact: at most 8 significant bits
    return (q.view(np.uint32) >> 16).astype(np.uint16)


def block_forward(layer, r, w_pre=None, post_norm=True, w_post=None, gate=None, scale=1.0, eps=1e-6, n_bits=None):
    """(r' float64, n bf16 bits): the block on the residual stream r; ``n_bits`` overrides the layer's input."""
    n = round_bf16(rms_norm(r, w_pre, eps)) if n_bits is None else n_bits
    y = L.forward(dict(layer, x=n), keep_intermediates=False)["y"]
    return residual(r, y, post_norm, w_post, gate, scale, eps), n
