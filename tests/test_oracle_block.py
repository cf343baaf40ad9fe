"""Pins of the block's oracle: closed forms, torch's own rounding, invariances."""

import numpy as np
import torch

from oracle import block as OB


def test_rms_norm_closed_forms():
    v = np.full((2, 128), -3.0)
    assert np.allclose(OB.rms_norm(v, eps=1e-30), -1.0, rtol=1e-15)
    assert np.all(OB.rms_norm(np.zeros((1, 128)), eps=1e-6) == 0)
    one = np.zeros((1, 256))
    one[0, 7] = 5.0
    n = OB.rms_norm(one, w=np.full(256, 2.0), eps=1e-30)
    assert np.isclose(n[0, 7], 2.0 * 16.0, rtol=1e-14) and np.count_nonzero(n) == 1


def test_rms_norm_is_scale_free_and_has_unit_rms():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(3, 384))
    a, b = OB.rms_norm(v, eps=1e-30), OB.rms_norm(1e3 * v, eps=1e-30)
    assert np.allclose(a, b, rtol=1e-12)
    assert np.allclose(np.mean(a * a, 1), 1.0, rtol=1e-12)


def test_residual_terms():
    rng = np.random.default_rng(1)
    r, y = rng.normal(size=(4, 128)), rng.normal(size=(4, 128))
    assert np.array_equal(OB.residual(r, y, post_norm=False, scale=0.0), r)
    assert np.allclose(OB.residual(r, y, post_norm=False, scale=0.5) - r, 0.5 * y, rtol=1e-12)
    g = rng.normal(size=128)
    per_token = OB.residual(r, y, gate=np.tile(g, (4, 1)))
    assert np.array_equal(per_token, OB.residual(r, y, gate=g))


def test_round_bf16_equals_torch():
    rng = np.random.default_rng(2)
    v = np.concatenate([rng.normal(size=4000) * np.exp2(rng.integers(-30, 30, 4000)), [0.0, -0.0, 1.00390625, -1.01171875]])
    v32 = v.astype(np.float32)
    ref = torch.from_numpy(v32).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    got = OB.round_bf16(v32.astype(np.float64))
    assert np.array_equal(got & 0x7FFF, ref & 0x7FFF) and np.array_equal(got[v32 != 0], ref[v32 != 0])
