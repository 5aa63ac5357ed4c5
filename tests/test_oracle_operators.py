"""Pins of the oracle's MXFP4 quantizer and balance loss (CPU): exact-rational
search, invariants, torch's automatic gradient in float64."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import balance as B
from oracle import formats as F

MAGS = [Fraction(m) for m in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]


def _rows(seed, R=24, K=96):
    g = np.random.default_rng(seed)
    v = (g.standard_normal((R, K)) * np.exp(g.uniform(-25, 25, (R, 1)))).astype(np.float32)
    v[0] = 0.0
    v[1, :32] = np.float32(1e-45)
    v[2] = np.resize(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9], np.float32), K)
    v[3, 40] = np.float32(3.4e38)
    return v


def test_mxfp4_codes_are_nearest():
    """Scale by the definition and every code by search over the eight
    magnitudes, ties to the even code, in rationals."""
    v = _rows(0)
    codes, scales = F.quantize_mxfp4(v)
    nib = F.unpack_nibbles(codes)
    for r in range(v.shape[0]):
        for b in range(v.shape[1] // 32):
            block = [Fraction(float(x)) for x in v[r, 32 * b:32 * b + 32]]
            amax = max(abs(x) for x in block)
            E = -127
            if amax:
                E = 0
                while Fraction(2) ** (E + 1) <= amax:
                    E += 1
                while Fraction(2) ** E > amax:
                    E -= 1
                E = min(max(E - 2, -127), 127)
            assert int(scales[r, b]) == E + 127
            for j, x in enumerate(block):
                q = abs(x) / Fraction(2) ** E
                best = min(range(8), key=lambda c: (abs(MAGS[c] - q), c % 2))
                got = int(nib[r, 32 * b + j])
                assert got & 7 == best
                assert got >> 3 == int(np.signbit(v[r, 32 * b + j]))


def test_mxfp4_representable_is_lossless_and_error_bounded():
    g = np.random.default_rng(1)
    codes = g.integers(0, 256, (16, 64), dtype=np.uint8)
    codes[:, ::16] = 0x77                        # each block holds its largest magnitude
    scales = g.integers(10, 240, (16, 4), dtype=np.uint8)
    v = F.dequantize_mxfp4(codes, scales)
    c2, s2 = F.quantize_mxfp4(v.astype(np.float32))
    assert np.array_equal(F.dequantize_mxfp4(c2, s2), v) and np.array_equal(s2, scales)
    x = _rows(2)[4:]
    d = F.dequantize_mxfp4(*F.quantize_mxfp4(x)).reshape(-1, 32)
    x = x.astype(np.float64).reshape(-1, 32)
    amax = np.abs(x).max(1, keepdims=True)
    # a block's maximum is below 8 X: at most half the gap of 2 below 6, at most 2 above it
    assert (np.abs(d - x) <= amax / 4).all()


@pytest.mark.parametrize("norm,scale", [(True, 1.0), (True, 2.5), (False, 0.5)])
def test_balance_against_automatic_gradient(norm, scale):
    g = np.random.default_rng(3)
    T, E, k, bounds = 23, 14, 3, [0, 5, 5, 17, 23]
    z = g.standard_normal((T, E)) * 2
    ids = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    mask = (g.random(T) < 0.8).astype(np.uint8)
    mask[0] = 1
    d_w, d_loss = g.standard_normal((T, k)), np.linspace(0.5, 2, 4)
    ref = B.balance_forward(z, ids, E, k, bounds, mask)
    dz, _ = B.balance_backward(z, ids, ref, d_loss, E, k, bounds, mask, d_w, norm, scale)
    zt = torch.from_numpy(z).requires_grad_()
    s = torch.sigmoid(zt)
    p = s / s.sum(1, keepdim=True)
    sel = torch.gather(s, 1, torch.from_numpy(ids).long())
    w = scale * (sel / sel.sum(1, keepdim=True) if norm else sel)
    live = torch.from_numpy(mask.astype(np.float64))
    total = (w * torch.from_numpy(d_w) * live[:, None]).sum()
    for q in range(4):
        toks = [t for t in range(bounds[q], bounds[q + 1]) if mask[t]]
        count = np.bincount(ids[toks].reshape(-1), minlength=E) if toks else np.zeros(E, int)
        assert np.array_equal(count, ref["counts"][q]) and ref["live"][q] == len(toks)
        if toks:
            loss = E / (k * len(toks)) * (torch.from_numpy(count.astype(np.float64)) * p[toks].mean(0)).sum()
            assert abs(float(loss.detach()) - ref["loss"][q]) <= 1e-12 * ref["loss"][q]
            total = total + d_loss[q] * loss
        else:
            assert ref["loss"][q] == 0
    total.backward()
    # float64 on both sides: sums of a few dozen terms of order one
    assert np.abs(dz - zt.grad.numpy()).max() <= 1e-12
    assert (dz[mask == 0] == 0).all()


def test_balance_is_one_when_even():
    E, k = 8, 2
    z = np.zeros((16, E))
    ids = (np.arange(32).reshape(16, 2) % E).astype(np.int32)
    assert B.balance_forward(z, ids, E, k)["loss"][0] == pytest.approx(1.0, abs=1e-15)


def test_mxfp4_scale_255_is_nan():
    """E8M0 has no value 2^128: byte 255 is its NaN, for every code of the block."""
    codes = np.resize(np.arange(256, dtype=np.uint8), (3, 16))
    got = F.dequantize_mxfp4(codes, np.array([[254], [255], [0]], np.uint8))
    assert np.isnan(got[1]).all() and np.isfinite(got[[0, 2]]).all()
    assert np.abs(got[0]).max() == 6.0 * 2.0 ** 127
