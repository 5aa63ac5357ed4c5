"""Host-side checks of the MXFP4 format, the grouped product and the balance
loss: the documented statuses come back without a GPU; and the oracle's own
pins for them."""
import ctypes
import os

import numpy as np
import pytest

import block_scaled_expert_amd as bse
from oracle import balance as B
from oracle import formats as F

P = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bse.LIB_PATH):
        from block_scaled_expert_amd import build
        build.build()
    return bse.load()


def _cfg(**kw):
    return bse.Config(**{**dict(fmt="mxfp4", max_tokens=64), **kw}).c()


def test_mxfp4_config(lib):
    cc = _cfg()
    assert lib.moe_validate_config(ctypes.byref(cc)) == 0
    cc.fmt = 3
    assert lib.moe_validate_config(ctypes.byref(cc)) == -5
    # a quantized row: half a byte and 1/32 byte of scale per element; [gate | up] in fp32 between the products
    sizes = {f: bse.workspace_size(bse.Config(fmt=f, max_tokens=1024)) for f in ("mxfp8", "mxfp4")}
    assert sizes["mxfp4"] - sizes["mxfp8"] == 8192 * 2 * 2304 * 4 - 8192 * 2304 // 2 - 1024 * 4608 // 2
    # canonical weights only
    w = bse.CWeights(0x4000, 0x5000, 0x6000, 0x7000, None, 0)
    d = bse.CWeights(0x14000, 0x15000, 0x16000, 0x17000, None, 0)
    cc = _cfg()
    assert lib.moe_prepare_weights(ctypes.byref(cc), ctypes.byref(w), ctypes.byref(d), None) == -5
    w.layout = 1
    n = bse.workspace_size(bse.Config(fmt="mxfp4", max_tokens=64))
    assert lib.moe_forward(ctypes.byref(cc), P, 8, P, P, ctypes.byref(w), P, P, n, None, None) == -1


def test_group_product_arguments(lib):
    base = dict(fmt=4, a=P, a_sc=P, a_rows=8, ids=None, div=1, M=8, w=P, w_sc=P, G=2, N=64, K=128, off=P, dt=0, out=P)

    def call(**kw):
        v = {**base, **kw}
        return lib.moe_group_product(v["fmt"], v["a"], v["a_sc"], v["a_rows"], v["ids"], v["div"], v["M"], v["w"],
                                     v["w_sc"], v["G"], v["N"], v["K"], v["off"], v["dt"], v["out"], None)

    for fmt in (0, 1, 2, 3, 5):
        assert call(fmt=fmt) == -5
    odd = ctypes.c_void_p(0x100008)
    for kw in (dict(dt=2), dict(M=-1), dict(a_rows=-1), dict(a_rows=0), dict(G=0), dict(G=1025), dict(N=0), dict(K=0),
               dict(K=48), dict(K=-32), dict(K=1 << 21), dict(N=(1 << 20) + 1), dict(ids=P, div=0), dict(a=None),
               dict(a_sc=None), dict(w=None), dict(w_sc=None), dict(off=None), dict(out=None), dict(a=odd),
               dict(w=odd), dict(out=odd), dict(off=ctypes.c_void_p(0x100002)), dict(M=(1 << 26) + 1)):
        assert call(**kw) == -1, kw
    assert call(M=0, a=None, w=None, out=None) == 0


def test_balance_arguments(lib):
    cc = _cfg(num_experts=64, top_k=4)
    r = ctypes.byref(cc)
    n = ctypes.c_size_t(0)
    assert lib.moe_balance_workspace_size(r, 100, 1, None) == -1
    assert lib.moe_balance_workspace_size(r, -1, 1, ctypes.byref(n)) == -1
    assert lib.moe_balance_workspace_size(r, 100, 0, ctypes.byref(n)) == -1
    assert lib.moe_balance_workspace_size(r, 100, 65536, ctypes.byref(n)) == -1
    assert lib.moe_balance_workspace_size(None, 100, 1, ctypes.byref(n)) == -1
    assert lib.moe_balance_workspace_size(r, 100, 3, ctypes.byref(n)) == 0 and n.value > 0

    def fwd(dt=1, z=P, T=100, ids=P, off=P, S=3, mask=None, counts=P, live=P, probs=P, loss=P, ws=P, nb=n.value):
        return lib.moe_balance_forward(r, dt, z, T, ids, off, S, mask, counts, live, probs, loss, ws, nb, None)

    odd = ctypes.c_void_p(0x100002)
    for kw in (dict(dt=2), dict(z=None), dict(T=-1), dict(ids=None), dict(off=None), dict(S=0), dict(counts=None),
               dict(live=None), dict(probs=None), dict(loss=None), dict(ws=None), dict(z=odd), dict(ids=odd),
               dict(ws=ctypes.c_void_p(0x100080)), dict(T=(1 << 26) + 1)):
        assert fwd(**kw) == -1, kw
    assert fwd(nb=n.value - 1) == -3

    def bwd(dt=1, z=P, T=100, ids=P, off=P, S=3, mask=None, counts=P, live=P, dl=P, dw=P, dz=P):
        return lib.moe_balance_backward(r, dt, z, T, ids, off, S, mask, counts, live, dl, dw, dz, None)

    for kw in (dict(dt=2), dict(z=None), dict(T=-1), dict(ids=None), dict(off=None), dict(counts=None),
               dict(live=None), dict(dl=None), dict(dz=None), dict(dz=odd), dict(S=0)):
        assert bwd(**kw) == -1, kw
    assert bwd(T=0, z=None, dz=None) == 0
    for kw in (dict(num_experts=0), dict(num_experts=1025), dict(num_experts=3, top_k=4), dict(top_k=0),
               dict(top_k=33)):
        bad = _cfg(**{**dict(num_experts=64, top_k=4), **kw})
        assert lib.moe_balance_workspace_size(ctypes.byref(bad), 100, 1, ctypes.byref(n)) == -1, kw


def test_route_logits_arguments(lib):
    cc = _cfg()
    r, n = ctypes.byref(cc), bse.workspace_size(bse.Config(fmt="mxfp4", max_tokens=64))
    assert lib.moe_route_logits(r, 65, P, n, P, None) == -4
    assert lib.moe_route_logits(r, -1, P, n, P, None) == -1
    assert lib.moe_route_logits(r, 8, None, n, P, None) == -1
    assert lib.moe_route_logits(r, 8, P, n - 1, P, None) == -3
    assert lib.moe_route_logits(r, 8, P, n, None, None) == -1
    assert lib.moe_route_logits(r, 0, P, n, None, None) == 0


# -- the oracle's pins --------------------------------------------------------

def test_oracle_mxfp4_is_nearest():
    """Every element's code is a nearest grid value, ties to the even code, and
    the scale puts the block's maximum in [4, 8)."""
    g = np.random.default_rng(0)
    v = (g.standard_normal((40, 64)) * np.exp(g.uniform(-30, 30, (40, 1)))).astype(np.float32)
    c, s = F.quantize_mxfp4(v)
    back = F.dequantize_mxfp4(c, s)
    step = np.ldexp(1.0, s.astype(np.int64) - 127)[..., None]
    q = v.reshape(40, 2, 32).astype(np.float64) / step
    top = np.abs(q).max(-1)
    assert ((top >= 4) & (top < 8)).all()
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    grid = np.concatenate([-grid[:0:-1], grid])
    best = np.abs(q[..., None] - grid).min(-1)
    assert np.array_equal(np.abs(back.reshape(40, 2, 32) / step - q), best)
    ties = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4], np.float32)
    c, s = F.quantize_mxfp4(ties)
    assert s[0, 0] == 127
    assert np.array_equal(F.dequantize_mxfp4(c, s)[0, :8], [0, 1, 1, 2, 2, 4, 4, 6])


def test_oracle_balance_closed_forms():
    """Balanced routing under equal logits gives loss 1; the gradient over a
    row of softmax-like shares sums to what the formula's factors give; the
    gradient matches differences."""
    E, k, T = 8, 2, 8
    z = np.full((T, E), -0.3)
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    f = B.balance_forward(z, ids, E, k)
    assert np.allclose(f["loss"], 1.0, rtol=1e-14) and (f["counts"] == T * k // E).all()
    g = np.random.default_rng(3)
    z = g.standard_normal((T, E)) * 2
    d_w, bounds, mask = g.standard_normal((T, k)), [0, 3, 3, T], np.array([1, 0, 1, 1, 1, 1, 0, 1])
    for norm, scale in ((True, 1.0), (True, 2.0), (False, 0.5)):
        f = B.balance_forward(z, ids, E, k, bounds, mask)
        d_loss = np.array([0.7, 1.1, 1.9])
        dz, _ = B.balance_backward(z, ids, f, d_loss, E, k, bounds, mask, d_w, norm, scale)
        at = lambda zz: B.balance_loss(zz, ids, d_loss, E, k, f["counts"], bounds, mask, d_w, norm, scale)  # noqa: E731
        h = 1e-6
        num = np.zeros_like(z)
        for i in np.ndindex(z.shape):
            up, dn = z.copy(), z.copy()
            up[i] += h
            dn[i] -= h
            num[i] = (at(up) - at(dn)) / (2 * h)
        assert np.abs(num - dz).max() <= 1e-8
        assert (dz[mask == 0] == 0).all()
        total = float((f["loss"] * d_loss).sum())
        only = B.balance_loss(z, ids, d_loss, E, k, f["counts"], bounds, mask)
        assert abs(total - only) <= 1e-12 * abs(total)


def test_decode_arguments(lib):
    """moe_decode_weights: what its vector accesses need is refused otherwise."""
    def call(fmt=4, codes=P, scales=P, gs=P, out=P, rows=2, cols=64):
        return lib.moe_decode_weights(fmt, codes, scales, gs, 1, 1, 1, rows, cols, out, None)

    at = ctypes.c_void_p
    for kw in (dict(out=at(0x100004)), dict(out=at(0x100008)), dict(codes=at(0x100004)), dict(out=None),
               dict(codes=None), dict(scales=None), dict(cols=48), dict(rows=0)):
        assert call(**kw) == -1, kw
    assert call(fmt=3) == -5
