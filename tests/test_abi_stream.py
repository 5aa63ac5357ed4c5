"""Host-side checks of the residual norm, the sorted rows, the 4-bit
matrix-vector product and the forward of quantized tokens: the documented
statuses come back without a GPU."""
import ctypes
import os

import pytest

import block_scaled_expert_amd as bse

P = ctypes.c_void_p(0x100000)
AT = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bse.LIB_PATH):
        from block_scaled_expert_amd import build
        build.build()
    return bse.load()


def test_group_matvec_arguments(lib):
    base = dict(glu=None, fmt=1, xt=0, x=P, rows=8, ids=None, div=1, M=8, w=P, sc=P, gs=P, group=1, stride=1, G=2, N=64, K=128,
                off=P, ot=0, out=P)

    def call(**kw):
        v = {**base, **kw}
        glu = None if v["glu"] is None else ctypes.byref(v["glu"])
        return lib.moe_group_matvec(glu, v["fmt"], v["xt"], v["x"], v["rows"], v["ids"], v["div"], v["M"], v["w"], v["sc"],
                                    v["gs"], v["group"], v["stride"], v["G"], v["N"], v["K"], v["off"], v["ot"], v["out"], None)

    for fmt in (0, 2, 3, 5):
        assert call(fmt=fmt) == -5
    odd = AT(0x100008)
    for kw in (dict(xt=2), dict(ot=-1), dict(M=-1), dict(M=(1 << 26) + 1), dict(rows=-1), dict(rows=0), dict(G=0), dict(G=1025),
               dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=48), dict(K=1 << 21), dict(ids=P, div=0), dict(x=None),
               dict(w=None), dict(sc=None), dict(off=None), dict(out=None), dict(gs=None), dict(group=0), dict(group=3),
               dict(group=2, stride=1), dict(x=odd), dict(w=odd), dict(out=odd), dict(sc=AT(0x100002)), dict(gs=AT(0x100001)),
               dict(off=AT(0x100002)), dict(ids=AT(0x100002)), dict(M=1 << 26, N=1 << 10)):
        assert call(**kw) == -1, kw
    glu = bse.Config(cap=7.0).c()
    assert call(glu=glu, N=63) == -1
    glu.cap = 0.0
    assert call(glu=glu) == -1
    glu.cap_form = 4
    assert call(glu=glu) == -1
    assert call(M=0, x=None, w=None, out=None) == 0
    # MXFP4 has no fp32 scale: a bad one is not looked at
    assert call(fmt=4, M=0, gs=None, group=0, stride=0) == 0


def test_norm_arguments(lib):
    def fwd(cfg=None, dt=0, x=P, rt=0, res=P, T=4, cols=64, w=P, eps=1e-6, ro=P, y=P, rstd=P, codes=None, sc=None, gs=None):
        return lib.moe_norm_forward(None if cfg is None else ctypes.byref(cfg), dt, x, rt, res, T, cols, w, eps, ro, y, rstd,
                                    codes, sc, gs, None)

    inf, nan = float("inf"), float("nan")
    for kw in (dict(dt=2), dict(rt=-1), dict(dt=1, rt=0), dict(T=-1), dict(T=(1 << 21) + 1), dict(cols=0), dict(cols=65537),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=inf), dict(eps=nan), dict(x=None), dict(w=None), dict(y=None),
               dict(codes=P), dict(sc=P), dict(gs=P), dict(x=AT(0x100001)), dict(y=AT(0x100001)), dict(res=AT(0x100001)),
               dict(rt=1, res=AT(0x100002)), dict(rt=1, ro=AT(0x100002)), dict(w=AT(0x100002)), dict(rstd=AT(0x100002))):
        assert fwd(**kw) == -1, kw
    assert fwd(T=0, x=None) == 0
    nv, mx = bse.Config(fmt="nvfp4").c(), bse.Config(fmt="mxfp8").c()
    enc = dict(codes=P, sc=P, gs=P)
    for kw in (dict(cfg=mx), dict(cfg=mx, codes=P), dict(cfg=nv, codes=P, sc=P), dict(cfg=mx, cols=48, **enc),
               dict(cfg=mx, **{**enc, "codes": AT(0x100008)}), dict(cfg=mx, x=AT(0x100008), **enc),
               dict(cfg=mx, y=AT(0x100008), **enc), dict(cfg=mx, res=AT(0x100008), **enc), dict(cfg=mx, ro=AT(0x100008), **enc),
               dict(cfg=mx, w=AT(0x100008), **enc), dict(cfg=nv, **{**enc, "gs": AT(0x100002)}),
               dict(cfg=bse.Config(fmt="nvfp4", act_gs=1).c(), **enc), dict(cfg=bse.Config(top_k=0).c(), **enc)):
        assert fwd(**kw) == -1, kw
    bad = bse.Config(fmt="mxfp8").c()
    bad.fmt = 3
    assert fwd(cfg=bad, **enc) == -5

    n = ctypes.c_size_t(0)
    size = lib.moe_norm_workspace_size
    assert size(4, 64, ctypes.byref(n)) == 0 and n.value >= 4 * 64 * 4
    assert size(-1, 64, ctypes.byref(n)) == -1 and size(4, 0, ctypes.byref(n)) == -1 and size(4, 64, None) == -1
    assert size(4, 64, ctypes.byref(n)) == 0

    def bwd(dt=0, dy=P, rt=0, res=P, dn=P, T=4, cols=64, w=P, rstd=P, dr=P, dx=P, dw=P, ws=P, nb=n.value):
        return lib.moe_norm_backward(dt, dy, rt, res, dn, T, cols, w, rstd, dr, dx, dw, ws, nb, None)

    for kw in (dict(dt=2), dict(rt=2), dict(dt=1, rt=0), dict(T=-1), dict(cols=0), dict(dy=None), dict(res=None), dict(w=None),
               dict(rstd=None), dict(dr=None), dict(ws=None), dict(ws=AT(0x100080)), dict(dw=AT(0x100002)), dict(dy=AT(0x100001)),
               dict(rt=1, dr=AT(0x100002)), dict(rt=1, dn=AT(0x100002)), dict(dx=AT(0x100001)), dict(rstd=AT(0x100002))):
        assert bwd(**kw) == -1, kw
    assert bwd(nb=n.value - 1) == -3
    assert bwd(T=0, dw=None, ws=None, nb=0) == 0


def test_rows_arguments(lib):
    def sort(dt=0, x=P, T=4, k=2, cols=64, pos=P, M=8, out=P):
        return lib.moe_sort_rows(dt, x, T, k, cols, pos, M, out, None)

    def sort_back(dt=0, d=P, M=8, pos=P, T=4, k=2, cols=64, dx=P):
        return lib.moe_sort_rows_backward(dt, d, M, pos, T, k, cols, dx, None)

    def combine(yt=0, y=P, M=8, pos=P, w=P, T=4, k=2, cols=64, ot=0, out=P):
        return lib.moe_combine_rows(yt, y, M, pos, w, T, k, cols, ot, out, None)

    def back(ot=0, d=P, yt=0, y=P, M=8, pos=P, w=P, T=4, k=2, cols=64, dy=P, dw=P):
        return lib.moe_combine_rows_backward(ot, d, yt, y, M, pos, w, T, k, cols, dy, dw, None)

    for f in (sort, sort_back, combine, back):
        for kw in (dict(T=-1), dict(T=(1 << 21) + 1), dict(k=0), dict(k=33), dict(cols=0), dict(cols=65537), dict(M=-1),
                   dict(M=(1 << 26) + 1), dict(pos=None), dict(pos=AT(0x100002))):
            assert f(**kw) == -1, (f, kw)
        assert f(T=0) == 0
    for kw in (dict(dt=2), dict(x=None), dict(out=None), dict(x=AT(0x100001)), dict(dt=1, out=AT(0x100002))):
        assert sort(**kw) == -1, kw
    assert sort(M=0, out=None) == 0                    # no row is local
    for kw in (dict(dt=2), dict(d=None), dict(dx=None), dict(d=AT(0x100001)), dict(dt=1, dx=AT(0x100002))):
        assert sort_back(**kw) == -1, kw
    for kw in (dict(yt=2), dict(ot=2), dict(y=None), dict(out=None), dict(yt=1, y=AT(0x100002)), dict(out=AT(0x100001)),
               dict(w=AT(0x100002))):
        assert combine(**kw) == -1, kw
    for kw in (dict(yt=2), dict(ot=2), dict(d=None), dict(y=None), dict(dy=None, dw=None), dict(d=AT(0x100001)),
               dict(yt=1, y=AT(0x100002)), dict(yt=1, dy=AT(0x100002)), dict(dw=AT(0x100002)), dict(w=AT(0x100002))):
        assert back(**kw) == -1, kw


def test_forward_quantized_arguments(lib):
    cfg = bse.Config(fmt="mxfp8", max_tokens=64)
    cc, n = cfg.c(), bse.workspace_size(cfg)
    w = bse.CWeights(0x4000, 0x5000, 0x6000, 0x7000, None, 0)

    def call(codes=P, sc=P, gs=None, T=8, ids=P, tw=P, weights=w, out=P, ws=P, nb=n, c=cc):
        return lib.moe_forward_quantized(ctypes.byref(c), codes, sc, gs, T, ids, tw, ctypes.byref(weights), out, ws, nb, None,
                                         None)

    for kw in (dict(codes=None), dict(sc=None), dict(T=-1), dict(ids=None), dict(tw=None), dict(out=None), dict(ws=None),
               dict(codes=AT(0x100008)), dict(sc=AT(0x100008)), dict(out=AT(0x100008))):
        assert call(**kw) == -1, kw
    assert call(T=65) == -4 and call(nb=n - 1) == -3 and call(T=0, codes=None) == 0
    nv = bse.Config(fmt="nvfp4", max_tokens=64)
    wn = bse.CWeights(0x4000, 0x5000, 0x6000, 0x7000, 0x8000, 0)
    nn = bse.workspace_size(nv)
    assert call(c=nv.c(), weights=wn, nb=nn, gs=None) == -1
    assert call(c=nv.c(), weights=wn, nb=nn, gs=AT(0x100002)) == -1


def test_config_holds_its_fields_alone():
    """The structure that a call took leaves no trace in the Config, its copies
    and pickles, and follows the fields."""
    import copy
    import dataclasses
    import pickle

    import block_scaled_expert_amd as bse
    cfg = bse.Config(top_k=4)
    before = dict(vars(cfg))
    assert cfg.ref()._obj.top_k == 4 and cfg.ref() is cfg.ref()
    assert vars(cfg) == before and bse.Config(**vars(cfg)) == cfg == dataclasses.replace(cfg)
    for twin in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
        assert twin == cfg
        twin.top_k = 2
        assert twin.ref()._obj.top_k == 2 and cfg.ref()._obj.top_k == 4
    cfg.top_k = 3
    assert cfg.ref()._obj.top_k == 3
    cfg.act_gs_static = [1.0, 1.0]
    cfg.ref()
    cfg.act_gs_static[0] = 2.0
    assert cfg.ref()._obj.act_gs_static[0] == 2.0
