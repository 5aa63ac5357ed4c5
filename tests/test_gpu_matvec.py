"""moe_group_matvec against the float64 product of x and the decoded weights."""
import numpy as np
import pytest

from oracle import formats as F
from tests._util import to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _weights(g, fmt, G, N, K, mats):
    codes = g.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        return codes, g.integers(119, 123, (G, N, K // 32), dtype=np.uint8), None
    sc = g.integers(1, 0x7F, (G, N, K // 16), dtype=np.uint8)
    return codes, sc, (g.random((G, mats)) * 1e-3 + 1e-4).astype(np.float32)


def _values(fmt, codes, sc):
    """float64 values without the fp32 scale."""
    if fmt == "mxfp4":
        return F.dequantize_mxfp4(codes, sc)
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(nib & 8, -1.0, 1.0) * mag[nib & 7]
    return v * np.repeat(F.e4m3_decode(sc).astype(np.float64), 16, -1)


def _x(g, rows, K, dtype):
    """(tensor, float64 values) of rows of uneven size."""
    import torch
    v = (g.standard_normal((rows, K)) * np.exp(g.uniform(-2, 2, (rows, 1)))).astype(np.float32)
    v[:, ::11] *= 20
    t = torch.from_numpy(v).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    return t, t.double().cpu().numpy()


def _sizes(g, G, M, kind):
    if kind == "one":
        n = np.zeros(G, np.int64)
        n[G // 2] = M
        return n
    if kind == "even":
        return np.array([M // G + (i < M % G) for i in range(G)])
    return g.multinomial(M, g.dirichlet(np.full(G, 0.3)))


def _cap(form, c, g, u):
    """(h, |dh/dg|, |dh/du|) of the capped SwiGLU, the slopes as upper bounds."""
    if form == 0:
        g2, u2 = c * np.tanh(g / c), c * np.tanh(u / c)
    elif form == 1:
        g2, u2 = np.minimum(g, c), np.clip(u, -c, c)
    else:
        g2, u2 = g, u
    silu = g2 / (1 + np.exp(np.minimum(-g2, 700.0)))
    h = silu * u2
    if form == 2:
        h = c * np.tanh(h / c)
    return h, 1.1 * np.abs(u2), np.abs(silu)      # |silu'| < 1.1; the caps' slopes are at most 1


def _check(bse, g, fmt, dtype, out_dtype, G, M, N, K, kind, glu=None, div=0, x_rows=None):
    import torch
    mats = 2 if glu is not None else 1
    codes, sc, gs = _weights(g, fmt, G, N, K, mats)
    rows = M if x_rows is None else x_rows
    x, xv = _x(g, rows, K, dtype)
    offsets = np.concatenate([[0], np.cumsum(_sizes(g, G, M, kind))])
    ids = g.permutation(M) if div else None
    src = np.arange(M) if ids is None else ids // div
    cols = N // 2 if glu is not None else N
    out = torch.full((M + 3, cols), float("nan"), dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32, device="cuda")
    kw = {} if gs is None else dict(gs=to_dev(gs), gs_group=mats, gs_stride=mats)
    bse.group_matvec(fmt, x, to_dev(codes), to_dev(sc), to_dev(offsets.astype(np.int32)), out[:M], swiglu=glu,
                     row_ids=None if ids is None else to_dev(ids.astype(np.int32)), id_div=max(div, 1), **kw)
    got = out.double().cpu().numpy()
    assert np.isnan(got[M:]).all()
    # Products of bf16 parts and weights are exact.  Each matrix instruction adds 32 of k to the fp32 sum, by a
    # last place (2^-23) of the magnitudes at most; fp32 x takes three of them.
    rel = ((3 if dtype == "f32" else 1) * (K / 32 + 1) + 2) * 2.0 ** -23
    for i in range(G):
        lo, hi = offsets[i], offsets[i + 1]
        if lo == hi:
            continue
        wv = _values(fmt, codes[i], sc[i])
        if gs is not None:
            wv = wv * np.repeat(gs[i].astype(np.float64), N // mats)[:, None]
        xs = xv[src[lo:hi]]
        ref, size = xs @ wv.T, np.abs(xs) @ np.abs(wv).T
        tol = rel * size
        if glu is not None:
            h, dg, du = _cap(glu.cap_form, glu.cap, ref[:, :cols], ref[:, cols:])
            # the epilogue's own error: tanh 2e-6, of which silu and the product pass on 6 times that for the gate
            # (|g| silu'/silu grows to c - 1), the exponential and the reciprocal 2e-6
            tol = dg * tol[:, :cols] + du * tol[:, cols:] + 2e-5 * np.abs(h)
            ref = h
        if out_dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        bad = ~(np.abs(got[lo:hi] - ref) <= tol + 2.0 ** -126)
        assert not bad.any(), (i, np.argwhere(bad)[:4], got[lo:hi][bad][:4], ref[bad][:4], tol[bad][:4])
    return got


CASES = [
    # G, M, N, K, kind
    (1, 1, 1, 32, "even"), (1, 1, 64, 128, "even"), (1, 5, 17, 96, "even"), (1, 16, 200, 512, "even"),
    (1, 17, 130, 256, "even"), (3, 7, 64, 160, "uneven"), (5, 51, 1003, 352, "uneven"), (16, 40, 96, 2304, "uneven"),
    (48, 130, 256, 1184, "uneven"), (7, 70, 130, 640, "one"), (2, 200, 520, 768, "even"), (1, 33, 66, 4608, "even"),
    (1024, 60, 33, 64, "uneven"), (1, 2, 40, 20480, "even"), (1, 13, 40, 9248, "even"), (300, 2000, 70, 96, "uneven"),
    (64, 600, 1300, 64, "even"), (1, 2, 3, 262144, "even"), (1, 3, 70000, 64, "even"),
]


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("G,M,N,K,kind", CASES)
def test_product(gpu_lib, G, M, N, K, kind, fmt, dtype, out_dtype):
    _check(gpu_lib, np.random.default_rng(G * 7919 + M * 31 + N + K), fmt, dtype, out_dtype, G, M, N, K, kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("G,M,N,K,kind,glu", [
    # two and four sets of waves on the chunks; whole rows of chunks or not
    (8, 20, 1200, 1024, "uneven", False), (2, 9, 600, 1536, "uneven", True), (3, 9, 700, 800, "uneven", False),
    # many tiles a workgroup, 1 row a group
    (384, 400, 1500, 256, "uneven", False), (384, 450, 1800, 256, "uneven", True), (384, 420, 1500, 96, "uneven", False),
    # more rows: 16 at a time, in several panels, one and two tiles in turn
    (48, 300, 1100, 512, "uneven", False), (20, 100, 3000, 2304, "uneven", False), (24, 130, 2100, 1280, "uneven", True),
    (384, 1600, 1500, 256, "uneven", False), (30, 200, 1600, 1056, "one", False), (300, 1300, 1210, 160, "uneven", True),
])
def test_larger_calls(gpu_lib, G, M, N, K, kind, glu, fmt, dtype):
    _check(gpu_lib, np.random.default_rng(G * 7919 + M * 31 + N + K), fmt, dtype, "f32", G, M, N, K, kind,
           glu=gpu_lib.Config(cap=7.0) if glu else None)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("G,M,N,K,kind,glu,dtype", [
    # long rows in few groups: items of 4 fp32 rows in two and four sets of waves, two sets of 4 waves
    (1, 8, 4608, 3328, "even", False, "f32"), (1, 8, 4608, 3328, "even", True, "f32"), (1, 6, 600, 4608, "even", True, "f32"),
    (2, 9, 1100, 3360, "uneven", False, "f32"), (1, 8, 4600, 5120, "even", False, "bf16"), (1, 7, 4500, 5216, "even", True, "bf16"),
    # what x needs of LDS, in one panel and in several
    (2, 16, 4608, 1056, "even", False, "f32"), (1, 8, 16384, 3328, "even", False, "f32"), (3, 16, 5000, 1280, "uneven", True, "f32"),
])
def test_few_rows_of_long_groups(gpu_lib, G, M, N, K, kind, glu, dtype, fmt):
    _check(gpu_lib, np.random.default_rng(G * 7919 + M * 31 + N + K), fmt, dtype, "f32", G, M, N, K, kind,
           glu=gpu_lib.Config(cap=7.0) if glu else None)


@pytest.mark.parametrize("cap_form", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("G,M,N,K,kind", [(1, 1, 2, 32, "even"), (4, 9, 34, 96, "uneven"), (3, 40, 256, 512, "even"),
                                          (9, 20, 1006, 352, "uneven"), (2, 5, 130, 4608, "even")])
def test_swiglu(gpu_lib, G, M, N, K, kind, fmt, dtype, out_dtype, cap_form):
    cfg = gpu_lib.Config(cap_form=cap_form, cap=7.0)
    _check(gpu_lib, np.random.default_rng(G * 7919 + M * 31 + N + K), fmt, dtype, out_dtype, G, M, N, K, kind, glu=cfg)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("G,T,k,N,K", [(12, 1, 8, 100, 256), (12, 33, 4, 192, 416), (384, 5, 8, 64, 64)])
def test_gathered_rows(gpu_lib, G, T, k, N, K, fmt):
    _check(gpu_lib, np.random.default_rng(T * 13 + N), fmt, "bf16", "f32", G, T * k, N, K, "uneven", div=k, x_rows=T)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_outside(gpu_lib, fmt, glu):
    """A row id outside x gives a zero row, rows in no group keep what they
    held, offsets outside [0, M] are clamped."""
    import torch
    g = np.random.default_rng(5)
    G, M, N, K, T = 3, 24, 70, 224, 6
    codes, sc, gs = _weights(g, fmt, G, N, K, 1)
    x, xv = _x(g, T, K, "bf16")
    kw = {} if gs is None else dict(gs=to_dev(gs))
    kw["swiglu"] = gpu_lib.Config() if glu else None
    ids = g.permutation(M).astype(np.int32)

    def run(ids, offsets):
        out = torch.full((M, N // 2 if glu else N), float("nan"), device="cuda")
        gpu_lib.group_matvec(fmt, x, to_dev(codes), to_dev(sc), to_dev(np.array(offsets, np.int32)), out, row_ids=to_dev(ids),
                             id_div=4, **kw)
        return out.cpu().numpy()

    good = run(ids, [0, 5, 5, 20])
    assert np.isnan(good[20:]).all() and not np.isnan(good[:20]).any()
    bad = ids.copy()
    bad[1], bad[19] = -5, M
    got = run(bad, [0, 5, 5, 20])
    assert (got[1] == 0).all() and (got[19] == 0).all()
    keep = np.delete(np.arange(20), [1, 19])
    assert np.array_equal(got[keep], good[keep])
    # group 0 is [0, 5), group 1 [5, 0) and empty, group 2 [0, M)
    wide = run(ids, [-4, 5, 0, M + 50])
    assert not np.isnan(wide).any() and np.array_equal(wide[5:20], good[5:20])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_values(gpu_lib, dtype):
    """E8M0 scales at both ends against x at the other; fp32 x at the ends of
    its range; NaN scales and rows stay in their columns and rows."""
    import torch
    g = np.random.default_rng(9)
    G, M, N, K = 2, 6, 48, 256
    codes = g.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    off = to_dev(np.array([0, 2, M], np.int32))
    for lo, hi, scale in ((0, 3, 2.0 ** 100), (240, 246, 2.0 ** -110), (120, 124, 2.0 ** 124), (126, 130, 2.0 ** -120)):
        sc = g.integers(lo, hi, (G, N, K // 32), dtype=np.uint8)
        v = (np.clip(g.standard_normal((M, K)), -2, 2) * scale).astype(np.float32)
        x = torch.from_numpy(v).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
        out = torch.empty((M, N), device="cuda")
        gpu_lib.group_matvec("mxfp4", x, to_dev(codes), to_dev(sc), off, out)
        for i, (a, b) in enumerate(((0, 2), (2, M))):
            wv, xs = _values("mxfp4", codes[i], sc[i]), x[a:b].double().cpu().numpy()
            ref, size = xs @ wv.T, np.abs(xs) @ np.abs(wv).T
            tol = ((3 if dtype == "f32" else 1) * (K / 32 + 1) + 2) * 2.0 ** -23 * size
            # fp32 parts below bf16's normal range lose what lies under 2^-133
            tol += 0 if dtype == "bf16" else 2.0 ** -133 * np.abs(wv).sum(1)
            assert (np.abs(out[a:b].double().cpu().numpy() - ref) <= tol).all(), (lo, i)
    sc = g.integers(120, 124, (G, N, K // 32), dtype=np.uint8)
    sc[0, 5, 2] = 255
    x = torch.from_numpy(g.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    x[3, 7] = float("nan")
    out = torch.empty((M, N), device="cuda")
    gpu_lib.group_matvec("mxfp4", x, to_dev(codes), to_dev(sc), off, out)
    want = np.zeros((M, N), bool)
    want[3] = True
    want[:2, 5] = True
    assert np.array_equal(out.isnan().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_every_code_under_every_scale(gpu_lib, fmt):
    """x picks one column: out is the weight itself, exactly."""
    import torch
    G, N, K = 1, 256, 32
    codes = np.tile(np.arange(16, dtype=np.uint8) | np.arange(15, -1, -1).astype(np.uint8) << 4, (G, N, 1))
    sc = np.arange(256, dtype=np.uint8).reshape(1, 256, 1)
    if fmt == "nvfp4":
        sc = np.concatenate([sc, sc[:, ::-1]], -1)
    x = torch.zeros((32, K), dtype=torch.bfloat16, device="cuda")
    x[torch.arange(32), torch.arange(32)] = 1.0
    out = torch.empty((32, N), device="cuda")
    kw = dict(gs=torch.ones(1, device="cuda")) if fmt == "nvfp4" else {}
    gpu_lib.group_matvec(fmt, x, to_dev(codes), to_dev(sc), to_dev(np.array([0, 32], np.int32)), out, **kw)
    got = out.t().double().cpu().numpy()
    nan = np.repeat((sc[0] & 0x7F) == 0x7F, 16, -1).any(-1) if fmt == "nvfp4" else sc[0, :, 0] == 255
    with np.errstate(invalid="ignore", over="ignore"):
        want = _values(fmt, codes[0], sc[0])
        want = want.astype(np.float32).astype(np.float64)
    # a weight beyond bf16's (and fp32's) range is inf, and inf times the other columns' zeros NaN
    over = np.isinf(want).any(1) | (np.abs(want) > 3.38e38).any(1)
    fine = ~nan & ~over
    assert fine.sum() > 240
    assert np.array_equal(got[fine], want[fine])
    assert np.isnan(got[nan]).all()


def test_split_of_fp32_rows_is_exact(gpu_lib):
    """x of 24 significant bits against one-hot weights comes back unchanged."""
    import torch
    K = N = 64
    codes = np.zeros((1, N, K), np.uint8)
    codes[0, np.arange(N), np.arange(K)] = 2                  # 1.0
    packed = codes[..., ::2] | codes[..., 1::2] << 4
    sc = np.full((1, N, K // 32), 127, np.uint8)
    g = np.random.default_rng(3)
    v = (g.standard_normal((16, K)) * 10.0 ** g.uniform(-30, 38, (16, K))).astype(np.float32)
    v[0, 0], v[0, 1], v[0, 2] = 3.4028235e38, 1.9999999, -16777215.0
    out = torch.empty((16, N), device="cuda")
    gpu_lib.group_matvec("mxfp4", torch.from_numpy(v).cuda(), to_dev(packed), to_dev(sc), to_dev(np.array([0, 16], np.int32)), out)
    assert np.array_equal(out.cpu().numpy(), v)


def test_same_bits_every_run_and_any_company(gpu_lib):
    import torch
    g = np.random.default_rng(8)
    G, M, N, K = 4, 40, 96, 640
    codes, sc, gs = _weights(g, "nvfp4", G, N, K, 1)
    x, _ = _x(g, M, K, "bf16")
    args = (to_dev(codes), to_dev(sc))

    def run(offsets):
        out = torch.full((M, N), float("nan"), device="cuda")
        gpu_lib.group_matvec("nvfp4", x, *args, to_dev(np.array(offsets, np.int32)), out, gs=to_dev(gs))
        return out.cpu().numpy()

    first = run([0, 10, 20, 30, 40])
    for _ in range(3):
        assert np.array_equal(first, run([0, 10, 20, 30, 40]))
    assert np.array_equal(first[:10], run([0, 10, 10, 10, 10])[:10])
    assert np.array_equal(first[:3], run([0, 3, 3, 3, 3])[:3])


def test_binding_refusals(gpu_lib):
    import torch
    u8 = dict(dtype=torch.uint8, device="cuda")
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    w, sc, gs = torch.zeros((2, 8, 64), **u8), torch.zeros((2, 8, 8), **u8), torch.ones(2, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    out = torch.empty((4, 8), dtype=torch.float32, device="cuda")
    ok = ("nvfp4", x, w, sc, off, out)
    gpu_lib.group_matvec(*ok, gs=gs)
    for i, bad in ((0, "mxfp5"), (1, x.cpu()), (1, x.half()), (2, w[:1]), (3, sc[:, :, :4]), (4, off[:2]), (4, off.long()),
                   (5, out.half()), (5, out[:, :4])):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            gpu_lib.group_matvec(*args, gs=gs)
    for kw in ({}, dict(gs=gs[:1]), dict(gs=gs, gs_group=3), dict(gs=gs, gs_group=2), dict(gs=gs.double())):
        with pytest.raises(ValueError):
            gpu_lib.group_matvec(*ok, **kw)
    with pytest.raises(gpu_lib.MoeError) as e:
        gpu_lib.group_matvec("mxfp8", x, torch.zeros((2, 8, 128), **u8), torch.zeros((2, 8, 4), **u8), off, out)
    assert e.value.status == -5
    with pytest.raises(gpu_lib.MoeError):
        gpu_lib.group_matvec(*ok, gs=gs, row_ids=torch.zeros(4, dtype=torch.int32, device="cuda"), id_div=0)
