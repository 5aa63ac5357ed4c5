"""moe_group_matvec at the ends of the range, in both of its kernels."""
import numpy as np
import pytest

from oracle import formats as F
from tests._util import to_dev

pytestmark = pytest.mark.gpu

G, N, K = 2, 12288, 256
# rows: a mean group of 4 at most and of more, which take a kernel each
ROWS = {"few": 8, "many": 40}


def _values(fmt, codes, sc):
    if fmt == "mxfp4":
        return F.dequantize_mxfp4(codes, sc)
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(nib & 8, -1.0, 1.0) * mag[nib & 7]
    return v * np.repeat(F.e4m3_decode(sc).astype(np.float64), 16, -1)


def _x(v, dtype):
    import torch
    t = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    return t, t.double().cpu().numpy()


def _offsets(M):
    return np.array([0, M // 2 - 1, M], np.int32)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lo,hi,scale,gs", [
    # bytes of the block scales, size of x, fp32 scale.  2^-9 .. 2^-6 under the largest x: 16 products of
    # unscaled codes pass fp32's range, what the formula adds does not
    (1, 8, 2.0 ** 124, 2.0 ** -20), (1, 2, 2.0 ** 126, 2.0 ** -30),
    # 16 .. 448
    (0x58, 0x7F, 2.0 ** 110, 2.0 ** -20), (0x58, 0x7F, 2.0 ** -90, 2.0 ** 10),
    # both small; the fp32 scale brings the sums back
    (1, 8, 2.0 ** -80, 2.0 ** 60),
])
def test_nvfp4_ends(gpu_lib, lo, hi, scale, gs, dtype, rows):
    import torch
    M, g = ROWS[rows], np.random.default_rng(lo * 131 + hi)
    codes = g.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    sc = g.integers(lo, hi, (G, N, K // 16), dtype=np.uint8)
    x, xv = _x(np.clip(g.standard_normal((M, K)), -2, 2) * scale, dtype)
    off, out = _offsets(M), torch.empty((M, N), device="cuda")
    gpu_lib.group_matvec("nvfp4", x, to_dev(codes), to_dev(sc), to_dev(off), out, gs=torch.full((G,), gs, device="cuda"))
    got = out.double().cpu().numpy()
    # a lane's instructions one after the other (8 for each of 1 or 3 parts of x), 2 blocks, 4 additions across
    # lanes, gs: at most a last place (2^-23) of the magnitudes each
    rel = (8 * (3 if dtype == "f32" else 1) + 2 + 4 + 1) * 2.0 ** -23
    for i in range(G):
        a, b = off[i], off[i + 1]
        wv = _values("nvfp4", codes[i], sc[i])
        size = np.abs(xv[a:b]) @ np.abs(wv).T
        # the formula's sums are within fp32: no partial sum passes the magnitudes' total and its roundings
        assert size.max() * (1 + rel) < 2.0 ** 128
        ref, tol = xv[a:b] @ wv.T * gs, rel * size * gs
        bad = ~(np.abs(got[a:b] - ref) <= tol)
        assert not bad.any(), (i, int(bad.sum()), got[a:b][bad][:4], ref[bad][:4])


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("gs", [1.0, 2.0 ** 40])
def test_nvfp4_least_rows(gpu_lib, gs, rows):
    """bf16 x down to its least normal numbers under block scales around 1: products
    and sums below fp32's normal range."""
    import torch
    M, g = ROWS[rows], np.random.default_rng(77)
    codes = g.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    sc = g.integers(0x30, 0x40, (G, N, K // 16), dtype=np.uint8)
    x, xv = _x(np.clip(g.standard_normal((M, K)), -2, 2) * 2.0 ** -118, "bf16")
    off, out = _offsets(M), torch.empty((M, N), device="cuda")
    gpu_lib.group_matvec("nvfp4", x, to_dev(codes), to_dev(sc), to_dev(off), out, gs=torch.full((G,), gs, device="cuda"))
    got = out.double().cpu().numpy()
    for i in range(G):
        a, b = off[i], off[i + 1]
        wv = _values("nvfp4", codes[i], sc[i])
        ref, size = xv[a:b] @ wv.T * gs, np.abs(xv[a:b]) @ np.abs(wv).T * gs
        # as above; and each rounding below the normal range is one of 2^-149, of sums that are kept 2^-7 smaller
        tol = 15 * 2.0 ** -23 * size + 15 * 2.0 ** -142 * 2 * gs + 2.0 ** -149
        assert (np.abs(got[a:b] - ref) <= tol).all(), i


@pytest.mark.parametrize("cap_form", [0, 1, 2, 3])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_nan_under_every_cap(gpu_lib, fmt, dtype, rows, cap_form):
    """A NaN scale byte of a gate or an up row makes its column of the group's rows
    NaN, a NaN in x its row, whichever cap is taken."""
    import torch
    M, g = ROWS[rows], np.random.default_rng(5)
    codes = g.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    sc = g.integers(*((0x20, 0x50) if fmt == "nvfp4" else (119, 123)), (G, N, K // (16 if fmt == "nvfp4" else 32)), dtype=np.uint8)
    nan = 0x7F if fmt == "nvfp4" else 255
    sc[0, 37, 1] = nan                   # a gate row
    sc[1, N // 2 + 5, 2] = nan           # an up row
    v = g.standard_normal((M, K))
    v[2, 11] = float("nan")
    x, _ = _x(v, dtype)
    off, out = _offsets(M), torch.empty((M, N // 2), device="cuda")
    kw = dict(gs=torch.full((G,), 1e-2, device="cuda")) if fmt == "nvfp4" else {}
    gpu_lib.group_matvec(fmt, x, to_dev(codes), to_dev(sc), to_dev(off), out, swiglu=gpu_lib.Config(cap_form=cap_form, cap=7.0), **kw)
    want = np.zeros((M, N // 2), bool)
    want[2] = True
    want[:off[1], 37] = True
    want[off[1]:, 5] = True
    assert np.array_equal(out.isnan().cpu().numpy(), want)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mxfp4_weights_beyond_fp32(gpu_lib, dtype, rows):
    """A weight of 2^128 and more (scale bytes 253 and 254) is infinite: its outputs
    are infinite under bf16 rows; an fp32 row's parts may be zero, where infinity
    gives NaN, so they are infinite or NaN.  Other outputs are not touched."""
    import torch
    M, g = ROWS[rows], np.random.default_rng(6)
    codes = np.full((G, N, K // 2), 0x22, np.uint8)                        # 1.0
    sc = np.full((G, N, K // 32), 127, np.uint8)
    sc[0, 3], codes[0, 3, 5] = 254, 0x24                                   # 2^127 and one of 2^128
    codes[0, 3, :5] = codes[0, 3, 6:] = 0
    sc[1, 9], codes[1, 9] = 253, 0x77                                      # 6 * 2^126
    x, xv = _x(np.abs(g.standard_normal((M, K))) + 0.5, dtype)
    off, out = _offsets(M), torch.empty((M, N), device="cuda")
    gpu_lib.group_matvec("mxfp4", x, to_dev(codes), to_dev(sc), to_dev(off), out)
    got = out.cpu().numpy()
    mine = np.zeros((M, N), bool)
    mine[:off[1], 3] = mine[off[1]:, 9] = True
    assert np.isfinite(got[~mine]).all()
    assert (np.isposinf(got[mine]) if dtype == "bf16" else ~np.isfinite(got[mine])).all()
