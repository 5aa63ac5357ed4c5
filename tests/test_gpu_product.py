"""moe_group_product against the float64 product of the decoded operands."""
import numpy as np
import pytest

from oracle import formats as F
from tests._util import to_dev

pytestmark = pytest.mark.gpu


def _operand(g, rows, K, lo=120, hi=126):
    codes = g.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    return codes, g.integers(lo, hi, (rows, K // 32), dtype=np.uint8)


def _sizes(g, G, M, kind):
    if kind == "one":                     # every row in one group
        n = np.zeros(G, np.int64)
        n[G // 2] = M
        return n
    if kind == "even":
        return np.array([M // G + (i < M % G) for i in range(G)])
    p = g.dirichlet(np.full(G, 0.3))      # uneven, some groups empty
    return g.multinomial(M, p)


def _run(lib, a, asc, w, wsc, offsets, M, out_f32, ids=None, div=1, fill=np.nan):
    import torch
    out = torch.full((M, w.shape[1]), fill, dtype=torch.float32 if out_f32 else torch.bfloat16, device="cuda")
    lib.group_product("mxfp4", to_dev(a), to_dev(asc), to_dev(w), to_dev(wsc), to_dev(offsets.astype(np.int32)), out,
                      row_ids=None if ids is None else to_dev(ids.astype(np.int32)), id_div=div)
    torch.cuda.synchronize()
    return out.float().cpu().numpy()


def _check(got, a, asc, w, wsc, offsets, out_f32, src):
    """Products of the codes are exact; the sums are fp32 with at most one
    rounding per 128 of k and lane group, each bounded by 2^-22 of the terms'
    magnitudes; bf16 adds half an ulp (2^-8)."""
    K = a.shape[1] * 2
    av = F.dequantize_mxfp4(a, asc)
    for i in range(len(offsets) - 1):
        lo, hi = offsets[i], offsets[i + 1]
        if lo == hi:
            continue
        wv = F.dequantize_mxfp4(w[i], wsc[i])
        rows = av[src[lo:hi]]
        ref, size = rows @ wv.T, np.abs(rows) @ np.abs(wv).T
        tol = (K / 128 + 8) * 2.0 ** -22 * size + (0 if out_f32 else 2.0 ** -8 * np.abs(ref))
        bad = ~(np.abs(got[lo:hi] - ref) <= tol)
        assert not bad.any(), (i, np.argwhere(bad)[:4], got[lo:hi][bad][:4], ref[bad][:4])


CASES = [
    # G, M, N, K, kind
    (1, 1, 1, 32, "even"), (1, 1, 64, 128, "even"), (1, 5, 17, 96, "even"), (1, 130, 200, 512, "even"),
    (3, 7, 64, 160, "uneven"), (5, 231, 1003, 352, "uneven"), (16, 40, 96, 2304, "uneven"),
    (48, 600, 256, 1184, "uneven"), (7, 300, 130, 640, "one"), (2, 700, 520, 768, "even"), (1, 257, 256, 4608, "even"),
    (1024, 60, 33, 64, "uneven"), (4, 1100, 320, 544, "uneven"),
    # rows per group on both sides of every rule on the mean group
    (2, 32, 80, 256, "even"), (2, 34, 80, 256, "even"), (2, 96, 80, 256, "even"), (2, 98, 80, 256, "even"),
    (2, 128, 272, 256, "even"), (2, 130, 272, 288, "even"), (2, 514, 272, 384, "even"),
    # enough tiles for the largest tile
    (1, 12400, 1003, 96, "even"), (40, 2600, 1300, 672, "uneven"), (3, 8300, 1280, 160, "one"),
]


@pytest.mark.parametrize("out_f32", [True, False])
@pytest.mark.parametrize("G,M,N,K,kind", CASES)
def test_product(gpu_lib, G, M, N, K, kind, out_f32):
    g = np.random.default_rng(G * 7919 + M * 31 + N + K)
    a, asc = _operand(g, M, K)
    w, wsc = _operand(g, G * N, K)
    w, wsc = w.reshape(G, N, -1), wsc.reshape(G, N, -1)
    offsets = np.concatenate([[0], np.cumsum(_sizes(g, G, M, kind))])
    got = _run(gpu_lib, a, asc, w, wsc, offsets, M, out_f32)
    _check(got, a, asc, w, wsc, offsets, out_f32, np.arange(M))


@pytest.mark.parametrize("G,T,k,N,K", [(12, 1, 8, 100, 256), (12, 33, 4, 192, 416), (3, 400, 3, 300, 512),
                                       (2, 1, 2, 64, 4608)])
def test_gathered_rows(gpu_lib, G, T, k, N, K):
    """Row r reads token row_ids[r] // k; a row id outside A gives a zero row;
    rows in no group keep what they held."""
    g = np.random.default_rng(T * 13 + N)
    a, asc = _operand(g, T, K)
    w, wsc = _operand(g, G * N, K)
    w, wsc = w.reshape(G, N, -1), wsc.reshape(G, N, -1)
    M = T * k
    ids = g.permutation(M)
    live = M - (2 if M > 4 else 0)           # the last rows belong to no group
    offsets = np.concatenate([[0], np.cumsum(_sizes(g, G, live, "uneven"))])
    got = _run(gpu_lib, a, asc, w, wsc, offsets, M, True, ids, k)
    _check(got, a, asc, w, wsc, offsets, True, ids // k)
    assert np.isnan(got[live:]).all()
    bad = ids.copy()
    bad[0], bad[live - 1] = -5, T * k
    got = _run(gpu_lib, a, asc, w, wsc, offsets, M, True, bad, k)
    assert (got[0] == 0).all() and (got[live - 1] == 0).all()
    if live > 2:
        keep = np.delete(np.arange(live), [0, live - 1])
        again = _run(gpu_lib, a, asc, w, wsc, offsets, M, True, ids, k)
        assert np.array_equal(got[keep], again[keep])


@pytest.mark.parametrize("M", [3, 300])
def test_offsets_are_clamped(gpu_lib, M):
    """Offsets outside [0, M] take part up to the bounds; descending ones make
    an empty group."""
    G, N, K = 3, 70, 224
    g = np.random.default_rng(M)
    a, asc = _operand(g, M, K)
    w, wsc = _operand(g, G * N, K)
    w, wsc = w.reshape(G, N, -1), wsc.reshape(G, N, -1)
    got = _run(gpu_lib, a, asc, w, wsc, np.array([-4, 1, 0, M + 50]), M, True)
    # group 0 is [0, 1), group 1 [1, 0) and empty, group 2 [0, M): row 0 is in two groups, either may write it
    av = F.dequantize_mxfp4(a, asc)
    ref = av @ F.dequantize_mxfp4(w[2], wsc[2]).T
    size = np.abs(av) @ np.abs(F.dequantize_mxfp4(w[2], wsc[2])).T
    assert (np.abs(got[1:] - ref[1:]) <= (K / 128 + 8) * 2.0 ** -22 * size[1:]).all()


@pytest.mark.parametrize("M,G", [(6, 3), (600, 2)])
def test_extreme_scales(gpu_lib, M, G):
    """Scale bytes at both ends: tiny times huge stays exact, underflow goes
    to zero, 255 (E8M0's NaN) gives NaN in its row or column only."""
    N, K = 48, 256
    g = np.random.default_rng(5)
    a, asc = _operand(g, M, K, 1, 3)
    w, wsc = _operand(g, G * N, K, 250, 253)
    w, wsc = w.reshape(G, N, -1), wsc.reshape(G, N, -1)
    offsets = np.concatenate([[0], np.cumsum(_sizes(g, G, M, "even"))])
    got = _run(gpu_lib, a, asc, w, wsc, offsets, M, True)
    _check(got, a, asc, w, wsc, offsets, True, np.arange(M))
    asc[1, 3] = 255
    wsc[0, 5, 2] = 255
    got = _run(gpu_lib, a, asc, w, wsc, offsets, M, True)
    nan = np.isnan(got)
    want = np.zeros_like(nan)
    want[1] = True
    want[offsets[0]:offsets[1], 5] = True
    assert np.array_equal(nan, want)


def test_same_bits_every_run_and_any_company(gpu_lib):
    """A row's result does not depend on the run, nor on the other rows of its
    group while the same kernel takes it."""
    G, M, N, K = 4, 40, 96, 640
    g = np.random.default_rng(8)
    a, asc = _operand(g, M, K)
    w, wsc = _operand(g, G * N, K)
    w, wsc = w.reshape(G, N, -1), wsc.reshape(G, N, -1)
    offsets = np.array([0, 10, 20, 30, 40])
    first = _run(gpu_lib, a, asc, w, wsc, offsets, M, True)
    for _ in range(3):
        assert np.array_equal(first, _run(gpu_lib, a, asc, w, wsc, offsets, M, True))
    fewer = _run(gpu_lib, a, asc, w, wsc, np.array([0, 10, 10, 10, 10]), M, True)
    assert np.array_equal(first[:10], fewer[:10])


def test_another_stream(gpu_lib):
    """Enqueued on the current stream, in order with its other work."""
    import torch
    g = np.random.default_rng(4)
    a, asc = _operand(g, 9, 128)
    w, wsc = _operand(g, 32, 128)
    ta, tas, tw, tws = to_dev(a), to_dev(asc), to_dev(w[None]), to_dev(wsc[None])
    off = to_dev(np.array([0, 9], np.int32))
    out = torch.zeros((9, 32), dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        gpu_lib.group_product("mxfp4", ta, tas, tw, tws, off, out)
        twice = out * 2
    side.synchronize()
    ref = F.dequantize_mxfp4(a, asc) @ F.dequantize_mxfp4(w, wsc).T
    assert np.abs(twice.cpu().numpy() - 2 * ref).max() <= 2.0 ** -18 * np.abs(ref).max()


def test_binding_refusals(gpu_lib):
    import torch
    u8 = dict(dtype=torch.uint8, device="cuda")
    a, asc = torch.zeros((4, 64), **u8), torch.zeros((4, 4), **u8)
    w, wsc = torch.zeros((2, 8, 64), **u8), torch.zeros((2, 8, 4), **u8)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    out = torch.empty((4, 8), dtype=torch.float32, device="cuda")
    ok = ("mxfp4", a, asc, w, wsc, off, out)
    gpu_lib.group_product(*ok)
    for i, bad in ((0, "mxfp5"), (1, a.cpu()), (2, asc[:, :3]), (3, w[:1]), (4, wsc[:, :7]), (5, off[:2]),
                   (5, off.long()), (6, out.half())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            gpu_lib.group_product(*args)
    with pytest.raises(gpu_lib.MoeError) as e:
        gpu_lib.group_product("mxfp8", *ok[1:])
    assert e.value.status == -5
    with pytest.raises(gpu_lib.MoeError):
        gpu_lib.group_product(*ok, row_ids=torch.zeros(4, dtype=torch.int32, device="cuda"), id_div=0)


@pytest.mark.parametrize("out_f32", [True, False])
@pytest.mark.parametrize("G,M,N,K,kind", [(2, 20, 80, 256, "even"), (2, 21, 80, 256, "even"), (40, 400, 300, 1184, "uneven"),
                                          (40, 401, 300, 1184, "uneven"), (9, 90, 640, 4736, "one"),
                                          (24, 700, 1300, 480, "uneven"), (6, 90, 257, 32, "even")])
def test_mean_group_of_ten(gpu_lib, G, M, N, K, kind, out_f32):
    """Both sides of the streaming kernel's bound, with groups of more and of
    fewer rows than either kernel's tile."""
    test_product(gpu_lib, G, M, N, K, kind, out_f32)


@pytest.mark.parametrize("out_f32", [True, False])
@pytest.mark.parametrize("M,N,K", [(300, 70, 96), (300, 272, 160), (12400, 1003, 32)])
def test_rows_past_a_partial_tile(gpu_lib, M, N, K, out_f32):
    """Tiles of 128 rows that hold fewer: the rows after the group's last keep
    what they held, as do those after the end of out.  Both tile widths."""
    import torch
    g = np.random.default_rng(M + N)
    a, asc = _operand(g, M, K)
    w, wsc = _operand(g, N, K)
    ta, tas, tw, tws = to_dev(a), to_dev(asc), to_dev(w[None]), to_dev(wsc[None])
    for live in (1, 31, 33, 64, 66, 97, 127, 129, M):
        off = to_dev(np.array([0, live], np.int32))
        whole = torch.full((M + 160, N), float("nan"), dtype=torch.float32 if out_f32 else torch.bfloat16, device="cuda")
        gpu_lib.group_product("mxfp4", ta, tas, tw, tws, off, whole[:M])
        got = whole.float().cpu().numpy()
        assert np.isnan(got[live:]).all(), live
        if live <= 300:
            _check(got, a, asc, w[None], wsc[None], [0, live], out_f32, np.arange(M))
        else:
            assert not np.isnan(got[:live]).any()
