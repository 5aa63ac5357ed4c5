"""The norm's gradient where a workgroup has several rows, and the norm of rows
of every magnitude, against the definition in float64 (on the GPU, elementary
operations)."""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # fp32's half step
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}   # what storing a result adds
TINY = 2.0 ** -126
TYPES = [("bf16", "none"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "none"), ("f32", "f32")]


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rand(shape, seed, dtype, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(_dt(dtype))


def _groups(T, cols):
    """Workgroups of the gradient: rows are dealt out to them in turn."""
    return min(T, min(4096, max(512, 256 * 4608 // cols)))


def _close(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), int(bad.sum()))


def _gradient(dy, s, w, rstd, d_next):
    """d, its bound before it is stored, dw and the sums of its terms' magnitudes."""
    import torch
    T, cols = dy.shape
    d, tol = torch.empty((T, cols), dtype=torch.float64, device="cuda"), torch.empty((T, cols), dtype=torch.float64, device="cuda")
    dw, size_w = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    # roundings of the row's dot product: the additions of a lane (8 elements a piece, 8 pieces at most, and the
    # element behind them), across the wave (2 + 2 + 2) and the waves (15), dy n and the product with w
    adds = 65 + 6 + 15 + 2
    for i in range(0, T, 512):
        at = slice(i, min(T, i + 512))
        g, r = dy[at].double(), rstd[at].double()[:, None]
        n = s[at].double() * r
        a = g * w.double()
        d[at] = r * (a - n * (a * n).mean(1, keepdim=True))
        size = (a * n).abs().mean(1, keepdim=True)
        # a 1, n 1, the mean's own and the quotient 1, n dot 1, the difference 1, times rstd 1
        tol[at] = U * 1.001 * r * (3 * a.abs() + n.abs() * (adds + 5) * size) + TINY
        if d_next is not None:
            d[at] += d_next[at].double()
        tol[at] += U * d[at].abs()
        dw += (g * n).sum(0)
        size_w += (g * n).abs().sum(0)
    return d, tol, dw, size_w


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,cols", [
    (1300, 4608), (1030, 4603),        # 3 rows a workgroup in some, 2 in the others; on and off 8 elements
    (5000, 264), (9001, 259),          # 4096 and more workgroups
    (2600, 9216), (2050, 9215),        # 6 waves: 6 and 5 rows
    (1100, 16384), (1025, 16383),      # above 12288 columns no row is loaded ahead
    (515, 40008), (514, 65535),
])
def test_several_rows_a_workgroup(gpu_lib, T, cols, dtype, res):
    import torch
    bse, groups = gpu_lib, _groups(T, cols)
    assert T > groups and T % groups != 0
    kind = dtype if res == "none" else res
    s, dy, w = _rand((T, cols), 1, kind, 3.0), _rand((T, cols), 2, dtype, 1e-3), 1.0 + 0.1 * _rand((cols,), 3, "f32")
    d_next = None if res == "none" else _rand((T, cols), 4, res, 1e-3)
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    d, tol, want_dw, size = _gradient(dy, s, w, rstd, d_next)
    d_res, dx, dw = torch.full_like(s, float("nan")), torch.full_like(dy, float("nan")), torch.full_like(w, float("nan"))
    ws = torch.full((bse.norm_workspace_size(T, cols),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere
    bse.norm_backward(dy, s, w, rstd, d_res, ws, d_res_out=d_next, dx=dx, d_weight=dw)
    _close(d_res, d, tol + HALF[kind] * (d.abs() + tol))
    _close(dx, d, tol + HALF[dtype] * (d.abs() + tol))
    # rows of a workgroup one after the other, its row of partial sums in one of 128 runs, then 15 and 7 additions;
    # n and dy n
    adds = -(-T // groups) + -(-groups // 128) + 15 + 7 + 2
    _close(dw, want_dw, adds * U * 1.001 * size + TINY)
    # over what reaches the stream from further on
    if d_next is not None:
        bse.norm_backward(dy, s, w, rstd, d_next, ws, d_res_out=d_next, d_weight=dw)
        assert torch.equal(d_next, d_res)
    elif dtype == kind:
        bse.norm_backward(dy, s, w, rstd, dy, ws, d_weight=dw)
        assert torch.equal(dy, d_res)
    _close(dw, want_dw, adds * U * 1.001 * size + TINY)


def test_weight_gradient_of_very_many_rows(gpu_lib):
    """300000 x 2056: 586 rows a workgroup, fp32 partial sums of them."""
    import torch
    T, cols = 300000, 2056
    s, dy, w = _rand((T, cols), 1, "bf16"), _rand((T, cols), 2, "bf16"), torch.ones(cols, device="cuda")
    rstd = torch.cat([(p.double().square().mean(1) + 1e-6).rsqrt().float() for p in s.split(10000)])
    d, dw = torch.empty_like(s), torch.empty_like(w)
    gpu_lib.norm_backward(dy, s, w, rstd, d, gpu_lib.norm_workspace(T, cols), d_weight=dw)
    want, size = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, T, 10000):
        at = slice(i, i + 10000)
        t = dy[at].double() * s[at].double() * rstd[at].double()[:, None]
        want += t.sum(0)
        size += t.abs().sum(0)
    groups = _groups(T, cols)
    adds = -(-T // groups) + -(-groups // 128) + 15 + 7 + 2
    _close(dw, want, adds * U * 1.001 * size)


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,cols", [(1, 1), (3, 7), (5, 264), (3, 1003), (33, 4608), (3, 8200), (2, 16384), (2, 65535)])
def test_norm_within_a_rounding(gpu_lib, T, cols, dtype, res):
    """rstd and y carry their errors: what is left is the rounding to fp32 and, in
    bf16, the one that stores y."""
    import torch
    x = _rand((T, cols), 5, dtype)
    x[:, ::7] *= 20.0
    r = None if res == "none" else _rand((T, cols), 6, res, 3.0)
    w = 1.0 + 0.3 * _rand((cols,), 7, "f32")
    y, rstd = torch.full_like(x, float("nan")), torch.full((T,), float("nan"), device="cuda")
    s = x if r is None else torch.empty_like(r)
    gpu_lib.norm_forward(x, w, y, residual=r, res_out=None if r is None else s, rstd=rstd, eps=1e-6)
    if r is not None:
        total = x.double() + r.double()
        _close(s, total, (U + HALF[res]) * (1 + U) * total.abs())
    eps = float(torch.tensor(1e-6))
    want = (s.double().square().mean(1) + eps).rsqrt()
    # the sum of squares, its mean, the root and the quotient in 64 bits: far below 2^-20 of a half step
    _close(rstd, want, U * (1 + 2.0 ** -20) * want)
    exact = s.double() * want[:, None] * w.double()
    half = U * (1 + 2.0 ** -20)
    _close(y, exact, (half + HALF[dtype] * (1 + half)) * exact.abs() + TINY)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_where_the_carried_errors_underflow(gpu_lib, dtype):
    """Rows whose root mean square is near fp32's largest number, where 1 / rms and
    its remainder are subnormal, and elements far below their row's."""
    import torch
    T, cols = 4, 1000
    x = _rand((T, cols), 10, "f32").clamp(-3, 3)
    x[0] *= 2.0 ** 126
    x[1] *= 2.0 ** 110
    x[2, ::3] *= 2.0 ** -107
    x[3, ::3] *= 2.0 ** -120
    x = x.to(_dt(dtype))
    w = 1.0 + 0.3 * _rand((cols,), 11, "f32")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    gpu_lib.norm_forward(x, w, y, rstd=rstd, eps=1e-6)
    want = (x.double().square().mean(1) + float(torch.tensor(1e-6))).rsqrt()
    _close(rstd, want, U * (1 + 2.0 ** -20) * want + 2.0 ** -150)
    exact = x.double() * want[:, None] * w.double()
    # rstd as stored is off by U and half of 2^-149; two products and the sum of the rest
    rel = 4 * U + 2.0 ** -150 / want[:, None]
    _close(y, exact, (rel + HALF[dtype] * (1 + rel)) * exact.abs() + TINY)


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("cols", [264, 1003])
def test_zeros_keep_their_sign(gpu_lib, cols, dtype, res):
    """s r weight of a negative zero is a negative zero, and the other way round
    under a negative weight."""
    import torch
    x = _rand((4, cols), 12, dtype)
    x[:, ::3], x[:, 1::5], x[3] = -0.0, 0.0, -0.0
    r = None if res == "none" else torch.where(x == 0, x, torch.zeros_like(x)).to(_dt(res))
    w = 1.0 + 0.1 * _rand((cols,), 13, "f32")
    w[::4] *= -1.0
    y = torch.empty_like(x)
    gpu_lib.norm_forward(x, w, y, residual=r)
    zero = x == 0
    assert (y[zero] == 0).all()
    assert torch.equal(y.signbit()[zero], (x.signbit() ^ w.signbit())[zero])


@pytest.mark.parametrize("fmt,act_gs", [("mxfp8", 0), ("mxfp4", 0), ("nvfp4", 0), ("nvfp4", 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [96, 2048, 4608])
def test_codes_of_rows_with_nan_and_inf(gpu_lib, cols, dtype, fmt, act_gs):
    """Codes, scales and row scales of rows with a NaN, an infinity, an infinite
    sum of squares, tiny and huge values are quantize_act's of the stored y."""
    import torch
    bse, T = gpu_lib, 12
    x = _rand((T, cols), 8, dtype)
    w = 1.0 + 0.3 * _rand((cols,), 9, "f32")
    x[0, 5] = float("nan")
    x[1, 40] = float("inf")
    x[2, 33], x[2, 34] = float("-inf"), float("nan")
    x[3] = float("nan")
    x[4] *= 1e37
    x[5] *= 1e-30
    x[6] = 0.0
    x[7, 32:64] = 0.0
    x[8, ::2] = -0.0
    x[9] = 0.0
    x[9, 17] = 1e-38
    w[50], w[51], w[60] = float("inf"), float("nan"), 1e38     # in every row
    cfg = bse.Config(fmt=fmt, act_gs=act_gs, act_gs_static=(0.004, 1.0))
    per, block = cols if fmt == "mxfp8" else cols // 2, 16 if fmt == "nvfp4" else 32

    def buffers():
        return (torch.full((T, per), 0xAA, dtype=torch.uint8, device="cuda"),
                torch.full((T, cols // block), 0xAA, dtype=torch.uint8, device="cuda"), torch.full((T,), 7.0, device="cuda"))

    for gain in (torch.ones_like(w), w):
        y, got, want = torch.empty_like(x), buffers(), buffers()
        bse.norm_forward(x, gain, y, cfg=cfg, codes=got[0], scales=got[1], row_gs=got[2])
        bse.quantize_act(cfg, y, want[0], want[1], want[2])
        for name, a, b in zip(("codes", "scales", "row_gs"), got, want):
            same = (a == b) | (a.isnan() & b.isnan() if a.is_floating_point() else torch.zeros_like(a, dtype=torch.bool))
            assert same.all(), (name, (~same).nonzero()[:4].tolist())
