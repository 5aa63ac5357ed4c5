"""moe_norm_forward / _backward against float64, and their codes against
moe_quantize_act."""
import numpy as np
import pytest

from oracle import stream as S

pytestmark = pytest.mark.gpu

# What the sums of a row leave: at most 64 additions in a lane, 6 across the
# wave and 16 across the waves, each 2^-24 of a positive sum (or of the sum of
# magnitudes).
ADDS = 64 + 6 + 16
U = 2.0 ** -24          # fp32's half step
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}   # what storing a result adds
# a value below the normal range has a step of its own: fp32 2^-149, bf16 2^-133
TINY = 2.0 ** -126


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rand(shape, seed, dtype, scale=1.0, loud=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    if loud:
        x[:, ::7] *= 20.0
    return x.to(_dt(dtype)).cuda()


def _f64(t):
    return t.double().cpu().numpy()


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 31), (1, 64), (4, 96), (7, 512), (3, 1003), (2, 2048), (5, 2056), (2, 4608), (130, 4608),
          (3, 8200), (2, 16384), (1, 40008), (1, 65536), (2, 65535), (1100, 40)]
TYPES = [("bf16", "none"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "none"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,cols", SHAPES)
def test_forward_and_backward(gpu_lib, T, cols, dtype, res):
    import torch
    bse, eps = gpu_lib, 1e-5
    x = _rand((T, cols), 1 + cols, dtype, loud=True)
    r = None if res == "none" else _rand((T, cols), 2 + cols, res, 3.0)
    w = 1.0 + 0.1 * _rand((cols,), 3 + cols, "f32")
    y, rstd = torch.full_like(x, float("nan")), torch.full((T,), float("nan"), device="cuda")
    s = x if r is None else torch.full_like(r, float("nan"))
    bse.norm_forward(x, w, y, residual=r, res_out=None if r is None else s, rstd=rstd, eps=eps)
    if r is not None:
        ref = _f64(x) + _f64(r)
        assert (np.abs(_f64(s) - ref) <= (U + HALF[res]) * (1 + U) * np.abs(ref)).all()
    s64 = _f64(s)
    want, wr = S.norm_forward(s64, _f64(w), float(np.float32(eps)))
    # rstd: half of the mean square's error, then the root and the quotient (2 U each)
    rel = (ADDS / 2 + 1 + 4) * U
    assert (np.abs(_f64(rstd) - wr) <= rel * wr).all()
    assert (np.abs(_f64(y) - want) <= ((rel + 2 * U) + HALF[dtype]) * 1.001 * np.abs(want) + TINY).all()

    dy = _rand((T, cols), 4 + cols, dtype, 1e-3)
    d_next = None if r is None else _rand((T, cols), 5 + cols, res, 1e-3)
    kind = dtype if r is None else res
    d_res = torch.full((T, cols), float("nan"), dtype=_dt(kind), device="cuda")
    dx = torch.full_like(x, float("nan"))
    dw = torch.full((cols,), float("nan"), device="cuda")
    bse.norm_backward(dy, s, w, rstd, d_res, bse.norm_workspace(T, cols), d_res_out=d_next, dx=dx, d_weight=dw)
    g64, w64, r64 = _f64(dy), _f64(w), _f64(rstd)[:, None]
    d, want_dw = S.norm_backward(g64, s64, w64, r64[:, 0], None if d_next is None else _f64(d_next))
    n = s64 * r64
    a, size = np.abs(g64 * w64), np.abs(g64 * w64 * n).mean(1, keepdims=True)
    # dy w, n dot, their difference, times rstd, plus d_next: 5 roundings around the mean's own error
    tol = U * (r64 * (4 * a + np.abs(n) * (ADDS + 9) * size) + np.abs(d)) * 1.001 + TINY
    assert (np.abs(_f64(d_res) - d) <= tol + HALF[kind] * (np.abs(d) + tol)).all()
    assert (np.abs(_f64(dx) - d) <= tol + HALF[dtype] * (np.abs(d) + tol)).all()
    # a workgroup's rows one after the other (T / 1024), then at most 1024 / 8 partial rows and 8 runs; dy n: 2
    adds = T // 1024 + 1 + 128 + 8 + 2
    assert (np.abs(_f64(dw) - want_dw) <= adds * U * np.abs(g64 * n).sum(0) + TINY).all()


@pytest.mark.parametrize("fmt,act_gs", [("mxfp8", 0), ("mxfp4", 0), ("nvfp4", 0), ("nvfp4", 2)])
@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,cols", [(1, 32), (3, 96), (5, 480), (2, 2048), (33, 4608), (2, 8224), (1, 65536)])
def test_codes_are_those_of_the_stored_rows(gpu_lib, T, cols, dtype, res, fmt, act_gs):
    """Codes, scales and row scales bit for bit, with a zero row among the rows;
    and y, the stream and rstd as without codes."""
    import torch
    bse = gpu_lib
    cfg = bse.Config(fmt=fmt, act_gs=act_gs, act_gs_static=(0.004, 1.0))
    x = _rand((T, cols), 11 + cols, dtype, loud=True)
    r = None if res == "none" else _rand((T, cols), 12 + cols, res, 3.0)
    x[T // 2] = 0.0
    if r is not None:
        r[T // 2] = 0.0
    w = 1.0 + 0.3 * _rand((cols,), 13, "f32")

    def call(**kw):
        y, s, rstd = torch.empty_like(x), None if r is None else torch.empty_like(r), torch.empty(T, device="cuda")
        bse.norm_forward(x, w, y, residual=r, res_out=s, rstd=rstd, **kw)
        return [t for t in (y, s, rstd) if t is not None]

    def buffers():
        n = {"mxfp8": cols}.get(fmt, cols // 2)
        return (torch.full((T, n), 0xAA, dtype=torch.uint8, device="cuda"),
                torch.full((T, cols // (16 if fmt == "nvfp4" else 32)), 0xAA, dtype=torch.uint8, device="cuda"),
                torch.full((T,), 7.0, device="cuda"))

    got, want = buffers(), buffers()
    outs = call(cfg=cfg, codes=got[0], scales=got[1], row_gs=got[2])
    for a, b in zip(outs, call()):
        assert torch.equal(a, b)
    bse.quantize_act(cfg, outs[0], want[0], want[1], want[2])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # without y, and without the stream
    only = buffers()
    bse.norm_forward(x, w, residual=r, cfg=cfg, codes=only[0], scales=only[1], row_gs=only[2])
    for a, b in zip(only, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [4608, 1003])
def test_in_place_and_without_outputs(gpu_lib, cols):
    """The stream and y written over their inputs, gradients over theirs; a
    caller that wants only some outputs gets the same bits."""
    import torch
    bse, T = gpu_lib, 9
    x, r, w = _rand((T, cols), 1, "bf16"), _rand((T, cols), 2, "bf16"), _rand((cols,), 3, "f32")
    y, s, rstd = torch.empty_like(x), torch.empty_like(r), torch.empty(T, device="cuda")
    bse.norm_forward(x, w, y, residual=r, res_out=s, rstd=rstd)
    x2, r2 = x.clone(), r.clone()
    bse.norm_forward(x2, w, x2, residual=r2, res_out=r2)
    assert torch.equal(x2, y) and torch.equal(r2, s)
    x3, y3 = x.clone(), torch.empty_like(x)
    bse.norm_forward(x3, w, y3, residual=r, res_out=x3)          # the stream over x
    assert torch.equal(x3, s) and torch.equal(y3, y)
    wide = torch.empty((T, cols), device="cuda")
    bse.norm_forward(x, w, y3, res_out=wide)                     # no residual, an fp32 stream: x itself
    assert torch.equal(wide, x.float())

    dy, dn, ws = _rand((T, cols), 4, "bf16"), _rand((T, cols), 5, "bf16"), bse.norm_workspace(T, cols)
    d, dw = torch.empty_like(r), torch.empty_like(w)
    bse.norm_backward(dy, s, w, rstd, d, ws, d_res_out=dn, d_weight=dw)
    d2 = torch.empty_like(d)
    bse.norm_backward(dy, s, w, rstd, d2, d_res_out=dn)          # no weight gradient, no workspace
    assert torch.equal(d, d2)
    over = dn.clone()
    bse.norm_backward(dy, s, w, rstd, over, ws, d_res_out=over, d_weight=dw)
    assert torch.equal(over, d)
    over, dw2 = dy.clone(), torch.empty_like(w)
    bse.norm_backward(over, s, w, rstd, over, ws, d_res_out=dn, d_weight=dw2)
    assert torch.equal(over, d) and torch.equal(dw2, dw)


def test_extreme_rows(gpu_lib):
    """A zero row has 1 / sqrt(eps); NaN and inf stay in their row; magnitudes
    near the ends of what squares hold."""
    import torch
    bse, cols, eps = gpu_lib, 256, 1e-6
    x = _rand((7, cols), 1, "f32")
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 9] = float("inf")
    x[4] *= 1e15
    x[5] *= 1e-15
    w = torch.ones(cols, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(7, device="cuda")
    bse.norm_forward(x, w, y, rstd=rstd, eps=eps)
    assert (y[1] == 0).all() and abs(float(rstd[1]) - 1e3) <= 1e-3
    assert y[2].isnan().all() and rstd[2].isnan()
    assert float(rstd[3]) == 0.0 and y[3, 9].isnan() and (y[3].nan_to_num() == 0).all()
    for i in (0, 4, 5, 6):
        want = S.norm_forward(_f64(x[i:i + 1]), np.ones(cols), float(np.float32(eps)))[0][0]
        assert (np.abs(_f64(y[i]) - want) <= (ADDS / 2 + 7) * U * np.abs(want)).all(), i


@pytest.mark.parametrize("size", [1e30, 1e-15, 1e-25])
def test_squares_beyond_fp32(gpu_lib, size):
    """Rows whose squares leave fp32's range on either side (eps as far down)."""
    import torch
    cols, eps = 1003, 1e-38 if size < 1 else 1e-6
    x = _rand((3, cols), 2, "f32") * size
    w = 1.0 + 0.1 * _rand((cols,), 3, "f32")
    y, rstd = torch.empty_like(x), torch.empty(3, device="cuda")
    gpu_lib.norm_forward(x, w, y, rstd=rstd, eps=eps)
    want, wr = S.norm_forward(_f64(x), _f64(w), float(np.float32(eps)))
    assert (np.abs(_f64(y) - want) <= 4 * U * np.abs(want) + TINY).all()
    assert (np.abs(_f64(rstd) - wr) <= 2 * U * wr).all()


def test_a_normed_row_is_the_exact_one_rounded(gpu_lib):
    """y is the 64-bit result rounded to fp32 and then to the type, so the codes
    are those of the exact row."""
    import torch
    T, cols = 200, 4608
    x, r = _rand((T, cols), 1, "bf16", loud=True), _rand((T, cols), 2, "bf16", 3.0)
    w = 1.0 + 0.1 * _rand((cols,), 3, "f32")
    y, s = torch.empty_like(x), torch.empty_like(x)
    gpu_lib.norm_forward(x, w, y, residual=r, res_out=s)
    want = torch.from_numpy(S.norm_forward(_f64(s), _f64(w), float(np.float32(1e-6)))[0]).float().bfloat16()
    # off only where fp32 itself rounds to the other side: the carried errors leave 2^-46, below 1 in 10^6 elements
    assert int((y.cpu() != want).sum()) <= 1


def test_offsets_into_larger_arrays(gpu_lib):
    """Rows at addresses that are no multiple of 16 bytes; what lies around the
    outputs stays."""
    import torch
    bse, T, cols = gpu_lib, 5, 264
    whole = _rand((T * cols + 16,), 1, "bf16")
    x = whole[3:3 + T * cols].view(T, cols)
    w = torch.ones(cols + 1, device="cuda")[1:]
    y, rstd = torch.empty((T, cols), dtype=torch.bfloat16, device="cuda"), torch.empty(T, device="cuda")
    bse.norm_forward(x.clone(), w.clone(), y, rstd=rstd)
    out = torch.full((T * cols + 16,), 9.0, dtype=torch.bfloat16, device="cuda")
    bse.norm_forward(x, w, out[5:5 + T * cols].view(T, cols))
    assert torch.equal(out[5:5 + T * cols].view(T, cols), y)
    assert (out[:5] == 9).all() and (out[5 + T * cols:] == 9).all()


def test_no_rows(gpu_lib):
    import torch
    bse = gpu_lib
    x, w, dw = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda"), torch.full((64,), 5.0, device="cuda")
    bse.norm_forward(x, w, x, rstd=torch.empty(0, device="cuda"))
    bse.norm_backward(x, x, w, torch.empty(0, device="cuda"), x, bse.norm_workspace(0, 64), d_weight=dw)
    assert (dw == 0).all()


def test_same_bits_every_run(gpu_lib):
    import torch
    bse, T, cols = gpu_lib, 3000, 72
    x, w, dy = _rand((T, cols), 1, "f32"), _rand((cols,), 2, "f32"), _rand((T, cols), 3, "f32")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    bse.norm_forward(x, w, y, rstd=rstd)
    got = []
    for _ in range(3):
        ws = torch.full((bse.norm_workspace_size(T, cols),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere
        d, dw = torch.empty_like(x), torch.empty_like(w)
        bse.norm_backward(dy, x, w, rstd, d, ws, d_weight=dw)
        got.append((d, dw))
    for d, dw in got[1:]:
        assert torch.equal(d, got[0][0]) and torch.equal(dw, got[0][1])


def test_binding_refusals(gpu_lib):
    import torch
    bse = gpu_lib
    x, w = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    bse.norm_forward(x, w, y)
    h = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    for args, kw in (((x.half(), w, y), {}), ((x, w.half(), y), {}), ((x, w, h), {}), ((x, w[:32], y), {}),
                     ((x.t(), w, y), {}), ((x, w, y), dict(residual=x[:2])), ((x, w, y), dict(residual=x, res_out=h)),
                     ((x.cpu(), w, y), {}), ((x, w, y), dict(codes=torch.zeros((4, 64), dtype=torch.uint8, device="cuda"))),
                     ((x, w, y), dict(cfg="mxfp8", codes=torch.zeros((4, 32), dtype=torch.uint8, device="cuda")))):
        with pytest.raises(ValueError):
            bse.norm_forward(*args, **kw)
    for kw in (dict(residual=h), dict(eps=0.0), dict(cfg="mxfp8")):
        with pytest.raises(bse.MoeError):
            bse.norm_forward(x, w, y, **kw)
    rstd = torch.ones(4, device="cuda")
    with pytest.raises(bse.MoeError):
        bse.norm_backward(x, x, w, rstd, y, d_weight=torch.empty_like(w))   # no workspace
