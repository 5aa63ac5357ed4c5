"""moe_sort_rows, moe_combine_rows and their gradients against float64."""
import numpy as np
import pytest

from oracle import stream as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}
ADDS = 64 + 6 + 16      # of a row's dot product: a lane, the wave, the waves
TINY = 2.0 ** -126


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rand(shape, seed, dtype):
    import torch
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(_dt(dtype)).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _positions(T, k, live, M, seed):
    """live pairs at distinct rows below M, the others at -1."""
    g = np.random.default_rng(seed)
    pos = np.full(T * k, -1, np.int32)
    pos[g.permutation(T * k)[:live]] = g.permutation(M)[:live]
    return pos.reshape(T, k)


CASES = [
    # T, k, cols, live, M
    (1, 1, 1, 1, 1), (1, 1, 8, 0, 3), (1, 8, 64, 8, 8), (3, 2, 7, 4, 6), (5, 3, 40, 9, 20), (17, 4, 1003, 50, 68),
    (6, 32, 96, 150, 192), (33, 8, 2304, 200, 264), (20, 8, 4608, 160, 160), (4, 5, 8200, 13, 20), (2, 3, 65536, 5, 6),
    (2, 2, 65535, 3, 4), (300, 6, 136, 900, 1800), (9, 3, 520, 0, 0),
    (1024, 2, 72, 1500, 2048), (1030, 3, 1003, 2000, 3090), (1025, 2, 8, 2050, 2050), (1024, 1, 5, 700, 1024),
]


@pytest.mark.parametrize("dtype,y_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,k,cols,live,M", CASES)
def test_rows(gpu_lib, T, k, cols, live, M, dtype, y_dtype):
    import torch
    bse = gpu_lib
    pos = _positions(T, k, live, M, T + cols)
    at = torch.from_numpy(pos).cuda()
    x, y = _rand((T, cols), 1, dtype), _rand((M, cols), 2, y_dtype)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).cuda()
    named = np.zeros(M, bool)
    named[pos[pos >= 0]] = True
    y[torch.from_numpy(~named).cuda()] = float("nan")      # rows that no pair names play no part

    rows = torch.full((M, cols), 5.0, dtype=_dt(dtype), device="cuda")
    bse.sort_rows(x, at, rows)
    assert np.array_equal(_f64(rows), S.sort_rows(_f64(x), pos, np.full((M, cols), 5.0)))

    y0 = np.nan_to_num(_f64(y))
    for weights in (w, None):
        out = torch.full((T, cols), float("nan"), dtype=_dt(dtype), device="cuda")
        bse.combine_rows(y, at, weights, out)
        w64 = None if weights is None else _f64(w)
        want, size = S.combine_rows(y0, pos, w64), S.combine_rows(np.abs(y0), pos, w64)
        tol = k * U * size                      # one rounding an addition
        assert (np.abs(_f64(out) - want) <= tol + HALF[dtype] * (np.abs(want) + tol) + TINY).all()
    if y_dtype == dtype:
        dx = torch.full((T, cols), float("nan"), dtype=_dt(dtype), device="cuda")
        bse.sort_rows_backward(y, at, dx)
        assert torch.equal(dx, out)             # the sum with weights 1

    d = _rand((T, cols), 4, dtype)
    dy = torch.full((M, cols), 5.0, dtype=_dt(y_dtype), device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    bse.combine_rows_backward(d, y, at, w, dy, dw)
    want, want_w = S.combine_rows_backward(_f64(d), y0, pos, _f64(w), np.full((M, cols), 5.0))
    assert (np.abs(_f64(dy) - want) <= (U + HALF[y_dtype] * (1 + U)) * np.abs(want) + TINY).all()
    size = S.combine_rows_backward(np.abs(_f64(d)), np.abs(y0), pos, None, np.zeros((M, cols)))[1]
    assert (np.abs(_f64(dw) - want_w) <= ADDS * U * size + TINY).all()
    # either gradient on its own, and y's over y
    dy2, dw2 = torch.full_like(dy, 5.0), torch.full_like(dw, float("nan"))
    bse.combine_rows_backward(d, None, at, w, dy2)
    assert torch.equal(dy2, dy)
    bse.combine_rows_backward(d, y, at, w, None, dw2)
    assert torch.equal(dw2, dw)
    over = y.clone()
    bse.combine_rows_backward(d, over, at, w, over, dw2)
    assert torch.equal(over[torch.from_numpy(named).cuda()], dy[torch.from_numpy(named).cuda()]) and torch.equal(dw2, dw)


@pytest.mark.parametrize("cols", [64, 61])
def test_positions_outside(gpu_lib, cols):
    """Positions below 0 or from M on are not local, whatever their value."""
    import torch
    bse, T, k, M = gpu_lib, 4, 3, 6
    pos = np.array([[0, -7, 6], [2 ** 31 - 1, 1, 2], [-2 ** 31, -1, 100], [5, 3, 4]], np.int32)
    at, x, y = torch.from_numpy(pos).cuda(), _rand((T, cols), 1, "f32"), _rand((M, cols), 2, "f32")
    w = torch.full((T, k), 0.5, device="cuda")
    w[0, 1], w[2, 0] = float("nan"), float("inf")         # weights of pairs elsewhere play no part
    rows = torch.zeros((M, cols), device="cuda")
    bse.sort_rows(x, at, rows)
    assert torch.equal(rows, x[torch.tensor([0, 1, 1, 3, 3, 3], device="cuda")])
    out = torch.full((T, cols), float("nan"), device="cuda")
    bse.combine_rows(y, at, w, out)
    assert (out[2] == 0).all() and torch.equal(out[0], 0.5 * y[0]) and not out.isnan().any()
    dw, dy = torch.full((T, k), float("nan"), device="cuda"), torch.zeros_like(y)
    bse.combine_rows_backward(x, y, at, w, dy, dw)
    assert (dw.cpu().numpy()[(pos < 0) | (pos >= M)] == 0).all()
    assert torch.equal(dy[0], 0.5 * x[0]) and torch.equal(dy[3], 0.5 * x[3])


def test_offsets_into_larger_arrays(gpu_lib):
    """Arrays that start off 16 bytes; what lies around the outputs stays."""
    import torch
    bse, T, k, cols = gpu_lib, 6, 2, 72
    pos = torch.from_numpy(_positions(T, k, 12, 12, 1)).cuda()
    x = _rand((T * cols + 3,), 1, "bf16")[3:].view(T, cols)
    out = torch.full((12 * cols + 16,), 9.0, dtype=torch.bfloat16, device="cuda")
    rows = out[5:5 + 12 * cols].view(12, cols)
    bse.sort_rows(x, pos, rows)
    want = torch.empty((12, cols), dtype=torch.bfloat16, device="cuda")
    bse.sort_rows(x.clone(), pos, want)
    assert torch.equal(rows, want) and (out[:5] == 9).all() and (out[5 + 12 * cols:] == 9).all()
    a, b = torch.empty_like(x), torch.empty((T, cols), dtype=torch.bfloat16, device="cuda")
    bse.combine_rows(rows, pos, None, b)
    bse.combine_rows(want, pos, None, a.contiguous())
    assert torch.equal(b, (2 * x))                          # two slots of the same row


def test_the_layer_combines_alike(gpu_lib):
    """fp32 rows to a bf16 token: the sum in slot order, rounded once."""
    import torch
    bse, T, k, cols = gpu_lib, 50, 8, 256
    pos = _positions(T, k, 300, 400, 5)
    at, y = torch.from_numpy(pos).cuda(), _rand((400, cols), 1, "f32")
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2)).cuda()
    out = torch.empty((T, cols), dtype=torch.bfloat16, device="cuda")
    bse.combine_rows(y, at, w, out)
    acc = np.zeros((T, cols))
    yn, wn = y.cpu().numpy().astype(np.float64), w.cpu().numpy().astype(np.float64)
    for j in range(k):       # a fused multiply-add: one fp32 rounding a step (the 64-bit product and sum round below it)
        p = pos[:, j]
        acc = np.where((p >= 0)[:, None], (wn[:, j:j + 1] * yn[np.maximum(p, 0)] + acc).astype(np.float32).astype(np.float64), acc)
    want = torch.from_numpy(acc.astype(np.float32)).to(torch.bfloat16)
    assert (out.cpu() != want).float().mean() <= 1e-3       # double rounding in the 64-bit sum is rarer than that


def test_binding_refusals(gpu_lib):
    import torch
    bse = gpu_lib
    x, rows = torch.zeros((4, 64), device="cuda"), torch.zeros((8, 64), device="cuda")
    pos, w = torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    bse.sort_rows(x, pos, rows)
    bse.sort_rows(x, pos.view(-1), rows)
    for args in ((x, pos.long(), rows), (x, pos[:3].contiguous(), rows), (x, pos, rows[:, :32]), (x, pos, rows.half()),
                 (x.half(), pos, rows), (x, pos.view(-1)[:7], rows)):
        with pytest.raises(ValueError):
            bse.sort_rows(*args)
    with pytest.raises(ValueError):
        bse.combine_rows(rows, pos, w[:, :1].contiguous(), x)
    with pytest.raises(ValueError):
        bse.combine_rows(rows, pos, w.double(), x)
    with pytest.raises(ValueError):
        bse.combine_rows_backward(x, None, pos, w, None)
    with pytest.raises(bse.MoeError):
        bse.combine_rows_backward(x, rows, pos, w, None)
