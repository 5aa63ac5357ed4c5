"""Rows, norms and weights whose byte offsets pass 32 bits."""
import numpy as np
import pytest

from oracle import stream as S

pytestmark = pytest.mark.gpu


def _room(gib):
    import torch
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_norm_of_many_rows(gpu_lib):
    """300000 x 8192 bf16: 4.9 GB an array."""
    import torch
    _room(40)
    T, cols = 300000, 8192
    x = torch.randn((T, cols), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    gpu_lib.norm_forward(x, w, y, rstd=rstd)
    d, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    gpu_lib.norm_backward(y, x, w, rstd, d, gpu_lib.norm_workspace(T, cols), d_weight=dw)
    for t in (0, 131071, 131073, 262143, 262145, T - 1):
        want, r = S.norm_forward(x[t:t + 1].double().cpu().numpy(), np.ones(cols), 1e-6)
        assert (np.abs(y[t].double().cpu().numpy() - want[0]) <= 2.0 ** -8 * 1.01 * np.abs(want[0])).all()
        # dy = y, which is s r up to its rounding (2^-8 of each element): d is r times what that leaves
        dy, s = y[t:t + 1].double().cpu().numpy(), x[t:t + 1].double().cpu().numpy()
        ref, _ = S.norm_backward(dy, s, np.ones(cols), rstd[t:t + 1].double().cpu().numpy())
        tol = 2.0 ** -24 * float(rstd[t]) * 100 * (np.abs(dy) + np.abs(s)) + 2.0 ** -8 * np.abs(ref)
        assert (np.abs(d[t].double().cpu().numpy() - ref) <= tol).all()
    # the weight's gradient is the column sums of y n = n^2 up to roundings, near T
    assert (dw.cpu().numpy() > 0.9 * T).all() and (dw.cpu().numpy() < 1.1 * T).all()


def test_rows_of_many_pairs(gpu_lib):
    """262144 pairs of 9216 bf16: 4.8 GB."""
    import torch
    _room(40)
    T, k, cols = 32768, 8, 9216
    x = torch.randn((T, cols), device="cuda", dtype=torch.bfloat16)
    pos = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).int().cuda()
    rows = torch.zeros((T * k, cols), dtype=torch.bfloat16, device="cuda")
    gpu_lib.sort_rows(x, pos, rows)
    w = torch.full((T, k), 0.125, device="cuda")
    back = torch.empty_like(x)
    gpu_lib.combine_rows(rows, pos, w, back)
    assert torch.equal(back, x)                       # eight eighths of the same row
    p = pos.view(T, k).cpu().numpy()
    for t in (0, 1000, T - 1):
        for j in range(k):
            assert torch.equal(rows[int(p[t, j])], x[t])
    dy, dw = torch.zeros_like(rows), torch.empty((T, k), device="cuda")
    gpu_lib.combine_rows_backward(x, rows, pos, w, dy, dw)
    size = (x.double() ** 2).sum(1, keepdim=True)
    assert ((dw.double() - size).abs() <= 86 * 2.0 ** -24 * size).all()
    for t in (5, T - 2):
        assert torch.equal(dy[int(p[t, 3])], (x[t].float() * 0.125).bfloat16())
    dx = torch.empty_like(x)
    gpu_lib.sort_rows_backward(dy, pos, dx)
    assert torch.equal(dx, x)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_weights_past_four_gib(gpu_lib, fmt):
    """520 groups of 4096 x 4096: 4.4 GB of codes; the last group's rows."""
    import torch
    _room(20)
    G, N, K = 520, 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    nv = fmt == "nvfp4"
    sc = torch.randint(*((40, 80) if nv else (119, 123)), (G, N, K // (16 if nv else 32)), dtype=torch.uint8, device="cuda",
                       generator=g)
    gs = torch.full((G,), 0.5, device="cuda")
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[-1], off[-2] = 5, 2
    x = torch.randn((5, K), device="cuda", generator=g).bfloat16()
    out, alone = torch.empty((5, N), device="cuda"), torch.empty((5, N), device="cuda")
    gpu_lib.group_matvec(fmt, x, w, sc, off, out, gs=gs if nv else None)
    # the same rows with the two groups' matrices on their own: other workgroups, the same sums
    few = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    gpu_lib.group_matvec(fmt, x, w[-2:].clone(), sc[-2:].clone(), few, alone, gs=gs[-2:].clone() if nv else None)
    size = out.abs().max()
    assert float(size) > 0 and float((out - alone).abs().max()) <= K * 2.0 ** -23 * float(size)


@pytest.mark.parametrize("cols", [1003, 1000])
def test_streamed_sizes_give_the_same_rows(gpu_lib, cols):
    """Arrays past the last-level cache take streaming accesses: row for row the
    bits of smaller calls, at widths on and off 8 elements."""
    import torch
    _room(10)
    T, k = 70001, 4
    x, r = torch.randn((T, cols), device="cuda").bfloat16(), torch.randn((T, cols), device="cuda").bfloat16()
    w, dy = torch.rand(cols, device="cuda"), torch.randn((T, cols), device="cuda").bfloat16()

    def norm(x, r, dy):
        n = x.shape[0]
        y, s, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(n, device="cuda")
        gpu_lib.norm_forward(x, w, y, residual=r, res_out=s, rstd=rstd)
        d = torch.empty_like(x)
        gpu_lib.norm_backward(dy, s, w, rstd, d, d_res_out=r)
        return y, s, rstd, d

    whole = norm(x, r, dy)
    pos = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).int()
    pos[torch.randperm(T * k, generator=torch.Generator().manual_seed(2))[:T]] = -1
    at = pos.cuda()
    tw = torch.rand((T, k), device="cuda")
    rows = torch.randn((T * k, cols), device="cuda").bfloat16()
    out, dyr, dw = torch.empty_like(x), torch.zeros_like(rows), torch.empty_like(tw)
    gpu_lib.combine_rows(rows, at, tw, out)
    gpu_lib.combine_rows_backward(x, rows, at, tw, dyr, dw)
    back = torch.zeros_like(rows)
    gpu_lib.sort_rows(x, at, back)
    for lo in (0, 35000, T - 90):
        cut = slice(lo, lo + 90)
        for a, b in zip(whole, norm(x[cut].clone(), r[cut].clone(), dy[cut].clone())):
            assert torch.equal(a[cut], b)
        p = pos.view(T, k)[cut].flatten()
        live = (p >= 0).nonzero()[:, 0]
        few = torch.full_like(p, -1)
        few[live] = torch.arange(live.numel(), dtype=torch.int32)
        mine, here = few.cuda(), p[live].long().cuda()
        o2, d2, w2 = torch.empty_like(out[cut]), torch.zeros((live.numel(), cols), dtype=torch.bfloat16, device="cuda"), torch.empty((90, k), device="cuda")
        gpu_lib.combine_rows(rows[here].contiguous(), mine, tw[cut].contiguous(), o2)
        assert torch.equal(o2, out[cut])
        gpu_lib.combine_rows_backward(x[cut].contiguous(), rows[here].contiguous(), mine, tw[cut].contiguous(), d2, w2)
        assert torch.equal(d2, dyr[here]) and torch.equal(w2, dw[cut])
        assert torch.equal(back[here], x[cut][(live // k).cuda()])
