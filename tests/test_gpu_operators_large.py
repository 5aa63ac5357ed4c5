"""MXFP4, grouped product and balance loss on tensors whose byte offsets pass
32 bits: the ends of the outputs against the oracle, which sees those rows only."""
import numpy as np
import pytest

from oracle import balance as B
from oracle import formats as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,M,N,f32", [(1, (1 << 20) + 5, 2112, False),       # tiles; 4.4 GB of output
                                       (110, 1100, 1 << 20, True)])            # streamed; 4.6 GB
def test_product(gpu_lib, G, M, N, f32):
    import torch
    K = 32
    gen = torch.Generator(device="cuda").manual_seed(M)
    codes = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=gen)  # noqa: E731
    a, w = codes(M, K // 2), codes(G, N, K // 2)
    a_sc = torch.randint(120, 126, (M, 1), dtype=torch.uint8, device="cuda", generator=gen)
    w_sc = torch.randint(120, 126, (G, N, 1), dtype=torch.uint8, device="cuda", generator=gen)
    offsets = torch.tensor([M * i // G for i in range(G + 1)], dtype=torch.int32, device="cuda")
    out = torch.full((M, N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    gpu_lib.group_product("mxfp4", a, a_sc, w, w_sc, offsets, out)
    rows, cols = slice(M - 7, M), slice(N - 2000, N)
    got = out[rows, cols].float().cpu().numpy()
    first = out[:7, :2000].float().cpu().numpy()
    assert not torch.isnan(out[::997]).any()
    for o, r, c, g in ((got, rows, cols, G - 1), (first, slice(0, 7), slice(0, 2000), 0)):
        av = F.dequantize_mxfp4(a[r].cpu().numpy(), a_sc[r].cpu().numpy())
        wv = F.dequantize_mxfp4(w[g, c].cpu().numpy(), w_sc[g, c].cpu().numpy())
        ref, size = av @ wv.T, np.abs(av) @ np.abs(wv).T
        assert (np.abs(o - ref) <= (K / 128 + 8) * 2.0 ** -22 * size + (0 if f32 else 2.0 ** -8 * np.abs(ref))).all()


def test_encode_and_decode(gpu_lib):
    import torch
    R, K = 480_007, 4608                      # 2.2e9 elements, 4.4 GB of bf16, 8.8 of fp32
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    codes = torch.empty((1, R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, R, K // 32), dtype=torch.uint8, device="cuda")
    gpu_lib.encode_weights("mxfp4", x[None], codes, scales)
    for r in (slice(0, 9), slice(R - 9, R)):
        c, s = F.quantize_mxfp4(x[r].float().cpu().numpy())
        assert np.array_equal(codes[0, r].cpu().numpy(), c) and np.array_equal(scales[0, r].cpu().numpy(), s)
    tail = x[R - 9:].float().cpu().numpy()
    del x
    out = torch.empty((1, R, K), dtype=torch.float32, device="cuda")
    gpu_lib.decode_weights("mxfp4", codes, scales, out)
    assert np.array_equal(out[0, R - 9:].cpu().numpy(), F.dequantize_mxfp4(*F.quantize_mxfp4(tail)).astype(np.float32))


def test_balance(gpu_lib):
    """2.2e9 logits; the last sequence is 40 tokens and is checked whole."""
    import torch
    T, E, k, n = 2_200_040, 1024, 4, 40
    gen = torch.Generator(device="cuda").manual_seed(6)
    z = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=gen)
    bounds = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    cfg = gpu_lib.Config(num_experts=E, top_k=k)
    counts, live = torch.empty((2, E), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    probs, loss = torch.empty((2, E), device="cuda"), torch.empty(2, device="cuda")
    ws = gpu_lib.balance_workspace(cfg, T, 2)
    gpu_lib.balance_forward(cfg, z, ids, counts, live, probs, loss, ws, seq_offsets=bounds)
    dz = torch.empty_like(z)
    d_loss = torch.tensor([2.0, 3.0], device="cuda")
    gpu_lib.balance_backward(cfg, z, ids, counts, live, d_loss, dz, seq_offsets=bounds)
    zt, it = z[T - n:].float().cpu().numpy(), ids[T - n:].cpu().numpy()
    ref = B.balance_forward(zt, it, E, k)
    assert live.cpu().tolist() == [T - n, n]
    assert torch.equal(counts[0].long(), torch.bincount(ids[:T - n].reshape(-1).long(), minlength=E))
    assert np.array_equal(counts[1].cpu().numpy(), ref["counts"][0])
    tol = 2e-6 + n * 2.0 ** -24
    assert (np.abs(probs[1].cpu().numpy() - ref["probs"][0]) <= tol * ref["probs"][0]).all()
    assert abs(float(loss[1]) - ref["loss"][0]) <= (tol + 2e-6) * ref["loss"][0]
    want, size = B.balance_backward(zt, it, ref, np.array([3.0]), E, k)
    got = dz[T - n:].float().cpu().numpy()
    assert (np.abs(got - want) <= 4e-6 * size + 2.0 ** -8 * np.abs(want) + 1e-37).all()


def test_balance_of_a_long_sequence(gpu_lib):
    """Equal logits give 1/E however many tokens there are, though the rounding
    errors of equal terms do not average out.  Bound: a probability 2e-6; runs
    of at most 256 additions, joined over 32 runs, 4 waves, 32 slots of one
    lane group and 4 + 16 partial sums, each within 2^-24."""
    import torch
    T, E = 1 << 26, 5
    cfg = gpu_lib.Config(num_experts=E, top_k=1)
    z = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    ids = (torch.arange(T, dtype=torch.int32, device="cuda") % E).reshape(T, 1)
    counts, live = torch.empty((1, E), dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    probs, loss = torch.empty((1, E), device="cuda"), torch.empty(1, device="cuda")
    gpu_lib.balance_forward(cfg, z, ids, counts, live, probs, loss, gpu_lib.balance_workspace(cfg, T))
    assert live.cpu().tolist() == [T]
    assert counts[0].cpu().tolist() == [(T - e + E - 1) // E for e in range(E)]
    tol = 2e-6 + (256 + 32 + 4 + 32 + 20) * 2.0 ** -24
    assert (probs[0].double() * E - 1).abs().max().item() <= tol
    assert abs(loss[0].item() - 1) <= tol + 2e-6
