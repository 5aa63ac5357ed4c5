"""moe_balance_forward / moe_balance_backward against the float64 oracle.

Tolerances: a probability is a quotient of fp32 sigmoids (exponential,
reciprocal, the row's sum and its reciprocal): 2e-6 of itself.  A mean over n
tokens adds them in fp32 in runs no longer than RUN: RUN * 2^-24 more.  A
gradient's terms carry 4e-6 each; size is the sum of their magnitudes.  bf16
outputs add half an ulp."""
import numpy as np
import pytest

import synth
from oracle import balance as B
from oracle import formats as F
from tests._util import to_dev

pytestmark = pytest.mark.gpu

RUN = 256


def _inputs(seed, T, E, k, f32=True, spread=2.0):
    g = np.random.default_rng(seed)
    z = (g.standard_normal((T, E)) * spread).astype(np.float32)
    if not f32:
        z = F.bf16_bits_to_f32(synth.to_bf16_bits(z))
    ids = np.argsort(-z + g.standard_normal((T, E)), axis=1)[:, :k].astype(np.int32)
    d_w = g.standard_normal((T, k)).astype(np.float32)
    return z, ids, d_w


def _call(lib, z, ids, E, k, f32=True, bounds=None, mask=None, d_w=None, d_loss=None, norm=True, scale=1.0):
    import torch
    T = z.shape[0]
    S = 1 if bounds is None else len(bounds) - 1
    cfg = lib.Config(num_experts=E, top_k=k, norm_topk=norm, routed_scale=scale)
    zt = torch.from_numpy(z).cuda()
    zt = zt if f32 else zt.bfloat16()
    dev = lambda v, dt: None if v is None else to_dev(np.asarray(v, dtype=dt))  # noqa: E731
    idt, bt, mt, dwt = dev(ids, np.int32), dev(bounds, np.int32), dev(mask, np.uint8), dev(d_w, np.float32)
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    live = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((S, E), float("nan"), device="cuda")
    loss = torch.full((S,), float("nan"), device="cuda")
    ws = lib.balance_workspace(cfg, T, S)
    ws.fill_(0xEE)
    lib.balance_forward(cfg, zt, idt, counts, live, probs, loss, ws, seq_offsets=bt, token_mask=mt)
    dl = dev(np.linspace(0.5, 2.0, S) if d_loss is None else d_loss, np.float32)
    dz = torch.full_like(zt, float("nan"))
    lib.balance_backward(cfg, zt, idt, counts, live, dl, dz, d_topk_w=dwt, seq_offsets=bt, token_mask=mt)
    torch.cuda.synchronize()
    return dict(counts=counts.cpu().numpy(), live=live.cpu().numpy(), probs=probs.cpu().numpy(),
                loss=loss.cpu().numpy(), dz=dz.float().cpu().numpy(), d_loss=dl.cpu().numpy())


def _check(got, z, ids, E, k, f32=True, bounds=None, mask=None, d_w=None, norm=True, scale=1.0):
    ref = B.balance_forward(z, ids, E, k, bounds, mask)
    assert np.array_equal(got["counts"], ref["counts"])
    assert np.array_equal(got["live"], ref["live"])
    tol = 2e-6 + RUN * 2.0 ** -24
    assert (np.abs(got["probs"] - ref["probs"]) <= tol * ref["probs"] + 1e-38).all()
    assert (np.abs(got["loss"] - ref["loss"]) <= (tol + 2e-6) * ref["loss"]).all()
    dz, size = B.balance_backward(z, ids, ref, got["d_loss"], E, k, bounds, mask, d_w, norm, scale)
    lim = 4e-6 * size + (0 if f32 else 2.0 ** -8 * np.abs(dz)) + 1e-37
    bad = ~(np.abs(got["dz"] - dz) <= lim)
    assert not bad.any(), (np.argwhere(bad)[:4], got["dz"][bad][:4], dz[bad][:4])


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 384, 8), (5, 2, 2), (64, 384, 8), (33, 63, 3), (40, 64, 1),
                                   (17, 65, 5), (300, 130, 8), (21, 256, 6), (70, 513, 16), (19, 1024, 32),
                                   (1500, 40, 4)])
def test_one_sequence(gpu_lib, T, E, k, f32):
    z, ids, d_w = _inputs(T + E, T, E, k, f32)
    _check(_call(gpu_lib, z, ids, E, k, f32, d_w=d_w), z, ids, E, k, f32, d_w=d_w)


@pytest.mark.parametrize("norm,scale", [(True, 2.5), (False, 1.0), (False, 0.5)])
def test_gate_forms(gpu_lib, norm, scale):
    z, ids, d_w = _inputs(2, 50, 96, 6)
    _check(_call(gpu_lib, z, ids, 96, 6, d_w=d_w, norm=norm, scale=scale), z, ids, 96, 6, d_w=d_w, norm=norm,
           scale=scale)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,bounds", [
    (100, [0, 1, 1, 40, 100]),                 # lengths of one and zero
    (100, [0, 0, 100, 100]),                   # empty first and last
    (200, [10, 30, 150]),                      # tokens before and after every sequence
    (90, list(range(0, 91, 3))),               # many short sequences
    (1200, [0, 600, 601, 1200]),
])
def test_sequences_and_masks(gpu_lib, T, bounds, f32):
    E, k = 70, 4
    z, ids, d_w = _inputs(T, T, E, k, f32)
    mask = (np.random.default_rng(T).random(T) < 0.7).astype(np.uint8)
    mask[:min(bounds[1], T)] = 0               # the first sequence has no live token
    z[mask == 0] = np.nan                      # nothing of a masked token is read
    ids[mask == 0] = 1 << 30
    d_w[mask == 0] = np.nan
    for m in (mask, mask * 200):               # any non-zero byte is a token
        got = _call(gpu_lib, z, ids, E, k, f32, bounds, m, d_w)
        _check(got, z, ids, E, k, f32, bounds, mask, d_w)
    assert (got["dz"][mask == 0] == 0).all()


def test_no_gate_gradient_and_no_tokens(gpu_lib):
    z, ids, _ = _inputs(6, 30, 48, 4)
    _check(_call(gpu_lib, z, ids, 48, 4), z, ids, 48, 4)
    got = _call(gpu_lib, z[:0], ids[:0], 48, 4)
    assert (got["counts"] == 0).all() and (got["live"] == 0).all() and (got["loss"] == 0).all()
    assert (got["probs"] == 0).all()
    got = _call(gpu_lib, z, ids, 48, 4, mask=np.zeros(30))
    assert (got["loss"] == 0).all() and (got["probs"] == 0).all() and (got["dz"] == 0).all()


def test_extreme_logits(gpu_lib):
    """Experts switched off by -inf, rows far below zero (where the sigmoids
    themselves underflow), rows far above, +inf, a row of only -inf."""
    E, k = 100, 4
    z, ids, d_w = _inputs(7, 12, E, k)
    z[0, ::3] = -np.inf
    z[1] -= 60.0
    z[2] -= 300.0
    z[3] += 60.0
    z[4, 5] = np.inf
    z[5] = -np.inf
    z[6] = np.where(np.arange(E) == 3, -40.0, -np.inf)
    z[7] = np.linspace(-3.0e38, -1.0e38, E)
    z[8] = np.linspace(-40.0, 40.0, E)
    z[9] = -28.0
    z[10] = 0.0
    _check(_call(gpu_lib, z, ids, E, k, d_w=d_w), z, ids, E, k, d_w=d_w)
    _check(_call(gpu_lib, z, ids, E, k, d_w=d_w, norm=False), z, ids, E, k, d_w=d_w, norm=False)


def test_nan_stays_in_its_sequence(gpu_lib):
    E, k, bounds = 20, 2, [0, 10, 20]
    z, ids, d_w = _inputs(8, 20, E, k)
    z[3, 4] = np.nan
    got = _call(gpu_lib, z, ids, E, k, bounds=bounds, d_w=d_w)
    assert np.isnan(got["loss"][0]) and np.isfinite(got["loss"][1])
    assert np.isnan(got["dz"][3]).all() and np.isfinite(np.delete(got["dz"], 3, 0)).all()


def test_ids_out_of_range_and_repeated(gpu_lib):
    """Replayed routing: ids outside [0, E) are not counted and take no gate
    gradient; a repeated id counts and adds twice."""
    E, k = 30, 4
    z, ids, d_w = _inputs(9, 40, E, k)
    ids[0, 1], ids[1, 0], ids[2] = -1, E, -1
    ids[3, 1] = ids[3, 0]
    _check(_call(gpu_lib, z, ids, E, k, d_w=d_w), z, ids, E, k, d_w=d_w)


def test_against_differences(gpu_lib):
    """The gradient against central differences of the float64 loss, the
    counts held fixed.  The difference's own error: h^2/6 of the third
    derivative (below 10 of the terms' size) and 2^-50 of the loss over h."""
    E, k, T, bounds = 10, 3, 6, [0, 2, 6]
    z, ids, d_w = _inputs(10, T, E, k)
    mask = np.array([1, 1, 1, 0, 1, 1], np.uint8)
    got = _call(gpu_lib, z, ids, E, k, bounds=bounds, mask=mask, d_w=d_w, scale=1.5)
    fwd = B.balance_forward(z, ids, E, k, bounds, mask)
    _, size = B.balance_backward(z, ids, fwd, got["d_loss"], E, k, bounds, mask, d_w, True, 1.5)
    f = lambda zz: B.balance_loss(zz, ids, got["d_loss"], E, k, fwd["counts"], bounds, mask, d_w, True, 1.5)  # noqa: E731
    h, base = 1e-4, z.astype(np.float64)
    for t in range(T):
        for e in range(E):
            up, dn = base.copy(), base.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = (f(up) - f(dn)) / (2 * h)
            assert abs(got["dz"][t, e] - d) <= 4e-6 * size[t, e] + 10 * h * h * size[t].sum() + 2.0 ** -50 * 20 / h


def test_same_bits_and_graph(gpu_lib):
    """Every run gives the same bits, also replayed from a HIP graph with
    other work between the replays."""
    import torch
    E, k, T = 384, 8, 900
    z, ids, d_w = _inputs(11, T, E, k)
    first = _call(gpu_lib, z, ids, E, k, d_w=d_w)
    again = _call(gpu_lib, z, ids, E, k, d_w=d_w)
    for n in first:
        assert np.array_equal(first[n], again[n]), n
    cfg = gpu_lib.Config(num_experts=E, top_k=k)
    zt, idt, dwt = torch.from_numpy(z).cuda(), to_dev(ids), to_dev(d_w)
    ws = gpu_lib.balance_workspace(cfg, T)
    counts = torch.zeros((1, E), dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    probs, loss = torch.zeros((1, E), device="cuda"), torch.zeros(1, device="cuda")
    dl, dz = torch.full((1,), 0.5, device="cuda"), torch.zeros_like(zt)

    def step():
        gpu_lib.balance_forward(cfg, zt, idt, counts, live, probs, loss, ws)
        gpu_lib.balance_backward(cfg, zt, idt, counts, live, dl, dz, d_topk_w=dwt)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in (counts, live, probs, loss, dz):
            t.fill_(3)
        ws.fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(counts.cpu().numpy(), first["counts"]) and np.array_equal(loss.cpu().numpy(), first["loss"])
        assert np.array_equal(dz.cpu().numpy(), first["dz"]) and np.array_equal(probs.cpu().numpy(), first["probs"])


def test_binding_refusals(gpu_lib):
    import torch
    E, k, T = 16, 2, 5
    cfg = gpu_lib.Config(num_experts=E, top_k=k)
    z = torch.zeros((T, E), device="cuda")
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    counts = torch.zeros((1, E), dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    probs, loss = torch.zeros((1, E), device="cuda"), torch.zeros(1, device="cuda")
    ws = gpu_lib.balance_workspace(cfg, T)
    ok = [z, ids, counts, live, probs, loss, ws]
    gpu_lib.balance_forward(cfg, *ok)
    for i, bad in ((0, z.half()), (0, z[:, :8]), (0, z.t().contiguous().t()), (1, ids.long()), (2, counts[:, :4]),
                   (3, live.float()), (4, probs.cpu()), (5, loss.double())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            gpu_lib.balance_forward(cfg, *args)
    with pytest.raises(gpu_lib.MoeError) as e:
        gpu_lib.balance_forward(cfg, *ok[:6], ws[:256])
    assert e.value.status == -3
    with pytest.raises(ValueError):
        gpu_lib.balance_backward(cfg, z, ids, counts, live, loss, z.bfloat16())


# sizes on both sides of the one-launch forward's bounds (128 tokens; tokens
# times groups of 64 experts up to 384), sequences of unequal length in each
@pytest.mark.parametrize("T,E,k", [(64, 384, 8), (65, 384, 8), (24, 1024, 16), (25, 1024, 16), (128, 192, 4),
                                   (129, 64, 4), (2, 1024, 32)])
def test_few_and_more_tokens(gpu_lib, T, E, k):
    z, ids, d_w = _inputs(T * 3 + E, T, E, k)
    mask = (np.arange(T) % 5 != 3).astype(np.uint8)
    for bounds in (None, [0, 0, 1, T - 1, T], [1, 1, T]):
        _check(_call(gpu_lib, z, ids, E, k, bounds=bounds, mask=mask, d_w=d_w), z, ids, E, k, bounds=bounds,
               mask=mask, d_w=d_w)


def test_extremes_among_many_tokens(gpu_lib):
    """The extreme rows where the forward takes two launches: repeated over
    160 tokens, and a NaN that stays in its sequence."""
    E, k = 100, 4
    z, ids, d_w = _inputs(12, 160, E, k)
    z[0::16, ::3] = -np.inf
    z[1::16] -= 60.0
    z[2::16] -= 300.0
    z[3::16] += 60.0
    z[4::16, 5] = np.inf
    z[5::16] = -np.inf
    z[6::16] = np.where(np.arange(E) == 3, -40.0, -np.inf)
    z[7::16] = np.linspace(-3.0e38, -1.0e38, E)
    z[8::16] = -28.0
    _check(_call(gpu_lib, z, ids, E, k, d_w=d_w), z, ids, E, k, d_w=d_w)
    z[20, 4] = np.nan
    got = _call(gpu_lib, z, ids, E, k, bounds=[0, 80, 160], d_w=d_w)
    assert np.isnan(got["loss"][0]) and np.isfinite(got["loss"][1])
    assert np.isnan(got["dz"][20]).all() and np.isfinite(np.delete(got["dz"], 20, 0)).all()
