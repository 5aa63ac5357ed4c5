"""examples/router_tuning_mxfp4.py: the calls together, against moe_forward,
against differences of the balance loss, and over a run."""
import importlib.util
import os

import numpy as np
import pytest

from tests._util import OUT_RTOL

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "router_tuning_mxfp4.py")


@pytest.fixture
def tuning():
    spec = importlib.util.spec_from_file_location("router_tuning_mxfp4", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _layer(tuning, bse, T):
    import torch
    g = torch.Generator().manual_seed(3)
    cfg = bse.Config(hidden=384, ffn=128, num_experts=12, top_k=3, fmt="mxfp4", max_tokens=T)
    w13 = (torch.randn(12, 256, 384, generator=g) * 0.08).cuda()
    w2 = (torch.randn(12, 384, 128, generator=g) * 0.1).cuda()
    bounds = torch.tensor([0, 1, 1, T], dtype=torch.int32, device="cuda")
    x = torch.randn(T, 384, generator=g).bfloat16().cuda()
    w_router = (torch.randn(12, 384, generator=g) * 0.08).cuda()
    return tuning.Layer(cfg, tuning.Experts(cfg, w13, w2), T, bounds), x, w_router


@pytest.mark.parametrize("T", [1, 45])
def test_steps_match_the_layer(gpu_lib, tuning, T):
    import torch
    layer, x, w_router = _layer(tuning, gpu_lib, T)
    got = layer.forward(x, w_router.bfloat16())
    out = torch.empty((T, 384), dtype=torch.bfloat16, device="cuda")
    gpu_lib.forward(layer.cfg, x, layer.ids, layer.topk_w, layer.experts.as_weights(), out, layer.ws)
    err = (got - out.float()).abs().max() / out.float().abs().max()
    assert float(err) <= OUT_RTOL


def test_router_gradient_against_differences(gpu_lib, tuning):
    """The chain from the logits to both losses, differenced in 64 bits with
    the selection held: d_out . out + balance, out linear in the gate weights."""
    import torch
    T, E, eps = 45, 12, 1e-5
    layer, x, w_router = _layer(tuning, gpu_lib, T)
    out = layer.forward(x, w_router.bfloat16())
    d_out = torch.randn(out.shape, generator=torch.Generator().manual_seed(4)).cuda()
    layer.backward(x, d_out, 3.0)
    z, ids = layer.z.cpu().double().numpy(), layer.ids.cpu().numpy()
    share = (layer.expert_out.double() * d_out.double()[:, None]).sum(2).cpu().numpy()
    bounds = layer.bounds.cpu().numpy()
    counts = layer.counts.cpu().double().numpy()
    live = layer.live.cpu().numpy()

    def value(zz):
        s = 1.0 / (1.0 + np.exp(-zz))
        sel = np.take_along_axis(s, ids, 1)
        total = (sel / sel.sum(1, keepdims=True) * share).sum()
        p = s / s.sum(1, keepdims=True)
        for q in range(3):
            if live[q]:
                total += 3.0 / 3 * E / (3 * live[q]) * (counts[q] * p[bounds[q]:bounds[q + 1]].mean(0)).sum()
        return total

    dz = layer.dz.cpu().numpy()
    rng = np.random.default_rng(5)
    for _ in range(40):
        t, e = rng.integers(T), rng.integers(E)
        hi, lo = z.copy(), z.copy()
        hi[t, e] += eps
        lo[t, e] -= eps
        d = (value(hi) - value(lo)) / (2 * eps)
        # differences: eps^2 and 64-bit cancellation, below 1e-8 of the terms; dz: fp32 sums of k shares
        assert abs(dz[t, e] - d) <= 1e-5 * (np.abs(share[t]).max() + 1.0)


def test_run_lowers_both_losses(gpu_lib, tuning):
    history = tuning.run(steps=40)
    assert all(np.isfinite(a).all() for a in history)
    first, last = np.array(history[0]), np.array(history[-1])
    assert last[0] < first[0] and last[1] < first[1]
