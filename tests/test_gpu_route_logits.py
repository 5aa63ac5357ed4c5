"""moe_route_logits after either call that routes: the logits behind the
selection, the same bits from moe_route and from moe_route_forward (whose
small batches route in one launch in two of the formats)."""
import numpy as np
import pytest

import synth
from oracle import formats as F
from oracle import layer as L
from tests._util import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T", [1, 33, 256, 300])
def test_after_route_and_route_forward(gpu_lib, fmt, T):
    import torch
    H, Fd, E, k, seed, most = 512, 128, 96, 4, 11, 300
    x, wr, b = synth.tokens(seed, T, H), synth.router_weight(seed, E, H), synth.router_bias(seed, E)
    ews = [L.quantize_expert_weights(fmt, *synth.expert_float_weights(seed, e, H, Fd, 0.05)) for e in range(E)]
    wd = {n: to_dev(np.stack([np.asarray(e[n]) for e in ews])) for n in ews[0]}
    cfg = gpu_lib.Config(hidden=H, ffn=Fd, num_experts=E, top_k=k, fmt=fmt, max_tokens=most, norm_topk=False)
    xt = to_dev(x.view(np.int16)).view(torch.bfloat16)
    wrt, bt = to_dev(wr.view(np.int16)).view(torch.bfloat16), to_dev(b)
    got = []
    for one_call in (False, True):
        ws = gpu_lib.workspace(cfg)
        ws.fill_(0xEE)
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
        z = torch.full((T, E), float("nan"), device="cuda")
        if one_call:
            out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            gpu_lib.route_forward(cfg, xt, wrt, bt, ids, tw, None, wd, out, ws)
        else:
            gpu_lib.route(cfg, xt, wrt, bt, ids, tw, None, ws)
        gpu_lib.route_logits(cfg, T, z, ws)
        got.append((z.cpu().numpy(), ids.cpu().numpy(), tw.cpu().numpy()))
    for a, c in zip(*got):
        assert np.array_equal(a, c)
    z, ids, tw = got[0]
    ref = L.route(L.OracleConfig(hidden=H, ffn=Fd, num_experts=E, top_k=k, fmt=fmt), x, wr, b)["logits"]
    # fp32 sums of H bf16 products: H roundings of at most 2^-24 of the magnitudes' sum
    size = np.abs(F.bf16_bits_to_f32(x)).astype(np.float64) @ np.abs(F.bf16_bits_to_f32(wr)).astype(np.float64).T
    assert (np.abs(z - ref) <= H * 2.0 ** -24 * size).all()
    s = np.take_along_axis(1.0 / (1.0 + np.exp(-z.astype(np.float64))), ids.astype(np.int64), 1)
    assert np.abs(s - tw).max() <= 4e-7      # expf and the division, a few ulp of a score below 1
