"""MXFP4 on the GPU against the oracle: encoder (activations and matrices),
decoder, and the whole layer in the format.  Codes, scales and decoded values
must be bit-identical."""
import numpy as np
import pytest

import synth
from oracle import formats as F
from oracle import layer as L
from tests._util import OUT_RTOL, rel_err, to_dev

pytestmark = pytest.mark.gpu


def _rows(R, cols, seed, f32):
    g = np.random.default_rng(seed)
    v = g.standard_normal((R, cols)).astype(np.float32)
    v *= np.exp(g.uniform(-20, 20, (R, 1))).astype(np.float32)
    kinds = [lambda r: r * 0, lambda r: r * np.float32(1e-38), lambda r: np.full_like(r, 9.2e-41),
             lambda r: np.sign(r) * np.float32(3e38), lambda r: -np.abs(r),
             lambda r: np.resize(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0, 4.0], np.float32),
                                 r.size)]
    for i, f in enumerate(kinds):
        if i < R:
            v[i] = f(v[i])
    v[-1, ::3] = -0.0
    if not f32:
        v = F.bf16_bits_to_f32(synth.to_bf16_bits(v))
    return v


def _upload(v, f32):
    import torch
    if f32:
        return torch.from_numpy(v).cuda()
    return to_dev(synth.to_bf16_bits(v).view(np.int16)).view(torch.bfloat16)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("R,cols", [(1, 32), (7, 96), (64, 4608), (3, 2336), (257, 160)])
def test_encode_rows_bit_exact(gpu_lib, R, cols, f32):
    import torch
    v = _rows(R, cols, R + cols, f32)
    codes = torch.full((R, cols // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, cols // 32), 0xAA, dtype=torch.uint8, device="cuda")
    gpu_lib.quantize_act("mxfp4", _upload(v, f32), codes, scales)
    out = torch.empty((1, R, cols), dtype=torch.float32, device="cuda")
    gpu_lib.decode_weights("mxfp4", codes[None], scales[None], out)
    c, s = F.quantize_mxfp4(v)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(out[0].cpu().numpy(), F.dequantize_mxfp4(c, s).astype(np.float32))


def test_encode_nan_and_infinity(gpu_lib):
    """A NaN encodes as +0 and leaves its block's scale to the other elements;
    an infinity saturates at 6 times the largest scale."""
    import torch
    v = np.random.default_rng(1).standard_normal((4, 64)).astype(np.float32)
    v[0, 5] = np.nan
    v[1, :32] = np.nan
    v[2, 40], v[2, 41] = np.inf, -np.inf
    v[3, 0] = -np.nan
    codes = torch.empty((4, 32), dtype=torch.uint8, device="cuda")
    scales = torch.empty((4, 2), dtype=torch.uint8, device="cuda")
    gpu_lib.quantize_act("mxfp4", torch.from_numpy(v).cuda(), codes, scales)
    c, s = F.quantize_mxfp4(v)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_encode_matrices_and_every_code(gpu_lib):
    """Matrices through encode_weights; the decoder over every code under the
    smallest, a middle and the largest scale."""
    import torch
    v = _rows(3 * 40, 352, 9, True).reshape(3, 40, 352)
    codes = torch.empty((3, 40, 176), dtype=torch.uint8, device="cuda")
    scales = torch.empty((3, 40, 11), dtype=torch.uint8, device="cuda")
    gpu_lib.encode_weights("mxfp4", torch.from_numpy(v).cuda(), codes, scales)
    c, s = F.quantize_mxfp4(v)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    every = np.resize(np.arange(256, dtype=np.uint8), (1, 254, 16))
    sc = np.arange(254, dtype=np.uint8).reshape(1, 254, 1)      # up to 2^126: 4 and 6 overflow to inf there
    out = torch.empty((1, 254, 32), dtype=torch.float32, device="cuda")
    gpu_lib.decode_weights("mxfp4", to_dev(every), to_dev(sc), out)
    assert np.array_equal(out.cpu().numpy(), F.dequantize_mxfp4(every, sc).astype(np.float32))


def _layer(H, Fd, E, k, T, seed, **kw):
    x = synth.tokens(seed, T, H)
    wr, b = synth.router_weight(seed, E, H), synth.router_bias(seed, E)
    lo, n = kw.get("expert_begin", 0), kw.get("num_local") or E
    ews = [L.quantize_expert_weights("mxfp4", *synth.expert_float_weights(seed, e, H, Fd, 0.05))
           for e in range(lo, lo + n)]
    ocfg = L.OracleConfig(hidden=H, ffn=Fd, num_experts=E, top_k=k, fmt="mxfp4", expert_begin=lo, num_local=n)
    return x, wr, b, ews, ocfg


@pytest.mark.parametrize("call", ["forward", "fused", "route_forward", "noalloc"])
@pytest.mark.parametrize("H,Fd,E,k,T,local", [(256, 128, 16, 2, 16, None), (512, 384, 24, 4, 1, None),
                                              (256, 256, 12, 3, 700, (4, 5))])
def test_layer_mxfp4(gpu_lib, call, H, Fd, E, k, T, local):
    """The layer with MXFP4 experts, by every call that takes the format."""
    import torch
    kw = {} if local is None else dict(expert_begin=local[0], num_local=local[1])
    x, wr, b, ews, ocfg = _layer(H, Fd, E, k, T, 3, **kw)
    cfg = gpu_lib.Config(hidden=H, ffn=Fd, num_experts=E, top_k=k, fmt="mxfp4", max_tokens=T,
                         expert_begin=ocfg.expert_begin, num_local_experts=ocfg.num_local)
    ws = gpu_lib.workspace(cfg)
    xt = to_dev(x.view(np.int16)).view(torch.bfloat16)
    wrt = to_dev(wr.view(np.int16)).view(torch.bfloat16)
    wd = {n: to_dev(np.stack([e[n] for e in ews])) for n in ("w13", "w13_sc", "w2", "w2_sc")}
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    bt = to_dev(b)
    if call == "route_forward":
        gpu_lib.route_forward(cfg, xt, wrt, bt, ids, tw, None, wd, out, ws)
    else:
        gpu_lib.route(cfg, xt, wrt, bt, ids, tw, None, ws)
        if call == "noalloc":
            gpu_lib.forward_noalloc(cfg, xt, ids, tw, wd, out)
        else:
            gpu_lib.forward(cfg, xt, ids, tw, wd, out, ws, fused=call == "fused")
    torch.cuda.synchronize()
    ref = L.moe_layer(ocfg, x, wr, b, ews, topk_ids=ids.cpu().numpy(), topk_w=tw.cpu().numpy())["out"]
    assert rel_err(out.view(torch.int16).cpu().numpy().view(np.uint16), ref) <= OUT_RTOL


def test_route_logits_are_the_routers(gpu_lib):
    """z from the workspace: the scores the gate weights came from, for the
    split (small) and the tiled (large) router."""
    import torch
    for T in (5, 300):
        H, E, k = 512, 96, 4
        x, wr, b = synth.tokens(7, T, H), synth.router_weight(7, E, H), synth.router_bias(7, E)
        cfg = gpu_lib.Config(hidden=H, ffn=128, num_experts=E, top_k=k, fmt="mxfp4", max_tokens=T, norm_topk=False)
        ws = gpu_lib.workspace(cfg)
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
        z = torch.empty((T, E), dtype=torch.float32, device="cuda")
        gpu_lib.route(cfg, to_dev(x.view(np.int16)).view(torch.bfloat16),
                      to_dev(wr.view(np.int16)).view(torch.bfloat16), to_dev(b), ids, tw, None, ws)
        gpu_lib.route_logits(cfg, T, z, ws)
        ref = L.route(L.OracleConfig(hidden=H, ffn=128, num_experts=E, top_k=k, fmt="mxfp4"), x, wr, b)["logits"]
        # fp32 sums of H bf16 products: H roundings of at most 2^-24 of the magnitudes' sum
        size = np.abs(F.bf16_bits_to_f32(x)).astype(np.float64) @ np.abs(F.bf16_bits_to_f32(wr)).astype(np.float64).T
        assert (np.abs(z.cpu().numpy() - ref) <= H * 2.0 ** -24 * size).all()
        s = 1.0 / (1.0 + np.exp(-z.cpu().numpy().astype(np.float64)))
        got = np.take_along_axis(s, ids.cpu().numpy().astype(np.int64), 1)
        assert np.abs(got - tw.cpu().numpy()).max() <= 4e-7      # expf and the division, a few ulp of a score below 1


def test_decode_every_scale(gpu_lib):
    """Every code under every scale byte: 2^127 still decodes, 255 (E8M0's NaN)
    makes its whole block NaN, as it does in the product."""
    import torch
    codes = np.tile(np.arange(256, dtype=np.uint8), (1, 256, 1))          # 16 blocks a row: every byte
    sc = np.repeat(np.arange(256, dtype=np.uint8).reshape(1, 256, 1), 16, axis=2)
    out = torch.empty((1, 256, 512), dtype=torch.float32, device="cuda")
    gpu_lib.decode_weights("mxfp4", to_dev(codes), to_dev(sc), out)
    with np.errstate(over="ignore"):
        ref = F.dequantize_mxfp4(codes, sc).astype(np.float32)
    got = out.cpu().numpy()
    assert np.isnan(got[0, 255]).all() and not np.isnan(got[0, :255]).any()
    assert np.array_equal(got, ref, equal_nan=True)
