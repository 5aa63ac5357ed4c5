"""The capped SwiGLU that encodes h in the MXFP4 layer, element by element:
with one expert a token, gate weight 1 and the identity as down matrix, the
layer's output is h's decoded MXFP4 value."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import layer as L
from tests._util import to_dev

pytestmark = pytest.mark.gpu

REL = 2e-5      # of moe_cap_swiglu's values, the same device function (test_gpu_epilogue)


def _identity(E, H, Fd):
    """w2 [E][H][F]: 1.0 (code 2, scale 2^0) on the diagonal."""
    nib = np.zeros((H, Fd), np.uint8)
    nib[np.arange(Fd), np.arange(Fd)] = 2
    codes = nib[:, 0::2] | nib[:, 1::2] << 4
    return (np.broadcast_to(codes, (E, H, Fd // 2)).copy(), np.full((E, H, Fd // 32), 127, np.uint8))


# F past the 2048 columns of one workgroup, and below
@pytest.mark.parametrize("form", [L.CAP_SOFT_GATE_UP, L.CAP_HARD_GATE_UP, L.CAP_SOFT_OUT, L.CAP_NONE])
@pytest.mark.parametrize("Fd,T", [(2304, 37), (2176, 5), (384, 300)])
def test_h_is_the_capped_swiglu_encoded(gpu_lib, Fd, T, form):
    import torch
    E, H = 3, max(Fd, 512)
    g = np.random.default_rng(Fd + T + form)
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).cuda().bfloat16()
    w13 = to_dev(g.integers(0, 256, (E, 2 * Fd, H // 2), dtype=np.uint8))
    w13_sc = to_dev(g.integers(119, 126, (E, 2 * Fd, H // 32), dtype=np.uint8))     # gates on both sides of the cap
    w2, w2_sc = (to_dev(v) for v in _identity(E, H, Fd))
    ids = to_dev(g.integers(0, E, (T, 1)).astype(np.int32))
    cfg = gpu_lib.Config(hidden=H, ffn=Fd, num_experts=E, top_k=1, fmt="mxfp4", max_tokens=T, cap_form=form, cap=7.0)
    ws = gpu_lib.workspace(cfg)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    gpu_lib.forward(cfg, x, ids, torch.ones((T, 1), device="cuda"), dict(w13=w13, w13_sc=w13_sc, w2=w2, w2_sc=w2_sc),
                    out, ws)
    # [gate | up] as the layer's own product gives it
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    pairs, pos = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    gpu_lib.dispatch(cfg, ids, off, pairs, pos, ws)
    xq = torch.empty((T, H // 2), dtype=torch.uint8, device="cuda")
    xs = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    gpu_lib.quantize_act(cfg, x, xq, xs)
    gu = torch.empty((T, 2 * Fd), dtype=torch.float32, device="cuda")
    gpu_lib.group_product("mxfp4", xq, xs, w13, w13_sc, off, gu, row_ids=pairs)
    gu = gu[pos.long()].cpu().numpy()
    got = out.float().cpu().numpy().astype(np.float64)
    assert (got[:, Fd:] == 0).all()
    got = got[:, :Fd].reshape(T, -1, 32)

    ocfg = L.OracleConfig(hidden=H, ffn=Fd, num_experts=E, top_k=1, fmt="mxfp4", cap_form=form, cap=7.0)
    h = L.cap_swiglu(ocfg, gu[:, :Fd], gu[:, Fd:]).astype(np.float64)
    lo, hi = h * (1 - REL), h * (1 + REL)
    ends = [F.quantize_mxfp4(v.astype(np.float32)) for v in (lo, hi)]
    same = ends[0][1] == ends[1][1]               # blocks whose scale no error within REL moves
    assert same.mean() > 0.99
    # a value within REL of h rounds to one of the two ends' codes or between them
    a, b = (F.dequantize_mxfp4(*e).reshape(T, -1, 32) for e in ends)
    ok = (np.minimum(a, b) <= got) & (got <= np.maximum(a, b))
    assert ok[same].all(), np.argwhere(~ok & same[..., None])[:4]
    assert (a == b)[same].mean() > 0.99           # nearly all of them to one code
