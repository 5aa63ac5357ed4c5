"""The binding of the norm, the sorted rows, the matrix-vector product and the
forward of quantized tokens with tensors of two devices, on stand-ins for
tensors and library: every tensor of a call has to be on the current device."""
import pytest
import torch

import block_scaled_expert_amd as bse

U8, I32, F32, BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


class Stub:
    """What the binding looks at of a tensor on the GPU."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.device_index = dtype, torch.Size(shape), device

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)


class Library:
    """Counts the calls that reach the library."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


T, K, M, H = 4, 2, 8, 64
CFG = bse.Config(fmt="nvfp4", hidden=H, ffn=H, num_experts=2, top_k=K, max_tokens=T)
X, Y, POS, TW = (BF16, T, H), (F32, M, H), (I32, T, K), (F32, T, K)
CALLS = {
    "group_matvec": (lambda t: bse.group_matvec("nvfp4", t["x"], t["w"], t["sc"], t["off"], t["out"], gs=t["gs"], row_ids=t["ids"]),
                     dict(x=X, w=(U8, 2, 16, H // 2), sc=(U8, 2, 16, H // 16), off=(I32, 3), out=(F32, M, 16), gs=(F32, 2),
                          ids=(I32, M))),
    "norm_forward": (lambda t: bse.norm_forward(t["x"], t["w"], t["y"], residual=t["r"], res_out=t["s"], rstd=t["rstd"], cfg=CFG,
                                                codes=t["codes"], scales=t["sc"], row_gs=t["gs"]),
                     dict(x=X, w=(F32, H), y=X, r=X, s=X, rstd=(F32, T), codes=(U8, T, H // 2), sc=(U8, T, H // 16), gs=(F32, T))),
    "norm_backward": (lambda t: bse.norm_backward(t["dy"], t["s"], t["w"], t["rstd"], t["d"], t["ws"], d_res_out=t["n"], dx=t["dx"],
                                                  d_weight=t["dw"]),
                      dict(dy=X, s=X, w=(F32, H), rstd=(F32, T), d=X, ws=(U8, 4096), n=X, dx=X, dw=(F32, H))),
    "sort_rows": (lambda t: bse.sort_rows(t["x"], t["pos"], t["out"]), dict(x=X, pos=POS, out=(BF16, M, H))),
    "sort_rows_backward": (lambda t: bse.sort_rows_backward(t["d"], t["pos"], t["dx"]), dict(d=(BF16, M, H), pos=POS, dx=X)),
    "combine_rows": (lambda t: bse.combine_rows(t["y"], t["pos"], t["tw"], t["out"]), dict(y=Y, pos=POS, tw=TW, out=X)),
    "combine_rows_backward": (lambda t: bse.combine_rows_backward(t["d"], t["y"], t["pos"], t["tw"], t["dy"], t["dw"]),
                              dict(d=X, y=Y, pos=POS, tw=TW, dy=Y, dw=TW)),
    "forward_quantized": (lambda t: bse.forward_quantized(CFG, t["codes"], t["sc"], t["ids"], t["tw"],
                                                          {k: t[k] for k in ("w13", "w13_sc", "w2", "w2_sc", "gs")}, t["out"], t["ws"],
                                                          row_gs=t["row_gs"]),
                          dict(codes=(U8, T, H // 2), sc=(U8, T, H // 16), ids=POS, tw=TW, w13=(U8, 2, 2 * H, H // 2),
                               w13_sc=(U8, 2, 2 * H, H // 16), w2=(U8, 2, H, H // 2), w2_sc=(U8, 2, H, H // 16), gs=(F32, 2, 3),
                               out=X, ws=(U8, 4096), row_gs=(F32, T))),
}


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(bse, "load", lambda: lib)
    monkeypatch.setattr(bse, "_accessors", lambda: (lambda device: 0x10 + device, lambda: 0))
    return lib


@pytest.mark.parametrize("name", list(CALLS))
def test_every_tensor_is_on_the_current_device(library, name):
    call, args = CALLS[name]
    call({k: Stub(*a) for k, a in args.items()})
    assert library.calls == ["moe_" + name]
    library.calls.clear()
    for bad in args:
        with pytest.raises(ValueError, match="current device"):
            call({k: Stub(*a, device=1 if k == bad else 0) for k, a in args.items()})
        assert library.calls == [], bad
