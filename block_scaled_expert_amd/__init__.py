"""Python binding of libmoe.so, the gfx950 routed-expert MoE library.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels on the caller's current torch stream.  The functions mirror the C
ABI in include/moe.h (moe_route, moe_dispatch, moe_quantize_act,
moe_forward, moe_forward_fused, moe_forward_fused_status, moe_route_forward,
moe_forward_noalloc, moe_cap_swiglu, moe_workspace_size,
moe_noalloc_scratch_bytes, moe_check_arch, moe_status_string, the weight
encoder and decoder, moe_group_product, moe_group_matvec, moe_route_logits,
the router's balance loss with its gradient, the residual norm with its
gradient, moe_forward_quantized, and the sorted rows with their gradients).
Tensors must be contiguous and on the current CUDA (HIP) device; apart from
moe_forward_noalloc's fixed device array the library never allocates, so
callers pass outputs and a workspace.  The calls named from the norm on, and
moe_group_matvec, refuse a tensor of another device.

There is no fallback: if the built library is missing, load() raises.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("BSE_MOE_LIB") or os.path.join(HERE, "libmoe.so")

FMT_NVFP4, FMT_MXFP8, FMT_MXFP4 = 1, 2, 4
FMTS = {"nvfp4": FMT_NVFP4, "mxfp8": FMT_MXFP8, "mxfp4": FMT_MXFP4}
CAP_SOFT_GATE_UP, CAP_HARD_GATE_UP, CAP_SOFT_OUT, CAP_NONE = 0, 1, 2, 3
DTYPE_BF16, DTYPE_F32 = 0, 1
ACT_GS_PER_ROW, ACT_GS_PER_TENSOR, ACT_GS_STATIC = 0, 1, 2
ACT_GS_SCRATCH_BYTES = 1028   # moe_quantize_act's scratch for a per-tensor NVFP4 scale
STAGES = ("quant_x", "dispatch", "gate_up", "quant_h", "down", "combine")

EXPORTED = ("moe_status_string", "moe_check_arch", "moe_validate_config", "moe_workspace_size",
            "moe_quantize_act", "moe_route", "moe_dispatch", "moe_prepare_weights", "moe_forward",
            "moe_forward_fused", "moe_forward_fused_status", "moe_cap_swiglu", "moe_encode_weights",
            "moe_decode_weights", "moe_forward_noalloc", "moe_noalloc_scratch_bytes", "moe_route_forward",
            "moe_route_logits", "moe_balance_workspace_size", "moe_balance_forward", "moe_balance_backward",
            "moe_group_product", "moe_group_matvec", "moe_norm_forward", "moe_norm_workspace_size",
            "moe_norm_backward", "moe_forward_quantized", "moe_sort_rows", "moe_sort_rows_backward",
            "moe_combine_rows", "moe_combine_rows_backward")
LAYOUT_CANONICAL, LAYOUT_PACKED = 0, 1


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class CConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("expert_begin", ctypes.c_int32),
                ("num_local_experts", ctypes.c_int32), ("fmt", ctypes.c_int32), ("cap_form", ctypes.c_int32),
                ("cap", ctypes.c_float), ("norm_topk", ctypes.c_int32), ("routed_scale", ctypes.c_float),
                ("max_tokens", ctypes.c_int32), ("act_gs", ctypes.c_int32), ("act_gs_static", ctypes.c_float * 2)]


class CWeights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_sc", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_sc", ctypes.c_void_p), ("gs", ctypes.c_void_p), ("layout", ctypes.c_int32)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libmoe.so (built by block_scaled_expert_amd.build); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_scaled_expert_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_check_arch.argtypes = [ctypes.c_char_p]
    lib.moe_validate_config.argtypes = [ctypes.POINTER(CConfig)]
    lib.moe_workspace_size.argtypes = [ctypes.POINTER(CConfig), ctypes.POINTER(sz)]
    lib.moe_quantize_act.argtypes = [ctypes.POINTER(CConfig), i32, i32, vp, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.moe_cap_swiglu.argtypes = [ctypes.POINTER(CConfig), vp, vp, ctypes.c_int64, vp, vp]
    lib.moe_forward_fused_status.argtypes = [ctypes.POINTER(CConfig), i32, vp, sz, vp, vp]
    lib.moe_encode_weights.argtypes = [i32, i32, vp, i32, i32, i32, vp, vp, vp, i32, i32, vp, sz, vp]
    lib.moe_decode_weights.argtypes = [i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.moe_route.argtypes = [ctypes.POINTER(CConfig), vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_dispatch.argtypes = [ctypes.POINTER(CConfig), vp, i32, vp, vp, vp, vp, sz, vp]
    lib.moe_prepare_weights.argtypes = [ctypes.POINTER(CConfig), ctypes.POINTER(CWeights), ctypes.POINTER(CWeights),
                                        vp]
    lib.moe_forward.argtypes = [ctypes.POINTER(CConfig), vp, i32, vp, vp, ctypes.POINTER(CWeights), vp, vp,
                                sz, vp, vp]
    lib.moe_forward_fused.argtypes = lib.moe_forward.argtypes
    lib.moe_forward_noalloc.argtypes = [ctypes.POINTER(CConfig), vp, i32, vp, vp, ctypes.POINTER(CWeights), vp, vp]
    lib.moe_noalloc_scratch_bytes.argtypes = []
    lib.moe_route_forward.argtypes = [ctypes.POINTER(CConfig), vp, i32, vp, vp, vp, vp, vp, ctypes.POINTER(CWeights),
                                      vp, vp, sz, vp, vp]
    lib.moe_route_logits.argtypes = [ctypes.POINTER(CConfig), i32, vp, sz, vp, vp]
    lib.moe_balance_workspace_size.argtypes = [ctypes.POINTER(CConfig), i32, i32, ctypes.POINTER(sz)]
    lib.moe_balance_forward.argtypes = [ctypes.POINTER(CConfig), i32, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                        sz, vp]
    lib.moe_balance_backward.argtypes = [ctypes.POINTER(CConfig), i32, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                         vp]
    lib.moe_group_product.argtypes = [i32, vp, vp, i32, vp, i32, i32, vp, vp, i32, i32, i32, vp, i32, vp, vp]
    lib.moe_group_matvec.argtypes = [ctypes.POINTER(CConfig), i32, i32, vp, i32, vp, i32, i32, vp, vp, vp, i32, i32, i32,
                                     i32, i32, vp, i32, vp, vp]
    lib.moe_norm_forward.argtypes = [ctypes.POINTER(CConfig), i32, vp, i32, vp, i32, i32, vp, ctypes.c_float, vp, vp, vp,
                                     vp, vp, vp, vp]
    lib.moe_norm_workspace_size.argtypes = [i32, i32, ctypes.POINTER(sz)]
    lib.moe_norm_backward.argtypes = [i32, vp, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_forward_quantized.argtypes = [ctypes.POINTER(CConfig), vp, vp, vp, i32, vp, vp, ctypes.POINTER(CWeights), vp,
                                          vp, sz, vp, vp]
    lib.moe_sort_rows.argtypes = [i32, vp, i32, i32, i32, vp, i32, vp, vp]
    lib.moe_sort_rows_backward.argtypes = [i32, vp, i32, vp, i32, i32, i32, vp, vp]
    lib.moe_combine_rows.argtypes = [i32, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.moe_combine_rows_backward.argtypes = [i32, vp, i32, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp]
    for name in EXPORTED:
        if name != "moe_status_string":
            getattr(lib, name).restype = ctypes.c_int
    lib.moe_noalloc_scratch_bytes.restype = ctypes.c_size_t
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def check_arch(arch: str) -> int:
    return load().moe_check_arch(arch.encode())


@dataclass
class Config:
    hidden: int = 4608
    ffn: int = 2304
    num_experts: int = 384
    top_k: int = 8
    fmt: str = "nvfp4"
    expert_begin: int = 0
    num_local_experts: int | None = None
    cap_form: int = CAP_SOFT_GATE_UP
    cap: float = 7.0
    norm_topk: bool = True
    routed_scale: float = 1.0
    max_tokens: int = 64
    act_gs: int = ACT_GS_PER_ROW
    act_gs_static: tuple = (1.0, 1.0)

    @property
    def num_local(self) -> int:
        return self.num_experts if self.num_local_experts is None else self.num_local_experts

    def ref(self):
        """A reference to the C structure of the fields as they are now, for one
        call.  Structures are kept by the values they were built from (building
        one takes 1.9 us of a small call's 6, finding it 0.7)."""
        if type(self) is not Config:                 # a subclass may read them in another way
            return ctypes.byref(self.c())
        fields = _fields_of(self)
        try:
            by_ref = _structures.get(fields)
        except TypeError:                            # a list, say
            return ctypes.byref(self.c())
        if by_ref is None:
            by_ref = ctypes.byref(Config(*fields).c())
            # anything but these could change its value and still be found
            if _PLAIN.issuperset(map(type, fields)) and _PLAIN.issuperset(map(type, fields[-1])):
                if len(_structures) >= 64:
                    _structures.clear()
                _structures[fields] = by_ref
        return by_ref

    def c(self) -> CConfig:
        if self.fmt not in FMTS:
            raise ValueError(f"unknown format {self.fmt!r}")
        return CConfig(self.hidden, self.ffn, self.num_experts, self.top_k, self.expert_begin, self.num_local,
                       FMTS[self.fmt], self.cap_form, self.cap, int(bool(self.norm_topk)), self.routed_scale,
                       self.max_tokens, self.act_gs, (ctypes.c_float * 2)(*self.act_gs_static))


_fields_of = operator.attrgetter(*Config.__dataclass_fields__)
_structures: dict = {}      # Config.ref's, by the values of the fields
_PLAIN = frozenset((bool, int, float, str, type(None), tuple))


def _ok(status: int, what: str) -> None:
    if status != 0:
        raise MoeError(status, what)


@functools.lru_cache(maxsize=None)
def _accessors():
    import torch
    return torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _device() -> int:
    return _accessors()[1]()


def _stream(on=None) -> int:
    """The current stream's handle (on: the current device, where it is known).
    The raw accessors: building a Stream object takes 3 us, more than everything
    else around a small call."""
    stream, device = _accessors()
    return stream(device() if on is None else on)


def _ptr(t, dtype=None, shape=None, name="tensor", on=None):
    """t's address; on: the device that it must be on (None: any GPU)."""
    if t is None:
        return None
    if on is None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU")
    elif t.get_device() != on:
        raise ValueError(f"{name} must be on the current device ({on}), is on {t.get_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _code_cols(fmt: str, cols: int) -> int:
    """Bytes of a row of `cols` codes."""
    return cols if fmt == "mxfp8" else cols // 2


def _scale_cols(fmt: str, cols: int) -> int:
    """Scales of a row of `cols` elements."""
    return cols // (16 if fmt == "nvfp4" else 32)


def workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t(0)
    cc = cfg.c()
    _ok(load().moe_workspace_size(ctypes.byref(cc), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def workspace(cfg: Config, device="cuda"):
    import torch
    return torch.empty(workspace_size(cfg), dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=None)
def _default_config(fmt: str):
    cfg = Config(fmt=fmt)
    return cfg, cfg.c()


def quantize_act(cfg, x, codes, scales, row_gs=None, site: int = 0, ws=None) -> None:
    """NVFP4 / MXFP8 / MXFP4 quantization of a bf16 or fp32 [rows, cols] tensor in
    cfg's format and activation-scale mode (cfg: a Config, or a format name
    for the per-row default).  site 0: gate/up input x, 1: down input h.
    ws: uint8 scratch of at least ACT_GS_SCRATCH_BYTES for NVFP4 per-tensor
    scales."""
    import torch
    if isinstance(cfg, str):
        cfg, cc = _default_config(cfg)
    else:
        cc = cfg.c()
    rows, cols = x.shape
    dt = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(x.dtype)
    if dt is None:
        raise ValueError("x must be bfloat16 or float32")
    nv = cfg.fmt == "nvfp4"
    args = (ctypes.byref(cc), site, dt, _ptr(x, name="x"), rows, cols,
            _ptr(codes, torch.uint8, (rows, _code_cols(cfg.fmt, cols)), "codes"),
            _ptr(scales, torch.uint8, (rows, _scale_cols(cfg.fmt, cols)), "scales"),
            _ptr(row_gs, torch.float32, (rows,), "row_gs") if nv else None,
            _ptr(ws, torch.uint8, None, "ws"), 0 if ws is None else ws.numel(), _stream())
    _ok(load().moe_quantize_act(*args), "moe_quantize_act")


def cap_swiglu(cfg: Config, g, u, h) -> None:
    """The expert epilogue's capped SwiGLU on fp32 tensors of equal size."""
    import torch
    n = g.numel()
    cc = cfg.c()
    _ok(load().moe_cap_swiglu(ctypes.byref(cc), _ptr(g, torch.float32, None, "g"),
                              _ptr(u, torch.float32, (n,) if u.dim() == 1 else None, "u"), n,
                              _ptr(h, torch.float32, None, "h"), _stream()), "moe_cap_swiglu")


def forward_fused_status(cfg: Config, T: int, ws, err) -> None:
    """err (int32 device tensor of one element) <- the error word of the last
    moe_forward_fused call on ws for T tokens (0: every wait was met)."""
    import torch
    cc = cfg.c()
    _ok(load().moe_forward_fused_status(ctypes.byref(cc), T, _ptr(ws, torch.uint8, None, "ws"), ws.numel(),
                                        _ptr(err, torch.int32, (1,), "err"), _stream()),
        "moe_forward_fused_status")


def _check_gs(gs, nmat: int, group: int, stride: int) -> None:
    if gs is None or group < 1 or stride < group:
        raise ValueError("NVFP4 needs gs, gs_group >= 1 and gs_stride >= gs_group")
    need = ((nmat - 1) // group) * stride + (nmat - 1) % group + 1 if nmat > 0 else 0
    if gs.numel() < need:
        raise ValueError(f"gs must hold at least {need} floats")


def encode_weights(fmt: str, w, codes, scales, gs=None, gs_group: int = 1, gs_stride: int = 1,
                   ws=None) -> None:
    """Matrices w [nmat, rows, cols] (bf16 or fp32) to NVFP4 (one fp32 scale
    per matrix, recomputed from its max |w|, written to gs[(m // gs_group) *
    gs_stride + m % gs_group]; ws: int32 scratch of at least nmat elements)
    or MXFP8 / MXFP4.  codes / scales: uint8 [nmat, rows, cols/2 (MXFP8: cols)]
    and [nmat, rows, cols/32 (NVFP4: cols/16)]."""
    import torch
    nmat, rows, cols = w.shape
    dt = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(w.dtype)
    if dt is None:
        raise ValueError("w must be bfloat16 or float32")
    nv = fmt == "nvfp4"
    _ptr(w, name="w")
    if nv:
        _check_gs(gs, nmat, gs_group, gs_stride)
        if ws is None or ws.numel() < nmat:
            raise ValueError(f"ws must hold at least {nmat} int32")
    args = (FMTS[fmt], dt, _ptr(w), nmat, rows, cols,
            _ptr(codes, torch.uint8, (nmat, rows, _code_cols(fmt, cols)), "codes"),
            _ptr(scales, torch.uint8, (nmat, rows, _scale_cols(fmt, cols)), "scales"),
            _ptr(gs, torch.float32, None, "gs") if nv else None, gs_group, gs_stride,
            _ptr(ws, torch.int32, None, "ws") if nv else None,
            (ws.numel() * 4) if (nv and ws is not None) else 0, _stream())
    _ok(load().moe_encode_weights(*args), "moe_encode_weights")


def decode_weights(fmt: str, codes, scales, out, gs=None, gs_group: int = 1, gs_stride: int = 1) -> None:
    """The fp32 values [nmat, rows, cols] of encoded matrices (see encode_weights)."""
    import torch
    nmat, rows, cols = out.shape
    nv = fmt == "nvfp4"
    if nv:
        _check_gs(gs, nmat, gs_group, gs_stride)
    args = (FMTS[fmt], _ptr(codes, torch.uint8, (nmat, rows, _code_cols(fmt, cols)), "codes"),
            _ptr(scales, torch.uint8, (nmat, rows, _scale_cols(fmt, cols)), "scales"),
            _ptr(gs, torch.float32, None, "gs") if nv else None, gs_group, gs_stride, nmat, rows, cols,
            _ptr(out, torch.float32, None, "out"), _stream())
    _ok(load().moe_decode_weights(*args), "moe_decode_weights")


def route(cfg: Config, x, w_router, bias, topk_ids, topk_w, near_tie, ws) -> None:
    import torch
    T = x.shape[0]
    H, E, k = cfg.hidden, cfg.num_experts, cfg.top_k
    cc = cfg.c()
    _ok(load().moe_route(ctypes.byref(cc), _ptr(x, torch.bfloat16, (T, H), "x"), T,
                         _ptr(w_router, torch.bfloat16, (E, H), "w_router"),
                         _ptr(bias, torch.float32, (E,), "bias"),
                         _ptr(topk_ids, torch.int32, (T, k), "topk_ids"),
                         _ptr(topk_w, torch.float32, (T, k), "topk_w"),
                         _ptr(near_tie, torch.uint8, (T,), "near_tie"),
                         _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream()), "moe_route")


def route_logits(cfg: Config, T: int, z, ws) -> None:
    """z [T, E] fp32 <- the logits the last route / route_forward of T tokens
    on ws selected from."""
    import torch
    cc = cfg.c()
    _ok(load().moe_route_logits(ctypes.byref(cc), T, _ptr(ws, torch.uint8, None, "ws"), ws.numel(),
                                _ptr(z, torch.float32, (T, cfg.num_experts), "z"), _stream()), "moe_route_logits")


def balance_workspace_size(cfg: Config, T: int, S: int = 1) -> int:
    n = ctypes.c_size_t(0)
    cc = cfg.c()
    _ok(load().moe_balance_workspace_size(ctypes.byref(cc), T, S, ctypes.byref(n)), "moe_balance_workspace_size")
    return n.value


def balance_workspace(cfg: Config, T: int, S: int = 1, device="cuda"):
    import torch
    return torch.empty(balance_workspace_size(cfg, T, S), dtype=torch.uint8, device=device)


def _balance_args(cfg: Config, z, topk_ids, seq_offsets, token_mask):
    """Pointers shared by the two balance calls: (dtype, z, T, ids, seq_offsets, S, mask)."""
    import torch
    dt = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(z.dtype)
    if dt is None:
        raise ValueError("z must be bfloat16 or float32")
    T = z.shape[0]
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    return (dt, _ptr(z, None, (T, cfg.num_experts), "z"), T,
            _ptr(topk_ids, torch.int32, (T, cfg.top_k), "topk_ids"),
            _ptr(seq_offsets, torch.int32, (S + 1,), "seq_offsets"), S,
            _ptr(token_mask, torch.uint8, (T,), "token_mask"))


def balance_forward(cfg: Config, z, topk_ids, counts, live, probs, loss, ws, seq_offsets=None,
                    token_mask=None) -> None:
    """Per-expert counts [S, E] (int32), live tokens [S] (int32), mean
    probabilities [S, E] and balance loss [S] (fp32) of each sequence from the
    router logits z [T, E] (bf16 or fp32) and topk_ids.  seq_offsets: int32
    [S + 1] (None: one sequence); token_mask: uint8 [T], 0 = not a token.
    ws: balance_workspace(cfg, T, S)."""
    import torch
    args = _balance_args(cfg, z, topk_ids, seq_offsets, token_mask)
    S, E = args[5], cfg.num_experts
    cc = cfg.c()
    _ok(load().moe_balance_forward(ctypes.byref(cc), *args, _ptr(counts, torch.int32, (S, E), "counts"),
                                   _ptr(live, torch.int32, (S,), "live"),
                                   _ptr(probs, torch.float32, (S, E), "probs"),
                                   _ptr(loss, torch.float32, (S,), "loss"), _ptr(ws, torch.uint8, None, "ws"),
                                   ws.numel(), _stream()), "moe_balance_forward")


def balance_backward(cfg: Config, z, topk_ids, counts, live, d_loss, dz, d_topk_w=None, seq_offsets=None,
                     token_mask=None) -> None:
    """dz [T, E] (z's dtype) <- the gradient of sum(d_loss * loss) and, with
    d_topk_w [T, k] given, of the gate weights, with respect to the logits.
    counts, live: balance_forward's."""
    import torch
    args = _balance_args(cfg, z, topk_ids, seq_offsets, token_mask)
    T, S, E = args[2], args[5], cfg.num_experts
    cc = cfg.c()
    _ok(load().moe_balance_backward(ctypes.byref(cc), *args, _ptr(counts, torch.int32, (S, E), "counts"),
                                    _ptr(live, torch.int32, (S,), "live"),
                                    _ptr(d_loss, torch.float32, (S,), "d_loss"),
                                    _ptr(d_topk_w, torch.float32, (T, cfg.top_k), "d_topk_w"),
                                    _ptr(dz, z.dtype, (T, E), "dz"), _stream()), "moe_balance_backward")


def group_product(fmt: str, a, a_scales, w, w_scales, offsets, out, row_ids=None, id_div: int = 1) -> None:
    """out[r] = A[src(r)] @ W[g].T for rows r in [offsets[g], offsets[g+1]),
    src(r) = r, or row_ids[r] // id_div.  a / a_scales: uint8 codes
    [rows, K/2] and scales [rows, K/32]; w / w_scales: [G, N, K/2] and
    [G, N, K/32]; offsets int32 [G+1]; out [M, N] fp32 or bf16; row_ids int32
    [M].  fmt "mxfp4"."""
    import torch
    if fmt not in FMTS:
        raise ValueError(f"unknown format {fmt!r}")
    dt = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(out.dtype)
    if dt is None:
        raise ValueError("out must be bfloat16 or float32")
    M, N = out.shape
    G, K = w.shape[0], a.shape[1] * 2
    a_rows = a.shape[0]
    _ok(load().moe_group_product(FMTS[fmt], _ptr(a, torch.uint8, None, "a"),
                                 _ptr(a_scales, torch.uint8, (a_rows, K // 32), "a_scales"), a_rows,
                                 _ptr(row_ids, torch.int32, (M,), "row_ids"), id_div, M,
                                 _ptr(w, torch.uint8, (G, N, K // 2), "w"),
                                 _ptr(w_scales, torch.uint8, (G, N, K // 32), "w_scales"), G, N, K,
                                 _ptr(offsets, torch.int32, (G + 1,), "offsets"), dt, _ptr(out, None, None, "out"),
                                 _stream()), "moe_group_product")


@functools.lru_cache(maxsize=None)
def _dtypes() -> dict:
    import torch
    return {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _dtype(t, name: str) -> int:
    """MOE_DTYPE of a bf16 or fp32 tensor."""
    dt = _dtypes().get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return dt


def group_matvec(fmt: str, x, w, w_scales, offsets, out, gs=None, gs_group: int = 1, gs_stride: int = 1, row_ids=None,
                 id_div: int = 1, swiglu: Config | None = None) -> None:
    """out[r] = x[src(r)] @ W[g].T for rows r in [offsets[g], offsets[g+1]),
    src(r) = r, or row_ids[r] // id_div; x bf16 or fp32 [rows, K], W 4-bit.
    w / w_scales: uint8 codes [G, N, K/2] and scales [G, N, K/16] (fmt
    "nvfp4") or [G, N, K/32] ("mxfp4"); NVFP4: gs, gs_group and gs_stride as in
    encode_weights; offsets int32 [G+1]; out [M, N] fp32 or bf16; row_ids int32
    [M].  swiglu: a Config whose capped SwiGLU is taken over [gate | up], out is
    then [M, N/2]."""
    import torch
    on = _device()
    if fmt not in FMTS:
        raise ValueError(f"unknown format {fmt!r}")
    rows, K = x.shape
    G, N = w.shape[:2]
    M = out.shape[0]
    nv = fmt == "nvfp4"
    if nv:
        if gs_group < 1 or N % gs_group:
            raise ValueError("N must be a multiple of gs_group")
        _check_gs(gs, G * gs_group, gs_group, gs_stride)
    _ok(load().moe_group_matvec(None if swiglu is None else swiglu.ref(), FMTS[fmt], _dtype(x, "x"),
                                _ptr(x, None, None, "x", on), rows, _ptr(row_ids, torch.int32, (M,), "row_ids", on), id_div, M,
                                _ptr(w, torch.uint8, (G, N, _code_cols(fmt, K)), "w", on),
                                _ptr(w_scales, torch.uint8, (G, N, _scale_cols(fmt, K)), "w_scales", on),
                                _ptr(gs, torch.float32, None, "gs", on) if nv else None, gs_group, gs_stride, G, N, K,
                                _ptr(offsets, torch.int32, (G + 1,), "offsets", on), _dtype(out, "out"),
                                _ptr(out, None, (M, N if swiglu is None else N // 2), "out", on), _stream(on)),
        "moe_group_matvec")


def norm_forward(x, weight, y=None, residual=None, res_out=None, rstd=None, eps: float = 1e-6, cfg=None, codes=None,
                 scales=None, row_gs=None) -> None:
    """res_out = x + residual; y = res_out * rstd * weight, rstd = (mean of
    res_out^2 + eps)^-1/2 per row; and the codes of y in cfg's format (a Config,
    or a format name for the per-row default) as quantize_act writes them.
    x, y [T, cols] bf16 or fp32; residual, res_out [T, cols] of x's type or
    fp32; weight [cols] and rstd [T] fp32.  Without cfg no codes are written."""
    import torch
    on = _device()
    if isinstance(cfg, str):
        cfg = _default_config(cfg)[0]
    T, cols = x.shape
    res = residual if residual is not None else res_out
    res_type = None if res is None else res.dtype
    enc = (None, None, None)
    if cfg is not None:
        enc = (_ptr(codes, torch.uint8, (T, _code_cols(cfg.fmt, cols)), "codes", on),
               _ptr(scales, torch.uint8, (T, _scale_cols(cfg.fmt, cols)), "scales", on),
               _ptr(row_gs, torch.float32, (T,), "row_gs", on) if cfg.fmt == "nvfp4" else None)
    elif codes is not None or scales is not None or row_gs is not None:
        raise ValueError("codes, scales and row_gs need cfg")
    _ok(load().moe_norm_forward(None if cfg is None else cfg.ref(), _dtype(x, "x"), _ptr(x, None, None, "x", on),
                                _dtype(x if res is None else res, "residual"),
                                _ptr(residual, res_type, (T, cols), "residual", on), T, cols,
                                _ptr(weight, torch.float32, (cols,), "weight", on), eps,
                                _ptr(res_out, res_type, (T, cols), "res_out", on), _ptr(y, x.dtype, (T, cols), "y", on),
                                _ptr(rstd, torch.float32, (T,), "rstd", on), *enc, _stream(on)),
        "moe_norm_forward")


def norm_workspace_size(T: int, cols: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(load().moe_norm_workspace_size(T, cols, ctypes.byref(n)), "moe_norm_workspace_size")
    return n.value


def norm_workspace(T: int, cols: int, device="cuda"):
    import torch
    return torch.empty(norm_workspace_size(T, cols), dtype=torch.uint8, device=device)


def norm_backward(dy, res, weight, rstd, d_res, ws=None, d_res_out=None, dx=None, d_weight=None) -> None:
    """d_res [T, cols] (res's type) <- the gradient of the stream res that
    norm_forward normed (its res_out, or x without a residual), with d_res_out
    added: the gradient of the residual and of x.  dx: the same in dy's type.
    d_weight [cols] fp32 needs ws: norm_workspace(T, cols)."""
    import torch
    on = _device()
    T, cols = dy.shape
    _ok(load().moe_norm_backward(_dtype(dy, "dy"), _ptr(dy, None, None, "dy", on), _dtype(res, "res"),
                                 _ptr(res, None, (T, cols), "res", on), _ptr(d_res_out, res.dtype, (T, cols), "d_res_out", on),
                                 T, cols, _ptr(weight, torch.float32, (cols,), "weight", on),
                                 _ptr(rstd, torch.float32, (T,), "rstd", on), _ptr(d_res, res.dtype, (T, cols), "d_res", on),
                                 _ptr(dx, dy.dtype, (T, cols), "dx", on),
                                 _ptr(d_weight, torch.float32, (cols,), "d_weight", on),
                                 _ptr(ws, torch.uint8, None, "ws", on), 0 if ws is None else ws.numel(), _stream(on)),
        "moe_norm_backward")


def _slots(pair_pos, T: int) -> int:
    """Slots of a token in pair_pos ([T, top_k] or flat)."""
    shape = pair_pos.shape
    if len(shape) == 2 and shape[0] == T:
        k = shape[1]
    else:
        n = pair_pos.numel()
        if len(shape) != 1 or T > 0 and n % T:
            raise ValueError(f"pair_pos must hold top_k positions for each of {T} tokens")
        k = n // T if T > 0 else 1
    if k < 1:
        raise ValueError(f"pair_pos must hold top_k positions for each of {T} tokens")
    return k


def sort_rows(x, pair_pos, out) -> None:
    """out[pair_pos[t, j]] = x[t] for the local pairs (pair_pos: dispatch's,
    int32 [T * top_k]).  x [T, cols] and out [M, cols] of one type, bf16 or fp32."""
    import torch
    on = _device()
    T, cols = x.shape
    M = out.shape[0]
    _ok(load().moe_sort_rows(_dtype(x, "x"), _ptr(x, None, None, "x", on), T, _slots(pair_pos, T), cols,
                             _ptr(pair_pos, torch.int32, None, "pair_pos", on), M, _ptr(out, x.dtype, (M, cols), "out", on),
                             _stream(on)), "moe_sort_rows")


def sort_rows_backward(d_out, pair_pos, dx) -> None:
    """dx[t] = sum over the local pairs of d_out[pair_pos[t, j]]: sort_rows' gradient."""
    import torch
    on = _device()
    T, cols = dx.shape
    M = d_out.shape[0]
    _ok(load().moe_sort_rows_backward(_dtype(dx, "dx"), _ptr(d_out, dx.dtype, (M, cols), "d_out", on), M,
                                      _ptr(pair_pos, torch.int32, None, "pair_pos", on), T, _slots(pair_pos, T), cols,
                                      _ptr(dx, None, None, "dx", on), _stream(on)), "moe_sort_rows_backward")


def combine_rows(y, pair_pos, topk_w, out) -> None:
    """out[t] = sum over the local pairs of topk_w[t, j] * y[pair_pos[t, j]]
    (topk_w fp32 [T, top_k]; None: all 1).  y [M, cols], out [T, cols], each
    bf16 or fp32."""
    import torch
    on = _device()
    T, cols = out.shape
    M, k = y.shape[0], _slots(pair_pos, T)
    _ok(load().moe_combine_rows(_dtype(y, "y"), _ptr(y, None, (M, cols), "y", on), M,
                                _ptr(pair_pos, torch.int32, None, "pair_pos", on),
                                _ptr(topk_w, torch.float32, (T, k), "topk_w", on), T, k, cols, _dtype(out, "out"),
                                _ptr(out, None, None, "out", on), _stream(on)), "moe_combine_rows")


def combine_rows_backward(d_out, y, pair_pos, topk_w, dy, d_topk_w=None) -> None:
    """combine_rows' gradients: dy [M, cols] (y's type; may be y) and d_topk_w
    [T, top_k] fp32, either of them None.  y may be None where d_topk_w is."""
    import torch
    on = _device()
    T, cols = d_out.shape
    k = _slots(pair_pos, T)
    rows = y if y is not None else dy
    if rows is None:
        raise ValueError("dy or y must be given")
    M = rows.shape[0]
    _ok(load().moe_combine_rows_backward(_dtype(d_out, "d_out"), _ptr(d_out, None, None, "d_out", on), _dtype(rows, "y"),
                                         _ptr(y, None, (M, cols), "y", on), M, _ptr(pair_pos, torch.int32, None, "pair_pos", on),
                                         _ptr(topk_w, torch.float32, (T, k), "topk_w", on), T, k, cols,
                                         _ptr(dy, rows.dtype, (M, cols), "dy", on),
                                         _ptr(d_topk_w, torch.float32, (T, k), "d_topk_w", on), _stream(on)),
        "moe_combine_rows_backward")


def dispatch(cfg: Config, topk_ids, expert_offsets, sorted_pairs=None, pair_pos=None, ws=None) -> None:
    import torch
    T = topk_ids.shape[0]
    P = T * cfg.top_k
    cc = cfg.c()
    _ok(load().moe_dispatch(ctypes.byref(cc), _ptr(topk_ids, torch.int32, (T, cfg.top_k), "topk_ids"), T,
                            _ptr(expert_offsets, torch.int32, (cfg.num_local + 1,), "expert_offsets"),
                            _ptr(sorted_pairs, torch.int32, None, "sorted_pairs"),
                            _ptr(pair_pos, torch.int32, (P,), "pair_pos"),
                            _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream()), "moe_dispatch")


def weights_struct(cfg: Config, w: dict, on=None) -> CWeights:
    """w: dict of device tensors w13, w13_sc, w2, w2_sc (uint8), gs (fp32,
    NVFP4) and optionally layout (LAYOUT_CANONICAL by default).  on: the device
    that they must be on (None: any GPU)."""
    import torch
    H, F, n = cfg.hidden, cfg.ffn, cfg.num_local
    nv = cfg.fmt == "nvfp4"
    shapes = {
        "w13": (n, 2 * F, _code_cols(cfg.fmt, H)), "w13_sc": (n, 2 * F, _scale_cols(cfg.fmt, H)),
        "w2": (n, H, _code_cols(cfg.fmt, F)), "w2_sc": (n, H, _scale_cols(cfg.fmt, F)),
    }
    ptrs = {k: _ptr(w[k], torch.uint8, s, k, on) for k, s in shapes.items()}
    gs = _ptr(w["gs"], torch.float32, (n, 3), "gs", on) if nv else None
    return CWeights(ptrs["w13"], ptrs["w13_sc"], ptrs["w2"], ptrs["w2_sc"], gs, int(w.get("layout", LAYOUT_CANONICAL)))


def prepare_weights(cfg: Config, w: dict) -> dict:
    """Repack canonical expert weights into the packed layout (new device
    tensors of the same shapes; gs is shared)."""
    import torch
    src = weights_struct(cfg, w)
    out = {k: torch.empty_like(w[k]) for k in ("w13", "w13_sc", "w2", "w2_sc")}
    if "gs" in w:
        out["gs"] = w["gs"]
    out["layout"] = LAYOUT_PACKED
    dst = weights_struct(cfg, out)
    cc = cfg.c()
    _ok(load().moe_prepare_weights(ctypes.byref(cc), ctypes.byref(src), ctypes.byref(dst), _stream()),
        "moe_prepare_weights")
    return out


def forward(cfg: Config, x, topk_ids, topk_w, weights, out, ws, events=None, fused: bool = False) -> None:
    """weights: dict of device tensors or a CWeights built by weights_struct.
    events: optional list of 2*6 torch.cuda.Event (stage timing).
    fused: call moe_forward_fused (the expert half in one launch) instead of moe_forward."""
    import torch
    T = x.shape[0]
    H, k = cfg.hidden, cfg.top_k
    cw = weights if isinstance(weights, CWeights) else weights_struct(cfg, weights)
    ev = None
    if events is not None:
        if len(events) != 2 * len(STAGES):
            raise ValueError("events must hold 2 per stage")
        ev = (ctypes.c_void_p * len(events))(*[e.cuda_event if e is not None else None for e in events])
    cc = cfg.c()
    fn = load().moe_forward_fused if fused else load().moe_forward
    _ok(fn(ctypes.byref(cc), _ptr(x, torch.bfloat16, (T, H), "x"), T,
           _ptr(topk_ids, torch.int32, (T, k), "topk_ids"),
           _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(cw),
           _ptr(out, torch.bfloat16, (T, H), "out"), _ptr(ws, torch.uint8, None, "ws"),
           ws.numel(), _stream(), ev), "moe_forward_fused" if fused else "moe_forward")


def forward_quantized(cfg: Config, codes, scales, topk_ids, topk_w, weights, out, ws, row_gs=None, events=None) -> None:
    """forward on tokens quantized already (norm_forward with cfg, or
    quantize_act at site 0): codes, scales and, for NVFP4, row_gs."""
    import torch
    on = _device()
    T = codes.shape[0]
    H, k, nv = cfg.hidden, cfg.top_k, cfg.fmt == "nvfp4"
    cw = weights if isinstance(weights, CWeights) else weights_struct(cfg, weights, on)   # CWeights: plain addresses
    ev = None
    if events is not None:
        if len(events) != 2 * len(STAGES):
            raise ValueError("events must hold 2 per stage")
        ev = (ctypes.c_void_p * len(events))(*[e.cuda_event if e is not None else None for e in events])
    _ok(load().moe_forward_quantized(cfg.ref(), _ptr(codes, torch.uint8, (T, _code_cols(cfg.fmt, H)), "codes", on),
                                     _ptr(scales, torch.uint8, (T, _scale_cols(cfg.fmt, H)), "scales", on),
                                     _ptr(row_gs, torch.float32, (T,), "row_gs", on) if nv else None, T,
                                     _ptr(topk_ids, torch.int32, (T, k), "topk_ids", on),
                                     _ptr(topk_w, torch.float32, (T, k), "topk_w", on), ctypes.byref(cw),
                                     _ptr(out, torch.bfloat16, (T, H), "out", on), _ptr(ws, torch.uint8, None, "ws", on),
                                     ws.numel(), _stream(on), ev),
        "moe_forward_quantized")


def forward_noalloc(cfg: Config, x, topk_ids, topk_w, weights, out) -> None:
    """moe_forward_noalloc: moe_forward with the library's per-device scratch
    buffer as its workspace (no workspace argument, nothing allocated)."""
    import torch
    T = x.shape[0]
    H, k = cfg.hidden, cfg.top_k
    cw = weights if isinstance(weights, CWeights) else weights_struct(cfg, weights)
    cc = cfg.c()
    _ok(load().moe_forward_noalloc(ctypes.byref(cc), _ptr(x, torch.bfloat16, (T, H), "x"), T,
                                   _ptr(topk_ids, torch.int32, (T, k), "topk_ids"),
                                   _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(cw),
                                   _ptr(out, torch.bfloat16, (T, H), "out"), _stream()), "moe_forward_noalloc")


def noalloc_scratch_bytes() -> int:
    return int(load().moe_noalloc_scratch_bytes())


def route_forward(cfg: Config, x, w_router, bias, topk_ids, topk_w, near_tie, weights, out, ws, events=None) -> None:
    """moe_route_forward: routing and the forward in one call; for small
    batches routing, x quantization and dispatch are one launch."""
    import torch
    T = x.shape[0]
    H, E, k = cfg.hidden, cfg.num_experts, cfg.top_k
    cw = weights if isinstance(weights, CWeights) else weights_struct(cfg, weights)
    ev = None
    if events is not None:
        if len(events) != 2 * len(STAGES):
            raise ValueError("events must hold 2 per stage")
        ev = (ctypes.c_void_p * len(events))(*[e.cuda_event if e is not None else None for e in events])
    cc = cfg.c()
    _ok(load().moe_route_forward(ctypes.byref(cc), _ptr(x, torch.bfloat16, (T, H), "x"), T,
                                 _ptr(w_router, torch.bfloat16, (E, H), "w_router"),
                                 _ptr(bias, torch.float32, (E,), "bias"),
                                 _ptr(topk_ids, torch.int32, (T, k), "topk_ids"),
                                 _ptr(topk_w, torch.float32, (T, k), "topk_w"),
                                 _ptr(near_tie, torch.uint8, (T,), "near_tie"), ctypes.byref(cw),
                                 _ptr(out, torch.bfloat16, (T, H), "out"), _ptr(ws, torch.uint8, None, "ws"),
                                 ws.numel(), _stream(), ev), "moe_route_forward")
