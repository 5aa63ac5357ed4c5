"""Workloads of the operators around the expert products.

Three operators, each as a user's program calls it:

- ``norm``: the layer's input: ``norm_forward`` (residual addition,
  root-mean-square norm and, where asked for, the MXFP8 codes and scales of the
  normed rows) and, in training, ``norm_backward`` (gradients of the residual
  stream, of the input and of the weight).
- ``rows``: tokens sorted by expert and back: ``sort_rows`` and
  ``combine_rows`` (the gate weights applied) and, in training,
  ``combine_rows_backward`` and ``sort_rows_backward``.
- ``matvec``: ``group_matvec``, out[r] = x[src(r)] W[g(r)]^T for the few rows
  that an expert has in decoding, x in bf16 or fp32 and W in NVFP4 or MXFP4,
  with the capped SwiGLU of a gate/up product in the same pass where asked for.

``run`` computes them in elementary torch operations where ``own`` is false
and through ``block_scaled_expert_amd`` where it is true.  ``exact`` evaluates
the definitions in 64 bits, written apart from both.  MXFP8 codes and scales
come back as the 8-bit floats that they are.
"""
import math

import numpy as np
import torch

own = False

HIDDEN, FFN, EXPERTS, TOP_K = 4608, 2304, 384, 8   # the layer this library is built for
EPS, CAP = 1e-6, 7.0


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _norm(name, tokens, cols, dtype, residual, codes, train):
    """residual: type of the residual stream, "none" without one."""
    return {"name": name, "op": "norm", "tokens": tokens, "cols": cols, "dtype": dtype, "residual": residual,
            "codes": codes, "train": train}


def _rows(name, tokens, experts, local, top_k, cols, dtype, y_dtype, train):
    """local: how many of the experts are on this GPU (the first ones)."""
    return {"name": name, "op": "rows", "tokens": tokens, "experts": experts, "local": local, "top_k": top_k,
            "cols": cols, "dtype": dtype, "y_dtype": y_dtype, "train": train}


def _matvec(name, fmt, groups, active, tokens, top_k, rows, n, k, swiglu, dtype, out):
    """rows: rows of the product.  tokens > 0: row r reads token ids[r] // top_k
    (the pairs of a dispatch); tokens == 0: row r reads row r.  swiglu: n is the
    width of [gate | up], half of it comes out."""
    return {"name": name, "op": "matvec", "fmt": fmt, "groups": groups, "active": active, "tokens": tokens,
            "top_k": top_k, "rows": rows, "n": n, "k": k, "swiglu": swiglu, "dtype": dtype, "out": out}


def listed():
    return [
        # input of the layer for a 64-token decode batch: launch latency
        _norm("norm_decode", 64, HIDDEN, "bf16", "bf16", True, False),
        # the same for a 16384-token prefill chunk
        _norm("norm_prefill", 16384, HIDDEN, "bf16", "bf16", True, False),
        # a training batch with the residual stream kept in fp32
        _norm("norm_train", 16384, HIDDEN, "bf16", "f32", False, True),
        # odd sizes, fp32, no residual: rows that are no multiple of a vector
        _norm("norm_odd", 1537, 1003, "f32", "none", False, True),
        # 64 decode tokens to their experts and back, expert outputs in fp32 as the layer keeps them
        _rows("rows_decode", 64, EXPERTS, EXPERTS, TOP_K, HIDDEN, "bf16", "f32", False),
        # a 16384-token training batch on one GPU, both directions
        _rows("rows_train", 16384, EXPERTS, EXPERTS, TOP_K, HIDDEN, "bf16", "bf16", True),
        # one of eight expert-parallel shares of it: seven of eight pairs are elsewhere
        _rows("rows_share", 16384, EXPERTS, 48, TOP_K, HIDDEN, "bf16", "f32", True),
        # odd sizes, fp32, an uneven split
        _rows("rows_ragged", 999, 7, 5, 3, 1003, "f32", "f32", True),
        # one token's gate/up and SwiGLU over its 8 experts: single-stream decode
        _matvec("matvec_token", "nvfp4", EXPERTS, 8, 1, TOP_K, 8, 2 * FFN, HIDDEN, True, "bf16", "f32"),
        # the same for a 64-token decode batch; 283 experts have rows (the mean number under uniform routing)
        _matvec("matvec_decode", "nvfp4", EXPERTS, 283, 64, TOP_K, 512, 2 * FFN, HIDDEN, True, "bf16", "f32"),
        # down of a 192-token decode batch: fp32 rows already in expert order
        _matvec("matvec_down", "mxfp4", EXPERTS, 377, 0, TOP_K, 1536, HIDDEN, FFN, False, "f32", "f32"),
        # odd sizes: a few experts, one of them empty, width and depth off every tile size
        _matvec("matvec_ragged", "mxfp4", 5, 4, 17, 3, 51, 1003, 352, False, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rows", "matvec"])
    if op == "norm":
        codes = rng.random() < 0.4
        cols = 32 * _log(rng, 1, 512) if codes else _log(rng, 8, 16384)
        if not codes and rng.random() < 0.5:
            cols = (cols + 7) // 8 * 8
        tokens = _log(rng, 1, min(65536, 16384 * HIDDEN // cols))
        dtype = rng.choice(["bf16", "f32"])
        residual = rng.choice(["none", dtype, "f32"])
        return _norm("", tokens, cols, dtype, residual, codes, not codes and rng.random() < 0.7)
    if op == "rows":
        experts = _log(rng, 2, 1024)
        top_k = rng.randint(1, min(experts, 16))
        local = experts if rng.random() < 0.5 else rng.randint(1, experts)
        cols = _log(rng, 8, 8192)
        if rng.random() < 0.6:
            cols = (cols + 7) // 8 * 8
        tokens = _log(rng, 1, min(16384, 16384 * HIDDEN * TOP_K // (2 * cols * top_k)))
        return _rows("", tokens, experts, local, top_k, cols, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]),
                     rng.random() < 0.6)
    groups = _log(rng, 1, EXPERTS)
    k = 32 * _log(rng, 1, HIDDEN // 32)
    n = _log(rng, 2, 2 * FFN)
    if rng.random() < 0.5:
        n = (n + 63) // 64 * 64
    swiglu = rng.random() < 0.4
    n += n % 2 if swiglu else 0
    top_k = rng.randint(1, 8)
    rows = _log(rng, 1, min(2048, 64 * groups))
    tokens = 0
    if rng.random() < 0.5:      # rows gathered from tokens
        tokens = max(1, rows // top_k)
        rows = tokens * top_k
    return _matvec("", rng.choice(["nvfp4", "mxfp4"]), groups, rng.randint(1, min(groups, rows)), tokens, top_k, rows, n, k,
                   swiglu, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]))


_BYTES = {"bf16": 2, "f32": 4, "none": 0}


def work(case):
    el = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        t, c = case["tokens"], case["cols"]
        res = _BYTES[case["residual"]]
        # forward: x, residual and weight in; the new residual, y (codes and scales), 1 / rms out
        size = t * c * (el + 2 * res + el) + 4 * c + 4 * t
        size += t * (c + c // 32) if case["codes"] else 0
        if case["train"]:
            # backward: dy, the normed stream, what reaches it from further on, 1 / rms and weight in; its
            # gradient, the input's where that is of another type, and the weight's out
            size += t * c * (el + (3 * res if res else 2 * el) + (el if res > el else 0)) + 8 * c + 4 * t
        return {"bytes": size, "flops": t * c * (16 if case["train"] else 5)}
    if case["op"] == "rows":
        t, c, ye = case["tokens"], case["cols"], _BYTES[case["y_dtype"]]
        pairs = t * case["top_k"]
        here = pairs * case["local"] // case["experts"]
        # sort and combine: x and y in, sorted rows and the output out
        size = t * c * el + here * c * el + here * c * ye + t * c * el + 8 * pairs
        if case["train"]:
            # back: the output's gradient and y in, y's and the gate weights' out; the sorted rows' in, x's out
            size += t * c * el + 2 * here * c * ye + 8 * pairs + here * c * el + t * c * el
        return {"bytes": size, "flops": here * c * (7 if case["train"] else 2)}
    n, k = case["n"], case["k"]
    w = n * (k // 2 + k // (16 if case["fmt"] == "nvfp4" else 32))
    x = (case["tokens"] if case["tokens"] else case["rows"]) * k * el
    width = n // 2 if case["swiglu"] else n
    ids = 4 * case["rows"] if case["tokens"] else 0
    return {"bytes": case["active"] * w + x + ids + case["rows"] * width * _BYTES[case["out"]] + 4 * (case["groups"] + 1),
            "flops": 2 * case["rows"] * n * k}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _activations(rows, cols, g, dev):
    """N(0, 1) tokens, a few channels 20 times larger, as they reach an expert layer."""
    x = torch.randn((rows, cols), generator=g, device=dev)
    x[:, ::277] *= 20.0
    return x


def _group_sizes(case, seed):
    """Rows of each group: `active` groups have at least one, the rest follow a
    long-tailed popularity; deterministic in the seed."""
    r = np.random.default_rng(seed)
    sizes = np.zeros(case["groups"], dtype=np.int64)
    live = np.sort(r.permutation(case["groups"])[:case["active"]])
    sizes[live] = 1
    p = (1.0 + np.arange(case["active"])) ** -0.4
    sizes[live] += r.multinomial(case["rows"] - case["active"], r.permutation(p) / p.sum())
    return sizes, live


def _prepare_norm(case, g, dev):
    t, c, dt, res = case["tokens"], case["cols"], _DT[case["dtype"]], _DT.get(case["residual"])
    s = {"case": case, "x": _activations(t, c, g, dev).to(dt), "res": None, "d_next": None,
         "weight": 1.0 + 0.1 * torch.randn((c,), generator=g, device=dev)}
    if res is not None:
        s["res"] = (3.0 * torch.randn((t, c), generator=g, device=dev)).to(res)
    if case["train"]:
        s["dy"] = (1e-3 * torch.randn((t, c), generator=g, device=dev)).to(dt)
        if res is not None:
            s["d_next"] = (1e-3 * torch.randn((t, c), generator=g, device=dev)).to(res)
    if own:
        import block_scaled_expert_amd as bse
        s["y"] = torch.empty_like(s["x"])
        s["rstd"] = torch.empty((t,), device=dev)
        s["sum"] = None if res is None else torch.empty_like(s["res"])
        s["cfg"] = bse.Config(fmt="mxfp8") if case["codes"] else None
        s["codes"] = torch.empty((t, c), dtype=torch.uint8, device=dev) if case["codes"] else None
        s["scales"] = torch.empty((t, c // 32), dtype=torch.uint8, device=dev) if case["codes"] else None
        if case["train"]:
            s["ws"] = bse.norm_workspace(t, c)
            s["d_res"] = torch.empty((t, c), dtype=dt if res is None else res, device=dev)
            s["dx"] = torch.empty_like(s["x"]) if res is not None and res != dt else None
            s["d_weight"] = torch.empty_like(s["weight"])
    return s


def _prepare_rows(case, g, dev):
    t, k, c, dt, yt = case["tokens"], case["top_k"], case["cols"], _DT[case["dtype"]], _DT[case["y_dtype"]]
    score = torch.rand((t, case["experts"]), generator=g, device=dev) + 0.2 * torch.rand((case["experts"],), generator=g, device=dev)
    ids = torch.topk(score, k, dim=1)[1].flatten()
    order = torch.sort(ids, stable=True)[1]
    here = int((ids < case["local"]).sum())
    pos = torch.full((t * k,), -1, dtype=torch.int32, device=dev)
    pos[order[:here]] = torch.arange(here, dtype=torch.int32, device=dev)
    w = torch.rand((t, k), generator=g, device=dev) + 0.1
    s = {"case": case, "pos": pos, "pairs": order[:here].to(torch.int32), "topk_w": w / w.sum(1, keepdim=True),
         "x": _activations(t, c, g, dev).to(dt), "y": torch.randn((t * k, c), generator=g, device=dev).to(yt)}
    if case["train"]:
        s["d_out"] = (1e-3 * torch.randn((t, c), generator=g, device=dev)).to(dt)
        s["d_sorted"] = (1e-3 * torch.randn((t * k, c), generator=g, device=dev)).to(dt)
    if own:
        s["sorted"] = torch.zeros((t * k, c), dtype=dt, device=dev)   # rows of pairs elsewhere keep what they hold
        s["out"] = torch.empty_like(s["x"])
        if case["train"]:
            s["dy"], s["d_w"], s["dx"] = torch.zeros_like(s["y"]), torch.empty_like(s["topk_w"]), torch.empty_like(s["x"])
    return s


def _prepare_matvec(case, g, dev, seed):
    G, N, K, R = case["groups"], case["n"], case["k"], case["rows"]
    nv = case["fmt"] == "nvfp4"
    sizes, live = _group_sizes(case, seed)
    offsets = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    s = {"case": case, "live": torch.from_numpy(live).to(dev), "most": int(sizes.max()), "host_offsets": offsets.tolist(),
         "offsets": torch.from_numpy(offsets).to(dev),
         "w": torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=g, device=dev)}
    lo, hi = (0x60, 0x7F) if nv else (119, 122)        # E4M3 16 .. 448; 2^-8 .. 2^-6
    s["w_sc"] = torch.randint(lo, hi, (G, N, K // (16 if nv else 32)), dtype=torch.uint8, generator=g, device=dev)
    s["mats"] = 2 if case["swiglu"] else 1              # matrices with an fp32 scale of their own
    s["gs"] = (0.1 + 0.05 * torch.rand((G, 3), generator=g, device=dev)) / 2688 if nv else None
    s["x"] = _activations(case["tokens"] or R, K, g, dev).to(_DT[case["dtype"]])
    s["ids"] = torch.randperm(R, generator=g, device=dev).to(torch.int32) if case["tokens"] else None
    if own:
        import block_scaled_expert_amd as bse
        s["cfg"] = bse.Config(fmt=case["fmt"], cap=CAP) if case["swiglu"] else None
        s["out"] = torch.empty((R, N // 2 if case["swiglu"] else N), dtype=_DT[case["out"]], device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if case["op"] == "norm":
        return _prepare_norm(case, g, dev)
    if case["op"] == "rows":
        return _prepare_rows(case, g, dev)
    return _prepare_matvec(case, g, dev, seed)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _run_own(s):
    import block_scaled_expert_amd as bse
    case = s["case"]
    if case["op"] == "norm":
        bse.norm_forward(s["x"], s["weight"], s["y"], residual=s["res"], res_out=s["sum"], rstd=s["rstd"], eps=EPS,
                         cfg=s["cfg"], codes=s["codes"], scales=s["scales"])
        out = {"y": s["y"], "sum": s["sum"], "rstd": s["rstd"]}
        if case["codes"]:
            out["codes"] = s["codes"].view(torch.float8_e4m3fn)
            out["scales"] = s["scales"].view(torch.float8_e8m0fnu)
        if case["train"]:
            stream = s["x"] if s["sum"] is None else s["sum"]
            bse.norm_backward(s["dy"], stream, s["weight"], s["rstd"], s["d_res"], s["ws"], d_res_out=s["d_next"],
                              dx=s["dx"], d_weight=s["d_weight"])
            out.update(d_res=s["d_res"], dx=s["dx"], d_weight=s["d_weight"])
        return out
    if case["op"] == "rows":
        bse.sort_rows(s["x"], s["pos"], s["sorted"])
        bse.combine_rows(s["y"], s["pos"], s["topk_w"], s["out"])
        out = {"sorted": s["sorted"], "out": s["out"]}
        if case["train"]:
            bse.combine_rows_backward(s["d_out"], s["y"], s["pos"], s["topk_w"], s["dy"], s["d_w"])
            bse.sort_rows_backward(s["d_sorted"], s["pos"], s["dx"])
            out.update(dy=s["dy"], d_w=s["d_w"], dx=s["dx"])
        return out
    bse.group_matvec(case["fmt"], s["x"], s["w"], s["w_sc"], s["offsets"], s["out"], gs=s["gs"], gs_group=s["mats"],
                     gs_stride=3, row_ids=s["ids"], id_div=case["top_k"], swiglu=s["cfg"])
    return s["out"]


def _e4m3(q):
    """fp32 rounded half to even to E4M3 values, saturating at 448."""
    e = (torch.frexp(q)[1] - 1).clamp(min=-6)
    return torch.ldexp(torch.round(torch.ldexp(q, 3 - e)), e - 3).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _mxfp8(y):
    """Rows to E4M3 values and the power-of-two scales of their blocks of 32."""
    b = y.float().reshape(y.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 1 - 8).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    return _e4m3(torch.ldexp(b, -e)).reshape(y.shape), (e[..., 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _norm_plain(s):
    case = s["case"]
    dt = s["x"].dtype
    total = None if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    v = s["x"].float() if total is None else total.float()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    n = v * rstd[:, None]
    y = (n * s["weight"]).to(dt)
    out = {"y": y, "sum": total, "rstd": rstd}
    if case["codes"]:
        out["codes"], out["scales"] = _mxfp8(y)
    if case["train"]:
        dn = s["dy"].float() * s["weight"]
        d = rstd[:, None] * (dn - n * (dn * n).mean(1, keepdim=True))
        if s["d_next"] is not None:
            d = d + s["d_next"].float()
        other = total is not None and total.dtype != dt
        out.update(d_res=d.to(dt if total is None else total.dtype), dx=d.to(dt) if other else None,
                   d_weight=(s["dy"].float() * n).sum(0))
    return out


def _rows_plain(s):
    case = s["case"]
    t, k, c, dt = case["tokens"], case["top_k"], case["cols"], s["x"].dtype
    pairs = s["pairs"].long()
    here = pairs.numel()
    token = torch.div(pairs, k, rounding_mode="floor")
    place = s["pos"].long().clamp(min=0)
    on = (s["pos"] >= 0).float()
    rows = torch.zeros((t * k, c), dtype=dt, device=s["x"].device)
    rows[:here] = s["x"][token]
    w = s["topk_w"].flatten() * on
    back = s["y"].float()[place] * w[:, None]
    out = {"sorted": rows, "out": back.reshape(t, k, c).sum(1).to(dt)}
    if case["train"]:
        d = s["d_out"].float()[token]
        dy = torch.zeros_like(s["y"])
        dy[:here] = (d * s["topk_w"].flatten()[pairs][:, None]).to(dy.dtype)
        dw = torch.zeros((t * k,), device=d.device)
        dw[pairs] = (d * s["y"][:here].float()).sum(1)
        dx = (s["d_sorted"].float()[place] * on[:, None]).reshape(t, k, c).sum(1)
        out.update(dy=dy, d_w=dw.reshape(t, k), dx=dx.to(dt))
    return out


_MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _weights(s):
    """fp32 values of the matrices that have rows."""
    codes, sc = s["w"][s["live"]], s["w_sc"][s["live"]]
    table = torch.tensor(_MAGS + tuple(-m for m in _MAGS), dtype=torch.float32, device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).to(torch.int32)].reshape(*sc.shape, -1)
    if s["gs"] is None:
        v = torch.ldexp(v, sc.to(torch.int32)[..., None] - 127)
    else:
        v = v * sc.view(torch.float8_e4m3fn).float()[..., None]
        gs = s["gs"][s["live"]][:, :s["mats"]]
        v = v * gs.repeat_interleave(sc.shape[1] // s["mats"], 1)[..., None, None]
    return v.reshape(*codes.shape[:2], -1)


def _matvec_plain(s):
    case = s["case"]
    x = s["x"].float()
    first, last = s["offsets"][:-1][s["live"]].long(), s["offsets"][1:][s["live"]].long()
    row = first[:, None] + torch.arange(s["most"], device=x.device)          # [group][row of it]
    there = row < last[:, None]
    row = row.clamp(max=case["rows"] - 1)
    src = row if s["ids"] is None else torch.div(s["ids"].long()[row], case["top_k"], rounding_mode="floor")
    y = torch.bmm(_weights(s), x[src].transpose(1, 2).contiguous()).transpose(1, 2)
    if case["swiglu"]:
        g, u = y[..., :case["n"] // 2], y[..., case["n"] // 2:]
        g, u = CAP * torch.tanh(g / CAP), CAP * torch.tanh(u / CAP)
        y = g / (1.0 + torch.exp(-g)) * u
    out = torch.empty((case["rows"], y.shape[-1]), dtype=_DT[case["out"]], device=x.device)
    out[row[there]] = y[there].to(out.dtype)
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "rows": _rows_plain, "matvec": _matvec_plain}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _encoded64(y):
    """Blocks of 32 of the stored y: values on the E4M3 grid of their binade, and the steps."""
    b = y.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    step = torch.exp2((torch.floor(torch.log2(top)) - 8.0).clamp(-127.0, 127.0))
    q = b / step
    grid = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(q / grid) * grid).clamp(-448.0, 448.0).flatten(-2), step[..., 0]


def _norm64(s):
    case = s["case"]
    t, c = s["x"].shape
    dev, f64 = s["x"].device, torch.float64
    new = lambda *shape: torch.empty(shape, dtype=f64, device=dev)  # noqa: E731
    res = s["res"] is not None
    out = {"y": new(t, c), "sum": new(t, c) if res else None, "rstd": new(t)}
    if case["codes"]:
        out["codes"], out["scales"] = new(t, c), new(t, c // 32)
    if case["train"]:
        out.update(d_res=new(t, c), dx=None, d_weight=torch.zeros(c, dtype=f64, device=dev))
    w = s["weight"].double()
    for i in range(0, t, 2048):
        at = slice(i, min(t, i + 2048))
        v = s["x"][at].double()
        if res:
            v = v + s["res"][at].double()
            out["sum"][at] = v
            v = v.to(s["res"].dtype).double()     # the stream is normed as it is stored
        ms = (v ** 2).sum(1, keepdim=True) / c + EPS
        y = v * w / ms.sqrt()
        out["y"][at], out["rstd"][at] = y, ms[:, 0] ** -0.5
        if case["codes"]:
            out["codes"][at], out["scales"][at] = _encoded64(y.to(s["x"].dtype))
        if case["train"]:
            a = s["dy"][at].double()
            d = a * w / ms.sqrt() - v * (a * w * v).sum(1, keepdim=True) / (c * ms ** 1.5)
            out["d_res"][at] = d if s["d_next"] is None else d + s["d_next"][at].double()
            out["d_weight"] += (a * v / ms.sqrt()).sum(0)
    if case["train"] and res and s["res"].dtype != s["x"].dtype:
        out["dx"] = out["d_res"]
    return out


def _rows64(s):
    case = s["case"]
    t, k, c = case["tokens"], case["top_k"], case["cols"]
    dev, f64 = s["x"].device, torch.float64
    zero = lambda *shape: torch.zeros(shape, dtype=f64, device=dev)  # noqa: E731
    out = {"sorted": zero(t * k, c), "out": zero(t, c)}
    if case["train"]:
        out.update(dy=zero(t * k, c), d_w=zero(t, k), dx=zero(t, c))
    pos = s["pos"].view(t, k).long()
    for j in range(k):
        for i in range(0, t, 4096):
            tok = torch.nonzero(pos[i:i + 4096, j] >= 0)[:, 0] + i
            at, w = pos[tok, j], s["topk_w"][tok, j].double()[:, None]
            out["sorted"][at] = s["x"][tok].double()
            out["out"][tok] += w * s["y"][at].double()
            if case["train"]:
                d = s["d_out"][tok].double()
                out["dy"][at] = w * d
                out["d_w"][tok, j] = (d * s["y"][at].double()).sum(1)
                out["dx"][tok] += s["d_sorted"][at].double()
    return out


def _value64(codes, scales, nv):
    """Values of 4-bit codes under their block scales, from the bit fields, in 64 bits."""
    def fields(v, bits, bias, man):
        e, m = (v // 2 ** man) % 2 ** bits, v % 2 ** man
        low = m.double() * 2.0 ** (1 - bias - man)
        mag = torch.where(e == 0, low, (1.0 + m.double() / 2 ** man) * torch.exp2((e - bias).double()))
        return torch.where(v >= 2 ** (bits + man), -mag, mag)

    nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    step = fields(scales.to(torch.int64), 4, 7, 3) if nv else torch.exp2(scales.double() - 127.0)
    return fields(nib, 2, 1, 1) * step.repeat_interleave(16 if nv else 32, -1)


def _matvec64(s):
    case = s["case"]
    nv, half = case["fmt"] == "nvfp4", case["n"] // 2
    out = torch.zeros((case["rows"], half if case["swiglu"] else case["n"]), dtype=torch.float64, device=s["w"].device)
    src = torch.arange(case["rows"], device=out.device)
    if s["ids"] is not None:
        src = torch.div(s["ids"].long(), case["top_k"], rounding_mode="floor")
    for i in s["live"].tolist():
        lo, hi = s["host_offsets"][i], s["host_offsets"][i + 1]
        y = s["x"][src[lo:hi]].double() @ _value64(s["w"][i], s["w_sc"][i], nv).T
        if nv:
            y *= s["gs"][i, :s["mats"]].double().repeat_interleave(case["n"] // s["mats"])
        if case["swiglu"]:
            g, u = CAP * torch.tanh(y[:, :half] / CAP), CAP * torch.tanh(y[:, half:] / CAP)
            y = g * u * torch.sigmoid(g)
        out[lo:hi] = y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm64, "rows": _rows64, "matvec": _matvec64}[case["op"]](s)
