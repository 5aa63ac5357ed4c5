"""Workloads of the MXFP4 expert operators and of the router's balance loss.

Three operators, each as a user's program calls it:

- ``quantize``: rows of activations (``quantize_act``) or expert matrices
  (``encode_weights``) to MXFP4 (E2M1 codes, one E8M0 scale per 32 elements)
  and back to fp32 values (``decode_weights``), the round trip of
  quantisation-aware work; the values come out.
- ``product``: ``group_product``, out[r] = A[src(r)] W[g(r)]^T over rows
  grouped by expert, both operands MXFP4.
- ``balance``: one training step of the router's balance loss:
  ``balance_forward`` (per-expert counts, mean probabilities, loss of each
  sequence) and ``balance_backward`` (gradient of the logits, the gate
  weights' share included).

``run`` computes them in elementary torch operations where ``own`` is false
and through ``block_scaled_expert_amd`` where it is true.  ``exact`` evaluates
the definitions in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

HIDDEN, FFN, EXPERTS, TOP_K = 4608, 2304, 384, 8   # the layer this library is built for


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _quantize(name, mats, rows, cols, dtype, weights):
    return {"name": name, "op": "quantize", "mats": mats, "rows": rows, "cols": cols, "dtype": dtype,
            "weights": weights}


def _product(name, groups, active, tokens, top_k, rows, n, k, out):
    """rows: rows of the product.  tokens > 0: row r reads token ids[r] // top_k
    (the pairs of a dispatch); tokens == 0: row r reads row r."""
    return {"name": name, "op": "product", "groups": groups, "active": active, "tokens": tokens, "top_k": top_k,
            "rows": rows, "n": n, "k": k, "out": out}


def _balance(name, tokens, experts, top_k, seqs, masked, dtype, norm):
    return {"name": name, "op": "balance", "tokens": tokens, "experts": experts, "top_k": top_k, "seqs": seqs,
            "masked": masked, "dtype": dtype, "norm": norm}


def listed():
    return [
        # activations of a 64-token decode batch: launch latency
        _quantize("quantize_decode", 1, 64, HIDDEN, "bf16", False),
        # activations of a 16384-token prefill chunk
        _quantize("quantize_prefill", 1, 16384, HIDDEN, "bf16", False),
        # gate and up matrices of four experts after an update: a weight sync re-encodes them
        _quantize("encode_weights", 8, FFN, HIDDEN, "f32", True),
        # one token's gate/up product over its 8 experts: single-stream decode
        _product("product_token", EXPERTS, 8, 1, TOP_K, 8, 2 * FFN, HIDDEN, "f32"),
        # gate/up of a 64-token decode batch; 283 experts have rows (the mean number under uniform routing)
        _product("product_decode", EXPERTS, 283, 64, TOP_K, 512, 2 * FFN, HIDDEN, "f32"),
        # down of a 192-token decode batch: rows already in expert order
        _product("product_down", EXPERTS, 377, 0, TOP_K, 1536, HIDDEN, FFN, "bf16"),
        # one of eight expert-parallel shares of a 16384-token prefill chunk (48 experts)
        _product("product_prefill", 48, 48, 16384, TOP_K, 16384, 2 * FFN, HIDDEN, "bf16"),
        # odd sizes: a few experts, one of them empty, width and depth off every tile size
        _product("product_ragged", 5, 4, 77, 3, 231, 1003, 352, "bf16"),
        # router step of one short sequence
        _balance("balance_short", 64, EXPERTS, TOP_K, 1, 0.0, "f32", True),
        # 37 packed sequences of uneven length (some empty) with padding tokens, bf16 logits
        _balance("balance_packed", 4099, EXPERTS, TOP_K, 37, 0.1, "bf16", True),
        # router step over a 16384-token batch
        _balance("balance_batch", 16384, EXPERTS, TOP_K, 1, 0.0, "f32", True),
        # the largest training batch: 131072 tokens in 32 sequences
        _balance("balance_large", 131072, EXPERTS, TOP_K, 32, 0.02, "f32", True),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "balance"])
    if op == "quantize":
        weights = rng.random() < 0.4
        cols = 32 * _log(rng, 1, 160)
        if cols == 3072:
            cols += 32
        most = 8 * FFN * HIDDEN // cols
        mats = rng.randint(1, 8) if weights else 1
        rows = _log(rng, 1, min(40000, max(1, most // mats)))
        return _quantize("", mats, rows, cols, rng.choice(["bf16", "f32"]), weights)
    if op == "product":
        groups = _log(rng, 1, EXPERTS)
        k = 32 * _log(rng, 1, HIDDEN // 32)
        n = _log(rng, 1, 2 * FFN)
        if k == 3072:
            k += 32
        if rng.random() < 0.5:
            n = (n + 63) // 64 * 64
        if n == 3072:
            n += 1
        top_k = rng.randint(1, 8)
        if rng.random() < 0.5:      # rows gathered from tokens
            tokens = _log(rng, 1, 16384 // top_k)
            rows = tokens * top_k
        else:
            tokens, rows = 0, _log(rng, 1, 16384)
        active = rng.randint(1, min(groups, rows))
        return _product("", groups, active, tokens, top_k, rows, n, k, rng.choice(["bf16", "f32"]))
    experts = _log(rng, 2, 1024)
    top_k = rng.randint(1, min(experts, 16))
    tokens = _log(rng, 1, min(131072, 131072 * EXPERTS // experts))
    seqs = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(256, tokens)))
    masked = rng.choice([0.0, 0.0, 0.05, 0.5])
    return _balance("", tokens, experts, top_k, seqs, masked, rng.choice(["bf16", "f32"]), rng.random() < 0.8)


def work(case):
    if case["op"] == "quantize":
        e = case["mats"] * case["rows"] * case["cols"]
        # the input and the fp32 values, and codes and scales written and read back
        return {"bytes": e * (2 if case["dtype"] == "bf16" else 4) + 2 * (e // 2 + e // 32) + 4 * e, "flops": 2 * e}
    if case["op"] == "product":
        n, k = case["n"], case["k"]
        per = lambda rows: rows * (k // 2 + k // 32)  # noqa: E731
        a = per(case["tokens"] if case["tokens"] else case["rows"])
        ids = 4 * case["rows"] if case["tokens"] else 0
        out = case["rows"] * n * (2 if case["out"] == "bf16" else 4)
        return {"bytes": a + case["active"] * per(n) + out + ids + 4 * (case["groups"] + 1),
                "flops": 2 * case["rows"] * n * k}
    t, e, k, s = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    # forward: logits and ids in; counts, probabilities, loss out.  backward: logits, ids, the gate
    # weights' gradient and the counts in; the logits' gradient out
    el = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": 3 * t * e * el + t * k * (4 + 4 + 4) + s * e * (4 + 4 + 4) + 2 * t + 8 * s,
            "flops": 20 * t * e}


# --------------------------------------------------------------------------
# MXFP4 in elementary operations
# --------------------------------------------------------------------------

_MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x):
    """fp32 [..., cols] -> (codes uint8 [..., cols/2], scales uint8 [..., cols/32]):
    per block of 32 the scale 2^(floor(log2 max) - 2), elements to the nearest
    E2M1 value, ties to the even code, saturating at 6."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    expo = torch.frexp(amax)[1] - 1 - 2
    expo = torch.where(amax > 0, expo, torch.full_like(expo, -127)).clamp(-127, 127)
    q = torch.ldexp(b, -expo)
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(q)).to(torch.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (expo[..., 0] + 127).to(torch.uint8)


def _decode(codes, scales):
    """fp32 values of MXFP4 codes and scales."""
    table = torch.tensor(_MAGS + tuple(-m for m in _MAGS), dtype=torch.float32, device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).to(torch.int32)]
    v = v.reshape(*scales.shape, 32)
    return torch.ldexp(v, scales.to(torch.int32)[..., None] - 127).reshape(*codes.shape[:-1], -1)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _generator(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


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
    live = r.permutation(case["groups"])[:case["active"]]
    sizes[live] = 1
    p = (1.0 + np.arange(case["active"])) ** -0.4
    sizes[live] += r.multinomial(case["rows"] - case["active"], p / p.sum())
    return sizes


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _generator(seed, dev)
    s = {"case": case}
    if case["op"] == "quantize":
        m, r, c = case["mats"], case["rows"], case["cols"]
        x = torch.empty((m, r, c), dtype=_DT[case["dtype"]], device=dev)
        for i in range(m):
            x[i] = 0.02 * torch.randn((r, c), generator=g, device=dev) if case["weights"] else _activations(r, c, g, dev)
        s["x"] = x if case["weights"] else x[0]
        if own:
            s["codes"] = torch.empty((m, r, c // 2), dtype=torch.uint8, device=dev)
            s["scales"] = torch.empty((m, r, c // 32), dtype=torch.uint8, device=dev)
            s["values"] = torch.empty((m, r, c), dtype=torch.float32, device=dev)
    elif case["op"] == "product":
        G, N, K, R = case["groups"], case["n"], case["k"], case["rows"]
        sizes = _group_sizes(case, seed)
        offsets = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
        s["host_offsets"] = offsets.tolist()
        s["offsets"] = torch.from_numpy(offsets).to(dev)
        s["w"] = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=g, device=dev)
        s["w_sc"] = torch.randint(119, 122, (G, N, K // 32), dtype=torch.uint8, generator=g, device=dev)
        s["a"], s["a_sc"] = _encode(_activations(case["tokens"] or R, K, g, dev))
        s["ids"] = torch.randperm(R, generator=g, device=dev).to(torch.int32) if case["tokens"] else None
        if own:
            s["out"] = torch.empty((R, N), dtype=_DT[case["out"]], device=dev)
    else:
        import random
        T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
        r = random.Random(seed)
        z = torch.randn((T, E), generator=g, device=dev) * 1.4
        z += 0.5 * torch.randn((E,), generator=g, device=dev)      # experts of uneven popularity
        s["z"] = z.to(_DT[case["dtype"]])
        bias = 0.1 * torch.randn((E,), generator=g, device=dev)
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        for lo in range(0, T, 16384):
            sel = torch.sigmoid(s["z"][lo:lo + 16384].float()) + bias
            ids[lo:lo + 16384] = torch.topk(sel, k, dim=1)[1].to(torch.int32)
        s["ids"] = ids
        s["d_w"] = torch.randn((T, k), generator=g, device=dev) * 1e-3
        cuts = sorted(r.randint(0, T) for _ in range(S - 1))
        bounds = np.array([0] + cuts + [T], dtype=np.int32)
        s["host_bounds"] = bounds.tolist()
        s["bounds"] = torch.from_numpy(bounds).to(dev) if S > 1 else None
        if case["masked"]:
            s["mask"] = (torch.rand((T,), generator=g, device=dev) >= case["masked"]).to(torch.uint8)
            s["d_w"] *= s["mask"][:, None]
        else:
            s["mask"] = None
        s["d_loss"] = 1e-2 * (0.5 + torch.rand((S,), generator=g, device=dev))
        if own:
            import block_scaled_expert_amd as bse
            s["cfg"] = bse.Config(num_experts=E, top_k=k, norm_topk=case["norm"], max_tokens=T)
            s["ws"] = bse.balance_workspace(s["cfg"], T, S)
            s["counts"] = torch.empty((S, E), dtype=torch.int32, device=dev)
            s["live"] = torch.empty((S,), dtype=torch.int32, device=dev)
            s["probs"] = torch.empty((S, E), dtype=torch.float32, device=dev)
            s["loss"] = torch.empty((S,), dtype=torch.float32, device=dev)
            s["dz"] = torch.empty_like(s["z"])
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _run_own(s):
    import block_scaled_expert_amd as bse
    case = s["case"]
    if case["op"] == "quantize":
        if case["weights"]:
            bse.encode_weights("mxfp4", s["x"], s["codes"], s["scales"])
        else:
            bse.quantize_act("mxfp4", s["x"], s["codes"][0], s["scales"][0])
        bse.decode_weights("mxfp4", s["codes"], s["scales"], s["values"])
        return s["values"]
    if case["op"] == "product":
        bse.group_product("mxfp4", s["a"], s["a_sc"], s["w"], s["w_sc"], s["offsets"], s["out"], row_ids=s["ids"],
                          id_div=case["top_k"])
        return s["out"]
    bse.balance_forward(s["cfg"], s["z"], s["ids"], s["counts"], s["live"], s["probs"], s["loss"], s["ws"],
                        seq_offsets=s["bounds"], token_mask=s["mask"])
    bse.balance_backward(s["cfg"], s["z"], s["ids"], s["counts"], s["live"], s["d_loss"], s["dz"], d_topk_w=s["d_w"],
                         seq_offsets=s["bounds"], token_mask=s["mask"])
    return {"counts": s["counts"], "live": s["live"], "probs": s["probs"], "loss": s["loss"], "dz": s["dz"]}


def _segments(s):
    """Sequence of each token (int64), from the sequence bounds on the device."""
    T = s["z"].shape[0]
    if s["bounds"] is None:
        return torch.zeros((T,), dtype=torch.int64, device=s["z"].device)
    at = torch.arange(T, dtype=torch.int32, device=s["z"].device)
    return torch.searchsorted(s["bounds"][1:-1].contiguous(), at, right=True)


def _balance_plain(s):
    case = s["case"]
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    dev = s["z"].device
    seg, ids = _segments(s), s["ids"].long()
    live = torch.ones((T,), device=dev) if s["mask"] is None else s["mask"].float()
    n = torch.zeros((S,), device=dev).index_add_(0, seg, live)
    inv_n = torch.where(n > 0, 1.0 / n, torch.zeros_like(n))
    sg = torch.sigmoid(s["z"].float())
    p = sg / sg.sum(1, keepdim=True)
    hit = torch.zeros((T, E), device=dev).scatter_(1, ids, 1.0) * live[:, None]
    counts = torch.zeros((S, E), device=dev).index_add_(0, seg, hit)
    probs = torch.zeros((S, E), device=dev).index_add_(0, seg, p * live[:, None]) * inv_n[:, None]
    loss = (E / k) * inv_n * (counts * probs).sum(1)
    # gradient: the counts carry none
    gain = (s["d_loss"] * (E / k) * inv_n * inv_n)[:, None] * counts
    gt = gain[seg]
    slope = p * (1.0 - sg)
    dz = slope * (gt - (gt * p).sum(1, keepdim=True))
    sel = sg.gather(1, ids)
    if case["norm"]:
        w = sel / sel.sum(1, keepdim=True)
        dw = w * (s["d_w"] - (s["d_w"] * w).sum(1, keepdim=True))
    else:
        dw = sel * s["d_w"]
    dz.scatter_add_(1, ids, dw * (1.0 - sel))
    dz *= live[:, None]
    return {"counts": counts.to(torch.int32), "live": n.to(torch.int32), "probs": probs, "loss": loss,
            "dz": dz.to(s["z"].dtype)}


def run(state):
    if own:
        return _run_own(state)
    s, case = state, state["case"]
    if case["op"] == "quantize":
        x = s["x"].float()
        return _decode(*_encode(x)).reshape(case["mats"], case["rows"], case["cols"])
    if case["op"] == "product":
        a = _decode(s["a"], s["a_sc"])
        if s["ids"] is not None:
            a = a[(s["ids"] // case["top_k"]).long()]
        out = torch.empty((case["rows"], case["n"]), dtype=_DT[case["out"]], device=a.device)
        at = s["host_offsets"]
        for i in range(case["groups"]):
            if at[i + 1] > at[i]:
                out[at[i]:at[i + 1]] = torch.mm(a[at[i]:at[i + 1]], _decode(s["w"][i], s["w_sc"][i]).t())
        return out
    return _balance_plain(s)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _value64(codes, scales):
    """Values of MXFP4 codes from the bit fields, in 64 bits."""
    nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    e, m = (nib // 2) % 4, nib % 2
    mag = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2((e - 1).double()))
    step = torch.exp2(scales.double() - 127.0).repeat_interleave(32, -1)
    return torch.where(nib >= 8, -mag, mag) * step


def _rounded64(x):
    """x to its MXFP4 value: elements rounded half to even on the E2M1 grid of their binade."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    step = torch.exp2((torch.floor(torch.log2(top)) - 2.0).clamp(-127.0, 127.0))
    q = b / step
    grid = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=1.0))) - 1.0)
    return ((torch.round(q / grid) * grid).clamp(-6.0, 6.0) * step).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"] if case["weights"] else s["x"][None]
        out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for i in range(x.shape[0]):
            for lo in range(0, x.shape[1], 4096):
                out[i, lo:lo + 4096] = _rounded64(x[i, lo:lo + 4096])
        return out
    if case["op"] == "product":
        out = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=s["w"].device)
        src = torch.arange(case["rows"], device=out.device)
        if s["ids"] is not None:
            src = torch.div(s["ids"].long(), case["top_k"], rounding_mode="floor")
        at = s["host_offsets"]
        for i, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
            if lo < hi:
                rows = src[lo:hi]
                out[lo:hi] = _value64(s["a"][rows], s["a_sc"][rows]) @ _value64(s["w"][i], s["w_sc"][i]).T
        return out
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    z, dev = s["z"], s["z"].device
    counts = torch.zeros((S, E), dtype=torch.int64, device=dev)
    live = torch.zeros((S,), dtype=torch.int64, device=dev)
    probs = torch.zeros((S, E), dtype=torch.float64, device=dev)
    loss = torch.zeros((S,), dtype=torch.float64, device=dev)
    dz = torch.zeros((T, E), dtype=torch.float64, device=dev)
    for i, (lo, hi) in enumerate(zip(s["host_bounds"][:-1], s["host_bounds"][1:])):
        at = torch.arange(lo, hi, device=dev)
        if s["mask"] is not None:
            at = at[s["mask"][lo:hi] != 0]
        n = at.numel()
        if n == 0:
            continue
        zi, ids, dw = z[at].double(), s["ids"][at].long(), s["d_w"][at].double()
        sg = 1.0 / (1.0 + torch.exp(-zi))
        p = sg / sg.sum(1, keepdim=True)
        counts[i] = torch.bincount(ids.flatten(), minlength=E)
        live[i] = n
        probs[i] = p.mean(0)
        f = counts[i].double() * (E / (k * n))
        loss[i] = torch.dot(f, probs[i])
        g = f * (s["d_loss"][i].double() / n)
        d = p * (1.0 - sg) * (g - (p @ g)[:, None])
        c = sg.gather(1, ids)
        if case["norm"]:
            t = c.sum(1, keepdim=True)
            dc = dw / t - (dw * c).sum(1, keepdim=True) / t ** 2
        else:
            dc = dw
        d.scatter_add_(1, ids, dc * c * (1.0 - c))
        dz[at] = d
    return {"counts": counts, "live": live, "probs": probs, "loss": loss, "dz": dz}
