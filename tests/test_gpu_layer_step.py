"""The residual norm, the sorted rows, the 4-bit matrix-vector product and the
forward of quantized tokens together with routing, dispatch and the balance
loss: a serving step and a training step as a user's program runs them, eager,
captured into graphs, and on two streams at once."""
import numpy as np
import pytest

import synth
from oracle import balance as B
from oracle import formats as F
from oracle import layer as L
from oracle import stream as S

from _util import lib_cfg, stack_local, to_dev

pytestmark = pytest.mark.gpu


def _bf16(seed, *shape, scale=1.0):
    import torch
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16().cuda()


def _f64(t):
    return t.double().cpu().numpy()


# -- forward of quantized tokens ----------------------------------------------

QUANT = {
    "mxfp8_decode": synth.Workload("q1", "quantized", 20, 512, 48, 8, 256, "mxfp8", 41, weights="gaussian"),
    "mxfp8_large": synth.Workload("q2", "quantized", 700, 256, 8, 2, 128, "mxfp8", 42, weights="gaussian"),
    "nvfp4_decode": synth.Workload("q3", "quantized", 33, 512, 32, 4, 256, "nvfp4", 43, weights="gaussian"),
    "nvfp4_large": synth.Workload("q4", "quantized", 600, 256, 16, 8, 128, "nvfp4", 44, weights="gaussian"),
    "mxfp4": synth.Workload("q5", "quantized", 65, 256, 12, 3, 128, "mxfp4", 45, weights="gaussian"),
    "one_token": synth.Workload("q6", "quantized", 1, 256, 12, 3, 128, "mxfp8", 46, weights="gaussian"),
}


@pytest.mark.parametrize("key", list(QUANT))
def test_forward_of_normed_tokens(gpu_lib, key):
    """Codes from the norm give the layer's output on the normed tokens, bit for
    bit; a share of the experts too."""
    import torch
    bse, w = gpu_lib, QUANT[key]
    T, H = w.tokens, w.hidden
    stacked, _ = stack_local(w)
    for share in (False, True):
        kw = dict(expert_begin=w.experts // 3, num_local_experts=w.experts // 2) if share else {}
        cfg = bse.Config(hidden=H, ffn=w.ffn, num_experts=w.experts, top_k=w.top_k, fmt=w.fmt, cap=w.cap, max_tokens=T, **kw)
        lo, n = (w.experts // 3, w.experts // 2) if share else (0, w.experts)
        wd = {k: to_dev(v[lo:lo + n]) for k, v in stacked.items()}
        x, res, gain = _bf16(1, T, H), _bf16(2, T, H, scale=2.0), 1.0 + 0.1 * _bf16(3, H).float()
        y, s = torch.empty_like(x), torch.empty_like(x)
        per = {"mxfp8": H}.get(w.fmt, H // 2)
        codes = torch.empty((T, per), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, H // (16 if w.fmt == "nvfp4" else 32)), dtype=torch.uint8, device="cuda")
        row_gs = torch.empty(T, device="cuda")
        bse.norm_forward(x, gain, y, residual=res, res_out=s, cfg=cfg, codes=codes, scales=scales, row_gs=row_gs)
        ids = torch.stack([torch.randperm(w.experts, generator=torch.Generator().manual_seed(t))[:w.top_k] for t in range(T)])
        ids, tw = ids.int().cuda(), torch.rand((T, w.top_k), generator=torch.Generator().manual_seed(7)).cuda()
        want, got = torch.empty_like(x), torch.full_like(x, float("nan"))
        bse.forward(cfg, y, ids, tw, wd, want, bse.workspace(cfg))
        ws = torch.full((bse.workspace_size(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
        bse.forward_quantized(cfg, codes, scales, ids, tw, wd, got, ws, row_gs=row_gs)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), share
        if w.fmt != "mxfp4":
            packed = bse.prepare_weights(cfg, wd)
            bse.forward_quantized(cfg, codes, scales, ids, tw, packed, got.zero_(), ws, row_gs=row_gs)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)), share


# -- serving: unquantized activations, 4-bit weights --------------------------

class Serving:
    """norm -> route -> dispatch -> gate/up with SwiGLU -> down -> combine."""

    def __init__(self, bse, w, T):
        import torch
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.bse, self.w, self.T = bse, w, T
        self.cfg = lib_cfg(bse, w, max_tokens=T)
        self.stacked, _ = stack_local(w)
        self.wd = {k: to_dev(v) for k, v in self.stacked.items()}
        H, E, k = w.hidden, w.experts, w.top_k
        self.gain = 1.0 + 0.1 * _bf16(5, H).float()
        self.wr = torch.from_numpy(synth.router_weight(w.seed, E, H).view(np.int16)).view(torch.bfloat16).cuda()
        self.bias = torch.from_numpy(synth.router_bias(w.seed, E, w.bias)).cuda()
        self.x, self.res = _bf16(1, T, H), _bf16(2, T, H)
        self.ws = bse.workspace(self.cfg)
        self.s, self.y, self.out = new(T, H, dtype=torch.bfloat16), new(T, H, dtype=torch.bfloat16), new(T, H, dtype=torch.bfloat16)
        self.ids, self.tw = new(T, k, dtype=torch.int32), new(T, k)
        self.offsets, self.pairs, self.pos = (new(n, dtype=torch.int32) for n in (E + 1, T * k, T * k))
        self.h, self.d = new(T * k, w.ffn), new(T * k, H)
        self.gs13 = self.wd["gs"].view(-1) if "gs" in self.wd else None
        self.gs2 = None if self.gs13 is None else self.gs13[2:]

    def step(self):
        bse, cfg, f = self.bse, self.cfg, self.w.fmt
        bse.norm_forward(self.x, self.gain, self.y, residual=self.res, res_out=self.s)
        bse.route(cfg, self.y, self.wr, self.bias, self.ids, self.tw, None, self.ws)
        bse.dispatch(cfg, self.ids, self.offsets, self.pairs, self.pos, self.ws)
        bse.group_matvec(f, self.y, self.wd["w13"], self.wd["w13_sc"], self.offsets, self.h, gs=self.gs13, gs_group=2,
                         gs_stride=3, row_ids=self.pairs, id_div=self.w.top_k, swiglu=cfg)
        bse.group_matvec(f, self.h, self.wd["w2"], self.wd["w2_sc"], self.offsets, self.d, gs=self.gs2, gs_group=1,
                         gs_stride=3)
        bse.combine_rows(self.d, self.pos, self.tw, self.out)

    def expected(self):
        """float64 from the step's own routing and normed tokens."""
        w = self.w
        y, ids, tw = _f64(self.y), self.ids.cpu().numpy(), _f64(self.tw)
        mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])

        def values(codes, sc, gs):
            if w.fmt == "mxfp4":
                return F.dequantize_mxfp4(codes, sc)
            nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
            return np.where(nib & 8, -1.0, 1.0) * mag[nib & 7] * np.repeat(F.e4m3_decode(sc).astype(np.float64), 16, -1) * gs

        out = np.zeros((self.T, w.hidden))
        n = w.ffn
        for e in np.unique(ids):
            c = {k: v[e] for k, v in self.stacked.items()}
            gs = c.get("gs", np.ones(3)).astype(np.float64)
            w13, w2 = values(c["w13"], c["w13_sc"], 1.0), values(c["w2"], c["w2_sc"], gs[2])
            t, j = np.nonzero(ids == e)
            g, u = y[t] @ (w13[:n] * gs[0]).T, y[t] @ (w13[n:] * gs[1]).T
            g, u = w.cap * np.tanh(g / w.cap), w.cap * np.tanh(u / w.cap)
            out[t] += tw[t, j][:, None] * ((g / (1 + np.exp(-g)) * u) @ w2.T)
        return out


SERVE = {f: synth.Workload("s", "serving", 0, 512, 24, 4, 384, f, 51, weights="gaussian") for f in ("nvfp4", "mxfp4")}


@pytest.mark.parametrize("fmt", list(SERVE))
@pytest.mark.parametrize("T", [1, 5, 33])
def test_serving_step(gpu_lib, fmt, T):
    """Against float64: the epilogue's 2e-5 and the sums' rounding are far below
    bf16's half step, 2^-8 of a value of the output's size."""
    import torch
    p = Serving(gpu_lib, SERVE[fmt], T)
    p.step()
    torch.cuda.synchronize()
    want = p.expected()
    assert np.abs(_f64(p.out) - want).max() <= (2.0 ** -8 + 1e-4) * np.abs(want).max()
    y = S.norm_forward(_f64(p.s), _f64(p.gain), float(np.float32(1e-6)))[0]
    assert (np.abs(_f64(p.y) - y) <= (2.0 ** -8 + 1e-5) * np.abs(y)).all()


@pytest.mark.parametrize("fmt", list(SERVE))
def test_serving_step_in_two_graphs(gpu_lib, fmt):
    """Two captured steps with buffers of their own, replayed in turn and
    against other eager work: every replay is the eager step."""
    import torch
    T, graphs, steps = 9, [], []
    for i in range(2):
        p = Serving(gpu_lib, SERVE[fmt], T)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            p.step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.step()
        graphs.append(g)
        steps.append(p)
    eager = Serving(gpu_lib, SERVE[fmt], T)
    other = torch.randn(256, 256, device="cuda")
    for rep in range(3):
        for i, (g, p) in enumerate(zip(graphs, steps)):
            x = _bf16(100 + 10 * rep + i, T, p.w.hidden)
            p.x.copy_(x)
            eager.x.copy_(x)
            p.out.zero_()
            g.replay()
            eager.step()
            torch.cuda.synchronize()
            other = torch.tanh(other @ other.T / 256.0)
            for name in ("s", "y", "ids", "tw", "out"):
                assert torch.equal(getattr(p, name), getattr(eager, name)), (rep, i, name)


def test_two_streams_at_once(gpu_lib):
    """Steps on two streams, each with its own buffers, share nothing."""
    import torch
    steps = [Serving(gpu_lib, SERVE["nvfp4"], T) for T in (7, 12)]
    want = []
    for p in steps:
        p.step()
        torch.cuda.synchronize()
        want.append(p.out.clone())
        p.out.zero_()
    streams = [torch.cuda.Stream() for _ in steps]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for p, s in zip(steps, streams):
            with torch.cuda.stream(s):
                p.step()
    torch.cuda.synchronize()
    for p, w in zip(steps, want):
        assert torch.equal(p.out, w)


# -- training -------------------------------------------------------------------

class Training:
    """One block: s = x + res, normed; routed to dense experts out_e = h V_e^T,
    h = relu(row U_e^T) in torch, and back; the loss is <out, d_out> + <s, d_s> +
    the balance loss."""

    def __init__(self, bse, T=37, H=96, n=64, E=6, k=3, local=None):
        import torch
        new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        g = torch.Generator().manual_seed(3)
        rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        self.bse, self.T, self.H, self.E, self.k = bse, T, H, E, k
        self.local = E if local is None else local
        self.cfg = bse.Config(hidden=128, ffn=128, num_experts=E, top_k=k, num_local_experts=self.local, fmt="mxfp8", max_tokens=T)
        self.x, self.res, self.gain = rnd(T, H), rnd(T, H), 1.0 + 0.1 * rnd(H)
        self.R, self.U, self.V = rnd(E, H) * H ** -0.5, rnd(E, n, H) * H ** -0.5, rnd(E, H, n) * n ** -0.5
        self.d_out, self.d_s, self.d_loss = rnd(T, H), rnd(T, H), torch.full((1,), 0.7, device="cuda")
        P = T * k
        self.ws, self.nws, self.bws = bse.workspace(self.cfg), bse.norm_workspace(T, H), bse.balance_workspace(self.cfg, T)
        self.s, self.y, self.rstd, self.out = new(T, H), new(T, H), new(T), new(T, H)
        self.offsets, self.pairs, self.pos = (new(m, dtype=torch.int32) for m in (self.local + 1, P, P))
        self.rows, self.o, self.dy, self.d_rows = new(P, H), new(P, H), new(P, H), new(P, H)
        self.dw, self.dn, self.dz = new(T, k), new(T, H), new(T, E)
        self.counts, self.live, self.probs, self.loss = new(1, E, dtype=torch.int32), new(1, dtype=torch.int32), new(1, E), new(1)
        self.d_res, self.d_gain = new(T, H), new(H)

    def route(self):
        """The routing, chosen once and kept: the gradient is that of a fixed choice."""
        import torch
        self.forward_norm()
        z = self.y @ self.R.T
        self.ids = torch.topk(torch.sigmoid(z), self.k, dim=1)[1].int()
        self.bse.dispatch(self.cfg, self.ids, self.offsets, self.pairs, self.pos, self.ws)
        self.bounds = self.offsets.tolist()

    def forward_norm(self):
        self.bse.norm_forward(self.x, self.gain, self.y, residual=self.res, res_out=self.s, rstd=self.rstd, eps=1e-5)

    def step(self):
        import torch
        bse = self.bse
        self.forward_norm()
        self.z = self.y @ self.R.T
        sg = torch.sigmoid(self.z).gather(1, self.ids.long())
        self.tw = sg / sg.sum(1, keepdim=True)
        bse.sort_rows(self.y, self.pos, self.rows)
        hidden = []
        for e in range(self.local):
            at = slice(self.bounds[e], self.bounds[e + 1])
            hidden.append(torch.relu(self.rows[at] @ self.U[e].T))
            self.o[at] = hidden[e] @ self.V[e].T
        bse.combine_rows(self.o, self.pos, self.tw, self.out)
        bse.balance_forward(self.cfg, self.z, self.ids, self.counts, self.live, self.probs, self.loss, self.bws)
        # back
        bse.combine_rows_backward(self.d_out, self.o, self.pos, self.tw, self.dy, self.dw)
        for e in range(self.local):
            at = slice(self.bounds[e], self.bounds[e + 1])
            self.d_rows[at] = ((self.dy[at] @ self.V[e]) * (hidden[e] > 0)) @ self.U[e]
        bse.sort_rows_backward(self.d_rows, self.pos, self.dn)
        bse.balance_backward(self.cfg, self.z, self.ids, self.counts, self.live, self.d_loss, self.dz, d_topk_w=self.dw)
        self.dn += self.dz @ self.R
        bse.norm_backward(self.dn, self.s, self.gain, self.rstd, self.d_res, self.nws, d_res_out=self.d_s, d_weight=self.d_gain)

    def loss64(self, x, gain):
        """The loss in float64 under the step's routing and counts."""
        s = x + _f64(self.res)
        y = S.norm_forward(s, gain, float(np.float32(1e-5)))[0]
        z = y @ _f64(self.R).T
        ids = self.ids.cpu().numpy()
        sg = np.take_along_axis(1 / (1 + np.exp(-z)), ids, 1)
        tw = sg / sg.sum(1, keepdims=True)
        out = np.zeros_like(y)
        for e in range(self.local):
            t, j = np.nonzero(ids == e)
            out[t] += tw[t, j][:, None] * (np.maximum(y[t] @ _f64(self.U[e]).T, 0) @ _f64(self.V[e]).T)
        balance = B.balance_loss(z, ids, _f64(self.d_loss), self.E, self.k, self.counts.cpu().numpy())
        return (out * _f64(self.d_out)).sum() + (s * _f64(self.d_s)).sum() + balance


@pytest.mark.parametrize("local", [None, 4])
def test_training_step_gradient_is_the_difference_quotient(gpu_lib, local):
    """The gradients of x and of the norm's weight along random directions,
    against differences of the float64 loss.  The differences' own error is below
    1e-6 of the slopes' size (step 1e-5, third derivatives of order 10), fp32 sums
    of some hundred terms leave 1e-5."""
    import torch
    p = Training(gpu_lib, local=local)
    p.route()
    p.step()
    torch.cuda.synchronize()
    x, gain, h = _f64(p.x), _f64(p.gain), 1e-5
    g = np.random.default_rng(1)
    for _ in range(4):
        v = g.standard_normal(x.shape)
        slope = (p.loss64(x + h * v, gain) - p.loss64(x - h * v, gain)) / (2 * h)
        size = np.sqrt((_f64(p.d_res) ** 2).sum())
        assert abs((v * _f64(p.d_res)).sum() - slope) <= 1e-4 * size
        v = g.standard_normal(gain.shape)
        slope = (p.loss64(x, gain + h * v) - p.loss64(x, gain - h * v)) / (2 * h)
        assert abs((v * _f64(p.d_gain)).sum() - slope) <= 1e-4 * np.sqrt((_f64(p.d_gain) ** 2).sum())


def test_training_step_in_a_graph(gpu_lib):
    """Captured forward and backward, replayed with new inputs: the eager bits."""
    import torch
    p, eager = Training(gpu_lib), Training(gpu_lib)
    p.route()
    eager.route()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.step()
    for rep in range(3):
        d = torch.randn(p.x.shape, generator=torch.Generator().manual_seed(rep)).cuda()
        p.d_out.copy_(d)
        eager.d_out.copy_(d)
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        for name in ("out", "dw", "dn", "d_res", "d_gain"):
            assert torch.equal(getattr(p, name), getattr(eager, name)), (rep, name)


def test_tensors_of_another_device_are_refused(gpu_lib, monkeypatch):
    """Every call launches on the current device: tensors of another one are an
    error before anything is enqueued."""
    import torch
    bse = gpu_lib
    x, o, w = torch.zeros((2, 32), device="cuda"), torch.ones((2, 32), device="cuda"), torch.ones(32, device="cuda")
    pos, tw, r = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones((2, 1), device="cuda"), torch.ones(2, device="cuda")
    codes, sc = (torch.zeros((1, 4, n), dtype=torch.uint8, device="cuda") for n in (16, 1))
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    cfg = bse.Config(fmt="mxfp4", hidden=32, num_experts=1, top_k=1)
    bf = torch.zeros((2, 32), dtype=torch.bfloat16, device="cuda")
    stream, device = bse._accessors()
    monkeypatch.setattr(bse, "_accessors", lambda: (stream, lambda: device() + 1))
    for call in (lambda: bse.norm_forward(x, w, o), lambda: bse.norm_backward(x, x, w, r, o),
                 lambda: bse.sort_rows(x, pos, o), lambda: bse.sort_rows_backward(x, pos, o),
                 lambda: bse.combine_rows(x, pos, tw, o), lambda: bse.combine_rows_backward(x, x, pos, tw, o),
                 lambda: bse.group_matvec("mxfp4", x, codes, sc, off, o[:, :4].contiguous()),
                 lambda: bse.forward_quantized(cfg, codes[0, :2], sc[0, :2], pos, tw, bse.CWeights(), bf, codes.view(-1))):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert (o == 1).all()
