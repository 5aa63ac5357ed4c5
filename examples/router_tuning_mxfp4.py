"""Tunes a router over frozen MXFP4 experts on one GPU.

The experts are encoded to MXFP4 once.  Each step routes a batch of packed
sequences, runs the experts through the grouped product, and moves the router
towards a target output and an even load: the gate weights' gradient and the
balance loss's go through balance_backward into the logits, and from there
into the router's weights.

    python examples/router_tuning_mxfp4.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_expert_amd as bse  # noqa: E402


class Experts:
    """Frozen expert weights, gate and up rows of an expert one after the other."""

    def __init__(self, cfg, w13, w2):
        self.w13, self.w13_sc = self.encode(w13)
        self.w2, self.w2_sc = self.encode(w2)

    @staticmethod
    def encode(w):
        n, rows, cols = w.shape
        codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device=w.device)
        bse.encode_weights("mxfp4", w, codes, scales)
        return codes, scales

    def as_weights(self):
        return {"w13": self.w13, "w13_sc": self.w13_sc, "w2": self.w2, "w2_sc": self.w2_sc}


class Layer:
    """The layer's steps with the intermediate values a router's gradient needs."""

    def __init__(self, cfg, experts, T, bounds, device="cuda"):
        def new(shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        H, F, E, k, S = cfg.hidden, cfg.ffn, cfg.num_experts, cfg.top_k, bounds.numel() - 1
        P = T * k
        self.cfg, self.experts, self.T, self.bounds = cfg, experts, T, bounds
        self.ws, self.balance_ws = bse.workspace(cfg), bse.balance_workspace(cfg, T, S)
        self.bias = torch.zeros(E, device=device)
        self.ids, self.topk_w, self.z = new((T, k), torch.int32), new((T, k)), new((T, E))
        self.offsets, self.pairs, self.pos = new(E + 1, torch.int32), new(P, torch.int32), new(P, torch.int32)
        self.xq, self.xs = new((T, H // 2), torch.uint8), new((T, H // 32), torch.uint8)
        self.hq, self.hs = new((P, F // 2), torch.uint8), new((P, F // 32), torch.uint8)
        self.gu, self.h, self.y = new((P, 2 * F)), new((P, F)), new((P, H))
        self.counts, self.live = new((S, E), torch.int32), new(S, torch.int32)
        self.probs, self.balance, self.dz = new((S, E)), new(S), new((T, E))

    def forward(self, x, w_router):
        """The layer's output [T, hidden] in fp32."""
        cfg, e = self.cfg, self.experts
        bse.route(cfg, x, w_router, self.bias, self.ids, self.topk_w, None, self.ws)
        bse.route_logits(cfg, self.T, self.z, self.ws)
        bse.dispatch(cfg, self.ids, self.offsets, self.pairs, self.pos, self.ws)
        bse.quantize_act(cfg, x, self.xq, self.xs)
        bse.group_product("mxfp4", self.xq, self.xs, e.w13, e.w13_sc, self.offsets, self.gu, row_ids=self.pairs,
                          id_div=cfg.top_k)
        gate, up = self.gu.split(cfg.ffn, dim=1)
        bse.cap_swiglu(cfg, gate.contiguous().view(-1), up.contiguous().view(-1), self.h.view(-1))
        bse.quantize_act(cfg, self.h, self.hq, self.hs, site=1)
        bse.group_product("mxfp4", self.hq, self.hs, e.w2, e.w2_sc, self.offsets, self.y)
        self.expert_out = self.y[self.pos.long()].view(self.T, cfg.top_k, cfg.hidden)
        bse.balance_forward(cfg, self.z, self.ids, self.counts, self.live, self.probs, self.balance, self.balance_ws,
                            seq_offsets=self.bounds)
        return (self.topk_w[:, :, None] * self.expert_out).sum(1)

    def backward(self, x, d_out, balance_weight):
        """The gradient of the router's weights [experts, hidden]."""
        d_topk_w = (self.expert_out * d_out[:, None, :]).sum(2)
        d_balance = torch.full_like(self.balance, balance_weight / self.balance.numel())
        bse.balance_backward(self.cfg, self.z, self.ids, self.counts, self.live, d_balance, self.dz,
                             d_topk_w=d_topk_w, seq_offsets=self.bounds)
        return self.dz.t().contiguous() @ x.float()


def run(steps=40, T=512, hidden=256, ffn=128, experts=16, top_k=2, lr=0.02, balance_weight=0.1, seed=0, log=None):
    """[(task loss, mean balance loss)] per step.  The target is the output of
    the same experts under another router; the tuned one starts skewed towards
    a few experts."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).cuda()

    cfg = bse.Config(hidden=hidden, ffn=ffn, num_experts=experts, top_k=top_k, fmt="mxfp4", max_tokens=T)
    frozen = Experts(cfg, normal(experts, 2 * ffn, hidden) * hidden ** -0.5, normal(experts, hidden, ffn) * ffn ** -0.5)
    bounds = torch.tensor([0, T // 8, T // 2, T], dtype=torch.int32, device="cuda")
    layer = Layer(cfg, frozen, T, bounds)

    x = normal(T, hidden)
    x[:, 0] = 1.0
    x = x.bfloat16()
    teacher = normal(experts, hidden) * hidden ** -0.5
    target = layer.forward(x, teacher.bfloat16()).clone()
    student = teacher + normal(experts, hidden) * 0.25 * hidden ** -0.5
    student[: experts // 4, 0] += 1.0                      # the constant feature: favours the first experts
    m, v = torch.zeros_like(student), torch.zeros_like(student)
    scale = target.pow(2).mean()

    history = []
    for step in range(1, steps + 1):
        diff = layer.forward(x, student.bfloat16()) - target
        grad = layer.backward(x, 2.0 * diff / (diff.numel() * scale), balance_weight)
        history.append((float(diff.pow(2).mean() / scale), float(layer.balance.mean())))
        if log:
            log(f"step {step:3d}  task {history[-1][0]:.4f}  balance {history[-1][1]:.4f}")
        m.lerp_(grad, 0.1)
        v.lerp_(grad * grad, 0.01)
        student -= lr * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    run(ap.parse_args().steps, log=lambda s: print(s, flush=True))
