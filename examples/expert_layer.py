"""One expert-parallel transformer block's boundary, forward and backward, with the operators of libar, as a training
step would call them:

    partial products of N ranks -> all-reduce + residual + norm (8-bit checkpoint of the residual for the backward)
    -> router -> tokens sorted by expert -> rows dispatched -> one matrix product per expert -> rows combined onto the
    residual;   and all of it backwards.

The ranks are separate buffers on one GPU; expert e lives on rank e % ranks, so the gradient of the normed rows is a
partial one on every rank, which the norm's gradient sums. ExpertBlock's experts are one weight matrix each, whose products
are plain torch; GatedExpertBlock's are gated feed-forward blocks in libar's own products, with their gradients scaled down
to a norm. The router and the loss are plain torch. `python examples/expert_layer.py` runs a few steps of either and prints
the loss.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_reduce_reduction_ring_amd as ar  # noqa: E402

EPS = 1e-5


class ExpertBlock:
    """The buffers that a program keeps for one layer, and its two passes."""

    def __init__(self, ranks, tokens, hidden, experts, k, align=16, dtype=torch.bfloat16, device="cuda:0"):
        new = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device=device)
        i32, f32, nb = torch.int32, torch.float32, -(-hidden // ar.AR_FP8_BLOCK)
        self.ranks, self.align, self.experts = ranks, align, experts
        rows = ar.ar_expert_rows(tokens, k, experts, align)
        # forward
        self.normed, self.residual = [new(tokens, hidden) for _ in range(ranks)], new(tokens, hidden)
        self.rstd, self.saved, self.saved_scales = new(tokens, dt=f32), new(tokens, hidden, dt=torch.uint8), new(tokens, nb, dt=f32)
        self.offsets, self.counts = new(experts + 1, dt=i32), new(experts, dt=i32)
        self.pos, self.src = new(tokens, k, dt=i32), new(rows, dt=i32)
        # rows behind the last segment are never written and go through no product
        self.xs, self.ys = (torch.zeros(rows, hidden, dtype=dtype, device=device) for _ in range(2))
        self.out = new(tokens, hidden)
        self.sort_ws = new(max(1, ar.ar_expert_sort_workspace_size(tokens, k, experts)), dt=torch.uint8)
        # backward
        self.dys, self.dxs = torch.zeros_like(self.xs), torch.zeros_like(self.xs)
        self.dweights, self.dnormed = new(tokens, k, dt=f32), [new(tokens, hidden) for _ in range(ranks)]
        self.dparts, self.dgamma = [new(tokens, hidden) for _ in range(ranks)], new(hidden, dt=f32)
        self.norm_ws = new(ar.ar_allreduce_rmsnorm_bwd_workspace_size(tokens, hidden), dt=torch.uint8)

    def _segments(self):
        off = self.offsets.tolist()  # the experts' products are plain torch here, so the host has to know their rows
        return [(e, slice(off[e], off[e + 1])) for e in range(self.experts) if off[e + 1] > off[e]]

    def _to_experts(self, parts, residual, gamma, ids):
        """All-reduce, residual and norm, and the rows in the experts' order."""
        ar.ar_allreduce_rmsnorm(parts, gamma, self.normed, residual=residual, residual_out=self.residual, rstd=self.rstd,
                                saved=self.saved, saved_scales=self.saved_scales, eps=EPS)
        ar.ar_expert_sort(ids, self.offsets, self.counts, self.pos, self.src, align=self.align, workspace=self.sort_ws)
        self.pos_on = [torch.where(ids % self.ranks == r, self.pos, -1) for r in range(self.ranks)]
        ar.ar_expert_dispatch(self.normed[0], self.pos, self.offsets, self.counts, self.xs)

    def _from_experts(self, dout, gamma):
        """The gradient of _to_experts, from the experts' rows' gradients."""
        for r in range(self.ranks):  # dispatch's gradient: combine without weights, of the rank's own experts
            ar.ar_expert_combine(self.dxs, self.pos_on[r], self.dnormed[r])
        ar.ar_allreduce_rmsnorm_bwd(self.dnormed, self.saved, gamma, self.rstd, self.dparts, self.dgamma,
                                    saved_scales=self.saved_scales, residual_grad=dout, workspace=self.norm_ws)

    def forward(self, parts, residual, gamma, experts_w, ids, weights):
        """parts: the ranks' partial products [tokens, hidden]; ids, weights: the router's choices. The block's output
        (the new residual stream)."""
        self._to_experts(parts, residual, gamma, ids)
        for e, rows in self._segments():
            torch.mm(self.xs[rows], experts_w[e], out=self.ys[rows])
        ar.ar_expert_combine(self.ys, self.pos, self.out, weights=weights, addend=self.residual)
        return self.out

    def backward(self, dout, gamma, experts_w, weights):
        """The gradients of the ranks' partial products (and of the residual), gamma, the experts' weights and the
        router's weights. The norm's gradient starts from the 8-bit checkpoint of the residual."""
        ar.ar_expert_combine_bwd(dout, self.ys, self.pos, weights, self.offsets, self.counts, self.dys, self.dweights)
        dw = torch.zeros_like(experts_w)
        for e, rows in self._segments():
            torch.mm(self.xs[rows].t().contiguous(), self.dys[rows], out=dw[e])
            torch.mm(self.dys[rows], experts_w[e].t().contiguous(), out=self.dxs[rows])
        self._from_experts(dout, gamma)
        return self.dparts[0], self.dgamma, dw, self.dweights


class GatedExpertBlock(ExpertBlock):
    """The same with gated feed-forward experts, out_e(x) = (act(x Wg_e^T) * (x Wu_e^T)) Wd_e^T. The host knows nothing of
    the segments and waits for nothing, so forward and backward can be captured in graphs."""

    def __init__(self, ranks, tokens, hidden, inner, experts, k, align=16, dtype=torch.bfloat16, device="cuda:0", act=ar.AR_ACT_SILU):
        super().__init__(ranks, tokens, hidden, experts, k, align, dtype, device)
        self.act = act
        self.h, self.gate, self.up, self.dh, self.dgate, self.dup = (
            torch.zeros(self.xs.shape[0], inner, dtype=dtype, device=device) for _ in range(6))
        # gate and up projections are one tensor, [experts, 2 inner, hidden], and so are their gradients
        self.dw_in = torch.zeros(experts, 2 * inner, hidden, dtype=dtype, device=device)
        self.dw_out = torch.zeros(experts, hidden, inner, dtype=dtype, device=device)
        self.plan = ar.ar_grad_plan([self.dw_in, self.dw_out, self.dgamma])
        self.norm = torch.zeros(1, device=device)
        self.clip_ws = torch.zeros(ar.ar_grad_norm_workspace_size(self.plan.shape[0]), dtype=torch.uint8, device=device)

    def forward(self, parts, residual, gamma, w_in, w_out, ids, weights):
        self._to_experts(parts, residual, gamma, ids)
        inner, seg = self.h.shape[1], {"offsets": self.offsets, "counts": self.counts}
        ar.ar_expert_gated(self.xs, w_in[:, :inner], w_in[:, inner:], self.h, gate=self.gate, up=self.up, act=self.act, **seg)
        ar.ar_expert_linear(self.h, w_out, self.ys, **seg)
        ar.ar_expert_combine(self.ys, self.pos, self.out, weights=weights, addend=self.residual)
        return self.out

    def backward(self, dout, gamma, w_in, w_out, weights):
        """The gradients of the ranks' partial products, gamma, both weights and the router's weights."""
        inner, seg = self.h.shape[1], {"offsets": self.offsets, "counts": self.counts}
        ar.ar_expert_combine_bwd(dout, self.ys, self.pos, weights, self.offsets, self.counts, self.dys, self.dweights)
        ar.ar_expert_linear_bwd(self.dys, self.h, w_out, dxs=self.dh, dw=self.dw_out, **seg)
        ar.ar_expert_gated_bwd(self.dh, self.gate, self.up, self.xs, w_in[:, :inner], w_in[:, inner:], self.dgate, self.dup,
                               dxs=self.dxs, dw_gate=self.dw_in[:, :inner], dw_up=self.dw_in[:, inner:], act=self.act, **seg)
        self._from_experts(dout, gamma)
        return self.dparts[0], self.dgamma, self.dw_in, self.dw_out, self.dweights

    def clip(self, max_norm):
        """The weights' gradients scaled down to a norm of max_norm, in place; their norm before."""
        ar.ar_grad_clip(self.plan, max_norm, self.norm, workspace=self.clip_ws)
        return self.norm


def route(x, router, k):
    """The k experts that a linear router prefers for every token, and their softmax weights."""
    top, ids = (x.float() @ router).topk(k, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()


def main(steps=4, ranks=4, tokens=512, hidden=1024, experts=16, k=2):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda:0")
    block = ExpertBlock(ranks, tokens, hidden, experts, k)
    parts = [randn(tokens, hidden).bfloat16() for _ in range(ranks)]
    residual, target = randn(tokens, hidden).bfloat16(), randn(tokens, hidden)
    gamma, w = torch.ones(hidden, device="cuda:0"), (randn(experts, hidden, hidden) / hidden ** 0.5).bfloat16()
    ids, weights = route(residual, randn(hidden, experts), k)
    losses = []
    for step in range(steps):
        out = block.forward(parts, residual, gamma, w, ids, weights)
        diff = out.float() - target
        losses.append(diff.square().mean().item())
        dout = (diff * (2 * 4096 / diff.numel())).bfloat16()  # scaled up, as mixed-precision training does
        _, dgamma, dw, _ = block.backward(dout, gamma, w, weights)
        # steps of a fixed length, so the scale does not matter
        gamma -= 0.02 * gamma.norm() * dgamma / dgamma.norm()
        w -= (0.05 * w.float().norm() * dw.float() / dw.float().norm()).bfloat16()
        print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    return losses


def main_gated(steps=4, ranks=4, tokens=512, hidden=1024, inner=512, experts=16, k=2):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda:0")
    block = GatedExpertBlock(ranks, tokens, hidden, inner, experts, k)
    parts = [randn(tokens, hidden).bfloat16() for _ in range(ranks)]
    residual, target = randn(tokens, hidden).bfloat16(), randn(tokens, hidden)
    gamma, w_in = torch.ones(hidden, device="cuda:0"), (randn(experts, 2 * inner, hidden) / hidden ** 0.5).bfloat16()
    w_out = (randn(experts, hidden, inner) / inner ** 0.5).bfloat16()
    ids, weights = route(residual, randn(hidden, experts), k)
    losses = []
    for step in range(steps):
        out = block.forward(parts, residual, gamma, w_in, w_out, ids, weights)
        diff = out.float() - target
        losses.append(diff.square().mean().item())
        dout = (diff * (2 * 4096 / diff.numel())).bfloat16()
        _, dgamma, dw_in, dw_out, _ = block.backward(dout, gamma, w_in, w_out, weights)
        norm = block.clip(1.0).item()
        gamma -= 2.0 * dgamma
        w_in -= 2.0 * dw_in
        w_out -= 2.0 * dw_out
        print(f"gated, step {step}: loss {losses[-1]:.4f}, gradients' norm {norm:.3f}", flush=True)
    return losses


if __name__ == "__main__":
    main()
    main_gated()
