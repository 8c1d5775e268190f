"""One decoder layer's MoE half: residual addition + RMSNorm, router, experts.

    s = x + residual,  y = rmsnorm(s) w,  logits = y Wr^T,
    (ids, p) = top-k of the logits,  out = experts(y, ids, p)

``forward`` / ``backward`` are the training (or prefill) step over the grouped
expert layer, ``decode`` the step of a few tokens over the same weights. The
router's projection and its two gradients are plain library products; every
other step is a libmgq call. ``out`` and ``s`` leave as the next layer's x and
residual.
"""
from __future__ import annotations

import torch

from . import mgq
from .layer import ExpertLayer
from .workloads import Workload


class MoEBlock:
    def __init__(self, w: Workload, device, recipe: str | None = None, eps: float = 1e-5,
                 score: int = mgq.SCORE_SOFTMAX, renorm: bool = True, route_scale: float = 1.0, **layer_kw):
        self.w, self.eps = w, eps
        self.route = dict(score=score, renorm=renorm, scale=route_scale)
        self.experts = ExpertLayer(w, device, recipe, **layer_kw)
        d = self.dev = self.experts.dev
        T, H, E = w.T, w.H, w.E
        self.norm_w = torch.ones(H, dtype=torch.bfloat16, device=d)
        self.router_w = torch.zeros(E, H, dtype=torch.float32, device=d)
        # forward state that the backward reads
        self.s = torch.empty(T, H, dtype=torch.bfloat16, device=d)
        self.y = torch.empty(T, H, dtype=torch.bfloat16, device=d)
        self.rstd = torch.empty(T, device=d)
        self.logits = torch.empty(T, E, device=d)
        self.topk_idx = torch.empty(T, w.k, dtype=torch.int32, device=d)
        self.probs = torch.empty(T, w.k, device=d)
        if self.experts.train:
            self.dlogits = torch.empty(T, E, device=d)
            self.dx = torch.empty(T, H, dtype=torch.bfloat16, device=d)
            self.dnorm_w = torch.empty(H, device=d)
            self.ws = torch.empty(max(16, mgq.add_rmsnorm_bwd_workspace_size(T, H)), dtype=torch.uint8, device=d)

    def load(self, w1, w2, norm_w, router_w):
        """bf16 expert weights [E, 2F, H] and [E, H, F] (quantised here), norm weight
        [H] bf16, router weight [E, H] float32."""
        self.experts.quantize_weights(w1, w2)
        self.norm_w.copy_(norm_w)
        self.router_w.copy_(router_w)

    def forward(self, x, residual=None):
        """(out, s) of the workload's T tokens (x, residual bf16 [T, H])."""
        mgq.add_rmsnorm_quantize(x, self.norm_w, self.eps, residual=residual, sum_out=self.s, y=self.y, rstd=self.rstd)
        torch.matmul(self.y.float(), self.router_w.t(), out=self.logits)
        mgq.router_topk(self.logits, self.topk_idx, self.probs, **self.route)
        return self.experts.forward(self.y, self.topk_idx, self.probs), self.s

    def backward(self, dout, dsum=None):
        """dx (also the residual's gradient) of the last forward, from the gradients of
        out and of s. Weight gradients: experts.dw1 / dw2, drouter_w, dnorm_w."""
        dy = self.experts.backward(dout, self.probs)
        mgq.router_topk_bwd(self.logits, self.topk_idx, self.experts.dprobs, self.dlogits, **self.route)
        self.drouter_w = torch.matmul(self.dlogits.t(), self.y.float())
        dy = torch.addmm(dy.float(), self.dlogits, self.router_w).to(torch.bfloat16)
        mgq.add_rmsnorm_bwd(dy, self.s, self.norm_w, self.rstd, self.dx, self.dnorm_w, self.ws, dsum=dsum)
        return self.dx

    def decode(self, x, residual=None):
        """(out, s) of 1 to 128 new tokens."""
        T = x.shape[0]
        s, y = torch.empty_like(x), torch.empty_like(x)
        idx = torch.empty(T, self.w.k, dtype=torch.int32, device=self.dev)
        probs = torch.empty(T, self.w.k, device=self.dev)
        mgq.add_rmsnorm_quantize(x, self.norm_w, self.eps, residual=residual, sum_out=s, y=y)
        mgq.router_topk(torch.matmul(y.float(), self.router_w.t()), idx, probs, **self.route)
        self.few = (y, idx, probs)           # of the last decode step
        return self.experts.forward_few(y, idx, probs), s
