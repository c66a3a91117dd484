"""A mixture-of-experts layer around the balanced router: the path that runs
routing, the exchange and the experts' 8-bit products together.

Each token's K experts are the largest biased scores of its router, its
output is the gate-weighted sum of what its experts' matrices make of it:

    s = sigmoid(h wr^T);  e_k, g_k = the K largest of s + b, s[e_k] / sum s[e_k]
    out = sum_k g_k (h w[e_k]^T)

``step`` of the bias (``update_bias``) is the exact quantile update of the
live tokens' own scores; ``backward`` gives the gradients of sum(out * dout) +
dloss * loss, with the loss of sequence-wise balance.  Every step below is a
libqb call; this module only owns buffers and orders the calls.
"""
from __future__ import annotations

import torch
from torch.autograd.graph import increment_version

from . import qb


class ExpertLayer:
    """Router weight wr bf16 [E, H] (E of 32 to 256, as qb_router_scores takes), expert matrices w float [E, M, H] (held in
    8 bits, in both orders), bias b float [E]; buffers for N tokens a call.  The experts' products hold their sums in 32
    bits; exact=False lets them use the faster instruction that drops some (see qb_fp8_product).

    Results are the layer's own buffers, which its next call writes again.  One forward at a time is followed by its
    backward, which reads that forward's h, seq_off and valid again: they are not copied, and one that torch or a layer
    has written since is an error."""

    def __init__(self, wr: torch.Tensor, w: torch.Tensor, K: int, N: int, coef: float = 0.0, B: int = 1,
                 exact: bool = True):
        E, M, H = w.shape
        self.wr, self.K, self.N, self.coef, self.exact = wr, K, N, coef, exact
        kw = dict(device=w.device)

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, **kw)

        def eighth(lead, rows, cols, scale_rows=None):
            return (new(lead + (rows, qb.fp8_ld(cols)), qb.F8),
                    new(lead + (rows if scale_rows is None else scale_rows, qb.fp8_sld(cols)), torch.uint8))

        blocks = lambda n: -(-n // qb.FP8_BLOCK)  # noqa: E731
        self.wq, self.ws = eighth((E,), M, H, blocks(M))
        self.wt, self.wts = eighth((E,), H, M, blocks(H))
        self.load_weights(w)
        self.b = torch.zeros(E, dtype=torch.float32, **kw)
        # an expert's rows begin at a multiple of 128, so that no block of the gradient's sums spans two
        R = qb.qb_dispatch_rows(N, K, E, qb.FP8_BLOCK)
        self.s = new((N, E), torch.float32)
        self.topk, self.pos = new((N, K), torch.int32), new((N, K), torch.int32)
        self.gate, self.dgate = new((N, K), torch.float32), new((N, K), torch.float32)
        self.count, self.weight = new((B, E), torch.int32), new((B, E), torch.float32)
        self.loss = new((1,), torch.float32)
        self.balance_ws = new((qb.qb_balance_workspace_bytes(N, E, B),), torch.uint8)
        self.dispatch_ws = new((qb.qb_dispatch_workspace_bytes(N, K, E),), torch.uint8)
        self.off, self.row_src = new((E + 1,), torch.int32), new((R,), torch.int32)
        self.xq, self.xs = eighth((), R, H)
        self.xt, self.xts = eighth((), H, R)
        self.dq, self.ds = eighth((), R, M)
        self.dt, self.dts = eighth((), M, R)
        self.rows, self.drows = new((R, M), torch.bfloat16), new((R, M), torch.bfloat16)
        self.dx_rows = new((R, H), torch.bfloat16)
        self.out, self.dx = new((N, M), torch.bfloat16), new((N, H), torch.bfloat16)
        self.dw, self.dlogits = new((E, M, H), torch.float32), new((N, E), torch.float32)
        self.alpha = new((N,), torch.float32)
        self.h, self.seqs, self.versions = None, {}, {}
        self.eqb = qb.EqbBuffers(1, E, device=w.device, lead=False)

    def load_weights(self, w: torch.Tensor, stream=None):
        """Lay the experts' matrices out again, as after an optimizer step."""
        qb.qb_fp8_quantize_weight(w, self.wq, self.ws, self.wt, self.wts, stream=stream)

    def forward(self, h: torch.Tensor, seq_off=None, valid=None, stream=None) -> torch.Tensor:
        """out bf16 [N, M] of hidden states h bf16 [N, H]; `loss` and `count`
        afterwards hold the balance loss and the per-expert counts of the
        sequences.  Padding (valid 0) goes to no expert, and its out is 0."""
        self.h, seqs = None, dict(seq_off=seq_off, valid=valid)
        qb.qb_router_scores(h, self.wr, self.s, stream=stream)
        qb.qb_balance_forward(self.s, self.b, self.K, self.topk, gate=self.gate, count=self.count, weight=self.weight,
                              loss=self.loss, ws=self.balance_ws, coef=self.coef, **seqs, stream=stream)
        qb.qb_dispatch(self.topk, self.b.numel(), qb.FP8_BLOCK, self.off, self.row_src, self.pos, self.dispatch_ws,
                       stream=stream)
        qb.qb_fp8_quantize(h, self.xq, self.xs, row_src=self.row_src, stream=stream)
        qb.qb_fp8_product(self.xq, self.xs, self.wq, self.ws, self.rows, off=self.off, exact=self.exact, stream=stream)
        qb.qb_combine(self.rows, self.pos, self.out, gate=self.gate, stream=stream)
        increment_version(self.out)
        self.h, self.seqs = h, seqs
        self.versions = {n: t._version for n, t in dict(h=h, **seqs).items() if t is not None and not t.is_inference()}
        return self.out

    def _forward_done(self):
        if self.h is None:
            raise RuntimeError("there was no forward")

    def backward(self, dout: torch.Tensor, dloss=None, stream=None):
        """Gradients of the last forward: dx bf16 [N, H] through the experts, dw
        float [E, M, H] and dlogits float [N, E] of the router's logits (whose
        own product with wr is the caller's)."""
        self._forward_done()
        for name, version in self.versions.items():
            if dict(h=self.h, **self.seqs)[name]._version != version:
                raise RuntimeError(f"{name} was written after the forward, and backward reads it again")
        qb.qb_combine_backward(dout, self.rows, self.pos, self.row_src, self.drows, gate=self.gate, dgate=self.dgate,
                               stream=stream)
        qb.qb_fp8_quantize(self.drows, self.dq, self.ds, stream=stream)
        qb.qb_fp8_product(self.dq, self.ds, self.wt, self.wts, self.dx_rows, off=self.off, exact=self.exact,
                          stream=stream)
        qb.qb_combine(self.dx_rows, self.pos, self.dx, stream=stream)
        qb.qb_fp8_quantize_cols(self.h, self.xt, self.xts, row_src=self.row_src, stream=stream)
        qb.qb_fp8_quantize_cols(self.drows, self.dt, self.dts, stream=stream)
        qb.qb_fp8_weight_grad(self.dt, self.dts, self.xt, self.xts, self.dw, off=self.off, stream=stream)
        qb.qb_balance_backward(self.s, self.topk, weight=self.weight, dloss=dloss, dgate=self.dgate,
                               dlogits=self.dlogits, **self.seqs, stream=stream)
        increment_version((self.dx, self.dw, self.dlogits))
        return self.dx, self.dw, self.dlogits

    def update_bias(self, stream=None):
        """The exact quantile update of b from the scores of the last forward's
        live tokens (with seq_off or valid, the others' rows of s are cleared)."""
        self._forward_done()
        masked = any(t is not None for t in self.seqs.values())
        self.eqb.reset(stream)
        qb.eqb_update(self.s, self.b, self.K, self.alpha, self.eqb, stream=stream, topk=self.topk if masked else None)
