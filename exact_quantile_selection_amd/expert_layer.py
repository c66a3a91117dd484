"""A mixture-of-experts layer around the balanced router: the path that runs
routing, the exchange and the experts' products together.

Each token's K experts are the largest biased scores of its router, its
output is the gate-weighted sum of what its experts' matrices make of it:

    s = sigmoid(h wr^T);  e_k, g_k = the K largest of s + b, s[e_k] / sum s[e_k]
    out = sum_k g_k (h w[e_k]^T)

``step`` of the bias (``update_bias``) is the exact quantile update of the
live tokens' own scores; ``backward`` gives the gradients of sum(out * dout) +
dloss * loss, with the loss of sequence-wise balance; ``orthogonalized`` turns a
gradient or momentum of the experts' matrices into their update.  Every step
below is a libqb call; this module only owns buffers and orders the calls.
"""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.graph import increment_version

from . import qb


def _on(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class ExpertLayer:
    """Router weight wr bf16 [E, H] (E of 32 to 256, as qb_router_scores takes), expert matrices w float [E, M, H], bias b
    float [E]; buffers for N tokens a call.  `held` says how the matrices are held and their products computed:

    * "e4m3": 8 bits, in both orders.  The products hold their sums in 32 bits; exact=False lets them use the faster
      instruction that drops some (see qb_fp8_product).
    * "bf16": one copy in bfloat16, which the gradient of the rows reads across.
    * "e2m1": 4 bits with a scale for each 32, in both orders, for the products with the matrices; their gradient is
      computed from the rows in bfloat16.

    Results are the layer's own buffers, which its next call writes again.  One forward at a time is followed by its
    backward, which reads that forward's h, seq_off and valid again, and the matrices: they are not copied, and one that
    torch or a layer has written since is an error."""

    def __init__(self, wr: torch.Tensor, w: torch.Tensor, K: int, N: int, coef: float = 0.0, B: int = 1,
                 exact: bool = True, held: str = "e4m3"):
        if held not in ("e4m3", "bf16", "e2m1"):
            raise ValueError(f"held={held!r}, expected 'e4m3', 'bf16' or 'e2m1'")
        if held != "e4m3" and not exact:
            raise ValueError("exact=False is a choice of the 8-bit products alone")
        E, M, H = w.shape
        self.wr, self.K, self.N, self.coef, self.exact, self.held = wr, K, N, coef, exact, held
        kw = dict(device=w.device)

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, **kw)

        def eighth(lead, rows, cols, scale_rows=None):
            return (new(lead + (rows, qb.fp8_ld(cols)), qb.F8),
                    new(lead + (rows if scale_rows is None else scale_rows, qb.fp8_sld(cols)), torch.uint8))

        def fourth(lead, rows, cols):
            return new(lead + (rows, qb.fp4_ld(cols)), torch.uint8), new(lead + (rows, qb.fp4_sld(cols)), torch.uint8)

        blocks = lambda n: -(-n // qb.FP8_BLOCK)  # noqa: E731
        if held == "e4m3":
            self.wq, self.ws = eighth((E,), M, H, blocks(M))
            self.wt, self.wts = eighth((E,), H, M, blocks(H))
        elif held == "e2m1":
            self.wq, self.ws = fourth((E,), M, H)
            self.wt, self.wts = fourth((E,), H, M)
        else:
            self.w = new((E, M, H), torch.bfloat16)
        self.load_weights(w)
        self.b = torch.zeros(E, dtype=torch.float32, **kw)
        # in 8 bits an expert's rows begin at a multiple of 128, so that no block of the gradient's sums spans two
        self.align = qb.FP8_BLOCK if held == "e4m3" else 1
        R = qb.qb_dispatch_rows(N, K, E, self.align)
        self.s = new((N, E), torch.float32)
        self.topk, self.pos = new((N, K), torch.int32), new((N, K), torch.int32)
        self.gate, self.dgate = new((N, K), torch.float32), new((N, K), torch.float32)
        self.count, self.weight = new((B, E), torch.int32), new((B, E), torch.float32)
        self.loss = new((1,), torch.float32)
        self.balance_ws = new((qb.qb_balance_workspace_bytes(N, E, B),), torch.uint8)
        self.dispatch_ws = new((qb.qb_dispatch_workspace_bytes(N, K, E),), torch.uint8)
        self.off, self.row_src = new((E + 1,), torch.int32), new((R,), torch.int32)
        if held == "e4m3":
            self.xq, self.xs = eighth((), R, H)
            self.xt, self.xts = eighth((), H, R)
            self.dq, self.ds = eighth((), R, M)
            self.dt, self.dts = eighth((), M, R)
        else:
            self.grad_ws = new((qb.qb_bf16_weight_grad_workspace_bytes(R, M, H, E),), torch.uint8)
            if held == "e2m1":
                self.xq, self.xs = fourth((), R, H)
                self.dq, self.ds = fourth((), R, M)
        self.rows, self.drows = new((R, M), torch.bfloat16), new((R, M), torch.bfloat16)
        self.dx_rows = new((R, H), torch.bfloat16)
        self.out, self.dx = new((N, M), torch.bfloat16), new((N, H), torch.bfloat16)
        self.dw, self.dlogits = new((E, M, H), torch.float32), new((N, E), torch.float32)
        self.alpha = new((N,), torch.float32)
        self.h, self.seqs, self.versions = None, {}, {}
        self.has_dw, self.o, self.ortho_ws = False, None, None
        self.eqb = qb.EqbBuffers(1, E, device=w.device, lead=False)

    def load_weights(self, w: torch.Tensor, stream=None):
        """Lay the experts' matrices out again, as after an optimizer step."""
        if self.held == "e4m3":
            qb.qb_fp8_quantize_weight(w, self.wq, self.ws, self.wt, self.wts, stream=stream)
        elif self.held == "e2m1":
            qb.qb_fp4_quantize_weight(w, self.wq, self.ws, self.wt, self.wts, stream=stream)
        else:
            if w.shape != self.w.shape:                # copy_ would broadcast it
                raise ValueError(f"w has shape {tuple(w.shape)}, expected {tuple(self.w.shape)}")
            with _on(stream), torch.no_grad():         # (of a parameter too)
                self.w.copy_(w)
            return
        increment_version((self.wq, self.ws, self.wt, self.wts))

    def forward(self, h: torch.Tensor, seq_off=None, valid=None, stream=None) -> torch.Tensor:
        """out bf16 [N, M] of hidden states h bf16 [N, H]; `loss` and `count`
        afterwards hold the balance loss and the per-expert counts of the
        sequences.  Padding (valid 0) goes to no expert, and its out is 0."""
        self.h, seqs = None, dict(seq_off=seq_off, valid=valid)
        qb.qb_router_scores(h, self.wr, self.s, stream=stream)
        qb.qb_balance_forward(self.s, self.b, self.K, self.topk, gate=self.gate, count=self.count, weight=self.weight,
                              loss=self.loss, ws=self.balance_ws, coef=self.coef, **seqs, stream=stream)
        qb.qb_dispatch(self.topk, self.b.numel(), self.align, self.off, self.row_src, self.pos, self.dispatch_ws,
                       stream=stream)
        if self.held == "e4m3":
            qb.qb_fp8_quantize(h, self.xq, self.xs, row_src=self.row_src, stream=stream)
            qb.qb_fp8_product(self.xq, self.xs, self.wq, self.ws, self.rows, off=self.off, exact=self.exact,
                              stream=stream)
        elif self.held == "e2m1":
            qb.qb_fp4_quantize(h, self.xq, self.xs, row_src=self.row_src, stream=stream)
            qb.qb_fp4_product(self.xq, self.xs, self.wq, self.ws, self.rows, off=self.off, stream=stream)
        else:
            qb.qb_bf16_product(h, self.w, self.rows, off=self.off, row_src=self.row_src, stream=stream)
        qb.qb_combine(self.rows, self.pos, self.out, gate=self.gate, stream=stream)
        increment_version(self.out)
        self.h, self.seqs = h, seqs
        self.versions = {n: t._version for n, t in self._read_again().items() if t is not None and not t.is_inference()}
        return self.out

    def _read_again(self):
        """What backward reads that its forward read."""
        return dict(h=self.h, **self.seqs, w=self.w if self.held == "bf16" else self.wt)

    def _forward_done(self):
        if self.h is None:
            raise RuntimeError("there was no forward")

    def backward(self, dout: torch.Tensor, dloss=None, stream=None):
        """Gradients of the last forward: dx bf16 [N, H] through the experts, dw
        float [E, M, H] and dlogits float [N, E] of the router's logits (whose
        own product with wr is the caller's)."""
        self._forward_done()
        now = self._read_again()
        for name, version in self.versions.items():
            if now[name]._version != version:
                raise RuntimeError(f"{name} was written after the forward, and backward reads it again")
        qb.qb_combine_backward(dout, self.rows, self.pos, self.row_src, self.drows, gate=self.gate, dgate=self.dgate,
                               stream=stream)
        if self.held == "e4m3":
            qb.qb_fp8_quantize(self.drows, self.dq, self.ds, stream=stream)
            qb.qb_fp8_product(self.dq, self.ds, self.wt, self.wts, self.dx_rows, off=self.off, exact=self.exact,
                              stream=stream)
        elif self.held == "e2m1":
            qb.qb_fp4_quantize(self.drows, self.dq, self.ds, stream=stream)
            qb.qb_fp4_product(self.dq, self.ds, self.wt, self.wts, self.dx_rows, off=self.off, stream=stream)
        else:
            qb.qb_bf16_product(self.drows, self.w, self.dx_rows, off=self.off, transposed=True, stream=stream)
        qb.qb_combine(self.dx_rows, self.pos, self.dx, stream=stream)
        if self.held == "e4m3":
            qb.qb_fp8_quantize_cols(self.h, self.xt, self.xts, row_src=self.row_src, stream=stream)
            qb.qb_fp8_quantize_cols(self.drows, self.dt, self.dts, stream=stream)
            qb.qb_fp8_weight_grad(self.dt, self.dts, self.xt, self.xts, self.dw, off=self.off, stream=stream)
        else:
            qb.qb_bf16_weight_grad(self.drows, self.h, self.dw, off=self.off, row_src=self.row_src, ws=self.grad_ws,
                                   stream=stream)
        self.has_dw = True
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

    def orthogonalized(self, update=None, steps: int = 5, poly=(3.4445, -4.7750, 2.0315), stream=None,
                       exact: bool = True) -> torch.Tensor:
        """o bf16 [E, M, H]: each expert's matrix of `update` float [E, M, H] (a momentum, say; the last backward's dw by
        default) orthogonalised as qb_orthogonalize does, whose `exact` is this one.  The first call makes its buffers, on its stream; the next one
        writes o again."""
        if update is None:
            if not self.has_dw:
                raise RuntimeError("there was no backward")
            update = self.dw
        if update.shape != self.dw.shape:
            raise ValueError(f"update has shape {tuple(update.shape)}, expected {tuple(self.dw.shape)}")
        if self.o is None:
            with _on(stream):
                self.o = torch.empty_like(self.dw, dtype=torch.bfloat16)
                self.ortho_ws = torch.empty((qb.qb_orthogonalize_workspace_bytes(*self.dw.shape),), dtype=torch.uint8,
                                            device=self.dw.device)
        qb.qb_orthogonalize(update, self.o, self.ortho_ws, steps=steps, poly=poly, stream=stream, exact=exact)
        increment_version(self.o)
        return self.o
