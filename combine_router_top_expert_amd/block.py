"""A transformer block's MoE half: RMS norm of the residual stream, then the layer.

``RMSNorm`` owns the buffers of ``mok_norm_fwd`` / ``mok_norm_bwd``;
``MoEBlock`` puts one in front of a ``MoELayer`` for training, and in front of
the 4-bit experts (``decode.MoEDecoder``) for serving.  Neither does arithmetic
of its own.  The calls share their buffers: the caller orders calls on
different streams, and replays of captured ones.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import make_config, mok_norm_bwd, mok_norm_bwd_ws_bytes, mok_norm_fwd
from .layer import MoELayer, _dt
from .streams import StreamUser


class RMSNorm(StreamUser):
    """``weight`` [d] in the layer's type (prec "f32": float32, else bfloat16)
    and buffers for up to ``rows`` rows.  res_type: "f32" or "bf16" rows of the
    residual stream (bf16 not with prec "f32").  mx: rows also as MX blocks."""

    def __init__(self, weight: torch.Tensor, rows: int, prec="bf16", res_type="bf16", eps=1e-6, mx=False,
                 with_bwd=True):
        self.device, self.d, self.rows, self.eps = weight.device, weight.numel(), rows, eps
        self.act, self.res_dt = _dt(prec), torch.float32 if res_type == "f32" else torch.bfloat16
        if prec == "f32" and res_type != "f32":
            raise ValueError("an fp32 layer has an fp32 residual stream")
        self._expect("weight", weight, self.act, (self.d,))
        if rows < 0 or self.d % 64 or not self.d:
            raise ValueError(f"rows >= 0 and d a multiple of 64 expected, got {rows} and {self.d}")
        self.weight = weight
        self.cfg = make_config(1, 1, self.d, 1, 1, 64, 1, prec, 0)
        # (not filled: a fill could still be on its way when another stream writes)
        new = lambda dt, *n: torch.empty(*n, dtype=dt, device=self.device)  # noqa: E731
        self.res = new(self.res_dt, rows, self.d)       # the residual stream behind the addition
        self.y = new(self.act, rows, self.d)
        self.rstd = new(torch.float32, rows)
        self.codes = new(torch.uint8, rows, self.d) if mx else None
        self.scales = new(torch.uint8, rows, self.d // 32) if mx else None
        self.T = 0
        self.with_bwd = with_bwd
        if with_bwd:
            self.d_r = new(self.res_dt, rows, self.d)
            # the same gradient in the layer's type, where that is another one
            self.d_x = self.d_r if self.act == self.res_dt else new(self.act, rows, self.d)
            self.dw = torch.zeros(self.d, dtype=torch.float32, device=self.device)
            with torch.cuda.device(self.device):
                self.ws = new(torch.uint8, mok_norm_bwd_ws_bytes(self.cfg, max(rows, 1)))
        self._ready()

    def forward(self, x: Optional[torch.Tensor], res: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x [T, d] (the layer's type) added to res [T, d] (the stream's type);
        one of them may be None.  Returns y [T, d]; res, rstd, codes and scales
        hold the rest in their first T rows.  All are overwritten by the next
        call."""
        T = self._rows_of(x, res)
        with torch.cuda.device(self.device):
            self._enter(stream)
            self._hold(stream, x, res)
            mok_norm_fwd(self.cfg, T, x, res, self.weight, self.eps, self.res, self.y, self.codes, self.scales,
                         self.rstd, stream)
        self.T = T
        return self.y[:T]

    def _rows_of(self, x, res) -> int:
        """How many rows a forward of x and res has; refuses what it could not read."""
        first = x if x is not None else res
        if first is None or first.dim() != 2:
            raise ValueError("rows [T, d] expected")
        T = first.shape[0]
        if T > self.rows:
            raise ValueError(f"{T} rows, and buffers for {self.rows}")
        if x is not None:
            self._expect("x", x, self.act, (T, self.d))
        if res is not None:
            self._expect("res", res, self.res_dt, (T, self.d))
        return T

    def backward(self, dy: torch.Tensor, d_res: Optional[torch.Tensor] = None, accumulate=False, stream=None):
        """The gradient of the last forward's res (and x): dy [T, d] reaches
        y, d_res [T, d] (the stream's type) reaches the residual stream behind
        the addition, or None.  Returns d_r [T, d] in the stream's type; d_x
        holds it in the layer's type and dw the weight's, with accumulate added
        to what dw holds."""
        if not self.with_bwd:
            raise RuntimeError("RMSNorm(with_bwd=False)")
        self._expect("dy", dy, self.act, (self.T, self.d))
        if d_res is not None:
            self._expect("d_res", d_res, self.res_dt, (self.T, self.d))
        with torch.cuda.device(self.device):
            self._enter(stream)
            self._hold(stream, dy, d_res)
            mok_norm_bwd(self.cfg, self.T, dy, self.res, self.weight, self.rstd, d_res, self.d_r,
                         None if self.d_x is self.d_r else self.d_x, self.dw, accumulate, self.ws, stream)
        return self.d_r[:self.T]


class MoEBlock(StreamUser):
    """res <- res + delta, out = layer(norm(res)): the norm of the layer's own
    sources, then the layer; ``decode`` for the rows of a few tokens.  ``out`` is the next block's delta.  Other sources'
    rows are given to the layer by their owners (``layer.xs``)."""

    def __init__(self, layer: MoELayer, weight: torch.Tensor, res_type="bf16", eps=1e-6):
        self.layer, self.device = layer, layer.device
        self.own = list(range(layer.own_lo, layer.own_lo + layer.own_n))
        prec = "f32" if layer.prec == "f32" else "bf16"
        if weight.numel() != layer.d:
            raise ValueError(f"norm weight of {layer.d} elements expected, got {weight.numel()}")
        if weight.device != layer.status.device:
            raise ValueError(f"norm weight on {weight.device}, and the layer on {layer.status.device}")
        # (before the norms: their calls come after what made them)
        self.dw_norm = torch.zeros(layer.d, dtype=torch.float32, device=weight.device) if layer.with_bwd else None
        self.norms = [RMSNorm(weight, layer.T_src, prec, res_type, eps, with_bwd=layer.with_bwd) for _ in self.own]
        self.weight, self.eps = weight, eps
        self._decode_norms = {}
        for n in self.norms:
            n.dw = self.dw_norm
        self._ready()

    def set_inputs(self, w_router, bias, e2l, w_gate, w_up, w_down, other_xs=None, other_topk=None):
        """The layer's weights; other_xs: {source: rows} of the sources that are not its own."""
        xs = [None] * self.layer.S
        for s, n in zip(self.own, self.norms):
            xs[s] = n.y
        for s, x in (other_xs or {}).items():
            xs[s] = x
        self.layer.set_inputs(xs, w_router, bias, e2l, w_gate, w_up, w_down, other_topk)

    def _per_source(self, what, rows):
        if len(rows) != len(self.norms):
            raise ValueError(f"{what}: one tensor for each of {len(self.norms)} own sources expected, got {len(rows)}")

    @property
    def res(self) -> List[torch.Tensor]:
        """The residual stream behind this block's addition, per own source."""
        return [n.res for n in self.norms]

    def forward(self, res, delta=None, stream=None):
        """res, delta: per own source [T_src, d]; delta None for the first block.  Returns the layer's outputs."""
        delta = [None] * len(self.norms) if delta is None else delta
        self._per_source("res", res)
        self._per_source("delta", delta)
        for n, r, x in zip(self.norms, res, delta):
            T = n._rows_of(x, r)
            if T != self.layer.T_src:         # the layer routes all rows of n.y
                raise ValueError(f"{T} rows, and the layer has {self.layer.T_src} of every source")
        with torch.cuda.device(self.layer.device):
            for i, n in enumerate(self.norms):
                n.forward(delta[i], res[i], stream)
            self.layer.forward(stream)
        return [self.layer.out[s] for s in self.own]

    def backward(self, d_out, d_res=None, stream=None, router_grad=True, balance=False, d_loss=None):
        """d_out: per source of the layer, the gradient of its outputs; d_res:
        per own source, the gradient that reaches the residual stream behind
        this block's addition, or None.  Returns the gradients of res and delta
        (the stream's type; ``norms[i].d_x`` in the layer's); dw_norm and the
        layer's gradients are overwritten.  balance: the gradient of the
        layer's last ``balance_loss`` (d_loss its weights, None = ones) is in
        all of them; the layer's own ``balance_backward`` would come after the
        norm has read d_x, and refuses."""
        L = self.layer
        for n in self.norms:                  # (all of it before the layer's gradients are written)
            if n.T != L.T_src:
                raise RuntimeError(f"backward of the block's own forward: a norm's last one had {n.T} rows, not {L.T_src}")
        if d_res is not None:
            self._per_source("d_res", d_res)
            for n, t in zip(self.norms, d_res):
                if t is not None:
                    n._expect("d_res", t, n.res_dt, (n.T, n.d))
        if balance:
            if not router_grad:
                raise ValueError("balance adds to the router's gradient: router_grad")
            if getattr(L, "_bal", None) is None:
                raise RuntimeError("balance needs the layer's balance_loss before it")
            L._check(d_loss, torch.float32, 2)
        with torch.cuda.device(L.device):
            L.backward(d_out, stream, router_grad)
            if balance:
                L.balance_backward(d_loss, stream)
            L._d_x_read = True
            if not self.norms:                # no rows: the sum over them is zero
                self._enter(stream)
                with torch.cuda.stream(self._torch_stream(stream)):
                    self.dw_norm.zero_()
            return [n.backward(L.d_x[s], None if d_res is None else d_res[i], i > 0, stream)
                    for i, (s, n) in enumerate(zip(self.own, self.norms))]

    def decode(self, decoder, res, delta=None, stream=None):
        """The block for a few tokens: res (the residual stream, fp32 or bf16)
        and delta [T, d] bf16 or None, T up to the decoder's tokens.  The
        experts read the norm's rows in MX blocks.  Returns out [T, d] bf16;
        ``decode_norm.res`` is the stream behind the addition.  Buffers are
        kept per decoder size and stream type, so that a captured call's stay."""
        if self.layer.prec == "f32":
            raise ValueError("4-bit experts are for bf16 and MXFP8 layers")
        key = (decoder.tokens, res.dtype)
        with torch.cuda.device(self.layer.device):
            if key not in self._decode_norms:
                kind = "f32" if res.dtype == torch.float32 else "bf16"
                self._decode_norms[key] = n = RMSNorm(self.weight, decoder.tokens, "bf16", kind, self.eps, mx=True,
                                                      with_bwd=False)
                n._after_current(stream, n.res, n.y, n.rstd, n.codes, n.scales)
            n = self.decode_norm = self._decode_norms[key]
            y = n.forward(delta, res, stream)
            return decoder(y, n.codes[:n.T], n.scales[:n.T], stream)
