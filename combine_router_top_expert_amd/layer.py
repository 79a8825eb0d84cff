"""Device buffers of one MoE layer instance, allocated with torch.

``MoELayer`` owns the caller-side memory the C ABI expects (configuration,
weights, forward state, staging rows, outputs, gradients, workspace, device
status word) and calls ``mok_layer_fwd`` / ``mok_layer_bwd``, and for training the
balance loss (``mok_balance_fwd`` / ``mok_balance_bwd``) with the router
projection's backward (``mok_router_bwd``).  It does no arithmetic of its own.
The calls share the layer's buffers: the caller orders calls on different
streams, and replays of captured ones.
"""
from __future__ import annotations

from typing import List, Optional

import numpy as np
import torch

from . import (MAX_SOURCES, AuxStream, make_balance, make_config, make_state, make_weights,
               mok_balance_bwd, mok_balance_fwd, mok_balance_ws_bytes, mok_checkpoint_pack,
               mok_checkpoint_unpack, mok_layer_bwd, mok_layer_bwd_checkpoint, mok_layer_fwd,
               mok_prepare_bwd, mok_mx_quantize, mok_router_bwd, mok_router_bwd_ws_bytes,
               mok_tune_fwd, mok_workspace_bytes, STATUS)
from .streams import StreamUser


def _dt(prec: str):
    return torch.float32 if prec == "f32" else torch.bfloat16


def to_device(a: np.ndarray, prec: str, device) -> torch.Tensor:
    """Storage array from the input generator (fp32 values or bf16 bits) -> device tensor."""
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16).copy()).to(device).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


class MoELayer(StreamUser):
    def __init__(self, S, T_src, d, E, k, I, E_local, prec, R_cap, own_lo, own_n, device="cuda",
                 ring_bytes=0, minibatch_rows=256, comm_wgs=0, gemm_wgs=0, with_bwd=True,
                 wait_limit_us=0, two_streams=True, bwd_ring_bytes=0, transposed_weights=True,
                 keep_logits=False, checkpoint=False, scratch: Optional["MoELayer"] = None):
        """checkpoint: what the backward needs of the expert FFN is kept in 8
        bits after the forward (ck_codes, ck_scales), and ab and h are scratch;
        scratch: a layer of the same sizes whose ab and h this one uses too, so
        that a stack of layers holds one pair: their calls on different
        streams, and replays of captured ones, are ordered by the caller.  (An
        MXFP8 layer keeps its own h, which holds 8-bit codes already.)"""
        assert S <= MAX_SOURCES
        if checkpoint and not with_bwd:
            raise ValueError("a checkpoint is for the backward: with_bwd")
        if scratch is not None:
            mine = dict(S=S, T_src=T_src, I=I, prec=prec, R_cap=R_cap)
            where = torch.empty(0, device=device).device          # with its number ("cuda" names the current one)
            if not (checkpoint and scratch.checkpoint) or where != scratch.status.device or any(
                    getattr(scratch, n) != v for n, v in mine.items()):
                raise ValueError("scratch is shared between checkpointing layers of the same sizes, type and device")
        self.S, self.T_src, self.d, self.E, self.k, self.I = S, T_src, d, E, k, I
        self.E_local, self.prec, self.R_cap = E_local, prec, R_cap
        self.own_lo, self.own_n = own_lo, own_n
        self.device = torch.device(device)
        self.cfg = make_config(S, T_src, d, E, k, I, E_local, prec, R_cap, minibatch_rows,
                               ring_bytes, comm_wgs, gemm_wgs, wait_limit_us, bwd_ring_bytes)
        dev = self.device
        act = _dt(prec)
        N = S * T_src * k
        self.topk_idx = torch.zeros(max(N, 1), dtype=torch.int32, device=dev)
        self.topk_gate = torch.zeros(max(N, 1), dtype=torch.float32, device=dev)
        self.counts = torch.zeros(E_local, dtype=torch.int32, device=dev)
        self.offsets = torch.zeros(E_local + 1, dtype=torch.int32, device=dev)
        self.row_src = torch.zeros(max(R_cap, 1), dtype=torch.int32, device=dev)
        self.dest_row = torch.zeros(max(N, 1), dtype=torch.int32, device=dev)
        if prec == "mxfp8":
            self.h = torch.zeros(max(R_cap, 1) * I, dtype=torch.uint8, device=dev)
        elif scratch is None:
            self.h = torch.zeros(max(R_cap, 1), I, dtype=act, device=dev)
        if scratch is not None:
            self.ab = scratch.ab
            if prec != "mxfp8":
                self.h = scratch.h
        else:
            self.ab = torch.zeros(max(R_cap, 1), 2 * I, dtype=act, device=dev) if with_bwd or prec != "mxfp8" else None
        self.checkpoint = checkpoint
        if checkpoint:
            self.ck_codes = torch.zeros(max(R_cap, 1), 2 * I, dtype=torch.uint8, device=dev)
            self.ck_scales = torch.zeros(max(R_cap, 1), I // 16, dtype=torch.uint8, device=dev)
        out_dt = torch.float32 if prec == "f32" else torch.bfloat16
        self.staging = [torch.zeros(T_src * k, d, dtype=out_dt, device=dev) for _ in range(S)]
        self.out = [torch.zeros(T_src, d, dtype=out_dt, device=dev) if own_lo <= s < own_lo + own_n
                    else None for s in range(S)]
        self.ws = torch.zeros(max(mok_workspace_bytes(self.cfg), 256), dtype=torch.uint8,
                              device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        # the bf16 backward runs its side work on a second stream (mok_aux)
        self.aux = None
        if two_streams and with_bwd and prec == "bf16" and not bwd_ring_bytes:
            self.aux = AuxStream(dev)
            self.aux.attach(self.cfg)
        # MXFP8: h holds E4M3 codes; its scales are kept for the backward
        self.h_scale = (torch.zeros(max(R_cap, 1) * I // 32, dtype=torch.uint8, device=dev)
                        if prec == "mxfp8" and with_bwd else None)
        # the router's logits, for the balance loss (balance_loss)
        self.logits = (torch.zeros(max(S * T_src, 1), E, dtype=torch.float32, device=dev)
                       if keep_logits else None)
        self.state = make_state(self.topk_idx, self.topk_gate, self.counts, self.offsets,
                                self.row_src, self.dest_row, self.h, self.ab, self.h_scale,
                                self.logits)
        self.with_bwd = with_bwd
        self._bal_bufs = {}
        self._d_x_read = False   # a block's norm has taken d_x on
        self.d_bias = None       # the balance losses' gradient of a router bias
        # bf16 backward: the weights also transposed (mok_prepare_bwd), so dh
        # and dx read them k-contiguous (bit-identical either way)
        self.transposed_weights = transposed_weights
        if with_bwd:
            self.d_gate = torch.zeros(max(N, 1), dtype=torch.float32, device=dev)
            self.dx_stage = [torch.zeros(T_src * k, d, dtype=act, device=dev) for _ in range(S)]
            self.d_x = [torch.zeros(T_src, d, dtype=act, device=dev) if own_lo <= s < own_lo + own_n
                        else None for s in range(S)]
            self.dw_gate = torch.zeros(E_local, I, d, dtype=torch.float32, device=dev)
            self.dw_up = torch.zeros(E_local, I, d, dtype=torch.float32, device=dev)
            self.dw_down = torch.zeros(E_local, d, I, dtype=torch.float32, device=dev)
            self.dw_router = torch.zeros(E, d, dtype=torch.float32, device=dev)
        self._ready()

    # ---------------------------------------------------------------- inputs
    def set_inputs(self, xs: List[torch.Tensor], w_router, bias, e2l, w_gate, w_up, w_down,
                   other_topk: Optional[List] = None):
        """xs: S device tensors [T_src, d]; other_topk: per non-own source
        (topk_idx [T_src, k] int32, topk_gate [T_src, k] fp32) numpy arrays.
        What the layer forms of the weights is formed on the current stream."""
        self.xs = xs
        self.w_router = w_router
        self.bias = bias
        self.e2l = e2l
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        per = self.T_src * self.k
        for s in range(self.S):
            if self.own_lo <= s < self.own_lo + self.own_n:
                continue
            idx, g = other_topk[s]
            self.topk_idx[s * per:(s + 1) * per] = torch.from_numpy(idx.reshape(-1)).to(self.device)
            self.topk_gate[s * per:(s + 1) * per] = torch.from_numpy(g.reshape(-1)).to(self.device)
        if self.prec == "mxfp8":
            self._quantize_weights()
        elif self.prec == "bf16" and self.with_bwd and self.transposed_weights:
            E, d, I = self.E_local, self.d, self.I
            self.wt = [torch.empty(E * I * d, dtype=torch.bfloat16, device=self.device),
                       torch.empty(E * d * 2 * I, dtype=torch.bfloat16, device=self.device)]
            self.update_weights()
            self.weights = make_weights(w_gate, w_up, w_down, wt_down=self.wt[0],
                                        wt_gu=self.wt[1])
        else:
            self.weights = make_weights(w_gate, w_up, w_down)
        self._ready()

    def set_peer_slots(self, s: int, y: torch.Tensor, d_gate: torch.Tensor,
                       dx: Optional[torch.Tensor] = None):
        """What the GPUs holding remote experts write back to own source s:
        y [T_src*k, d] into its staging rows, d_gate [T_src*k] and dx
        [T_src*k, d] into its reverse-dispatch rows.  The layer overwrites the
        rows of local slots on every pass, so only remote slots keep them."""
        per = self.T_src * self.k
        self.staging[s].copy_(y)
        if self.with_bwd:
            self.d_gate[s * per:(s + 1) * per].copy_(d_gate)
            if dx is not None:
                self.dx_stage[s].copy_(dx)

    def update_weights(self, stream=None):
        """After the expert weights were written in place (an optimizer step):
        forms what the layer keeps beside them again -- the backward's
        transposed copies, the MX codes -- in the same buffers.  A layer in
        fp32, or in bf16 without transposed weights, keeps nothing."""
        with torch.cuda.device(self.device):
            self._enter(stream)
            w = (self.w_gate, self.w_up, self.w_down)
            if self.prec == "mxfp8":
                for t, (codes, scales) in zip(w, self.wq):
                    mok_mx_quantize(t.numel() // t.shape[-1], t.shape[-1], t, codes, scales, stream)
                if self.with_bwd:
                    mok_prepare_bwd(self.cfg, *w, *self.wt, stream)
            elif self.prec == "bf16" and self.with_bwd and self.transposed_weights:
                mok_prepare_bwd(self.cfg, *w, self.wt[0], None, self.wt[1], None, stream)

    def _quantize_weights(self):
        """MX-quantise the expert weights (off the timed path)."""
        self.wq = [(torch.empty(w.numel(), dtype=torch.uint8, device=self.device),
                    torch.empty(w.numel() // 32, dtype=torch.uint8, device=self.device))
                   for w in (self.w_gate, self.w_up, self.w_down)]
        q = self.wq
        t = [None] * 4
        if self.with_bwd:
            # the backward's transposed operands: W_down^T and [W_gate; W_up]^T
            E, d, I = self.E_local, self.d, self.I
            t = [torch.empty(E * I * d, dtype=torch.uint8, device=self.device),
                 torch.empty(E * I * d // 32, dtype=torch.uint8, device=self.device),
                 torch.empty(E * d * 2 * I, dtype=torch.uint8, device=self.device),
                 torch.empty(E * d * 2 * I // 32, dtype=torch.uint8, device=self.device)]
        self.wt = t
        self.update_weights()
        self.weights = make_weights(q[0][0], q[1][0], q[2][0], q[0][1], q[1][1], q[2][1], *t)

    # ---------------------------------------------------------------- passes
    def forward(self, stream=None):
        self._enter(stream)
        mok_layer_fwd(self.cfg, self.own_lo, self.own_n, self.xs, self.w_router, self.bias,
                      self.e2l, self.weights, self.state, self.staging, self.out, self.ws,
                      self.status, stream)
        self._keep(stream)

    def _keep(self, stream):
        """What the backward needs of the forward that just ran, in 8 bits."""
        if self.checkpoint:
            mok_checkpoint_pack(self.cfg, self.offsets, self.ab, self.ck_codes, self.ck_scales, stream)

    def tune(self, mbs=None, comms=None, reps=3, stream=None):
        """Pick the fused path's minibatch size and dispatch/GEMM split with
        mok_tune_fwd (off the timed path; synchronises).  The workspace grows
        to fit every candidate first.  Returns {(minibatch_rows, comm_wgs):
        ms per forward or None}; self.cfg holds the fastest pair after."""
        mbs = list(mbs) if mbs is not None else [64, 128, 256, 512, 1024, 2048, 4096]
        need = self.ws.numel()
        for mb in mbs:
            c = type(self.cfg).from_buffer_copy(self.cfg)
            c.minibatch_rows = mb
            need = max(need, mok_workspace_bytes(c))
        if need > self.ws.numel():
            self.ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
            self._ready()
        self._enter(stream)
        best, table = mok_tune_fwd(self.cfg, mbs, comms, reps, self.ws.numel(), self.own_lo,
                                   self.own_n, self.xs, self.w_router, self.bias, self.e2l,
                                   self.weights, self.state, self.staging, self.out, self.ws,
                                   self.status, stream)
        self.cfg.minibatch_rows = best.minibatch_rows
        self.cfg.comm_wgs = best.comm_wgs
        self.cfg.gemm_wgs = best.gemm_wgs
        self._keep(stream)
        return table

    def backward(self, d_out: List[torch.Tensor], stream=None, router_grad=True):
        dw_router = self.dw_router if router_grad else None
        self._enter(stream)
        self._hold(stream, *d_out)
        self._d_x_read = False
        if self.checkpoint and self.prec == "bf16" and not self.cfg.bwd_ring_bytes:
            mok_layer_bwd_checkpoint(self.cfg, self.own_lo, self.own_n, d_out, self.xs, self.w_router, self.e2l,
                                     self.weights, self.state, self.ck_codes, self.ck_scales, self.staging,
                                     self.d_gate, self.dx_stage, self.d_x, self.dw_gate, self.dw_up, self.dw_down,
                                     dw_router, self.ws, self.status, stream)
            return
        if self.checkpoint:
            mok_checkpoint_unpack(self.cfg, self.offsets, self.ck_codes, self.ck_scales, self.ab,
                                  None if self.prec == "mxfp8" else self.h, stream)
        mok_layer_bwd(self.cfg, self.own_lo, self.own_n, d_out, self.xs, self.w_router, self.e2l,
                      self.weights, self.state, self.staging, self.d_gate, self.dx_stage, self.d_x,
                      self.dw_gate, self.dw_up, self.dw_down, dw_router, self.ws, self.status, stream)

    def _check(self, t, dt, n=None):
        """Refuses a tensor that a kernel could not read as n (any) values dt."""
        dev = self.logits.device
        if t is not None and (t.dtype != dt or not t.is_contiguous() or t.device != dev
                              or (n is not None and t.numel() != n) or t.numel() < 1):
            raise ValueError(f"contiguous {dt} tensor{'' if n is None else f' of {n}'} on {dev} expected, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")

    def balance_loss(self, alpha, beta=0.0, group_offsets=None, token_mask=None, stream=None):
        """Balance loss and z-loss of the last forward's own tokens (fp32 [2]
        on the device; needs keep_logits).  group_offsets: int32 [G+1] over
        the own rows (sequences), None = one group; token_mask: uint8 [own
        rows] or None.  Leaves counts_all [G, E], prob [G, E] and n_tok
        [G+2]; they and the losses are overwritten by the next call with as
        many groups (buffers are kept per number of groups, so that a captured
        call's stay)."""
        if self.logits is None:
            raise RuntimeError("balance_loss needs MoELayer(keep_logits=True)")
        T, dev = self.own_n * self.T_src, self.logits.device
        G = 0 if group_offsets is None else group_offsets.numel() - 1
        self._check(group_offsets, torch.int32)
        self._check(token_mask, torch.uint8, T)
        if group_offsets is not None and G < 1:
            raise ValueError("group_offsets needs at least two entries")
        self._bal = make_balance(alpha, beta, G, group_offsets, token_mask)
        self._bal_keep = (group_offsets, token_mask)
        with torch.cuda.device(self.device):
            rows = max(G, 1)
            if rows not in self._bal_bufs:
                e = lambda t, *n: torch.empty(*n, dtype=t, device=dev)  # noqa: E731
                self._bal_bufs[rows] = (e(torch.int32, rows, self.E), e(torch.float32, rows, self.E),
                                        e(torch.int32, rows + 2), e(torch.float32, 2),
                                        e(torch.uint8, mok_balance_ws_bytes(self.cfg, T, self._bal)))
                self._after_current(stream, *self._bal_bufs[rows])
            self._hold(stream, group_offsets, token_mask)
            self.counts_all, self.prob, self.n_tok, self.loss, self.ws_bal = self._bal_bufs[rows]
            lo = self.own_lo * self.T_src
            mok_balance_fwd(self.cfg, T, self._bal, self.logits[lo:], self.topk_idx[lo * self.k:],
                            self.counts_all, self.prob, self.n_tok, self.loss, self.ws_bal,
                            self.status, stream)
        return self.loss

    def balance_backward(self, d_loss=None, stream=None):
        """Adds the gradient of d_loss[0] * balance loss + d_loss[1] * z-loss
        (d_loss fp32 [2] on the device, None = ones) to d_x and dw_router,
        after backward() (in a block: MoEBlock.backward(balance=True)).  With a
        router bias, d_bias [E] becomes these losses' gradient of it; backward()
        forms none, so the share that comes through the gates is not in it."""
        if getattr(self, "_bal", None) is None or not self.with_bwd:
            raise RuntimeError("balance_backward needs balance_loss and backward before it")
        if self._d_x_read:
            raise RuntimeError("the block's norm has read d_x already: MoEBlock.backward(balance=True)")
        self._check(d_loss, torch.float32, 2)
        with torch.cuda.device(self.device):
            T, lo = self.own_n * self.T_src, self.own_lo * self.T_src
            if getattr(self, "d_logits", None) is None:
                self.d_logits = torch.empty(max(T, 1), self.E, dtype=torch.float32, device=self.device)
                self.ws_router = torch.empty(mok_router_bwd_ws_bytes(self.cfg, self.own_n),
                                             dtype=torch.uint8, device=self.device)
                self._after_current(stream, self.d_logits, self.ws_router)
            if self.bias is not None and self.d_bias is None:
                self.d_bias = torch.empty(self.E, dtype=torch.float32, device=self.device)
                self._after_current(stream, self.d_bias)
            d_bias = self.d_bias if self.bias is not None else None
            self._hold(stream, *self._bal_keep, d_loss)
            with torch.cuda.stream(self._torch_stream(stream)):
                if self._bal.G > 0:  # rows outside every group are not written: they add nothing
                    self.d_logits.zero_()
                if d_bias is not None:
                    d_bias.zero_()
            mok_balance_bwd(self.cfg, T, self._bal, self.logits[lo:], self.counts_all, self.n_tok,
                            d_loss, self.d_logits, self.status, stream)
            mok_router_bwd(self.cfg, self.own_lo, self.own_n, self.d_logits, self.xs, self.w_router,
                           self.d_x, self.dw_router, d_bias, True, self.ws_router, stream)

    def decoder(self, tokens):
        """The layer's form for up to `tokens` tokens at once: its local experts
        in 4 bits (a ``decode.MoEDecoder`` with the layer's router and weights
        as they are now)."""
        from .decode import MoEDecoder
        if self.prec == "f32":
            raise ValueError("4-bit experts are for bf16 and MXFP8 layers")
        return MoEDecoder(self.w_router, self.bias, self.e2l, self.w_gate, self.w_up, self.w_down, self.k, tokens)

    def check_status(self):
        st = int(self.status.item())
        if st != 0:
            raise RuntimeError(f"device status {STATUS.get(st, st)}")
