"""The layer's form for a few tokens: its experts with weights in 4 bits.

``MoEDecoder`` owns the 4-bit weights and the buffers of ``mok_route`` and
``mok_decode_ffn`` for up to ``tokens`` tokens.  It does no arithmetic of its
own.  Its weights are laid out on the stream that is current when it is made,
which its calls on other streams come after; its calls share their buffers: the
caller orders calls on different streams, and replays of captured ones.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (STATUS, make_config, make_w4, mok_decode_ffn, mok_decode_ws_bytes, mok_mxfp4_quantize, mok_route,
               mok_w4)
from .streams import StreamUser


class MoEDecoder(StreamUser):
    """w_router [E, d] bf16, bias [E] fp32 or None, expert_to_local [E] int32;
    w_gate, w_up [E_local, I, d], w_down [E_local, d, I] float32 or bfloat16,
    which are quantised (MXFP4) and not kept.  d and I multiples of 128."""

    def __init__(self, w_router, bias, expert_to_local, w_gate, w_up, w_down, k, tokens):
        self.device = w_router.device
        (self.E, self.d), (self.E_local, self.I, _) = w_router.shape, w_gate.shape
        self.k, self.tokens = k, tokens
        self._expect("w_router", w_router, torch.bfloat16, (self.E, self.d))
        if bias is not None:
            self._expect("bias", bias, torch.float32, (self.E,))
        self._expect("expert_to_local", expert_to_local, torch.int32, (self.E,))
        self.w_router, self.bias, self.e2l = w_router, bias, expert_to_local
        self.cfg = make_config(1, max(tokens, 1), self.d, self.E, k, self.I, self.E_local, "bf16", 0)
        need = mok_decode_ws_bytes(self.cfg, tokens)
        if need == 0 or self.d % 128 or self.I % 128:
            raise ValueError(f"tokens {tokens}, d {self.d}, I {self.I}, E {self.E}, k {k}, E_local {self.E_local}: "
                             "not a layer of 4-bit experts")
        new = lambda dt, *n: torch.empty(*n, dtype=dt, device=self.device)  # noqa: E731
        self.topk_idx, self.topk_gate = new(torch.int32, tokens, k), new(torch.float32, tokens, k)
        self.out = new(torch.bfloat16, tokens, self.d)
        self.ws = new(torch.uint8, need)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.weights: Optional[mok_w4] = None
        self.update_weights(w_gate, w_up, w_down)
        self._ready()

    def _buffers(self):
        return super()._buffers() + self.weights.tensors

    def update_weights(self, w_gate, w_up, w_down, stream=None):
        """Other expert weights of the same sizes in the place of the ones
        there: quantised on `stream` into the same memory, so captured calls
        read them."""
        s = self._torch_stream(stream)
        with torch.cuda.device(self.device), torch.cuda.stream(s):
            self._enter(stream)
            rows = []
            for name, w, shape in (("w_gate", w_gate, (self.E_local, self.I, self.d)),
                                   ("w_up", w_up, (self.E_local, self.I, self.d)),
                                   ("w_down", w_down, (self.E_local, self.d, self.I))):
                self._expect(name, w, w.dtype if w.dtype == torch.float32 else torch.bfloat16, shape)
                self._hold(stream, w)
                codes = torch.empty(*shape[:2], shape[2] // 2, dtype=torch.uint8, device=self.device)
                scales = torch.empty(*shape[:2], shape[2] // 32, dtype=torch.uint8, device=self.device)
                mok_mxfp4_quantize(shape[0] * shape[1], shape[2], w, codes, scales)
                rows.append((codes, scales))
            self.weights = make_w4(*(r[0] for r in rows), *(r[1] for r in rows), into=self.weights)

    def __call__(self, x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """x [T, d] bf16, T <= tokens, which the router reads, and the experts
        too unless codes [T, d] and scales [T, d/32] hold the rows in MX blocks
        (``RMSNorm(mx=True)``).  Returns out [T, d] bf16: the gate-weighted sum
        over the slots with a local expert, overwritten by the next call."""
        T = x.shape[0]
        if T > self.tokens:
            raise ValueError(f"{T} tokens, and buffers for {self.tokens}")
        if (codes is None) != (scales is None):
            raise ValueError("codes come with scales")
        self._expect("x", x, torch.bfloat16, (T, self.d))
        if codes is not None:
            self._expect("codes", codes, torch.uint8, (T, self.d))
            self._expect("scales", scales, torch.uint8, (T, self.d // 32))
        with torch.cuda.device(self.device):
            self._enter(stream)
            self._hold(stream, x, codes, scales)
            mok_route(self.cfg, T, x, self.w_router, self.bias, self.topk_idx, self.topk_gate, stream)
            mok_decode_ffn(self.cfg, T, x if codes is None else codes, scales, self.topk_idx, self.topk_gate, self.e2l,
                           self.weights, self.out, self.ws, self.status, stream)
        return self.out[:T]

    def check_status(self):
        st = int(self.status.item())
        if st != 0:
            raise RuntimeError(f"device status {STATUS.get(st, st)}")
