"""AdamW over the tensors of a model, through ``mok_grad_norm`` and ``mok_adamw``.

``AdamW`` owns what the C ABI expects from its caller: the moments (fp32, or
MX blocks of E4M3 codes with E8M0 scales), fp32 copies behind bf16 parameters,
the descriptors, the workspace.  It does no arithmetic of its own: one step is
the norm's launches (with ``max_norm``) and the update's.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence, Union

import torch

from . import (make_adamw, make_param, make_params, mok_adamw, mok_grad_norm,
               mok_grad_norm_ws_bytes)


class AdamW:
    """params: contiguous fp32 or bf16 tensors of one device, updated in place.

    weight_decay, state_bits: one value, or one per tensor.  state_bits 32 or 8
    (moments of a tensor in fp32, or in 8 bits).  master: keep fp32 copies of
    bf16 parameters, taken here: a step writes the parameters from them, so
    call take_params after writing parameters by other means; without them a bf16 parameter is rounded to nearest, or at
    random with random_params.  max_norm: clip the global gradient norm; a step
    whose norm is not finite is left out.  capturable: the step number (and the
    learning rate, see set_lr) live on the device, so a step captured in a
    graph advances at every replay; the number counts left-out steps too.

    Steps may run on several streams: a step, set_lr, bind and the two
    state_dict calls (these on the current stream) come after whatever the
    optimizer did before on another stream, and after a call other than a step
    the next step also waits for the current stream.  Replays of captured
    steps are ordered by the caller.
    """

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.01,
                 state_bits: Union[int, Sequence[int]] = 32, master: bool = True,
                 random_params: bool = False, max_norm: Optional[float] = None, seed: int = 0,
                 capturable: bool = False):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        if max_norm is not None and not max_norm > 0.0:
            raise ValueError(f"max_norm above zero (or None) expected, got {max_norm}")
        dev = self.params[0].device
        per = lambda v: list(v) if isinstance(v, (list, tuple)) else [v] * len(self.params)  # noqa: E731
        self.weight_decay, self.state_bits = per(weight_decay), per(state_bits)
        if len(self.weight_decay) != len(self.params) or len(self.state_bits) != len(self.params):
            raise ValueError("one weight_decay and state_bits per parameter")
        for p, bits in zip(self.params, self.state_bits):
            if p.device != dev or not p.is_contiguous():
                raise ValueError("parameters must be contiguous and on one device")
            if p.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError(f"float32 or bfloat16 expected, got {p.dtype}")
            if bits not in (8, 32):
                raise ValueError(f"state_bits 8 or 32 expected, got {bits}")
        ends = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size())
                      for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(ends, ends[1:])):
            raise ValueError("parameters overlap (the same one twice?): a step writes each by itself")
        self.device, self.max_norm = dev, max_norm
        self.step_count = 0
        self.master = [p.detach().float() if master and p.dtype == torch.bfloat16 else None
                       for p in self.params]
        z = lambda n, t: torch.zeros(n, dtype=t, device=dev)  # noqa: E731
        self.m, self.v, self.m_scale, self.v_scale = [], [], [], []
        for p, bits in zip(self.params, self.state_bits):
            n, t = p.numel(), torch.float32 if bits == 32 else torch.uint8
            self.m.append(z(n, t))
            self.v.append(z(n, t))
            self.m_scale.append(None if bits == 32 else z((n + 31) // 32, torch.uint8))
            self.v_scale.append(None if bits == 32 else z((n + 31) // 32, torch.uint8))
        self.norm = z(2, torch.float32)      # norm and clip factor of the last step
        self.dev_step = z(1, torch.int64) if capturable else None
        self.dev_lr = torch.full((1,), lr, dtype=torch.float64, device=dev) if capturable else None
        self.args = make_adamw(lr, betas[0], betas[1], eps, seed=seed, random_params=random_params,
                               dev_scale=self.norm[1:] if max_norm is not None else None,
                               dev_lr=self.dev_lr, dev_step=self.dev_step)
        self._held = self._ws = None
        # The stream of the last call, and an event behind a step on another
        # stream than the current one (a handle its owner may take down; 4 us
        # that steps on the current stream do not pay).
        self._last = self._event = None
        self._behind = True      # the current stream holds work that a step has to see
        self._seen, self._held_seen = set(), set()   # streams that _hold has named
        if dev.type == "cuda":
            with torch.cuda.device(dev):
                self._last = torch.cuda.current_stream()
                self._seen.add(self._last)

    def _after_last(self, s):
        """Work on `s` from here on comes after the calls before.  Not in a
        capture, which waits for nothing outside it."""
        if s != self._last:
            if self._event is not None:
                s.wait_event(self._event)
            else:
                s.wait_stream(self._last)

    def _hold(self, s):
        """Memory of what a step on `s` works on is not given to others before
        it is done, though every owner lets it go."""
        if s not in self._seen:
            self._seen.add(s)
            for ts in (self.m, self.v, self.m_scale, self.v_scale, self.master,
                       [self.norm, self.dev_step, self.dev_lr, self._ws]):
                for t in ts:
                    if t is not None:
                        t.record_stream(s)
        if s not in self._held_seen:
            self._held_seen.add(s)
            for p, g in self._held:
                p.record_stream(s)
                g.record_stream(s)

    @contextlib.contextmanager
    def _on_current(self):
        """Work of a call other than a step, on the current stream."""
        self._behind = True
        if self.device.type != "cuda":
            yield
            return
        with torch.cuda.device(self.device):
            cur = torch.cuda.current_stream()
            eager = not torch.cuda.is_current_stream_capturing()
            if eager:
                self._after_last(cur)
            yield
            if eager:
                self._last, self._event = cur, None

    def state_dict(self) -> dict:
        """Moments and fp32 copies (the tensors themselves), step number and
        the seed of the random rounding."""
        with self._on_current():
            step = int(self.dev_step.item()) if self.dev_step is not None else self.step_count
        return {"step": step, "seed": self.args.seed, "m": self.m, "v": self.v, "m_scale": self.m_scale,
                "v_scale": self.v_scale, "master": self.master}

    def load_state_dict(self, state: dict):
        """Copies a state_dict of an optimizer over tensors of the same sizes
        and kinds into this one's buffers (their addresses stay) and goes on
        with its step number and seed (steps captured before keep theirs)."""
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            mine, theirs = getattr(self, name), state[name]
            if len(mine) != len(theirs) or any(
                    (a is None) != (b is None) or (a is not None and (a.numel() != b.numel() or a.dtype != b.dtype))
                    for a, b in zip(mine, theirs)):
                raise ValueError(f"state of other tensors: {name}")
        with self._on_current():
            for name in ("m", "v", "m_scale", "v_scale", "master"):
                for a, b in zip(getattr(self, name), state[name]):
                    if a is not None:
                        a.copy_(b.detach().view(a.shape))
            self.step_count = int(state["step"])
            self.args.seed = int(state.get("seed", self.args.seed))   # (older states hold none)
            if self.dev_step is not None:
                self.dev_step.fill_(self.step_count)

    def take_params(self):
        """Takes the parameters as they are now (weights loaded into them, say)
        into the fp32 copies, whose next step would write the former ones."""
        with self._on_current():
            for p, w in zip(self.params, self.master):
                if w is not None:
                    w.copy_(p.detach())

    def set_lr(self, lr: float):
        self.args.lr = lr
        if self.dev_lr is not None:
            with self._on_current():
                self.dev_lr.fill_(lr)

    def bind(self, grads: Sequence[torch.Tensor]):
        """Descriptors for these gradient tensors (kept: step() without
        arguments reads them again).  They name the memory that parameters and
        gradients have now, which is held: a tensor that is given other memory
        afterwards (its .data) has to be bound again."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("one gradient per parameter")
        for p, g in zip(self.params, grads):
            if g.device != self.device:
                raise ValueError(f"gradient on {g.device}, parameters on {self.device}")
        held = [(p.detach(), g.detach()) for p, g in zip(self.params, grads)]
        self._desc = make_params([
            make_param(p=p, g=g, m=m, v=v, master=w, m_scale=ms, v_scale=vs, weight_decay=wd)
            for (p, g), m, v, w, ms, vs, wd in zip(held, self.m, self.v, self.master, self.m_scale,
                                                   self.v_scale, self.weight_decay)])
        self._held = held
        self._held_seen.clear()
        if self.max_norm is not None and self._ws is None:   # (its size follows from the parameters')
            with self._on_current():
                self._ws = torch.empty(mok_grad_norm_ws_bytes(self._desc), dtype=torch.uint8,
                                       device=self.device)
                self._seen.clear()

    def step(self, grads: Optional[Sequence[torch.Tensor]] = None, grad_scale: float = 1.0,
             stream=None):
        """One step on `stream` (a torch stream; None: the device's current
        one).  grads: gradients to bind, or None for those bound before.
        Gradients are multiplied by grad_scale > 0 (the norm is taken
        before, and clipped to max_norm / grad_scale; both have to be fp32
        values)."""
        f32 = ctypes.c_float(grad_scale).value       # as the kernels take it
        if not 0.0 < f32 < math.inf:
            raise ValueError(f"grad_scale above zero, finite in fp32, expected, got {grad_scale}")
        limit = 0.0 if self.max_norm is None else self.max_norm / grad_scale
        if self.max_norm is not None and not ctypes.c_float(limit).value > 0.0:
            raise ValueError(f"max_norm / grad_scale = {limit} is zero in fp32: nothing would be clipped")
        if grads is not None:
            self.bind(grads)
        if self._held is None:
            raise RuntimeError("step() before any gradients were bound")
        if self.device.type != "cuda":
            raise ValueError(f"a step needs parameters on a GPU, not on {self.device}")
        with torch.cuda.device(self.device):
            cur = torch.cuda.current_stream()
            s = cur if stream is None else stream
            if s.device != self.device:
                raise ValueError(f"stream on {s.device}, parameters on {self.device}")
            side = s != cur
            joins = captured = torch.cuda.is_current_stream_capturing()
            if side and not captured:
                with torch.cuda.stream(s):
                    captured = torch.cuda.is_current_stream_capturing()
            if self.dev_step is None and captured:
                raise RuntimeError("a captured step needs AdamW(capturable=True): its number would stand still")
            if not captured:
                self._after_last(s)
                if side or s not in self._seen:
                    self._hold(s)
            if side and (joins or (self._behind and not captured)):
                s.wait_stream(cur)
            if not captured:
                self._behind = False
            if self.max_norm is not None:
                mok_grad_norm(self._desc, limit, self.norm, self._ws, s)
            self.step_count += 1
            self.args.step = self.step_count
            self.args.grad_scale = grad_scale
            if self.dev_step is not None:
                with torch.cuda.stream(s):
                    self.dev_step.add_(1)
            mok_adamw(self._desc, self.args, s)
            if joins and side:       # a capture's branches come together again
                cur.wait_stream(s)
            if not captured:
                self._last = s
                self._event = s.record_event() if side else None
