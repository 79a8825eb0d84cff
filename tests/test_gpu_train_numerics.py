"""Numerics of the training entry points where a plain comparison at ordinary
sizes does not reach: gradients whose leading bits cancel, second moments at
the bottom of fp32's range, long column sums.

Tolerances as in test_gpu_train (U = 2^-24, half a step of fp32); what a test
adds to them is derived in its docstring.
"""
import math

import pytest
import torch

import combine_router_top_expert_amd as mok
from test_gpu_train import DEV, U, _gen, _log, _within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("E", [2, 64, 65, 128, 129, 200, 256, 257, 512])
@pytest.mark.parametrize("add", [False, True])
def test_router_bwd_dx_takes_every_bit_of_the_gradient(E, add):
    """Two gradients of a token cancel to 2^-12 of themselves and meet equal
    rows of W, so d_x is what their last bits leave.  The bf16 parts of both
    make six nonzero products, exact in fp32, with at most seven additions
    (the base among them) off by a step, 2 U of the magnitudes, each: 14 U,
    taken as 16 U; then the bf16 rounding.  A gradient without its last eight
    bits is off by up to 128 U."""
    _log("router_bwd cancel", E, add)
    S, T_src, d = 2, 77, 192
    T, g = S * T_src, _gen(E)
    a = (1 + torch.rand(T, generator=g)) * torch.where(torch.rand(T, generator=g) < 0.5, -1.0, 1.0)
    b = -(a.double() * (1 - 2.0 ** -12 * torch.rand(T, generator=g).double())).float()
    pair = torch.stack([torch.randperm(E, generator=g)[:2] for _ in range(T)])
    dz = torch.zeros(T, E).scatter_(1, pair, torch.stack([a, b], 1))
    s = torch.randn(d, generator=g).bfloat16()
    w = s.expand(E, d).contiguous()
    x = [torch.randn(T_src, d, generator=g).bfloat16() for _ in range(S)]
    dx0 = [(torch.randn(T_src, d, generator=g) * 2.0 ** -12).bfloat16() for _ in range(S)]
    cfg = mok.make_config(S, T_src, d, E, 1, 64, 1, "bf16", 0)
    ws = torch.full((mok.mok_router_bwd_ws_bytes(cfg, S),), 0xFF, dtype=torch.uint8, device=DEV)
    ref = (a.double() + b.double())[:, None] * s.double()
    if add:
        ref = ref + torch.cat(dx0).double()
    mag = (a.double().abs() + b.double().abs())[:, None] * s.double().abs()
    for with_dw in (True, False):     # the products together and alone
        dx = [t.to(DEV) for t in dx0]
        dw = torch.zeros(E, d, device=DEV) if with_dw else None
        mok.mok_router_bwd(cfg, 0, S, dz.to(DEV), [t.to(DEV) for t in x], w.to(DEV), dx, dw, None, add, ws)
        torch.cuda.synchronize()
        _within(torch.cat(dx), ref, (2.0 ** -8 + 2 * U) * ref.abs() + 16 * U * mag, f"d_x, dw {with_dw}")


@pytest.mark.parametrize("E", [130, 256, 300, 512])
def test_router_bwd_dx_repeats_itself(E):
    """Waves that share a row's experts exchange their sums: the same bytes
    from every call, for tokens that fill no block and columns of one step."""
    _log("router_bwd repeat", E)
    for T, d in ((1, 64), (63, 64), (65, 128), (1000, 576)):
        g = _gen(T)
        cfg = mok.make_config(1, T, d, E, 1, 64, 1, "bf16", 0)
        dz, w = torch.randn(T, E, generator=g).to(DEV), torch.randn(E, d, generator=g).bfloat16().to(DEV)
        x = torch.randn(T, d, generator=g).bfloat16().to(DEV)
        ws = torch.empty(mok.mok_router_bwd_ws_bytes(cfg, 1), dtype=torch.uint8, device=DEV)
        first = None
        for _ in range(5):
            dx, dw = torch.full((T, d), 9.0, dtype=torch.bfloat16, device=DEV), torch.zeros(E, d, device=DEV)
            mok.mok_router_bwd(cfg, 0, 1, dz, [x], w, [dx], dw, None, False, ws)
            torch.cuda.synchronize()
            if first is None:
                first = dx
                zd, wd = dz.double().cpu(), w.double().cpu()
                ref = zd @ wd
                _within(dx, ref, 2.0 ** -8 * ref.abs() + (3 * E + 2) * U * (zd.abs() @ wd.abs()), (T, d))
            assert torch.equal(dx, first), (T, d)
