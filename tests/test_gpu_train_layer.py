"""The layer's training calls together, where a plain step does not reach:
the router's bias.  Tolerances as in test_gpu_train."""
import pytest
import torch

import combine_router_top_expert_amd as mok
from combine_router_top_expert_amd.layer import MoELayer
from test_gpu_train import DEV, U, _gen, _log, _within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prec", ["f32", "bf16"])
@pytest.mark.parametrize("off", [None, [0, 100, 290]], ids=str)
def test_balance_backward_of_a_router_bias(prec, off):
    """d_bias is the losses' gradient of the bias, from autograd in 64 bits on
    the kept logits, whatever an earlier call left there, and d_x and
    dw_router are those of the same call without it.  Its error is that of a
    column of d_logits (96 U of p times weights, here by the largest term of
    each) and one rounding."""
    _log("bias", prec, off)
    S, T, d, E, k, I = 1, 300, 64, 8, 2, 64
    gen, dt = _gen(17), torch.float32 if prec == "f32" else torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=gen).to(DEV, dt)  # noqa: E731
    L = MoELayer(S, T, d, E, k, I, E, prec, T * k, 0, 1, device=DEV, keep_logits=True)
    bias = torch.randn(E, generator=gen).to(DEV)
    L.set_inputs([rnd(T, d)], rnd(E, d), bias, torch.arange(E, dtype=torch.int32, device=DEV), rnd(E, I, d),
                 rnd(E, I, d), rnd(E, d, I))
    offd = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    dout, dl = [rnd(T, d)], torch.tensor([2.0, 0.5], device=DEV)
    L.forward()
    L.backward(dout)
    before = [L.d_x[0].clone(), L.dw_router.clone()]
    for _ in range(2):
        L.balance_loss(0.5, 0.01, offd)
        L.backward(dout)
        L.balance_backward(dl)
    torch.cuda.synchronize()
    L.check_status()
    z = L.logits.cpu().double()
    idx = L.topk_idx.view(T, k).cpu().long()
    b = torch.zeros(E, dtype=torch.float64, requires_grad=True)
    p = torch.softmax(z + b, 1)
    groups = [0, T] if off is None else off
    G, N = len(groups) - 1, groups[-1] - groups[0]
    total, size = 0.0, torch.zeros(E, dtype=torch.float64)
    for lo, hi in zip(groups, groups[1:]):
        n = hi - lo
        w = 2.0 * 0.5 * torch.bincount(idx[lo:hi].reshape(-1), minlength=E).double() * E / (k * n * n * G)
        lse = torch.logsumexp(z[lo:hi] + b, 1)
        total = total + (p[lo:hi] * w).sum() + 0.5 * 0.01 / N * lse.square().sum()
        size = size + (p[lo:hi] * (2 * w.max() + 0.01 / N * (1 + lse.abs()[:, None]))).sum(0).detach()
    ref, = torch.autograd.grad(total, b)
    _within(L.d_bias, ref, 192 * U * size + U * ref.abs(), "d_bias")
    # the other outputs: the entry point without a bias gradient
    cfg, ws = L.cfg, torch.empty(mok.mok_router_bwd_ws_bytes(L.cfg, 1), dtype=torch.uint8, device=DEV)
    mok.mok_router_bwd(cfg, 0, 1, L.d_logits, L.xs, L.w_router, [before[0]], before[1], None, True, ws)
    torch.cuda.synchronize()
    assert torch.equal(L.d_x[0], before[0]) and torch.equal(L.dw_router, before[1])


def test_layer_without_a_bias_has_no_gradient_of_it():
    S, T, d, E, k, I = 1, 64, 64, 4, 1, 64
    rnd = lambda *s: torch.randn(*s, generator=_gen(1)).to(DEV)  # noqa: E731
    L = MoELayer(S, T, d, E, k, I, E, "f32", T * k, 0, 1, device=DEV, keep_logits=True)
    L.set_inputs([rnd(T, d)], rnd(E, d), None, torch.arange(E, dtype=torch.int32, device=DEV), rnd(E, I, d),
                 rnd(E, I, d), rnd(E, d, I))
    L.forward()
    L.balance_loss(0.5, 0.01)
    L.backward([rnd(T, d)])
    L.balance_backward()
    torch.cuda.synchronize()
    L.check_status()
    assert L.d_bias is None
