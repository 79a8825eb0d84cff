"""Blocks with the calls around them that a training program makes."""
import pytest
import torch

import combine_router_top_expert_amd as mok
from combine_router_top_expert_amd.block import MoEBlock
from combine_router_top_expert_amd.layer import MoELayer
from test_gpu_block import _grads, _layer
from test_gpu_train import DEV, _gen, _log

pytestmark = pytest.mark.gpu


def _block_in_64(res, delta, wn, wr, wg, wu, wd, k, eps):
    """r, out, balance loss (times 1 / alpha) and z-loss (times 1 / beta) of a block, all its rows one group."""
    r = res + delta
    y = r * (r.square().mean(1, keepdim=True) + eps).rsqrt() * wn
    z = y @ wr.t()
    top = z.topk(k, 1)
    gate = torch.softmax(top.values, 1)
    out = 0.0
    for e in range(wr.shape[0]):
        g = (gate * (top.indices == e)).sum(1, keepdim=True)
        a, b = y @ wg[e].t(), y @ wu[e].t()
        out = out + g * ((a * torch.sigmoid(a) * b) @ wd[e].t())
    n, E = z.shape
    share = torch.bincount(top.indices.reshape(-1), minlength=E).double() / (k * n)
    return r, out, E * (share * torch.softmax(z, 1).mean(0)).sum(), torch.logsumexp(z, 1).square().mean()


def test_block_gradients_with_balance_losses():
    """Two fp32 blocks whose layers have balance and z-losses, against autograd in 64 bits: the losses' gradients
    reach the residual stream, the first block and the norms' weights.  Errors as without the losses (a chain of
    about ten products of at most 192 terms: below 1e-4 of a result's norm); their own are those of a softmax row,
    96 u.  The losses weigh enough for every gradient to differ by a hundredth without them (asserted)."""
    _log("block balance")
    S, T, d, E, k, I, eps, alpha, beta = 2, 70, 128, 8, 2, 192, 1e-6, 4000.0, 300.0
    gen = _gen(22)
    rnd = lambda *s, std=1.0: (std * torch.randn(*s, generator=gen)).to(DEV)  # noqa: E731
    blocks, refs, plain = [], [], []
    for _ in range(2):
        L = MoELayer(S, T, d, E, k, I, E, "f32", S * T * k, 0, S, device=DEV, keep_logits=True)
        wn = 1 + rnd(d, std=0.2)
        w = [rnd(E, d, std=d ** -0.5), rnd(E, I, d, std=d ** -0.5), rnd(E, I, d, std=d ** -0.5), rnd(E, d, I, std=I ** -0.5)]
        b = MoEBlock(L, wn, "f32", eps)
        b.set_inputs(w[0], None, torch.arange(E, dtype=torch.int32, device=DEV), *w[1:])
        blocks.append(b)
        refs.append([t.double().requires_grad_() for t in (wn, *w)])
        plain.append([t.double().requires_grad_() for t in (wn, *w)])
    res, delta = [rnd(T, d, std=2.0) for _ in range(S)], [rnd(T, d) for _ in range(S)]
    dout, dres = [rnd(T, d) for _ in range(S)], [rnd(T, d) for _ in range(S)]
    dl = torch.tensor([2.0, 0.5], device=DEV)
    o1 = blocks[0].forward(res, delta)
    blocks[1].forward(blocks[0].res, o1)
    losses = [b.layer.balance_loss(alpha, beta) for b in blocks]
    g2 = blocks[1].backward(dout, dres, balance=True, d_loss=dl)
    g1 = blocks[0].backward([n.d_x for n in blocks[1].norms], g2, balance=True)
    torch.cuda.synchronize()
    for b in blocks:
        b.layer.check_status()

    def in_64(ws, weight):
        R, D = (torch.cat(t).double().requires_grad_() for t in (res, delta))
        r, out, b1, z1 = _block_in_64(R, D, *ws[0], k, eps)
        r, out, b2, z2 = _block_in_64(r, out, *ws[1], k, eps)
        total = (out * torch.cat(dout).double()).sum() + (r * torch.cat(dres).double()).sum()
        (total + weight * (alpha * b1 + beta * z1 + 2.0 * alpha * b2 + 0.5 * beta * z2)).backward()
        return R.grad, D.grad, torch.stack([alpha * b1, beta * z1, alpha * b2, beta * z2]).detach().cpu().view(2, 2)
    R, D, want = in_64(refs, 1.0)
    R0, _, _ = in_64(plain, 0.0)
    near = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert near(R0, R) > 1e-2
    for got, ref in ((torch.cat(g1), R), (torch.cat(g1), D), (torch.stack(losses).cpu(), want)):
        assert near(got, ref) < 1e-4
    for b, ref, bare in zip(blocks, refs, plain):
        L = b.layer
        for i, (got, w) in enumerate(zip((b.dw_norm, L.dw_router, L.dw_gate, L.dw_up, L.dw_down), ref)):
            assert near(got, w.grad) < 1e-4, i
        assert all(near(bare[i].grad, ref[i].grad) > 1e-2 for i in (0, 1))


@pytest.mark.parametrize("mb,slots", [(64, 3), (128, 1)])
def test_layers_that_checkpoint_with_a_ring_backward(mb, slots):
    """Two layers that share ab and h, whose backward goes through a ring: both unpack their checkpoint into the shared
    buffers.  The gradients are the bytes of the ring's and of the one-launch backward on what the checkpoints stand
    for, and of the backward that reads the checkpoint itself."""
    _log("ring checkpoint", mb, slots)
    d, I, E = 128, 192, 8
    ring = dict(minibatch_rows=mb, bwd_ring_bytes=(64 * E + 64) * d * 2 + 768 + slots * mb * (2 * d + 2 * I) * 2)
    A, dout = _layer("bf16", 3, checkpoint=True, **ring)
    B, _ = _layer("bf16", 4, checkpoint=True, scratch=A, **ring)
    A.forward()
    B.forward()                                # ab and h now hold B's
    for L in (B, A):
        L.backward(dout)
    got = [_grads(L) for L in (A, B)]
    for L, seed, g in ((A, 3, got[0]), (B, 4, got[1])):
        L.check_status()
        for kw in (ring, {}):
            P, _ = _layer("bf16", seed, **kw)
            P.forward()
            mok.mok_checkpoint_unpack(P.cfg, P.offsets, L.ck_codes, L.ck_scales, P.ab, P.h)
            P.backward(dout)
            for i, (a, b) in enumerate(zip(g, _grads(P))):
                assert torch.equal(a, b), i
        C, _ = _layer("bf16", seed, checkpoint=True)
        C.forward()
        C.backward(dout)
        for i, (a, b) in enumerate(zip(g, _grads(C))):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("prec", ["f32", "bf16"])
def test_captured_step_with_balance_losses(prec):
    """Forward, losses and backward(balance=True) of two sources, captured: every replay gives the eager bytes for
    the rows that are there then."""
    _log("captured balance", prec)
    S, T, d, E, k, I = 2, 70, 128, 8, 2, 192
    gen, dt = _gen(5), torch.float32 if prec == "f32" else torch.bfloat16
    rnd = lambda *s, std=1.0: (std * torch.randn(*s, generator=gen)).to(DEV, dt)  # noqa: E731
    w = [rnd(E, d, std=d ** -0.5), rnd(E, I, d, std=d ** -0.5), rnd(E, I, d, std=d ** -0.5), rnd(E, d, I, std=I ** -0.5)]
    wn = (1 + 0.2 * torch.randn(d, generator=gen)).to(DEV, dt)

    def build():
        L = MoELayer(S, T, d, E, k, I, E, prec, S * T * k, 0, S, device=DEV, keep_logits=True, two_streams=False)
        b = MoEBlock(L, wn, "f32")
        b.set_inputs(w[0], None, torch.arange(E, dtype=torch.int32, device=DEV), *w[1:])
        return b
    rows = [[(2 * torch.randn(T, d, generator=gen)).to(DEV) for _ in range(S)] for _ in range(3)]
    dout, dl = [rnd(T, d) for _ in range(S)], torch.tensor([300.0, 20.0], device=DEV)

    def step(b, res):
        out = b.forward(res)
        loss = b.layer.balance_loss(1.0, 1.0)
        g = b.backward(dout, balance=True, d_loss=dl)
        return [*out, loss, *g, b.dw_norm, b.layer.dw_router, b.layer.dw_gate]
    eager, b = build(), build()
    slot = [t.clone() for t in rows[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b, slot)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b, slot)
    for i in (0, 1, 2, 0):
        for t, r in zip(slot, rows[i]):
            t.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, rows[i])
        torch.cuda.synchronize()
        for j, (a, c) in enumerate(zip(got, want)):
            assert torch.equal(a, c), (i, j)
        assert not torch.equal(want[3], torch.zeros_like(want[3]))
    b.layer.check_status()


def test_calls_without_rows():
    """No tokens: the norm, its backward and the decoder return empty rows, and the weight's gradient is zero."""
    from combine_router_top_expert_amd.block import RMSNorm
    n = RMSNorm(torch.ones(128, device=DEV, dtype=torch.bfloat16), 4, "bf16", "f32", mx=True)
    x = torch.zeros(0, 128, device=DEV, dtype=torch.bfloat16)
    n.dw.fill_(float("nan"))
    assert n.forward(x).shape == (0, 128) and n.backward(x).shape == (0, 128)
    torch.cuda.synchronize()
    assert (n.dw == 0).all()
    L, _ = _layer("bf16", 11, d=128, I=128)
    dec = L.decoder(4)
    assert dec(x).shape == (0, 128)
    torch.cuda.synchronize()
    dec.check_status()
