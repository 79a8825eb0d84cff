"""The operators around the layer where element offsets pass 2^31 (and byte
offsets 2^32): rows that repeat, so that every row has to give the bytes of its
first copy, which the other tests hold against the formulas."""
import pytest
import torch

import combine_router_top_expert_amd as mok
from test_gpu_decode import _place, _ref, _routing, _run, _weights
from test_gpu_norm import _near
from test_gpu_train import DEV, U, _gen, _log

pytestmark = pytest.mark.gpu

BASE = 1000                                   # rows before they repeat


def _repeat(base, T):
    """base's rows again and again, T of them."""
    n = -(-T // base.shape[0])
    return base.repeat(n, *[1] * (base.dim() - 1))[:T].contiguous()


def _repeats(t, base, what):
    """Every row of t is the one BASE rows before it, and the first ones are base's."""
    a, b = t.view(torch.uint8), base.view(torch.uint8)
    assert torch.equal(a[:BASE], b[:BASE]), what
    for lo in range(BASE, a.shape[0], 16 * BASE):
        part = a[lo:lo + 16 * BASE]
        n = part.shape[0] // BASE * BASE
        assert bool((part[:n].view(-1, *b.shape) == b).all()), (what, lo)
        assert torch.equal(part[n:], b[:part.shape[0] - n]), (what, lo)


def test_norm():
    T, d = 133000, 16384                      # 2.18e9 elements
    _log("large norm", T, d)
    g = _gen(1)
    x, res = torch.randn(BASE, d, generator=g).to(DEV, torch.bfloat16), torch.randn(BASE, d, generator=g).to(DEV, torch.bfloat16)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV, torch.bfloat16)

    def run(n, x, res):
        cfg = mok.make_config(1, 1, d, 1, 1, 64, 1, "bf16", 0)
        new = lambda dt, *s: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
        r, y, c, s, rstd = new(x.dtype, n, d), new(x.dtype, n, d), new(torch.uint8, n, d), new(torch.uint8, n, d // 32), new(torch.float32, n)
        mok.mok_norm_fwd(cfg, n, x, res, w, 1e-6, r, y, c, s, rstd)
        dr, dw = new(x.dtype, n, d), new(torch.float32, d)
        mok.mok_norm_bwd(cfg, n, x, r, w, rstd, res, dr, None, dw, False,
                         new(torch.uint8, mok.mok_norm_bwd_ws_bytes(cfg, n)))
        torch.cuda.synchronize()
        return (r, y, c, s, rstd[:, None], dr), dw
    base, _ = run(BASE, x, res)
    got, dw = run(T, _repeat(x, T), _repeat(res, T))
    for i, (a, b) in enumerate(zip(got, base)):
        _repeats(a, a[:BASE].clone(), i)
        if i < 5:                             # (the backward of so few rows is another kernel)
            assert torch.equal(a[:BASE].view(torch.uint8), b.view(torch.uint8)), i
    # the weight's gradient of 133 copies, with test_gpu_norm's bound
    r, rstd = base[0].double(), base[4].double()
    t = x.double() * r * rstd
    want = 133 * t.sum(0)
    _near(dw, want, 133 * 72 * U * t.abs().sum(0) + 2 * U * want.abs(), "d_w")


def test_checkpoint():
    R, I = 800000, 1408                       # 2.25e9 elements of a | b
    _log("large checkpoint", R, I)
    g = _gen(2)
    ab = torch.randn(BASE, 2 * I, generator=g).to(DEV, torch.bfloat16)
    dh = torch.randn(BASE, I, generator=g).to(DEV, torch.bfloat16)

    def run(n, ab, dh):
        cfg = mok.make_config(1, 1, 64, 1, 1, I, 1, "bf16", n)
        off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        new = lambda dt, *s: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
        c, s, back, h = new(torch.uint8, n, 2 * I), new(torch.uint8, n, I // 16), new(ab.dtype, n, 2 * I), new(ab.dtype, n, I)
        mok.mok_checkpoint_pack(cfg, off, ab, c, s)
        mok.mok_checkpoint_unpack(cfg, off, c, s, back, h)
        dab = new(ab.dtype, n, 2 * I)
        mok.mok_checkpoint_swiglu_bwd(cfg, off, c, s, dh, I, dab, None)
        # dh in the first halves of dab's own rows
        own = new(ab.dtype, n, 2 * I)
        own[:, :I] = dh
        mok.mok_checkpoint_swiglu_bwd(cfg, off, c, s, own, 2 * I, own, None)
        torch.cuda.synchronize()
        return c, s, back, h, dab, own
    base = run(BASE, ab, dh)
    assert torch.equal(base[4], base[5])
    got = run(R, _repeat(ab, R), _repeat(dh, R))
    for i, (a, b) in enumerate(zip(got, base)):
        _repeats(a, b, i)


def test_decode():
    T, d, I, E, k, L = 280000, 1024, 1024, 8, 8, 8        # 2.24e6 items: 2.3e9 elements of h and of y
    _log("large decode", T, d, I, E, k, L)
    w, e2l = _weights(L, d, I, 3), _place(E, L, 1)
    topk, gate = _routing(BASE, E, k, 2)
    x = torch.randn(BASE, d, generator=_gen(4)).to(DEV, torch.bfloat16)
    out, st = _run(_repeat(x, T), None, _repeat(topk, T), _repeat(gate, T), e2l, w, d, I, L)
    assert st == 0
    ref, bound = _ref(x.double(), topk, gate, e2l, w, d, I)
    _near(out[:BASE], ref, bound, "out")
    _repeats(out, out[:BASE].clone(), "out")
