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
from test_gpu_train import DEV, U, _codes32, _e4m3, _gen, _log, _scales, _within, _words

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


# ------------------------------------------------------------------ AdamW
def _tiny_grads(n, seed):
    """Gradients whose second moments lie on both sides of 2^-102 and of
    2^-126, blocks of 32 of one size and blocks of all."""
    g = _gen(seed)
    size = 10.0 ** (torch.rand(n // 32, 1, generator=g).double() * 10 - 22)
    size = torch.where(torch.rand(n // 32, 1, generator=g) < 0.3,
                       10.0 ** (torch.rand(n // 32, 32, generator=g).double() * 10 - 22), size)
    return (torch.randn(n // 32, 32, generator=g).double() * size).float().view(-1)


def test_adamw_8bit_roots_of_tiny_second_moments():
    """Codes and scales of both moments, bit for bit against the formula with
    every operation rounded to fp32 by itself, for |g| down to 1e-22 and an
    eps that hides nothing of what is stored; gradients, then none (the roots
    decay by sqrt(beta2) and no faster)."""
    _log("adamw tiny 8 bits")
    n, seed = 32 * 500, 3
    grads = _tiny_grads(n, 5)
    z8 = lambda k: torch.zeros(k, dtype=torch.uint8, device=DEV)  # noqa: E731
    p, g = torch.zeros(n, device=DEV), grads.to(DEV)
    mc, vc, ms, vs = z8(n), z8(n), z8(n // 32), z8(n // 32)
    params = mok.make_params([mok.make_param(p=p, g=g, m=mc, v=vc, m_scale=ms, v_scale=vs)])
    f = lambda v: torch.tensor(v, dtype=torch.float32)  # noqa: E731
    b1, b2, c1, c2 = f(0.9), f(0.999), f(1 - 0.9), f(1 - 0.999)
    m, r = torch.zeros(n), torch.zeros(n)
    for step in range(1, 9):
        if step == 4:
            g.zero_()
            grads = torch.zeros(n)
        mok.mok_adamw(params, mok.make_adamw(1e-3, 0.9, 0.999, 1e-8, step=step, seed=seed))
        torch.cuda.synchronize()
        m, r = b1 * m + c1 * grads, torch.sqrt(b2 * (r * r) + c2 * (grads * grads))
        w = torch.from_numpy(_words(n, 0, step, seed)[0])
        for x, u, code, sc, name in ((m, w & 0xFFFF, mc, ms, "m"), (r, w >> 16, vc, vs, "v")):
            want, exps = _codes32(x, u.double() / 65536, x is r)
            assert torch.equal(sc.cpu(), exps), (step, name)
            assert torch.equal(code.cpu() & 0x7F, want), (step, name)
        m = _e4m3(mc).float() * _scales(ms, n).float()
        r = _e4m3(vc).float() * _scales(vs, n).float()
    assert float(r[r > 0].min()) < 2.0 ** -63


@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-15, 1e-12])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_update_of_tiny_second_moments(eps, bits):
    """The first step's update for the same gradients: m and v are products
    rounded to fp32 (v by up to half of fp32's smallest subnormal), root,
    correction, sum, reciprocal and the last two products add a few U: 16 U
    of the update and the root's share of v's own rounding."""
    _log("adamw tiny update", eps, bits)
    n = 32 * 500
    grads = _tiny_grads(n, 6)
    p, g = torch.zeros(n, device=DEV), grads.to(DEV)
    z = lambda k, dt: torch.zeros(k, dtype=dt, device=DEV)  # noqa: E731
    dt, sc = (torch.uint8, n // 32) if bits == 8 else (torch.float32, None)
    params = mok.make_params([mok.make_param(p=p, g=g, m=z(n, dt), v=z(n, dt),
                                             m_scale=sc and z(sc, dt), v_scale=sc and z(sc, dt))])
    mok.mok_adamw(params, mok.make_adamw(1.0, 0.9, 0.999, eps, step=1))
    torch.cuda.synchronize()
    f = lambda v: torch.tensor(v, dtype=torch.float32)  # noqa: E731
    m, v = (f(1 - 0.9) * grads).double(), (f(1 - 0.999) * (grads * grads)).double()   # as they are rounded
    keep = v > 0
    assert float(v[keep].min()) < 2.0 ** -126 and int((v[keep] > 2.0 ** -102).sum()) > n // 10
    want = -m / (1 - 0.9) / (v.sqrt() / math.sqrt(1 - 0.999) + eps)
    _within(p.cpu()[keep], want[keep], 16 * U * want[keep].abs(), "p")


# ------------------------------------------------------------------ balance
def _balance_fwd(z, topk, k, beta, off=None):
    T, E = z.shape
    G = 1 if off is None else len(off) - 1
    cfg = mok.make_config(1, T, 64, E, k, 64, 1, "f32", 0)
    offd = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    bal = mok.make_balance(1.0, beta, 0 if off is None else G, offd)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    counts, n_tok, st = i32(G, E), i32(G + 2), i32(1)
    prob, loss = torch.zeros(G, E, device=DEV), torch.zeros(2, device=DEV)
    ws = torch.full((mok.mok_balance_ws_bytes(cfg, T, bal),), 0xFF, dtype=torch.uint8, device=DEV)
    mok.mok_balance_fwd(cfg, T, bal, z, topk, counts, prob, n_tok, loss, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return prob.cpu(), loss.cpu()


def test_balance_column_sums_of_many_rows():
    """A million equal rows: every lane adds the same value again and again,
    whose rounding then goes one way.  The mean is a single row's p but for
    32 additions in fp32 (31 U), a rounding to fp32 before and after two sums
    over waves (4 U) and the mean's own (U): 36 U."""
    T, E = 1 << 20, 512
    _log("balance many rows", T, E)
    row = torch.randn(1, E, generator=_gen(2)).to(DEV)
    one, _ = _balance_fwd(row, torch.zeros(1, 1, dtype=torch.int32, device=DEV), 1, 0.0)
    many, _ = _balance_fwd(row.expand(T, E).contiguous(), torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1, 0.0)
    _within(many, one.double(), 36 * U * one.double(), "prob")


@pytest.mark.parametrize("T, off", [(200, None), (5000, None), (5000, [0, 100, 4990])], ids=str)
def test_balance_z_loss_of_large_logits(T, off):
    """lse^2 = 1.6e37 in every row: the mean is an fp32 value though the sum
    over a chunk is not.  lse is off by 2 U, its square by 4 U, and the loss
    is rounded once."""
    _log("balance large lse", T, off)
    E = 8
    z = torch.full((T, E), 4e18, device=DEV)
    _, loss = _balance_fwd(z, torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1, 1.0, off)
    want = (z[0, 0].double().cpu() + math.log(E)) ** 2
    _within(loss[1], want, 6 * U * want, "z-loss")
