"""The training entry points on the GPU against plain forms in 64 bits:
balance loss with counts and gradient, the router's logits, the router
projection's backward, the global gradient norm, AdamW with 32- and 8-bit
moments, and a training step that runs them together.

Tolerances (u = 2^-24, half a step of fp32):
  * a probability: the argument z - max is rounded once (u |z - max|), expf is
    good to 2 ulp (4 u), the sum of E positive terms to its depth (a lane's 8
    values and 6 exchanges: 14 u), reciprocal and product to 3 u.  With
    |z - max| <= 40 here: 61 u, taken as 64 u;
  * the gradient p ((w - sum p w) + c lse): the terms |w| and sum p|w| carry
    the error of p (64 u) and of their own sums and products (16 u), lse that
    of the sum of exponentials (24 u absolute) and a logf and an add (4 u
    |lse|): bound 96 u p (|w| + sum p|w|) * 2 + 96 u p |c| (1 + |lse|);
  * losses and mean probabilities are sums of positive terms: 64 u from p, u
    per row that a lane adds within a chunk and one rounding;
  * matrix products: n terms give at most (n + 2) u sum |a||b|, a result in
    bf16 half a step (2^-8 |ref|) more; where fp32 operands are split into
    bf16 parts, 2^-16 sum |a||b| (two parts, bf16 results) or 2^-23 (three);
  * AdamW, element by element: m and v are one product, one fused
    multiply-add, a scaled gradient and constants rounded to fp32 (8 u of the
    summed magnitudes); p 4 u |p| + 24 u |update|.
"""
import math

import numpy as np
import pytest
import torch

import combine_router_top_expert_amd as mok
from combine_router_top_expert_amd import synth
from combine_router_top_expert_amd.layer import MoELayer
from combine_router_top_expert_amd.optim import AdamW

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def _log(*a):
    print("[train]", *a, flush=True)


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _within(got, ref, bound, what=""):
    """|got - ref| <= bound element by element (both NaN counts as equal)."""
    got, ref = got.detach().cpu().double(), ref.double()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(ref)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    over = ~same & ~((got - ref).abs() <= bound)
    if over.any():
        i = int(torch.nonzero(over.reshape(-1))[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} off, first at {i}: "
                             f"{got.reshape(-1)[i]} against {ref.reshape(-1)[i]} "
                             f"(bound {bound.reshape(-1)[i]})")


# ------------------------------------------------------------------ balance
def _balance_ref(z, topk, E, k, alpha, beta, off, mask, d_loss, dz0):
    """Definition in 64 bits: losses, counts, prob, n_tok, d_logits and its error bound."""
    z = z.double()
    T = z.shape[0]
    off = [0, T] if off is None else off
    G = len(off) - 1
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    keep = keep & (z != -math.inf).any(1)
    rows = [torch.arange(off[g], off[g + 1])[keep[off[g]:off[g + 1]]] for g in range(G)]
    n = [len(r) for r in rows]
    N, Gp = sum(n), sum(x > 0 for x in n)
    counts, prob = torch.zeros(G, E, dtype=torch.int64), torch.zeros(G, E, dtype=torch.float64)
    dz, bound = dz0.double().clone(), torch.zeros(T, E, dtype=torch.float64)
    if T:
        dz[off[0]:off[G]] = 0
    loss = torch.zeros(2, dtype=torch.float64)
    for g in range(G):
        r = rows[g]
        if not n[g]:
            continue
        lse = torch.logsumexp(z[r], 1)
        p = torch.softmax(z[r], 1)
        ids = topk[r].reshape(-1).long()
        counts[g] = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        f = counts[g].double() * E / (k * n[g])
        prob[g] = p.mean(0)
        loss[0] += alpha * (f * prob[g]).sum() / Gp
        loss[1] += beta * (lse * lse).sum() / N
        w, c = alpha * d_loss[0] * f / (n[g] * Gp), 2 * beta * d_loss[1] / N
        dz[r] = p * (w - (p @ w)[:, None]) + p * (c * lse)[:, None]
        wc = (w - w.mean()).abs()
        bound[r] = 192 * U * p * (wc + (p @ wc)[:, None]) + 96 * U * p * abs(c) * (1 + lse.abs())[:, None]
    return loss, counts, prob, n + [N, Gp], dz, bound


def _balance_run(z, topk, E, k, alpha, beta, off, mask, d_loss, dz0, shift=0, inplace=False):
    T = z.shape[0]
    cfg = mok.make_config(1, T, 64, E, k, 64, 1, "f32", 0)

    def put(t):  # `shift` elements into an allocation: rows that do not start on 16 bytes
        buf = torch.zeros(t.numel() + shift, dtype=t.dtype, device=DEV)
        v = buf[shift:].view(t.shape)
        v.copy_(t)
        return v
    zd, dz = put(z), put(dz0)
    td = topk.to(DEV)
    offd = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    md = None if mask is None else mask.to(DEV)
    G = 1 if off is None else len(off) - 1
    bal = mok.make_balance(alpha, beta, 0 if off is None else G, offd, md)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    counts = torch.full((G, E), -7, dtype=torch.int32, device=DEV)
    prob, loss = nan(G, E), nan(2)
    n_tok = torch.full((G + 2,), -7, dtype=torch.int32, device=DEV)
    ws = torch.full((mok.mok_balance_ws_bytes(cfg, T, bal),), 0xFF, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dl = None if d_loss is None else torch.tensor(d_loss, dtype=torch.float32, device=DEV)
    mok.mok_balance_fwd(cfg, T, bal, zd, td, counts, prob, n_tok, loss, ws, st)
    if inplace:
        dz = zd
    mok.mok_balance_bwd(cfg, T, bal, zd, counts, n_tok, dl, dz, st)
    torch.cuda.synchronize()
    return loss.cpu(), counts.cpu(), prob.cpu(), n_tok.cpu(), dz.cpu(), int(st.item())


def _logits(T, E, k, seed, dead=0):
    g = _gen(seed)
    z = 2 * torch.randn(T, E, generator=g)
    if dead:
        z[:, torch.randperm(E, generator=g)[:dead]] = -math.inf
    topk = torch.topk(z, k, dim=1).indices.to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    return z, topk


BALANCE = [
    # T, E, k, offsets, masked share, dead experts
    (1, 1, 1, None, 0, 0),
    (1, 8, 2, None, 0, 0),
    (512, 8, 2, None, 0, 0),
    (3, 512, 16, None, 0, 100),
    (257, 511, 3, None, 0.3, 0),
    (1000, 64, 6, [0, 1, 1, 500, 963], 0.1, 3),
    (333, 61, 5, [2, 100, 101, 102, 333], 0.5, 0),
    (700, 260, 8, [0, 350, 700], 0, 0),
    (90, 2, 1, [0, 45, 90], 0, 0),
    (200, 3, 2, [10, 10, 10, 190], 0.9, 0),
    (4097, 256, 8, None, 0, 0),
    (64, 5, 1, list(range(65)), 0.2, 0),
    (130, 100, 4, [0, 130], 0, 0),
    (130, 33, 16, None, 0.2, 0),
    (100, 17, 2, None, 0, 0),
    # many chunks and groups: empty groups at both ends and between, groups of one row, one long
    (3000, 256, 8, [0, 0, 0, 1, 2, 17, 17, 2900, 2990, 2990], 0.1, 0),
    (2500, 512, 2, [3] + list(range(3, 2400, 7)) + [2499], 0, 0),
    (40000, 16, 4, [0, 39999, 39999, 40000], 0, 0),
    # many rows: two to a wave where 33 to 64 units of 16 bytes hold one
    (65537, 132, 4, [5, 5, 21, 30000, 65530], 0.1, 7),
    (65600, 256, 2, None, 0, 0),
]


@pytest.mark.parametrize("case", BALANCE, ids=str)
@pytest.mark.parametrize("shift", [0, 1])
def test_balance_against_definition(case, shift):
    T, E, k, off, masked, dead = case
    _log("balance", case, shift)
    z, topk = _logits(T, E, k, seed=T * 1000 + E, dead=dead)
    mask = (torch.rand(T, generator=_gen(3)) >= masked).to(torch.uint8) if masked else None
    if mask is not None:  # what is masked is never used
        z[mask == 0] = float("nan")
    dz0 = torch.full((T, E), 7.0)
    d_loss = [1.5, -0.75]
    ref = _balance_ref(z, topk, E, k, 1e-2, 1e-3, off, mask, d_loss, dz0)
    got = _balance_run(z, topk, E, k, 1e-2, 1e-3, off, mask, d_loss, dz0, shift)
    assert got[5] == 0
    assert torch.equal(got[1].long(), ref[1])
    assert got[3].tolist() == ref[3]
    most = max([b - a for a, b in zip(off, off[1:])] if off else [T])
    sums = (64 + min(most, 256) + 2) * U      # a chunk adds at most 256 rows per lane here
    _within(got[2], ref[2], sums * ref[2], "prob")
    lse2 = 2 * (28 * U) + sums                # lse^2: twice the relative error of lse >= 1, here
    _within(got[0][:1], ref[0][:1], sums * ref[0][:1], "balance loss")
    _within(got[0][1:], ref[0][1:], lse2 * (ref[0][1:] + 1e-3), "z-loss")
    _within(got[4], ref[4], ref[5], "d_logits")


def test_balance_default_weights_and_in_place():
    """d_loss NULL is ones; d_logits may overwrite the logits."""
    T, E, k = 301, 48, 4
    _log("balance in place")
    z, topk = _logits(T, E, k, seed=5)
    for inplace in (False, True):
        ref = _balance_ref(z, topk, E, k, 0.5, 0.25, None, None, [1.0, 1.0], torch.zeros(T, E))
        got = _balance_run(z, topk, E, k, 0.5, 0.25, None, None, None, torch.zeros(T, E), inplace=inplace)
        _within(got[4], ref[4], ref[5], "d_logits")


@pytest.mark.parametrize("groups", [None, [0, 0], [0, 40, 40]], ids=str)
def test_balance_nothing_counts(groups):
    """No tokens, only empty groups, or every row masked: zeros, no NaN."""
    _log("balance empty", groups)
    T, E, k = (0 if groups != [0, 40, 40] else 40), 6, 2
    z, topk = _logits(T, E, k, seed=1)
    mask = torch.zeros(T, dtype=torch.uint8) if T else None
    got = _balance_run(z, topk, E, k, 1.0, 1.0, groups, mask, [1.0, 1.0], torch.full((T, E), 3.0))
    assert got[0].tolist() == [0.0, 0.0] and not got[1].any() and not got[2].any()
    assert not got[3].any() and not got[4].any() and got[5] == 0


def test_balance_rows_of_minus_infinity_and_nan():
    """A row of -inf does not count; a NaN or +inf logit of a counted row
    reaches its losses and gradient (also in a row of NaN alone)."""
    _log("balance inf/nan")
    T, E, k = 20, 8, 2
    z, topk = _logits(T, E, k, seed=2)
    z[3] = -math.inf
    ref = _balance_ref(z, topk, E, k, 1e-2, 1e-3, None, None, [1.0, 1.0], torch.zeros(T, E))
    got = _balance_run(z, topk, E, k, 1e-2, 1e-3, None, None, [1.0, 1.0], torch.full((T, E), 9.0))
    assert got[3].tolist() == [T - 1, T - 1, 1] and torch.equal(got[1].long(), ref[1])
    _within(got[4], ref[4], ref[5], "d_logits")
    assert not got[4][3].any()
    for bad in (float("nan"), math.inf):
        zb = z.clone()
        zb[5, 1] = bad
        got = _balance_run(zb, topk, E, k, 1e-2, 1e-3, None, None, [1.0, 1.0], torch.zeros(T, E))
        assert torch.isnan(got[0]).all() and torch.isnan(got[4][5]).all()
        assert torch.isfinite(got[4][6]).all()
    zb = z.clone()
    zb[5] = float("nan")
    got = _balance_run(zb, topk, E, k, 1e-2, 1e-3, None, None, [1.0, 1.0], torch.zeros(T, E))
    assert got[3][0] == T - 1 and torch.isnan(got[0]).all()


@pytest.mark.parametrize("E", [8, 60, 256])
def test_balance_rows_at_the_ends_of_the_range(E):
    """Rows whose logits are all, or but for some, a type's lowest value (a
    finite mask), and rows near the largest: maximum times log2 e passes
    fp32's range there.  The z-loss weight is zero (lse^2 is not finite)."""
    _log("balance ends", E)
    T, k = 90, 2
    z, topk = _logits(T, E, k, seed=6)
    low = [torch.finfo(t).min for t in (torch.float32, torch.bfloat16, torch.float16)]
    for i, v in enumerate(low + [3.0e38, torch.finfo(torch.float32).max]):
        z[10 * i] = v
        z[10 * i + 1, : E // 2] = v
        z[10 * i + 2, 1:] = v
    z[70], z[70, 3] = low[0], low[0] / 2
    z[71], z[71, ::2] = 3.0e38, torch.nextafter(torch.tensor(3.0e38), torch.tensor(0.0))
    for i, v in enumerate((-1e9, 1e9, -1e7, 3e7, -1e12, 1e20)):
        z[72 + i] += v
    ref = _balance_ref(z, topk, E, k, 1e-2, 0.0, [0, 40, T], None, [1.0, 1.0], torch.zeros(T, E))
    got = _balance_run(z, topk, E, k, 1e-2, 0.0, [0, 40, T], None, [1.0, 1.0], torch.full((T, E), 9.0))
    assert got[5] == 0 and got[3].tolist() == ref[3] and torch.equal(got[1].long(), ref[1])
    # p: 2^-22 of itself (exponential, reciprocal, the exponent's rounding up to
    # 2^-24 of 25 beyond which p is below 2^-36 of the row), sums of E terms
    _within(got[2], ref[2], 64 * U * ref[2] + 2.0 ** -36, "prob")
    _within(got[0], ref[0], 64 * U * ref[0].abs() + 1e-9, "loss")
    _within(got[4], ref[4], ref[5] + 2.0 ** -36, "d_logits")


def test_balance_bad_ids_and_offsets_are_latched():
    _log("balance latches")
    T, E, k = 50, 8, 2
    z, topk = _logits(T, E, k, seed=4)
    bad = topk.clone()
    bad[3, 0], bad[7, 1], bad[9] = -1, E, topk[9, 0]      # and one expert twice in a row
    ref = _balance_ref(z, bad, E, k, 1e-2, 1e-3, None, None, [1.0, 1.0], torch.zeros(T, E))
    got = _balance_run(z, bad, E, k, 1e-2, 1e-3, None, None, [1.0, 1.0], torch.zeros(T, E))
    assert got[5] == -6 and torch.equal(got[1].long(), ref[1])
    for off in ([0, 30, 20, 50], [0, 20, 51], [-1, 20, 50], [0, 51], [50, 0]):
        got = _balance_run(z, topk, E, k, 1e-2, 1e-3, off, None, [1.0, 1.0], torch.full((T, E), 3.0))
        assert got[5] == -8
        assert not got[0].any() and not got[1].any() and not got[2].any() and not got[3].any()
        assert (got[4] == 3.0).all()


def test_balance_gradient_against_differences():
    """The losses along a direction: (L(z + h v) - L(z - h v)) / 2h = <dz, v>.
    The losses are fp32 sums good to about 80 u; with h = 2^-6 that is 80 u
    |L| / h, and the third derivative leaves h^2 (|v| <= 1, all factors of
    order L)."""
    _log("balance differences")
    T, E, k, h = 128, 16, 2, 2.0 ** -6
    z, topk = _logits(T, E, k, seed=8)
    v = torch.rand(T, E, generator=_gen(9)) * 2 - 1
    off = [0, 50, 128]
    dz = _balance_run(z, topk, E, k, 1.0, 0.1, off, None, [1.0, 1.0], torch.zeros(T, E))[4].double()
    up, dn = (_balance_run(z + s * h * v, topk, E, k, 1.0, 0.1, off, None, None, torch.zeros(T, E))[0].double().sum()
              for s in (1, -1))
    slope = float((up - dn) / (2 * h))
    assert abs(slope - float((dz * v.double()).sum())) <= 80 * U * float(up) / h + h * h * float(up)


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("case", [("f32", 70, 128, 3, 2), ("bf16", 129, 64, 1, 1), ("bf16", 300, 256, 61, 5),
                                  ("bf16", 33, 256, 512, 16), ("f32", 1, 64, 8, 2)], ids=str)
def test_route_logits(case):
    """Same routing bytes as mok_route; the logits of the fp32 chain (d
    fused multiply-adds and the bias: at most (d + 1) u sum |x||w|)."""
    prec, T, d, E, k = case
    _log("logits", case)
    dt = torch.float32 if prec == "f32" else torch.bfloat16
    g = _gen(T + E)
    x, w, b = (torch.randn(T, d, generator=g).to(dt), torch.randn(E, d, generator=g).to(dt),
               torch.randn(E, generator=g))
    cfg = mok.make_config(1, T, d, E, k, 64, 1, prec, 0)
    out = []
    for keep in (False, True):
        idx = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        gate = torch.full((T, k), float("nan"), device=DEV)
        z = torch.full((T, E), float("nan"), device=DEV) if keep else None
        mok.mok_route_logits(cfg, T, x.to(DEV), w.to(DEV), b.to(DEV), idx, gate, z)
        torch.cuda.synchronize()
        out.append((idx.cpu(), gate.cpu(), z))
    plain = (torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV))
    mok.mok_route(cfg, T, x.to(DEV), w.to(DEV), b.to(DEV), *plain)
    for idx, gate, _ in out:
        assert torch.equal(idx, plain[0].cpu()) and torch.equal(gate, plain[1].cpu())
    z = out[1][2].cpu()
    ref = x.double() @ w.double().t() + b.double()
    _within(z, ref, (d + 1) * U * (x.double().abs() @ w.double().abs().t() + b.double().abs()), "logits")
    assert torch.equal(torch.gather(z, 1, out[1][0].long()), torch.sort(z, 1, descending=True).values[:, :k])


ROUTER = [
    # prec, S, own_lo, own_n, T_src, d, E
    ("f32", 1, 0, 1, 512, 256, 8),
    ("f32", 3, 1, 2, 37, 192, 61),
    ("f32", 1, 0, 1, 1, 64, 1),
    ("bf16", 1, 0, 1, 1, 64, 1),
    ("bf16", 4, 1, 2, 65, 128, 64),
    ("bf16", 1, 0, 1, 700, 320, 256),
    ("bf16", 2, 0, 2, 1000, 1024, 31),
    ("bf16", 1, 0, 1, 129, 64, 512),
    ("bf16", 1, 0, 1, 128, 128, 130),
    ("bf16", 2, 0, 2, 16, 64, 65),
    ("bf16", 1, 0, 1, 64, 192, 300),
    ("bf16", 3, 0, 3, 8192, 128, 192),
    ("bf16", 8, 0, 8, 3, 448, 200),
    ("bf16", 1, 0, 1, 5000, 128, 100),
    ("bf16", 1, 0, 1, 260, 7168, 72),
]


@pytest.mark.parametrize("case", ROUTER, ids=str)
@pytest.mark.parametrize("add", [False, True])
def test_router_bwd(case, add):
    prec, S, lo, n, T_src, d, E = case
    _log("router_bwd", case, add)
    dt = torch.float32 if prec == "f32" else torch.bfloat16
    g = _gen(d + E)
    T = n * T_src
    dz = torch.randn(T, E, generator=g) * torch.exp(2 * torch.randn(T, E, generator=g)) * 1e-4
    xs = [torch.randn(T_src, d, generator=g).to(dt) for _ in range(S)]
    w = torch.randn(E, d, generator=g).to(dt)
    dx0 = [torch.randn(T_src, d, generator=g).to(dt) for _ in range(S)]
    dw0, db0 = torch.randn(E, d, generator=g), torch.randn(E, generator=g)
    cfg = mok.make_config(S, T_src, d, E, 1, 64, 1, prec, 0)
    dx, dw, db = [t.to(DEV) for t in dx0], dw0.to(DEV), db0.to(DEV)
    ws = torch.full((mok.mok_router_bwd_ws_bytes(cfg, n),), 0xFF, dtype=torch.uint8, device=DEV)
    mok.mok_router_bwd(cfg, lo, n, dz.to(DEV), [t.to(DEV) for t in xs], w.to(DEV), dx, dw, db, add, ws)
    torch.cuda.synchronize()
    zd, xd, wd = dz.double(), torch.cat(xs[lo:lo + n]).double(), w.double()
    base = 1.0 if add else 0.0
    mag_x, mag_w = zd.abs() @ wd.abs(), zd.abs().t() @ xd.abs()
    ref = zd @ wd + base * torch.cat(dx0[lo:lo + n]).double()
    half = 0.0 if prec == "f32" else 2.0 ** -8
    split = 0.0 if prec == "f32" else 2.0 ** -16
    _within(torch.cat([dx[s].cpu() for s in range(lo, lo + n)]), ref,
            ((E + 2) * U + split) * mag_x + (half + 2 * U) * ref.abs() + U * mag_x, "d_x")
    for s in range(S):  # other sources' buffers are not touched
        if not lo <= s < lo + n:
            assert torch.equal(dx[s].cpu(), dx0[s])
    refw = zd.t() @ xd + base * dw0.double()
    _within(dw, refw, ((T + 2) * U + 2 * U) * mag_w + 2 * U * refw.abs(), "dw_router")
    refb = zd.sum(0) + base * db0.double()
    _within(db, refb, 2 * U * (zd.abs().sum(0) + refb.abs()), "d_bias")


def test_router_bwd_parts_and_repeat():
    """Any of the three outputs may be left out; the same call gives the same
    bytes; no own rows leave zeros, or what was there."""
    _log("router_bwd parts")
    S, T_src, d, E = 2, 600, 256, 40
    g = _gen(1)
    dz = torch.randn(S * T_src, E, generator=g).to(DEV)
    xs = [torch.randn(T_src, d, generator=g).bfloat16().to(DEV) for _ in range(S)]
    w = torch.randn(E, d, generator=g).bfloat16().to(DEV)
    cfg = mok.make_config(S, T_src, d, E, 1, 64, 1, "bf16", 0)
    ws = torch.full((mok.mok_router_bwd_ws_bytes(cfg, S),), 0xFF, dtype=torch.uint8, device=DEV)

    def run(dx=True, dw=True, db=True):
        o = ([torch.full((T_src, d), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(S)],
             torch.full((E, d), 5.0, device=DEV), torch.full((E,), 5.0, device=DEV))
        mok.mok_router_bwd(cfg, 0, S, dz, xs, w, o[0] if dx else None, o[1] if dw else None,
                           o[2] if db else None, False, ws)
        torch.cuda.synchronize()
        return o

    full = run()
    for dx, dw, db in ((True, True, True), (True, False, False), (False, True, False), (False, False, True),
                       (False, True, True)):
        o = run(dx, dw, db)
        for s in range(S):
            assert torch.equal(o[0][s], full[0][s] if dx else torch.full_like(o[0][s], 5.0))
        assert torch.equal(o[1], full[1] if dw else torch.full_like(o[1], 5.0))
        assert torch.equal(o[2], full[2] if db else torch.full_like(o[2], 5.0))
    for add in (False, True):
        dw, db = torch.full((E, d), 5.0, device=DEV), torch.full((E,), 5.0, device=DEV)
        mok.mok_router_bwd(cfg, 0, 0, None, None, None, None, dw, db, add, ws)
        torch.cuda.synchronize()
        assert (dw == (5.0 if add else 0.0)).all() and (db == (5.0 if add else 0.0)).all()


def test_router_bwd_non_finite_rows_stay_in_their_rows():
    """A token of NaN gradients spoils its own d_x row, and all of dw; a NaN
    weight row spoils d_x only."""
    _log("router_bwd nan")
    T, d, E = 100, 128, 8
    g = _gen(2)
    dz = torch.randn(T, E, generator=g)
    dz[17, 2] = float("nan")
    dz[40, 3] = math.inf
    x, w = torch.randn(T, d, generator=g).bfloat16(), torch.randn(E, d, generator=g).bfloat16()
    cfg = mok.make_config(1, T, d, E, 1, 64, 1, "bf16", 0)
    ws = torch.empty(mok.mok_router_bwd_ws_bytes(cfg, 1), dtype=torch.uint8, device=DEV)
    dx, dw = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV), torch.zeros(E, d, device=DEV)
    mok.mok_router_bwd(cfg, 0, 1, dz.to(DEV), [x.to(DEV)], w.to(DEV), [dx], dw, None, False, ws)
    torch.cuda.synchronize()
    ok = torch.ones(T, dtype=torch.bool)
    ok[17] = ok[40] = False
    assert torch.isfinite(dx.cpu()[ok].float()).all()
    assert torch.isnan(dx.cpu()[17].float()).all() and not torch.isfinite(dx.cpu()[40].float()).any()
    keep = [e for e in range(E) if e not in (2, 3)]
    assert torch.isfinite(dw.cpu()[keep]).all()
    assert torch.isnan(dw.cpu()[2]).all() and not torch.isfinite(dw.cpu()[3]).any()


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_grad_norm(dt):
    """Sums in 64 bits, one rounding to fp32 each for norm and factor; more
    tensors than a launch takes, empty and unaligned ones."""
    _log("norm", dt)
    g = _gen(6)
    sizes = [0, 1, 7, 8, 31, 2048, 8191, 8192, 8193, 100000] + [3 + 5 * i for i in range(95)] + [0]
    ts = []
    for i, n in enumerate(sizes):
        buf = torch.zeros(n + 3, dtype=dt, device=DEV)
        v = buf[i % 4:][:n] if n else buf[:0]
        v.copy_(torch.randn(n, generator=g))
        ts.append(v)
    for max_norm in (1.0, 1e6, 0.0):
        params = mok.make_params([mok.make_param(g=t) for t in ts])
        ws = torch.full((mok.mok_grad_norm_ws_bytes(params),), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.full((2,), -1.0, device=DEV)
        mok.mok_grad_norm(params, max_norm, out, ws)
        torch.cuda.synchronize()
        ref = math.sqrt(sum(float(t.double().square().sum()) for t in ts))
        want = min(1.0, max_norm / (ref + 1e-6)) if max_norm > 0 else 1.0
        assert abs(float(out[0]) - ref) <= 2 * U * ref
        assert abs(float(out[1]) - want) <= 4 * U * want


def test_grad_norm_extremes():
    """Values whose squares leave fp32's range, none at all, and non-finite ones."""
    _log("norm extremes")

    def run(ts, max_norm=1.0):
        params = mok.make_params([mok.make_param(g=t) for t in ts])
        ws = torch.empty(max(mok.mok_grad_norm_ws_bytes(params), 8), dtype=torch.uint8, device=DEV)
        out = torch.full((2,), -1.0, device=DEV)
        mok.mok_grad_norm(params, max_norm, out, ws)
        return out.cpu()
    big = torch.full((1000,), 1e25, device=DEV)
    assert abs(float(run([big])[0]) / (1e25 * math.sqrt(1000)) - 1) < 1e-6
    tiny = torch.full((1000,), 1e-30, device=DEV)
    assert abs(float(run([tiny])[0]) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6
    assert run([]).tolist() == [0.0, 1.0]
    for bad in (float("nan"), math.inf, -math.inf):
        t = torch.ones(3000, device=DEV)
        t[2999] = bad
        o = run([big, t])
        assert not math.isfinite(float(o[0])) and math.isnan(float(o[1]))
    o = run([torch.full((100,), 3e38, device=DEV)])    # the norm itself overflows
    assert math.isinf(float(o[0])) and math.isnan(float(o[1]))


# ------------------------------------------------------------------ AdamW
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8)
G64 = 0x9E3779B97F4A7C15
M64 = (1 << 64) - 1


def _mix(z):
    with np.errstate(over="ignore"):
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def _words(n, tensor, step, seed, start=0):
    """(w for the moments, w for p) of elements start .. start + n, as the header defines them."""
    one = lambda v: np.array([v & M64], dtype=np.uint64)  # noqa: E731
    key = int(_mix(one(int(_mix(one(seed + tensor))[0]) + step * G64))[0])
    i = np.arange(start, start + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = _mix(np.uint64(key) + (i // np.uint64(8) + np.uint64(1)) * np.uint64(G64))
    a, b, j = z & np.uint64(0xFFFFFFFF), z >> np.uint64(32), i % np.uint64(8)
    lim = np.uint64(0xFFFFFFFF)
    return ((a + j * b) & lim).astype(np.int64), ((b + j * a) & lim).astype(np.int64)


def _e4m3(code):
    return code.cpu().view(torch.float8_e4m3fn).double()


def _scales(s, n):
    return (2.0 ** (s.cpu().double() - 127)).repeat_interleave(32)[:n]


def _round_range(x, u, sh, eps):
    """Codes' values that rounding |x| 2^-sh by u may give with x off by eps |x|
    (and by 2^-20 of a code's step, the last bit kept below a subnormal code)."""
    out = []
    for sgn in (-1, 1):
        y = x.abs() * (1 + sgn * eps) * 2.0 ** -sh
        step = 2.0 ** (torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
        out.append((torch.floor(y / step + u + sgn * 2.0 ** -20) * step).clamp_max(448.0))
    return out


class _Case:
    """One tensor's state before a step, on the CPU."""

    def __init__(self, n, p_type, g_type, bits, seed, wd=0.1, shift=0):
        g = _gen(seed)
        rnd = lambda s: torch.randn(n, generator=g) * s  # noqa: E731
        self.n, self.bits, self.wd, self.p_type = n, bits, wd, p_type
        self.g = rnd(1e-2) * torch.exp(rnd(2.0))
        if n > 40:
            self.g[33:40] = 0.0
        if g_type == "bf16":
            self.g = self.g.bfloat16()
        p = rnd(0.1)
        self.master = p if p_type == "master" else None
        self.p = p if p_type == "f32" else p.bfloat16()
        m, r = rnd(1e-2) * torch.exp(rnd(2.0)), (rnd(1e-2) * torch.exp(rnd(2.0))).abs()
        self.ms = self.vs = None
        if bits == 8:
            blocks = (n + 31) // 32
            self.ms = torch.randint(110, 120, (blocks,), generator=g).to(torch.uint8)
            self.vs = torch.randint(110, 120, (blocks,), generator=g).to(torch.uint8)
            self.m = torch.randint(-126, 127, (n,), generator=g)
            self.m = torch.where(self.m < 0, 128 - self.m, self.m).to(torch.uint8)
            self.v = torch.randint(0, 127, (n,), generator=g).to(torch.uint8)
        else:
            self.m, self.v = m, r * r
        self.shift = shift

    def put(self, t):
        if t is None:
            return None
        buf = torch.zeros(t.numel() + self.shift, dtype=t.dtype, device=DEV)
        v = buf[self.shift:]
        v.copy_(t)
        return v

    def to_device(self):
        self.d = {k: self.put(getattr(self, k)) for k in ("p", "g", "master", "m", "v")}
        for k in ("ms", "vs"):
            t = getattr(self, k)
            self.d[k] = None if t is None else t.to(DEV)
        d = self.d
        return mok.make_param(p=d["p"], g=d["g"], m=d["m"], v=d["v"], master=d["master"], m_scale=d["ms"],
                              v_scale=d["vs"], weight_decay=self.wd)

    def check(self, tensor, step, seed, scale, random):
        n, h, d = self.n, HYPER, self.d
        g = self.g.double() * scale
        p0 = (self.p if self.master is None else self.master).double()
        if self.bits == 8:
            m0, v0 = _e4m3(self.m) * _scales(self.ms, n), (_e4m3(self.v) * _scales(self.vs, n)) ** 2
        else:
            m0, v0 = self.m.double(), self.v.double()
        m = h["beta1"] * m0 + (1 - h["beta1"]) * g
        v = h["beta2"] * v0 + (1 - h["beta2"]) * g * g
        c1, c2 = 1 - h["beta1"] ** step, 1 - h["beta2"] ** step
        den = v.sqrt() / math.sqrt(c2) + h["eps"]
        upd = h["lr"] / c1 * m / den
        p = p0 * (1 - h["lr"] * self.wd) - upd
        mag_m = h["beta1"] * m0.abs() + (1 - h["beta1"]) * g.abs()
        # the update's error: that of m relative to den, and 24 u of its own
        pb = 4 * U * p0.abs() + 24 * U * upd.abs() + h["lr"] / c1 * 8 * U * mag_m / den
        what = f"n={n} {self.p_type} bits={self.bits}"
        w, wp = (torch.from_numpy(t) for t in _words(n, tensor, step, seed))
        if self.p_type == "f32":
            _within(d["p"], p, pb, "p " + what)
        else:
            if self.master is not None:
                _within(d["master"], p, pb, "master " + what)
                assert torch.equal(d["p"].cpu(), d["master"].cpu().bfloat16())
            elif random:
                u = (wp >> 16).double() / 65536
                lo, hi = [], []
                for sgn, out in ((-1, lo), (1, hi)):
                    a = p.abs() + sgn * pb
                    ulp = 2.0 ** (torch.floor(torch.log2(a.clamp_min(1e-37))) - 7)
                    out.append(torch.floor(a / ulp + u) * ulp)
                got = d["p"].cpu().double().abs()
                assert ((got >= lo[0]) & (got <= hi[0])).all(), what
            else:
                _within(d["p"], p, 2.0 ** -8 * p.abs() + pb, "p " + what)
        if self.bits == 32:
            _within(d["m"], m, 8 * U * mag_m, "m " + what)
            _within(d["v"], v, 8 * U * v, "v " + what)
            return
        for val, code, sc, u, err in ((m, d["m"], d["ms"], (w & 0xFFFF).double() / 65536, 8 * U * mag_m),
                                      (v.sqrt(), d["v"], d["vs"], (w >> 16).double() / 65536, 8 * U * v.sqrt())):
            blocks = (n + 31) // 32
            a = torch.zeros(blocks * 32, dtype=torch.float64)
            a[:n] = val.abs()
            amax, eb = a.view(-1, 32).amax(1), 16 * U
            sh = sc.cpu().double() - 127
            top = amax > 0
            assert (amax[top] * (1 - eb) <= 448 * 2.0 ** sh[top]).all(), what            # it fits,
            assert (amax[top] * (1 + eb) > 448 * 2.0 ** (sh[top] - 1)).all(), what       # and no smaller one does
            rel = (err / val.abs().clamp_min(1e-300)).clamp_max(1.0)
            lo, hi = _round_range(val, u, sh.repeat_interleave(32)[:n], rel)
            got = _e4m3(code)
            assert ((got.abs() >= lo) & (got.abs() <= hi.clamp_min(2.0 ** -9 if val is not m else 0.0))).all(), what
            some = (val != 0) & (got != 0) & (val.abs() > err)
            assert torch.equal(torch.sign(got[some]), torch.sign(val[some])), what
        live = v.sqrt() > 1e-30
        assert (_e4m3(d["v"])[live] > 0).all(), what    # never a divisor of zero


ADAM_SIZES = [1, 5, 8, 31, 32, 33, 100, 2048, 2049, 8192, 30001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g_type", ["f32", "bf16"])
@pytest.mark.parametrize("p_type", ["f32", "bf16", "master"])
def test_adamw_one_step(p_type, g_type, bits):
    """Every size in one call, aligned and not, against the formula in 64 bits."""
    _log("adamw", p_type, g_type, bits)
    step, seed, scale = 7, 99, 0.375
    cases = [_Case(n, p_type, g_type, bits, 10 * i + s, wd=0.1 * (i % 3), shift=s)
             for i, n in enumerate(ADAM_SIZES) for s in (0, 1, 8)]
    params = mok.make_params([c.to_device() for c in cases])
    dev = torch.tensor([scale], device=DEV)
    random = p_type == "bf16" and bits == 8
    mok.mok_adamw(params, mok.make_adamw(**HYPER, step=step, seed=seed, dev_scale=dev, random_params=random))
    torch.cuda.synchronize()
    for t, c in enumerate(cases):
        c.check(t, step, seed, scale, random)


def _codes32(x, u, root):
    """E4M3 codes (without sign) and exponents of fp32 values in blocks of 32, each rounded down or up by its u."""
    b = x.double().abs().view(-1, 32)
    top = b.amax(1)
    sh = torch.ceil(torch.log2((top / 448).clamp_min(2.0 ** -127)))
    y = (b * torch.exp2(-sh)[:, None]).view(-1)
    q = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    val = torch.floor(y / q + u) * q
    if root:
        val = torch.where((y > 0) & (val < 2.0 ** -9), 2.0 ** -9, val)
    return val.to(torch.float8_e4m3fn).view(torch.uint8), (sh + 127).to(torch.uint8)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_moments_are_the_formula_in_32_bits(bits):
    """What a step stores of the moments, bit for bit against the formula with
    every product, sum and root rounded to fp32 by itself, over two steps."""
    _log("adamw bits", bits)
    n, step, seed, scale = 32 * 8000, 4, 21, 0.375
    c = _Case(n, "f32", "f32", bits, 5)
    c.g[33:40] = 1e-3
    params = mok.make_params([c.to_device()])
    f = lambda v: torch.tensor(v, dtype=torch.float32)  # noqa: E731
    b1, b2, c1, c2 = f(HYPER["beta1"]), f(HYPER["beta2"]), f(1 - HYPER["beta1"]), f(1 - HYPER["beta2"])
    gs = c.g * f(scale)
    if bits == 8:
        m = _e4m3(c.m).float() * _scales(c.ms, n).float()
        r = _e4m3(c.v).float() * _scales(c.vs, n).float()
    else:
        m, v = c.m, c.v
    for k in (step, step + 1):
        mok.mok_adamw(params, mok.make_adamw(**HYPER, step=k, seed=seed, grad_scale=scale))
        torch.cuda.synchronize()
        d = c.d
        if bits == 32:
            m, v = b1 * m + c1 * gs, b2 * v + c2 * (gs * gs)
            assert torch.equal(d["m"].cpu(), m) and torch.equal(d["v"].cpu(), v)
            continue
        m, r = b1 * m + c1 * gs, torch.sqrt(b2 * (r * r) + c2 * (gs * gs))
        w = torch.from_numpy(_words(n, 0, k, seed)[0])
        for x, u, code, sc in ((m, w & 0xFFFF, d["m"], d["ms"]), (r, w >> 16, d["v"], d["vs"])):
            want, exps = _codes32(x, u.double() / 65536, x is r)
            assert torch.equal(sc.cpu(), exps)
            assert torch.equal(code.cpu() & 0x7F, want)
            if x is m:
                live = want > 0
                assert torch.equal((code.cpu() >> 7)[live], (m < 0).to(torch.uint8)[live])
        m = _e4m3(d["m"]).float() * _scales(d["ms"], n).float()
        r = _e4m3(d["v"]).float() * _scales(d["vs"], n).float()


def test_adamw_many_tensors_of_mixed_kinds():
    """More tensors than one launch takes, kinds mixed, empty ones between."""
    _log("adamw mixed")
    kinds = [("f32", "f32", 32), ("bf16", "bf16", 8), ("master", "f32", 8), ("bf16", "f32", 32),
             ("f32", "bf16", 8)]
    cases = [_Case(0 if i % 11 == 5 else 17 * i + 1, *kinds[i % 5], seed=i) for i in range(131)]
    params = mok.make_params([c.to_device() for c in cases])
    mok.mok_adamw(params, mok.make_adamw(**HYPER, step=3, seed=1, grad_scale=2.0))
    torch.cuda.synchronize()
    for t, c in enumerate(cases):
        if c.n:
            c.check(t, 3, 1, 2.0, False)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_skips_on_a_nan_factor(bits):
    _log("adamw skip", bits)
    c = _Case(1000, "master", "f32", bits, 3)
    params = mok.make_params([c.to_device()])
    before = {k: None if t is None else t.clone() for k, t in c.d.items()}
    nan = torch.tensor([float("nan")], device=DEV)
    mok.mok_adamw(params, mok.make_adamw(**HYPER, step=1, dev_scale=nan))
    torch.cuda.synchronize()
    for k, t in c.d.items():
        assert t is None or torch.equal(t.view(torch.uint8), before[k].view(torch.uint8)), k


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_non_finite_gradients_stay_with_their_element(bits):
    _log("adamw non-finite", bits)
    n = 96
    c = _Case(n, "f32", "f32", bits, 4)
    c.g[5], c.g[40], c.g[70] = float("nan"), math.inf, -math.inf
    params = mok.make_params([c.to_device()])
    mok.mok_adamw(params, mok.make_adamw(**HYPER, step=1))
    torch.cuda.synchronize()
    bad = torch.zeros(n, dtype=torch.bool)
    bad[[5, 40, 70]] = True
    p = c.d["p"].cpu()
    assert torch.isnan(p[bad]).all() and torch.isfinite(p[~bad]).all()
    m = _e4m3(c.d["m"]) if bits == 8 else c.d["m"].cpu()
    assert not torch.isfinite(m[bad]).any() and torch.isfinite(m[~bad]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_from_zero_states(bits):
    """First steps from zeroed moments, zero gradients among them: an element
    that never saw a gradient only decays."""
    _log("adamw first", bits)
    n = 300
    g = torch.zeros(n, device=DEV)
    g[::3] = torch.randn(100, generator=_gen(1)).to(DEV)
    p = torch.ones(n, device=DEV)
    opt = AdamW([p], lr=1e-2, weight_decay=0.5, state_bits=bits)
    for _ in range(4):
        opt.step([g])
    torch.cuda.synchronize()
    idle = torch.ones(n, dtype=torch.bool)
    idle[::3] = False
    want = (1 - 1e-2 * 0.5) ** 4
    assert ((p.cpu()[idle] - want).abs() <= 16 * U).all()
    moved = (p.cpu()[~idle] - want).abs()
    assert (moved > 1e-3).all() and torch.isfinite(p).all()


def test_adamw_8bit_moments_follow_a_slow_average():
    """The mean of the random rounding: with a constant gradient, sqrt(v)
    from zero follows |g| sqrt(1 - beta2^t) though a step moves it by far less
    than half of one code.  Averages over 32768 elements; a single element
    spreads by about 1/6 of its value, the mean by less than 1e-3 of it, and
    rounding changes the mean of r^2 only by the spread's square: 6 %."""
    _log("adamw slow")
    n, steps, b2 = 32768, 300, 0.999
    g = torch.ones(n, device=DEV)
    opt = AdamW([torch.zeros(n, device=DEV)], state_bits=8, weight_decay=0.0)
    opt.bind([g])
    for _ in range(steps):
        opt.step()
    torch.cuda.synchronize()
    r = _e4m3(opt.v[0]) * _scales(opt.v_scale[0], n)
    want = math.sqrt(1 - b2 ** steps)
    assert abs(float(r.mean()) / want - 1) < 0.06
    m = _e4m3(opt.m[0]) * _scales(opt.m_scale[0], n)
    assert abs(float(m.mean()) - 1) < 0.01


@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_adamw_tiny_second_moments_with_tiny_eps(eps):
    """v down to fp32's subnormals where no eps hides it: the update from the
    moments that the step stored, in 64 bits."""
    _log("adamw tiny v", eps)
    n, step = 4096, 3
    gen = _gen(3)
    g = torch.randn(n, generator=gen) * 10.0 ** torch.linspace(-21, -16, n)
    g[g == 0] = 1e-19
    p, m, v = torch.zeros(n), 0.1 * g, 0.5 * g * g
    d = [t.to(DEV) for t in (p, g, m, v)]
    params = mok.make_params([mok.make_param(p=d[0], g=d[1], m=d[2], v=d[3])])
    mok.mok_adamw(params, mok.make_adamw(1.0, 0.9, 0.99, eps, step=step))
    torch.cuda.synchronize()
    m, v = d[2].cpu().double(), d[3].cpu().double()
    keep = v > 0
    assert int(keep.sum()) > n // 2 and float(v[keep].min()) < 2.0 ** -126
    want = -m / (1 - 0.9 ** step) / (v.sqrt() / math.sqrt(1 - 0.99 ** step) + eps)
    # root, product with the correction, sum, reciprocal, two products
    _within(d[0].cpu()[keep], want[keep], 16 * U * want[keep].abs(), "p")


def test_adamw_captured_steps_match_eager():
    """A captured step (norm, clip, update, step number and learning rate on
    the device) replayed with eager work in between equals eager steps, bit
    for bit."""
    _log("adamw graph")
    gen = _gen(12)
    base = [torch.randn(n, generator=gen).to(DEV, dt) for n, dt in
            ((5000, torch.bfloat16), (333, torch.float32), (64, torch.bfloat16))]
    grads = [[torch.randn(p.numel(), generator=gen).to(DEV) for p in base] for _ in range(4)]

    def make():
        ps = [p.clone() for p in base]
        return ps, AdamW(ps, lr=1e-2, state_bits=[8, 32, 8], max_norm=0.5, seed=5, capturable=True)
    eager, oe = make()
    for i, gs in enumerate(grads):
        oe.set_lr(1e-2 / (i + 1))
        oe.step(gs)
    torch.cuda.synchronize()
    graph, og = make()
    slot = [t.clone() for t in grads[0]]
    og.bind(slot)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        og.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        og.step()
    for i in range(1, 4):
        for s, t in zip(slot, grads[i]):
            s.copy_(t)
        og.set_lr(1e-2 / (i + 1))
        torch.cuda.synchronize()
        cg.replay()
        torch.cuda.synchronize()
    for a, b in zip(eager + oe.m + oe.v + [oe.norm], graph + og.m + og.v + [og.norm]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del cg


def test_balance_and_router_captured_match_eager():
    """Both entry points in one graph, replayed on changed logits."""
    _log("balance graph")
    T, E, k, d = 700, 40, 4, 128
    cfg = mok.make_config(1, T, d, E, k, 64, 1, "bf16", 0)
    z, topk = _logits(T, E, k, seed=3)
    zd, td = z.to(DEV), topk.to(DEV)
    off = torch.tensor([0, 100, 650], dtype=torch.int32, device=DEV)
    bal = mok.make_balance(1e-2, 1e-3, 2, off)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.randn(T, d, generator=_gen(1)).bfloat16().to(DEV)
    w = torch.randn(E, d, generator=_gen(2)).bfloat16().to(DEV)
    o = dict(counts=i32(2, E), prob=torch.zeros(2, E, device=DEV), n_tok=i32(4), loss=torch.zeros(2, device=DEV),
             dz=torch.zeros(T, E, device=DEV), dx=torch.zeros(T, d, dtype=torch.bfloat16, device=DEV),
             dw=torch.zeros(E, d, device=DEV), db=torch.zeros(E, device=DEV))
    ws = torch.empty(mok.mok_balance_ws_bytes(cfg, T, bal), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(mok.mok_router_bwd_ws_bytes(cfg, 1), dtype=torch.uint8, device=DEV)
    st = i32(1)

    def step():
        mok.mok_balance_fwd(cfg, T, bal, zd, td, o["counts"], o["prob"], o["n_tok"], o["loss"], ws, st)
        mok.mok_balance_bwd(cfg, T, bal, zd, o["counts"], o["n_tok"], None, o["dz"], st)
        mok.mok_router_bwd(cfg, 0, 1, o["dz"], [x], w, [o["dx"]], o["dw"], o["db"], False, ws2)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        step()
    for rep in range(3):
        zd.copy_(torch.randn(T, E, generator=_gen(20 + rep)))
        step()
        torch.cuda.synchronize()
        want = {n: t.clone() for n, t in o.items()}
        for t in o.values():
            t.fill_(9)
        o["dz"][650:] = want["dz"][650:]
        torch.cuda.synchronize()
        cg.replay()
        torch.cuda.synchronize()
        for n, t in o.items():
            assert torch.equal(t, want[n]), (rep, n)
    assert int(st.item()) == 0
    del cg


# ------------------------------------------------------------------ beyond 32 bits
def test_balance_beyond_32_bit_offsets():
    """More than 2^31 logits: counts and the last rows against the definition."""
    T, E, k = (1 << 22) + 1000, 512, 1
    _log("balance large", T, E)
    cfg = mok.make_config(1, T, 64, E, k, 64, 1, "f32", 0)
    z = torch.zeros(T, E, device=DEV)
    tail = torch.randn(1000, E, generator=_gen(1))
    z[-1000:] = tail.to(DEV)
    topk = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    topk[-1000:] = torch.argmax(tail, 1, keepdim=True).to(torch.int32).to(DEV)
    off = torch.tensor([0, T - 1000, T], dtype=torch.int32, device=DEV)
    bal = mok.make_balance(1.0, 1e-3, 2, off)
    counts, n_tok = torch.zeros(2, E, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    prob, loss = torch.zeros(2, E, device=DEV), torch.zeros(2, device=DEV)
    ws = torch.empty(mok.mok_balance_ws_bytes(cfg, T, bal), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    mok.mok_balance_fwd(cfg, T, bal, z, topk, counts, prob, n_tok, loss, ws, st)
    mok.mok_balance_bwd(cfg, T, bal, z, counts, n_tok, None, z, st)      # in place
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and n_tok.tolist() == [T - 1000, 1000, T, 2]
    assert int(counts[0, 0]) == T - 1000 and int(counts[0].sum()) == T - 1000
    d = tail.double()
    lse = torch.logsumexp(d, 1)
    p = torch.exp(d - lse[:, None])
    c = torch.bincount(torch.argmax(tail, 1), minlength=E).double()
    w = c * E / (1000.0 * 1000 * 2)
    assert torch.equal(counts[1].cpu().double(), c)
    want = p * (w - (p @ w)[:, None]) + p * (2e-3 / T * lse)[:, None]
    wc = (w - w.mean()).abs()
    _within(z[-1000:], want, 192 * U * p * (wc + (p @ wc)[:, None]) + 96 * U * p * 2e-3 / T * (1 + lse.abs())[:, None], "tail")
    _within(prob[1], p.mean(0), 400 * U * p.mean(0), "prob")


def test_router_bwd_beyond_32_bit_offsets():
    """More than 2^31 token values: the last rows of d_x, and dw and db of
    gradients that live in the last rows alone."""
    T, d, E = 300_100, 7168, 2
    _log("router large", T, d)
    cfg = mok.make_config(1, T, d, E, 1, 64, 1, "bf16", 0)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    dz = torch.zeros(T, E, device=DEV)
    g = _gen(4)
    xt, zt, w = (torch.randn(100, d, generator=g).bfloat16(), torch.randn(100, E, generator=g),
                 torch.randn(E, d, generator=g).bfloat16())
    x[-100:], dz[-100:] = xt.to(DEV), zt.to(DEV)
    dx = torch.full((T, d), 9.0, dtype=torch.bfloat16, device=DEV)
    dw, db = torch.empty(E, d, device=DEV), torch.empty(E, device=DEV)
    ws = torch.empty(mok.mok_router_bwd_ws_bytes(cfg, 1), dtype=torch.uint8, device=DEV)
    mok.mok_router_bwd(cfg, 0, 1, dz, [x], w.to(DEV), [dx], dw, db, False, ws)
    torch.cuda.synchronize()
    assert not dx[:-100].any()
    zd = zt.double()
    ref = zd @ w.double()
    _within(dx[-100:], ref, 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 4 * U) * (zd.abs() @ w.double().abs()), "d_x")
    refw = zd.t() @ xt.double()
    _within(dw, refw, 104 * U * (zd.abs().t() @ xt.double().abs()) + 2 * U * refw.abs(), "dw")
    _within(db, zd.sum(0), 2 * U * zd.abs().sum(0), "db")


def test_optimizer_beyond_32_bit_offsets():
    """One tensor of more than 2^31 elements, bf16 with 8-bit moments: its
    last elements (their random words count from the tensor's start), and its
    norm."""
    n, m = (1 << 31) + 77, 333
    _log("adamw large", n)
    p, g = torch.zeros(n, dtype=torch.bfloat16, device=DEV), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    codes = [torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((n + 31) // 32, dtype=torch.uint8, device=DEV) for _ in range(2)]
    gt = torch.randn(m, generator=_gen(9)).bfloat16()
    g[-m:] = gt.to(DEV)
    params = mok.make_params([mok.make_param(p=p, g=g, m=codes[0], v=codes[1], m_scale=scales[0], v_scale=scales[1])])
    out = torch.zeros(2, device=DEV)
    ws = torch.empty(mok.mok_grad_norm_ws_bytes(params), dtype=torch.uint8, device=DEV)
    mok.mok_grad_norm(params, 0.0, out, ws)
    mok.mok_adamw(params, mok.make_adamw(**HYPER, step=1, seed=5))
    torch.cuda.synchronize()
    norm = float(gt.double().norm())
    assert abs(float(out[0]) - norm) <= 2 * U * norm
    gd = gt.double()
    want = -HYPER["lr"] * gd / (gd.abs() + HYPER["eps"])   # the first step from zero
    _within(p[-m:], want, 2.0 ** -8 * want.abs() + 48 * U * want.abs(), "p")
    assert not p[:-m].any()
    w = torch.from_numpy(_words(m, 0, 1, 5, start=n - m)[0])
    for val, code, sc, u in ((0.1 * gd, codes[0], scales[0], (w & 0xFFFF).double() / 65536),
                             (math.sqrt(1e-3) * gd.abs(), codes[1], scales[1], (w >> 16).double() / 65536)):
        at = torch.arange(n - m, n)
        sh = sc.cpu()[at // 32].double() - 127
        lo, hi = _round_range(val, u, sh, torch.full((m,), 16 * U, dtype=torch.float64))
        got = _e4m3(code[-m:]).abs()
        assert ((got >= lo) & (got <= hi.clamp_min(2.0 ** -9))).all()


# ------------------------------------------------------------------ together
def test_training_steps_of_the_layer():
    """Forward with kept logits, balance loss, backward, its gradient added,
    clipped AdamW on every weight, the kept copies formed again: two steps in
    fp32 against torch autograd in 64 bits on the same (fixed) routing.  The
    layer's own fp32 gradients are good to about 1e-5 of the largest; the
    first Adam steps divide by |g| itself, so an element's change is off by
    that share of the step where its gradient is not tiny."""
    _log("training steps")
    w = synth.WORKLOADS["C1"].replace(S=2, T_src=96, d=64, E=8, k=2, I=64, own=[0, 1])
    S, T, d, E, k, I = w.S, w.T_src, w.d, w.E, w.k, w.I
    gen = _gen(31)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen) * std  # noqa: E731
    xs = [rnd(T, d) for _ in range(S)]
    W = dict(wr=rnd(E, d, std=d ** -0.5), wg=rnd(E, I, d, std=d ** -0.5), wu=rnd(E, I, d, std=d ** -0.5),
             wd=rnd(E, d, I, std=I ** -0.5))
    dout = [rnd(T, d, std=0.05) for _ in range(S)]
    alpha, beta, lr, wdec, max_norm = 0.5, 0.01, 1e-2, 0.1, 0.7
    off = [0, 50, 180]
    mask = torch.ones(S * T, dtype=torch.uint8)
    mask[10:20] = 0
    dev = {n: t.to(DEV) for n, t in W.items()}
    L = MoELayer(S, T, d, E, k, I, E, "f32", S * T * k, 0, S, device=DEV, keep_logits=True)
    L.set_inputs([x.to(DEV) for x in xs], dev["wr"], None, torch.arange(E, dtype=torch.int32, device=DEV),
                 dev["wg"], dev["wu"], dev["wd"])
    names = ["wr", "wg", "wu", "wd"]
    opt = AdamW([dev[n] for n in names], lr=lr, weight_decay=wdec, max_norm=max_norm)
    offd, maskd = torch.tensor(off, dtype=torch.int32, device=DEV), mask.to(DEV)
    ref = {n: t.double().requires_grad_() for n, t in W.items()}
    mom = {n: (torch.zeros_like(t), torch.zeros_like(t)) for n, t in ref.items()}
    X, D = torch.cat(xs).double(), torch.cat(dout).double()
    for step in (1, 2):
        L.forward()
        loss = L.balance_loss(alpha, beta, offd, maskd).clone()
        L.backward([t.to(DEV) for t in dout])
        L.balance_backward()
        opt.step([L.dw_router, L.dw_gate, L.dw_up, L.dw_down])
        L.update_weights()
        torch.cuda.synchronize()
        L.check_status()
        idx = L.topk_idx.view(S * T, k).cpu().long()
        xr = X.clone().requires_grad_()
        z = xr @ ref["wr"].t()
        gate = torch.softmax(torch.gather(z, 1, idx), 1)
        out = torch.zeros(S * T, d, dtype=torch.float64)
        for e in range(E):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            h = torch.nn.functional.silu(xr[t] @ ref["wg"][e].t()) * (xr[t] @ ref["wu"][e].t())
            out = out.index_add(0, t, gate[t, j, None] * (h @ ref["wd"][e].t()))
        lb, lz, N = 0.0, 0.0, int(mask[off[0]:off[-1]].sum())
        for a, b in zip(off, off[1:]):
            r = torch.arange(a, b)[mask[a:b] != 0]
            f = torch.bincount(idx[r].reshape(-1), minlength=E).double() * E / (k * len(r))
            lb = lb + alpha * (f * torch.softmax(z[r], 1).mean(0)).sum() / 2
            lz = lz + beta * torch.logsumexp(z[r], 1).square().sum() / N
        _within(loss, torch.stack([lb, lz]).detach(), 2e-5 * torch.stack([lb, lz]).detach().abs(), "losses")
        total = (out * D).sum() + lb + lz
        grads = dict(zip(names + ["x"], torch.autograd.grad(total, [ref[n] for n in names] + [xr])))
        got = dict(wr=L.dw_router, wg=L.dw_gate, wu=L.dw_up, wd=L.dw_down, x=torch.cat(L.d_x))
        for n, gr in grads.items():
            _within(got[n], gr, 2e-5 * step * float(gr.abs().max()), f"gradient {n}")
        norm = math.sqrt(sum(float(grads[n].square().sum()) for n in names))
        assert abs(float(opt.norm[0]) / norm - 1) < 1e-5
        s = min(1.0, max_norm / (norm + 1e-6))
        with torch.no_grad():
            for n in names:
                m, v = mom[n]
                g = grads[n] * s
                m.mul_(0.9).add_(0.1 * g)
                v.mul_(0.999).add_(0.001 * g * g)
                ref[n].mul_(1 - lr * wdec).sub_(
                    lr / (1 - 0.9 ** step) * m / ((v / (1 - 0.999 ** step)).sqrt() + 1e-8))
                plain = v.sqrt() > 1e-3 * v.sqrt().max()      # gradients that are not tiny
                off_by = (dev[n].cpu().double() - ref[n]).abs()
                assert float(off_by[plain].max()) <= 0.05 * lr, n
                ref[n].copy_(dev[n].cpu().double())


def test_bf16_layer_keeps_its_copies_in_step():
    """After an optimizer step and update_weights, the layer's results are
    those of a fresh layer with the new weights, byte for byte (bf16 with
    transposed copies, and MXFP8)."""
    for prec in ("bf16", "mxfp8"):
        _log("update_weights", prec)
        S, T, d, E, k, I = 1, 160, 128, 4, 2, 128
        gen = _gen(7)
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).bfloat16().to(DEV)  # noqa: E731
        x, wr, dout = rnd(T, d), rnd(E, d, std=0.1), rnd(T, d, std=0.1)
        ws = [rnd(E, I, d, std=0.1), rnd(E, I, d, std=0.1), rnd(E, d, I, std=0.1)]

        def layer():
            L = MoELayer(S, T, d, E, k, I, E, prec, T * k, 0, 1, device=DEV, keep_logits=True)
            L.set_inputs([x], wr, None, torch.arange(E, dtype=torch.int32, device=DEV), *ws)
            return L

        def step(L):
            L.forward()
            L.balance_loss(1e-2, 1e-3)
            L.backward([dout])
            L.balance_backward()
            torch.cuda.synchronize()
            L.check_status()
            return [t.clone() for t in (L.out[0], L.d_x[0], L.dw_router, L.dw_gate, L.dw_up, L.dw_down, L.logits)]
        L = layer()
        step(L)
        opt = AdamW([wr, *ws], lr=1e-2, state_bits=[32, 8, 8, 8], max_norm=1.0)
        opt.step([L.dw_router, L.dw_gate, L.dw_up, L.dw_down])
        L.update_weights()
        for a, b in zip(step(L), step(layer())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), prec


def test_optimizer_refuses_a_captured_step_with_a_host_number(monkeypatch):
    opt = AdamW([torch.zeros(8, device=DEV)])
    opt.bind([torch.zeros(8, device=DEV)])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="capturable"):
        opt.step()


def _balance_layer():
    S, T, d, E, k, I = 1, 300, 64, 8, 2, 64
    gen = _gen(13)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    L = MoELayer(S, T, d, E, k, I, E, "f32", T * k, 0, 1, device=DEV, keep_logits=True)
    L.set_inputs([rnd(T, d)], rnd(E, d), None, torch.arange(E, dtype=torch.int32, device=DEV), rnd(E, I, d),
                 rnd(E, I, d), rnd(E, d, I))
    dout = [rnd(T, d)]
    off = [torch.tensor(o, dtype=torch.int32, device=DEV) for o in ([0, 100, 300], [0, 50, 90, 300])]
    return L, dout, off


def test_training_calls_on_a_side_stream():
    """Balance loss, its gradient and a clipped step on a stream other than
    the current one, whose buffers are made by these calls, while the current
    stream is busy: the bytes of the same calls on the current stream."""
    _log("side stream")

    def run(side):
        L, dout, off = _balance_layer()
        w = [t.clone() for t in (L.w_router, L.w_gate)]
        opt = AdamW(w, max_norm=0.1, state_bits=[32, 8])
        L.forward()
        L.backward(dout)
        torch.cuda.synchronize()
        busy = torch.ones(1 << 26, device=DEV)
        if side is not None:
            for _ in range(20):
                busy.mul_(1.0)
        loss = [L.balance_loss(0.5, 0.01, o, stream=side).clone() if side is None else
                L.balance_loss(0.5, 0.01, o, stream=side) for o in off]
        L.balance_backward(stream=side)
        opt.step([L.dw_router, L.dw_gate], stream=side)
        torch.cuda.synchronize()
        L.check_status()
        return [t.clone() for t in (*loss, L.d_x[0], L.dw_router, *w)]
    for a, b in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(a, b)


def test_captured_balance_keeps_its_buffers():
    """A captured call replayed after calls with other numbers of groups."""
    _log("balance buffers")
    L, dout, off = _balance_layer()
    L.forward()
    L.balance_loss(0.5, 0.01, off[0])
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        loss = L.balance_loss(0.5, 0.01, off[0])
    for i in range(3):
        other = L.balance_loss(0.5, 0.01, off[1]).clone()
        junk = [torch.full((n,), float("nan"), device=DEV) for n in (2, 4, 16, 24, 1000)]
        cg.replay()
        torch.cuda.synchronize()
        assert all(bool(torch.isnan(j).all()) for j in junk)
        replayed = loss.clone()
        assert torch.equal(replayed, L.balance_loss(0.5, 0.01, off[0])), i
        assert torch.equal(other, L.balance_loss(0.5, 0.01, off[1])), i


def test_balance_backward_forgets_rows_of_earlier_groups():
    """Rows outside the groups of this call add nothing, though they were in
    those of the call before."""
    _log("balance rows outside")

    def run(offs):
        L, dout, _ = _balance_layer()
        L.forward()
        for o in offs:
            L.balance_loss(0.5, 0.01, torch.tensor(o, dtype=torch.int32, device=DEV))
            L.backward(dout)
            L.balance_backward()
        torch.cuda.synchronize()
        return L.d_x[0].clone(), L.dw_router.clone()
    for a, b in zip(run([[20, 120]]), run([[0, 300], [20, 120]])):
        assert torch.equal(a, b)
