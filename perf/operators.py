"""The training-side operators of the MoE layer, as cases to be timed.

Four operators a training program calls around ``mok_layer_fwd`` /
``mok_layer_bwd``:

* ``balance``: the load-balance loss and the z-loss of the router's logits,
  the per-expert counts, and the gradient with respect to the logits
  (``mok_balance_fwd`` + ``mok_balance_bwd``);
* ``router``: the backward of the router projection for a dense gradient of
  the logits (``mok_router_bwd``): token gradient, router weight gradient,
  bias gradient;
* ``norm``: the global gradient norm and the clip factor over many tensors
  (``mok_grad_norm``);
* ``adamw``: one AdamW step over many tensors, moments in 32 bits or in MX
  blocks of 8 bits (``mok_adamw``).

``own`` false: their plain forms in elementary torch operations.  ``own``
true: the calls of this package.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32                                   # elements per shared exponent of an 8-bit moment
GOLD = -0x61C8864680B583EB                   # 0x9E3779B97F4A7C15 as a signed 64-bit number
MIX1 = -0x40A7B892E31B1A47                   # 0xBF58476D1CE4E5B9
MIX2 = -0x6B2FB644ECCEEE15                   # 0x94D049BB133111EB


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one step of the small fp32 layer (512 tokens, 8 experts, top-2): a call whose latency counts
        {"name": "balance_small", "op": "balance", "T": 512, "E": 8, "k": 2, "G": 1, "pad": 0,
         "masked": 0.0, "dead": 0, "skew": 0.0},
        # 16384 tokens over 64 experts, a balance loss per sequence: ragged sequences, padding masked,
        # rows behind the last sequence, three experts switched off (their logits are -inf)
        {"name": "balance_sequences", "op": "balance", "T": 16384, "E": 64, "k": 6, "G": 24, "pad": 37,
         "masked": 0.1, "dead": 3, "skew": 0.0},
        # all 32 x 4096 tokens of the 256-expert layer at once, skewed routing
        {"name": "balance_large", "op": "balance", "T": 131072, "E": 256, "k": 8, "G": 32, "pad": 0,
         "masked": 0.0, "dead": 0, "skew": 1.2},
        # the small fp32 layer's router
        {"name": "router_small_f32", "op": "router", "S": 1, "T_src": 512, "d": 256, "E": 8,
         "prec": "f32", "add": False},
        # the mid layer: 8 sources of 2048 tokens, 64 experts
        {"name": "router_mid", "op": "router", "S": 8, "T_src": 2048, "d": 2048, "E": 64,
         "prec": "bf16", "add": False},
        # one GPU's share of the 256-expert layer, added to what the layer's backward left
        {"name": "router_large_add", "op": "router", "S": 1, "T_src": 4096, "d": 7168, "E": 256,
         "prec": "bf16", "add": True},
        # gradients of 24 small layers: 120 tensors from 8 to a million elements
        {"name": "norm_many", "op": "norm", "layers": 24, "E": 8, "d": 256, "I": 512, "g": "bf16"},
        # fp32 gradients of the mid layer (64 experts of 3 x 1408 x 2048)
        {"name": "norm_large", "op": "norm", "layers": 1, "E": 64, "d": 2048, "I": 1408, "g": "f32"},
        # the small fp32 layer's step
        {"name": "adamw_small", "op": "adamw", "layers": 1, "E": 8, "d": 256, "I": 512, "p": "f32",
         "g": "f32", "bits": 32, "random": False},
        # 24 layers of bf16 parameters alone, rounded at random, moments in 8 bits
        {"name": "adamw_many_8bit", "op": "adamw", "layers": 24, "E": 7, "d": 192, "I": 448, "p": "bf16",
         "g": "bf16", "bits": 8, "random": True},
        # one GPU's share of the 256-expert layer (8 experts of 3 x 2048 x 7168), 8-bit moments
        {"name": "adamw_large_8bit", "op": "adamw", "layers": 1, "E": 8, "d": 7168, "I": 2048,
         "p": "master", "g": "f32", "bits": 8, "random": False},
        # the mid layer, bf16 parameters with fp32 copies, fp32 moments
        {"name": "adamw_large", "op": "adamw", "layers": 1, "E": 64, "d": 2048, "I": 1408,
         "p": "master", "g": "f32", "bits": 32, "random": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "router", "norm", "adamw"])
    if op == "balance":
        E = _log(rng, 2, 512)
        T = _log(rng, 1, min(131072, 131072 * 256 // E))
        G = min(T, _log(rng, 1, 64))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(16, E)), "G": G,
                "pad": rng.choice([0, min(T - 1, 5)]), "masked": rng.choice([0.0, 0.1, 0.5]),
                "dead": rng.choice([0, E // 8]), "skew": rng.choice([0.0, 1.2])}
    if op == "router":
        d, E = 64 * _log(rng, 1, 112), _log(rng, 2, 512)
        T = _log(rng, 1, max(1, min(65536, 4096 * 7168 * 256 // (d * max(E, 64)))))
        prec = rng.choice(["bf16", "bf16", "f32"])
        S = rng.choice([1, 1, 3, 8])
        T_src = max(1, (T if prec == "bf16" else max(1, T // 4)) // S)
        return {"op": op, "S": S, "T_src": T_src, "d": d, "E": E, "prec": prec,
                "add": rng.choice([False, True])}
    layers, E = _log(rng, 1, 24), _log(rng, 1, 64)
    d = 64 * _log(rng, 1, 64)
    room = 300_000_000 // (3 * layers * E * d)
    I = 64 * _log(rng, 1, max(1, min(64, room // 64)))
    g = rng.choice(["f32", "bf16"])
    if op == "norm":
        return {"op": op, "layers": layers, "E": E, "d": d, "I": I, "g": g}
    p = rng.choice(["f32", "bf16", "master"])
    return {"op": op, "layers": layers, "E": E, "d": d, "I": I, "p": p, "g": g,
            "bits": rng.choice([32, 8]), "random": p == "bf16" and rng.random() < 0.5}


def _sizes(c):
    """Elements of every tensor: per layer the three expert matrices, the router and its bias."""
    e = c["E"] * c["I"] * c["d"]
    return [n for _ in range(c["layers"]) for n in (e, e, e, c["E"] * c["d"], c["E"])]


def _places(sizes):
    """Offsets of the tensors in one flat buffer (each begins on a block) and its length."""
    at, n = [], 0
    for k in sizes:
        at.append(n)
        n += -(-k // BLOCK) * BLOCK
    return at, n


# ------------------------------------------------------------------ inputs
def _prepare_balance(c, r):
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=r)  # noqa: E731
    z = rnd(T, E) + c["skew"] * -torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    dead = torch.randperm(E, device=DEV, generator=r)[:min(c["dead"], E - k)]
    z[:, dead] = -math.inf
    idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
    cuts = torch.sort(torch.randint(0, T - c["pad"] + 1, (G - 1,), device=DEV, generator=r)).values
    off = torch.cat([torch.zeros(1, device=DEV), cuts, torch.full((1,), T - c["pad"], device=DEV)]).to(torch.int32)
    mask = (torch.rand(T, device=DEV, generator=r) >= c["masked"]).to(torch.uint8) if c["masked"] else None
    d_loss = 0.5 + torch.rand(2, device=DEV, generator=r)
    return {"logits": z, "topk_idx": idx, "offsets": off, "mask": mask, "d_loss": d_loss,
            "d_logits": torch.zeros(T, E, device=DEV), "alpha": 1e-2, "beta": 1e-3}


def _prepare_router(c, r):
    S, T, d, E = c["S"], c["T_src"], c["d"], c["E"]
    dt = torch.float32 if c["prec"] == "f32" else torch.bfloat16
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=r)  # noqa: E731
    # gradients of the logits as a balance loss gives them: probabilities times a centred weight
    dz = torch.softmax(rnd(S * T, E), dim=1) * rnd(S * T, E) * (1.0 / (S * T))
    s = {"d_logits": dz, "w_router": (rnd(E, d) / math.sqrt(d)).to(dt),
         "x": [rnd(T, d).to(dt) for _ in range(S)]}
    # what the layer's backward left there before, where the call adds to it
    s["d_x"] = [(rnd(T, d) * 1e-4).to(dt) if c["add"] else torch.empty(T, d, dtype=dt, device=DEV) for _ in range(S)]
    s["dw_router"] = rnd(E, d) * 1e-3 if c["add"] else torch.empty(E, d, device=DEV)
    s["d_bias"] = rnd(E) * 1e-3 if c["add"] else torch.empty(E, device=DEV)
    return s


def _blocks_from(v):
    """Nearest E4M3 codes and E8M0 scales of values (flat, whole blocks): a state to begin with."""
    b = v.view(-1, BLOCK)
    amax = b.abs().amax(1).clamp_min(1e-30)
    sh = torch.ceil(torch.log2(amax / 448.0))
    code = (b * torch.exp2(-sh)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return code.view(torch.uint8).reshape(-1), (sh + 127).to(torch.uint8)


def _prepare_step(c, r):
    sizes = _sizes(c)
    at, n = _places(sizes)
    rnd = lambda std: torch.randn(n, device=DEV, generator=r) * std  # noqa: E731
    real = torch.zeros(n, dtype=torch.bool, device=DEV)  # the gaps between tensors hold zeros
    for o, k in zip(at, sizes):
        real[o:o + k] = True
    g = rnd(1e-3).mul_(real)
    s = {"g": g.to(torch.bfloat16) if c["g"] == "bf16" else g, "sizes": sizes, "at": at}
    if c["op"] == "norm":
        s["max_norm"] = 1.0
        return s
    p = rnd(2e-2).mul_(real)
    s["p"] = p if c["p"] == "f32" else p.to(torch.bfloat16)
    s["master"] = p if c["p"] == "master" else None
    m, v = rnd(3e-4).mul_(real), rnd(1e-3).square_().mul_(real)
    if c["bits"] == 8:
        s["m"], s["m_scale"] = _blocks_from(m)
        s["v"], s["v_scale"] = _blocks_from(v.sqrt_())
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
    s["random"] = c["random"]
    s["scale"] = 0.5 + 0.5 * torch.rand(1, device=DEV, generator=r)   # the clip factor
    s["hyper"] = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1,
                  "step": 100, "seed": 1234 + c["layers"]}
    return s


def prepare(case, seed):
    r = torch.Generator(device=DEV)
    r.manual_seed(seed)
    op = case["op"]
    s = _prepare_balance(case, r) if op == "balance" else _prepare_router(case, r) if op == "router" else _prepare_step(case, r)
    s["case"] = case
    if own:
        _handles(case, s)
    return s


def _handles(c, s):
    """What a program keeps beside its tensors: configuration, descriptors, workspace, outputs."""
    import combine_router_top_expert_amd as mok
    zeros = lambda n, t: torch.zeros(max(n, 1), dtype=t, device=DEV)  # noqa: E731
    s["status"] = zeros(1, torch.int32)
    if c["op"] == "balance":
        cfg = mok.make_config(1, c["T"], 64, c["E"], c["k"], 64, 1, "bf16", 0)
        bal = mok.make_balance(s["alpha"], s["beta"], c["G"], s["offsets"], s["mask"])
        s["cfg"], s["bal"] = cfg, bal
        s["ws"] = zeros(mok.mok_balance_ws_bytes(cfg, c["T"], bal), torch.uint8)
        s["counts"] = torch.zeros(c["G"], c["E"], dtype=torch.int32, device=DEV)
        s["prob"] = torch.zeros(c["G"], c["E"], device=DEV)
        s["n_tok"] = zeros(c["G"] + 2, torch.int32)
        s["loss"] = zeros(2, torch.float32)
    elif c["op"] == "router":
        s["cfg"] = mok.make_config(c["S"], c["T_src"], c["d"], c["E"], 1, 64, 1, c["prec"], 0)
        s["ws"] = zeros(mok.mok_router_bwd_ws_bytes(s["cfg"], c["S"]), torch.uint8)
    else:
        cut = lambda t, per=1: [None] * len(s["at"]) if t is None else [  # noqa: E731
            t[o // per:o // per + -(-k // per)] for o, k in zip(s["at"], s["sizes"])]
        if c["op"] == "norm":
            s["params"] = mok.make_params([mok.make_param(g=g) for g in cut(s["g"])])
            s["ws"] = zeros(mok.mok_grad_norm_ws_bytes(s["params"]), torch.uint8)
            s["out"] = zeros(2, torch.float32)
        else:
            h = s["hyper"]
            s["params"] = mok.make_params([
                mok.make_param(p=p, g=g, m=m, v=v, master=w, m_scale=ms, v_scale=vs, weight_decay=h["weight_decay"])
                for p, g, m, v, w, ms, vs in zip(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]), cut(s["master"]),
                                                 cut(s["m_scale"], BLOCK), cut(s["v_scale"], BLOCK))])
            s["adamw"] = mok.make_adamw(h["lr"], h["beta1"], h["beta2"], h["eps"], step=h["step"], seed=h["seed"],
                                        dev_scale=s["scale"], random_params=s["random"])


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return (_plain_balance(s) if op == "balance" else _plain_router(s) if op == "router"
            else _plain_norm(s) if op == "norm" else _plain_adamw(s))


def _own(op, s):
    import combine_router_top_expert_amd as mok
    if op == "balance":
        T = s["case"]["T"]
        mok.mok_balance_fwd(s["cfg"], T, s["bal"], s["logits"], s["topk_idx"], s["counts"], s["prob"], s["n_tok"],
                            s["loss"], s["ws"], s["status"])
        mok.mok_balance_bwd(s["cfg"], T, s["bal"], s["logits"], s["counts"], s["n_tok"], s["d_loss"], s["d_logits"],
                            s["status"])
        return [s["loss"], s["counts"], s["prob"], s["n_tok"], s["d_logits"]]
    if op == "router":
        c = s["case"]
        mok.mok_router_bwd(s["cfg"], 0, c["S"], s["d_logits"], s["x"], s["w_router"], s["d_x"], s["dw_router"],
                           s["d_bias"], c["add"], s["ws"])
        return [s["dw_router"], s["d_bias"], s["d_x"]]
    if op == "norm":
        mok.mok_grad_norm(s["params"], s["max_norm"], s["out"], s["ws"])
        return s["out"]
    mok.mok_adamw(s["params"], s["adamw"])
    return _moments(s)


def _moments(s):
    """What the step wrote.  8-bit moments as what their codes (E4M3) and scales (powers of two) stand for."""
    out = [s["p"]] + ([] if s["master"] is None else [s["master"]])
    if s["m_scale"] is None:
        return out + [s["m"], s["v"]]
    return out + [s["m"].view(torch.float8_e4m3fn), s["m_scale"].view(torch.float8_e8m0fnu),
                  s["v"].view(torch.float8_e4m3fn), s["v_scale"].view(torch.float8_e8m0fnu)]


# ------------------------------------------------------------------ plain forms
def _plain_balance(s):
    c, z = s["case"], s["logits"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    group = torch.searchsorted(s["offsets"], torch.arange(T, device=DEV, dtype=torch.int32), right=True) - 1
    inside = (group >= 0) & (group < G)
    top = z.amax(1)
    live = inside & (top > -math.inf)
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)
    top = torch.where(live, top, 0.0)
    e = torch.exp(torch.where(live[:, None], z - top[:, None], -math.inf))
    total = e.sum(1)
    p = e / torch.where(live, total, 1.0)[:, None]
    lse = torch.where(live, top + torch.log(torch.where(live, total, 1.0)), 0.0)
    member = (group[None, :] == torch.arange(G, device=DEV)[:, None]) & live[None, :]
    psum = member.double() @ p.double()                        # long sums in 64 bits
    n = member.sum(1)
    slot = torch.where(live[:, None], group[:, None] * E + s["topk_idx"], G * E).reshape(-1)
    counts = torch.zeros(G * E + 1, dtype=torch.int32, device=DEV).index_add_(
        0, slot, torch.ones(T * k, dtype=torch.int32, device=DEV))[:-1].view(G, E)
    groups, N = (n > 0).sum(), n.sum()
    some = n.clamp_min(1).double()
    coef = torch.where(n > 0, E / (k * some * some * groups.clamp_min(1)), 0.0)
    loss = torch.stack([s["alpha"] * (coef * (counts * psum).sum(1)).sum(),
                        s["beta"] * lse.double().square().sum() / N.clamp_min(1)]).float()
    prob = (psum / some[:, None]).float()
    # the gradient: the weights are centred first (a constant per group drops out), so that
    # what is left of nearly equal counts is not a difference of large numbers
    w = ((s["alpha"] * s["d_loss"][0] * coef)[:, None] * (counts - (k * n / E)[:, None])).float()
    w = w[group.clamp(0, G - 1)]
    zc = (2.0 * s["beta"] * s["d_loss"][1] / N.clamp_min(1)) * lse
    dz = p * ((w - (p * w).sum(1, keepdim=True)) + zc[:, None])
    s["d_logits"].copy_(torch.where(inside[:, None], dz, s["d_logits"]))
    n_tok = torch.cat([n, N[None], groups[None]]).to(torch.int32)
    return [loss, counts, prob, n_tok, s["d_logits"]]


def _plain_router(s):
    c, dz = s["case"], s["d_logits"]
    x = torch.cat(s["x"]).float()
    dx, dw, db = dz @ s["w_router"].float(), dz.t() @ x, dz.sum(0, dtype=torch.float64).float()
    if c["add"]:
        dx, dw, db = torch.cat(s["d_x"]).float() + dx, s["dw_router"] + dw, s["d_bias"] + db
    s["dw_router"].copy_(dw)
    s["d_bias"].copy_(db)
    parts = [o.copy_(v) for o, v in zip(s["d_x"], dx.to(s["d_x"][0].dtype).split(c["T_src"]))]
    return [s["dw_router"], s["d_bias"], parts]


def _plain_norm(s):
    norm = s["g"].float().square().sum(dtype=torch.float64).sqrt()
    return torch.stack([norm, (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0)]).float()


def _mix(z):
    """The 64-bit finaliser of SplitMix64 (Steele, Lea and Flood, OOPSLA 2014) on int64, wrapping."""
    z = (z ^ ((z >> 30) & 0x3FFFFFFFF)) * MIX1
    z = (z ^ ((z >> 27) & 0x1FFFFFFFFF)) * MIX2
    return z ^ ((z >> 31) & 0x1FFFFFFFF)


def _words(s):
    """Random 32-bit words (a, b) of every group of 8 elements, and the element's place in it.  Element i of
    tensor t takes a + (i % 8) b for its moments and b + (i % 8) a for its parameter, of the word
    mix(key + (i / 8 + 1) gold), key = mix(mix(seed + t) + step gold)."""
    h, sizes = s["hyper"], s["sizes"]
    room = torch.tensor([-(-k // BLOCK) * (BLOCK // 8) for k in sizes], device=DEV)
    t = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), room, output_size=s["g"].numel() // 8)
    first = torch.cumsum(room, 0) - room
    q = torch.arange(t.numel(), device=DEV) - first[t]
    step = torch.tensor(h["step"], device=DEV)
    key = _mix(_mix(h["seed"] + torch.arange(len(sizes), device=DEV)) + step * GOLD)
    w = _mix(key[t] + (q + 1) * GOLD)
    return w & 0xFFFFFFFF, (w >> 32) & 0xFFFFFFFF


def _spread(a, b):
    j = torch.arange(8, device=DEV)
    return ((a[:, None] + j * b[:, None]) & 0xFFFFFFFF).reshape(-1)


def _from_blocks(code, scale):
    v = code.view(torch.float8_e4m3fn).float().view(-1, BLOCK)
    return (v * torch.exp2(scale.float() - 127.0)[:, None]).reshape(-1)


def _to_blocks(v, u, keep):
    """E4M3 codes and E8M0 scales of v: the smallest power of two that takes the block's largest magnitude to at
    most 448; each value rounded down or up by its u in [0, 1); keep: what is above zero stays above zero."""
    b = v.view(-1, BLOCK)
    mant, ex = torch.frexp(b.abs().amax(1))                   # amax = mant 2^ex, mant in [1/2, 1)
    sh = torch.where(mant > 0, ex - 9 + (mant > 0.875).int(), -127).clamp(-127, 127)
    y = (b.abs() * torch.exp2(-sh.float())[:, None]).reshape(-1)
    e = (torch.frexp(y).exponent - 1).clamp(-6, 8)
    n = torch.floor(torch.ldexp(y, 3 - e) + u)
    if keep:
        n = torch.where((v > 0) & (n < 1), 1.0, n)
    q = torch.copysign(torch.ldexp(n, e - 3), v)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), (sh + 127).to(torch.uint8)


def _plain_adamw(s):
    h = s["hyper"]
    b1, b2 = h["beta1"], h["beta2"]
    c1, c2 = 1.0 - b1 ** h["step"], 1.0 - b2 ** h["step"]
    g = s["g"].float() * s["scale"]
    p = s["p"].float() if s["master"] is None else s["master"]
    eight = s["m_scale"] is not None
    if eight:
        m, v = _from_blocks(s["m"], s["m_scale"]), _from_blocks(s["v"], s["v_scale"]).square()
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * (g * g)
    r = torch.sqrt(v)
    p = p * (1.0 - h["lr"] * h["weight_decay"]) - (h["lr"] / c1) * (m / (r * (1.0 / math.sqrt(c2)) + h["eps"]))
    if eight or s["random"]:
        a, b = _words(s)
    if eight:
        w = _spread(a, b)
        um, uv = (w & 0xFFFF).float() / 65536.0, (w >> 16).float() / 65536.0
        for dst, val in zip((s["m"], s["m_scale"], s["v"], s["v_scale"]), (*_to_blocks(m, um, False), *_to_blocks(r, uv, True))):
            dst.copy_(val)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if s["master"] is not None:
        s["master"].copy_(p)
    if s["random"]:  # bf16 bits: 16 random bits added below the last one kept
        bits = p.view(torch.int32).long() + (_spread(b, a) >> 16)
        s["p"].view(torch.int16).copy_((bits >> 16).to(torch.int16))
    else:
        s["p"].copy_(p)
    return _moments(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    if op == "balance":
        n = c["T"] * c["E"]
        return {"bytes": 8 * n + c["T"] * (4 * c["k"] + (1 if c["masked"] else 0)) + 8 * c["G"] * c["E"],
                "flops": 20 * n}
    if op == "router":
        T, e = c["S"] * c["T_src"], 4 if c["prec"] == "f32" else 2
        wide = 2 if c["add"] else 1
        return {"bytes": 4 * T * c["E"] + e * T * c["d"] * (1 + wide) + c["E"] * c["d"] * (e + 4 * wide),
                "flops": 4 * T * c["E"] * c["d"]}
    n = sum(_sizes(c))
    g = 4 if c["g"] == "f32" else 2
    if op == "norm":
        return {"bytes": g * n, "flops": 2 * n}
    moments = 16 if c["bits"] == 32 else 4 * (1 + 1 / BLOCK)
    weights = {"f32": 8, "bf16": 4, "master": 10}[c["p"]]
    return {"bytes": n * (g + moments + weights), "flops": 16 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_balance(case, s) if op == "balance" else _exact_router(case, s) if op == "router"
            else _exact_norm(s) if op == "norm" else _exact_adamw(s))


def _exact_balance(c, s):
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    z = s["logits"].double()
    off = s["offsets"].tolist()
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] != 0
    keep = keep & torch.isfinite(z).any(1)
    rows = [torch.arange(off[g], off[g + 1], device=DEV)[keep[off[g]:off[g + 1]]] for g in range(G)]
    N, groups = sum(len(r) for r in rows), sum(len(r) > 0 for r in rows)
    d0, d1 = (float(v) for v in s["d_loss"].double())
    counts = torch.zeros(G, E, dtype=torch.int64, device=DEV)
    prob = torch.zeros(G, E, dtype=torch.float64, device=DEV)
    dz = s["d_logits"].double()
    dz[off[0]:off[G]] = 0.0
    loss = torch.zeros(2, dtype=torch.float64, device=DEV)
    for g, r in enumerate(rows):
        n = len(r)
        if n == 0:
            continue
        lse = torch.logsumexp(z[r], 1)
        p = torch.exp(z[r] - lse[:, None])
        counts[g] = torch.bincount(s["topk_idx"][r].reshape(-1).long(), minlength=E)
        f = counts[g].double() * E / (k * n)
        prob[g] = p.mean(0)
        loss[0] += s["alpha"] * (f * prob[g]).sum() / groups
        loss[1] += s["beta"] * (lse * lse).sum() / N
        w = s["alpha"] * d0 * f / (n * groups)
        dz[r] = p * (w - (p @ w)[:, None]) + p * (2 * s["beta"] * d1 / N * lse)[:, None]
    n_tok = torch.tensor([len(r) for r in rows] + [N, groups], device=DEV)
    return [loss, counts, prob, n_tok, dz]


def _exact_router(c, s):
    dz, w = s["d_logits"].double(), s["w_router"].double()
    T = c["T_src"]
    keep = 1.0 if c["add"] else 0.0
    dw = s["dw_router"].double() * keep if c["add"] else torch.zeros(c["E"], c["d"], dtype=torch.float64, device=DEV)
    db = (s["d_bias"].double() if c["add"] else 0.0) + torch.ones(dz.shape[0], dtype=torch.float64, device=DEV) @ dz
    dx = []
    for i in range(c["S"]):
        part = dz[i * T:(i + 1) * T]
        dw = dw + torch.matmul(part.t(), s["x"][i].double())
        dx.append(torch.matmul(part, w) + (s["d_x"][i].double() if c["add"] else 0.0))
    return [dw, db, dx]


def _exact_norm(s):
    norm = torch.linalg.vector_norm(s["g"].double())
    return torch.stack([norm, torch.minimum(torch.ones_like(norm), s["max_norm"] / (norm + 1e-6))])


def _grid(v, u, keep):
    """v on the E4M3 grid of its blocks in 64 bits: (element values, scales)."""
    a = v.abs().view(-1, BLOCK)
    top = a.amax(1)
    sh = torch.ceil(torch.log2(torch.where(top > 0, top, 2.0 ** -200) / 448.0)).clamp(-127, 127)
    y = (a * 2.0 ** -sh[:, None]).reshape(-1)
    step = 2.0 ** (torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    n = torch.floor(y / step + u)
    if keep:
        n = torch.where((y > 0) & (n == 0), 1.0, n)
    return torch.sign(v) * n * step, 2.0 ** sh


def _exact_adamw(s):
    h = s["hyper"]
    t = h["step"]
    g = s["g"].double() * s["scale"].double()
    p0 = (s["p"] if s["master"] is None else s["master"]).double()
    eight = s["m_scale"] is not None
    m0, v0 = s["m"], s["v"]
    if eight:
        lift = lambda code, sc: code.view(torch.float8_e4m3fn).double() * (2.0 ** (sc.double() - 127)).repeat_interleave(BLOCK)  # noqa: E731
        m0, v0 = lift(m0, s["m_scale"]), lift(v0, s["v_scale"]) ** 2
    m = m0.double() * h["beta1"] + g * (1 - h["beta1"])
    v = v0.double() * h["beta2"] + g * g * (1 - h["beta2"])
    del m0, v0, g
    upd = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)).sqrt() + h["eps"])
    p = p0 - h["lr"] * h["weight_decay"] * p0 - h["lr"] * upd
    del p0, upd
    a = b = None
    if eight or s["random"]:
        a, b = _words(s)
    low = p  # the bf16 copy; its rounding is half a step or less, which 64 bits leave out
    if s["random"]:
        u = (_spread(b, a) >> 16).double() / 65536.0
        ulp = 2.0 ** (torch.floor(torch.log2(p.abs().clamp_min(1e-37))) - 7)
        low = torch.sign(p) * torch.floor(p.abs() / ulp + u) * ulp
    out = [low] + ([] if s["master"] is None else [p])
    if not eight:
        return out + [m, v]
    w = _spread(a, b)
    um, uv = (w & 0xFFFF).double() / 65536.0, (w >> 16).double() / 65536.0
    return out + [*_grid(m, um, False), *_grid(v.sqrt(), uv, True)]
