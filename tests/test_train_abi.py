"""Argument checks of the training entry points (balance loss, router
projection backward, gradient norm, AdamW) on the host: refused calls return
MOK_EINVAL before any GPU work, with dummy pointers that nothing reads."""
import ctypes
import os

import pytest
import torch

import combine_router_top_expert_amd as mok
from combine_router_top_expert_amd import build

EINVAL = -1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mok.LIB_PATH):
        build.build()
    return mok.lib()


def _cfg(**kw):
    base = dict(S=2, T_src=100, d=256, E=8, k=2, I=128, E_local=8, prec="bf16", R_cap=400)
    base.update(kw)
    return mok.make_config(**base)


def _bal(G=0, off=None, mask=None):
    return mok.mok_balance(0.01, 0.001, G, off, mask)


def _balance_fwd(L, cfg, T=10, bal=None, z=16, topk=16, out=(16, 16, 16, 16), ws=256):
    return L.mok_balance_fwd(ctypes.byref(cfg), T, ctypes.byref(bal or _bal()), z, topk, *out, ws,
                             None, None)


def test_balance_refusals(L):
    cfg = _cfg()
    assert _balance_fwd(L, _cfg(E=0)) == EINVAL
    assert _balance_fwd(L, cfg, T=-1) == EINVAL
    assert _balance_fwd(L, cfg, z=None) == EINVAL
    assert _balance_fwd(L, cfg, topk=None) == EINVAL
    for i in range(4):
        out = [16] * 4
        out[i] = None
        assert _balance_fwd(L, cfg, out=out) == EINVAL
    assert _balance_fwd(L, cfg, z=18) == EINVAL
    assert _balance_fwd(L, cfg, topk=18) == EINVAL
    assert _balance_fwd(L, cfg, ws=None) == EINVAL
    assert _balance_fwd(L, cfg, ws=4) == EINVAL                        # 8-byte partial sums
    assert _balance_fwd(L, cfg, bal=_bal(G=-1)) == EINVAL
    assert _balance_fwd(L, cfg, bal=_bal(G=3)) == EINVAL               # groups without offsets
    assert _balance_fwd(L, _cfg(T_src=1, k=8), T=1 << 29) == EINVAL    # counts beyond int32
    assert _balance_fwd(L, _cfg(T_src=1, k=1), T=(1 << 30) + 1) == EINVAL
    assert _balance_fwd(L, cfg, bal=_bal(G=1 << 29, off=16)) == EINVAL  # G * E beyond int32
    assert L.mok_balance_fwd(ctypes.byref(cfg), 10, None, 16, 16, 16, 16, 16, 16, 256, None,
                             None) == EINVAL
    b = ctypes.byref(_bal())
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, None, 16, 16, None, 16, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, 16, None, 16, None, 16, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, 16, 16, None, None, 16, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, 16, 16, 16, None, None, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, 18, 16, 16, None, 16, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, 16, 16, 16, 18, 16, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 10, b, 16, 16, 16, None, 18, None, None) == EINVAL
    assert L.mok_balance_bwd(ctypes.byref(cfg), 0, b, None, None, None, None, None, None, None) == 0


def test_balance_workspace(L):
    cfg = _cfg()
    one = mok.mok_balance_ws_bytes(cfg, 1, _bal())
    assert 0 < one <= mok.mok_balance_ws_bytes(cfg, 100000, _bal())
    assert mok.mok_balance_ws_bytes(cfg, 0, _bal()) > 0
    assert mok.mok_balance_ws_bytes(cfg, 100, _bal(G=2)) == 0          # no offsets
    assert mok.mok_balance_ws_bytes(_cfg(E=513), 100, _bal()) == 0
    assert mok.mok_balance_ws_bytes(cfg, 100, _bal(G=5000, off=16)) >= 5000 * 8 * 8


def _router(L, cfg, own=(0, 2), dz=16, x=16, w=16, dx=16, dw=16, db=16, ws=256):
    tab = lambda v: None if v is None else ctypes.cast((ctypes.c_void_p * cfg.S)(*([v] * cfg.S)), ctypes.c_void_p)  # noqa: E731
    return L.mok_router_bwd(ctypes.byref(cfg), *own, dz, tab(x), w, tab(dx), dw, db, 0, ws, None)


def test_router_bwd_refusals(L):
    cfg = _cfg()
    assert _router(L, _cfg(d=100)) == EINVAL
    assert _router(L, _cfg(d=(1 << 26) + 64, T_src=1)) == EINVAL
    assert _router(L, cfg, own=(1, 2)) == EINVAL          # past the last source
    assert _router(L, cfg, own=(-1, 1)) == EINVAL
    assert _router(L, cfg, dz=None) == EINVAL
    assert _router(L, cfg, dz=18) == EINVAL               # fp32 gradients, misaligned
    assert _router(L, cfg, w=None) == EINVAL
    assert _router(L, cfg, w=24) == EINVAL
    assert _router(L, cfg, x=None) == EINVAL
    assert _router(L, cfg, x=24) == EINVAL
    assert _router(L, cfg, dx=24) == EINVAL
    assert _router(L, cfg, dw=24) == EINVAL
    assert _router(L, cfg, db=18) == EINVAL
    assert _router(L, cfg, ws=None) == EINVAL
    assert _router(L, cfg, ws=24) == EINVAL
    # a table without an own entry
    tab = (ctypes.c_void_p * 2)(16, None)
    tp, full = ctypes.cast(tab, ctypes.c_void_p), ctypes.cast((ctypes.c_void_p * 2)(16, 16), ctypes.c_void_p)
    assert L.mok_router_bwd(ctypes.byref(cfg), 0, 2, 16, tp, 16, full, 16, None, 0, 256, None) == EINVAL
    assert L.mok_router_bwd(ctypes.byref(cfg), 0, 2, 16, full, 16, tp, 16, None, 0, 256, None) == EINVAL
    assert mok.mok_router_bwd_ws_bytes(cfg, 3) == 0
    assert mok.mok_router_bwd_ws_bytes(cfg, -1) == 0
    assert mok.mok_router_bwd_ws_bytes(cfg, 2) > 0


def _param(**kw):
    base = dict(p=16, g=16, master=None, m=16, v=16, m_scale=None, v_scale=None, n=100,
                p_type=mok.MOK_F32, g_type=mok.MOK_F32, state_bits=32, weight_decay=0.1)
    base.update(kw)
    return mok.mok_param(*[base[f] for f, _ in mok.mok_param._fields_])


def _adamw(L, params, **kw):
    a = mok.make_adamw(kw.pop("lr", 1e-3), **kw)
    arr = mok.make_params(params)
    return L.mok_adamw(len(params), arr, ctypes.byref(a), None)


BAD_PARAMS = [dict(n=-1), dict(n=(1 << 40) + 1), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p=18),
              dict(g=18), dict(m=18), dict(v=18), dict(p_type=2), dict(g_type=7),
              dict(state_bits=16), dict(state_bits=8), dict(state_bits=8, m_scale=16),
              dict(state_bits=8, v_scale=16), dict(master=16),
              dict(p_type=mok.MOK_BF16, master=18), dict(p_type=mok.MOK_BF16, p=17),
              dict(g_type=mok.MOK_BF16, g=17)]


@pytest.mark.parametrize("bad", BAD_PARAMS, ids=str)
def test_adamw_refuses_a_bad_tensor(L, bad):
    # the second of two, so that every entry is looked at before anything runs
    assert _adamw(L, [_param(), _param(**bad)]) == EINVAL


@pytest.mark.parametrize("bad", [dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                                 dict(eps=-1e-8), dict(lr=-1.0), dict(lr=float("nan")),
                                 dict(eps=float("nan")), dict(beta2=float("nan"))], ids=str)
def test_adamw_refuses_bad_constants(L, bad):
    assert _adamw(L, [_param()], **bad) == EINVAL


def test_adamw_and_norm_refusals(L):
    a = mok.make_adamw(1e-3)
    arr = mok.make_params([_param()])
    assert L.mok_adamw(-1, arr, ctypes.byref(a), None) == EINVAL
    assert L.mok_adamw(1, None, ctypes.byref(a), None) == EINVAL
    assert L.mok_adamw(1, arr, None, None) == EINVAL
    assert L.mok_adamw(0, None, ctypes.byref(a), None) == 0            # nothing to do
    assert L.mok_adamw(1, mok.make_params([_param(n=0, p=None, g=None, m=None, v=None)]),
                       ctypes.byref(a), None) == 0
    a.random_params = 2
    assert L.mok_adamw(1, arr, ctypes.byref(a), None) == EINVAL
    for bad in (dict(dev_scale=18), dict(dev_lr=20), dict(dev_step=20)):
        assert _adamw(L, [_param()], **bad) == EINVAL
    assert L.mok_grad_norm(1, arr, 1.0, 18, 16, None) == EINVAL
    assert L.mok_grad_norm(1, arr, 1.0, None, 16, None) == EINVAL
    assert L.mok_grad_norm(1, arr, 1.0, 16, None, None) == EINVAL
    assert L.mok_grad_norm(1, arr, 1.0, 16, 4, None) == EINVAL
    assert L.mok_grad_norm(-1, arr, 1.0, 16, 16, None) == EINVAL
    assert L.mok_grad_norm(1, mok.make_params([_param(g=None)]), 1.0, 16, 16, None) == EINVAL
    assert mok.mok_grad_norm_ws_bytes(mok.make_params([_param(n=-1)])) == 0
    # the norm needs the gradients only
    assert mok.mok_grad_norm_ws_bytes(mok.make_params([mok.make_param(g=torch.zeros(5))])) >= 8


def test_route_logits_checks_what_route_checks(L):
    cfg = _cfg()
    assert L.mok_route_logits(ctypes.byref(cfg), 10, None, 1, None, 1, 1, 1, None) == EINVAL
    assert L.mok_route_logits(ctypes.byref(cfg), 10, 1, 1, None, 1, None, 1, None) == EINVAL
    assert L.mok_route_logits(ctypes.byref(_cfg(d=96)), 10, 1, 1, None, 1, 1, 1, None) == EINVAL


def test_bindings_refuse_wrong_tensors():
    z = torch.zeros
    with pytest.raises(TypeError):
        mok.make_param(p=z(4, dtype=torch.float16), g=z(4), m=z(4), v=z(4))
    with pytest.raises(ValueError):
        mok.make_param(p=z(4), g=z(5), m=z(4), v=z(4))
    with pytest.raises(ValueError):
        mok.make_param(p=z(4, 4).t(), g=z(4, 4), m=z(16), v=z(16))
    # 8-bit moments: both scales, one byte per 32 elements, codes in bytes
    u8 = lambda n: z(n, dtype=torch.uint8)  # noqa: E731
    ok = dict(p=z(40), g=z(40), m=u8(40), v=u8(40), m_scale=u8(2), v_scale=u8(2))
    assert mok.make_param(**ok).state_bits == 8
    for bad in (dict(v_scale=None), dict(m_scale=u8(1)), dict(v_scale=u8(3)), dict(m=z(40))):
        with pytest.raises((ValueError, TypeError)):
            mok.make_param(**{**ok, **bad})
    with pytest.raises(TypeError):
        mok.make_param(p=z(4), g=z(4), m=z(4, dtype=torch.bfloat16), v=z(4))


def test_optimizer_refusals():
    from combine_router_top_expert_amd.optim import AdamW
    w = torch.zeros(8)
    with pytest.raises(ValueError):
        AdamW([])
    with pytest.raises(TypeError):
        AdamW([torch.zeros(8, dtype=torch.float16)])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4, 4).t()])
    with pytest.raises(ValueError):
        AdamW([w], state_bits=16)
    with pytest.raises(ValueError):
        AdamW([w], weight_decay=[0.1, 0.2])
    opt = AdamW([w])
    with pytest.raises(RuntimeError):
        opt.step()
    with pytest.raises(ValueError):
        opt.bind([w, w])
    with pytest.raises(ValueError):
        opt.bind([torch.zeros(9)])


def test_optimizer_state_moves_between_optimizers():
    from combine_router_top_expert_amd.optim import AdamW
    ps = [torch.randn(70).bfloat16(), torch.randn(33)]
    a, b = (AdamW([p.clone() for p in ps], state_bits=[8, 32]) for _ in range(2))
    for t in a.m + a.v + [a.m_scale[0], a.v_scale[0], a.master[0]]:
        t.copy_(torch.randint(0, 100, t.shape))
    a.step_count = 17
    b.load_state_dict(a.state_dict())
    assert b.step_count == 17
    for x, y in zip(a.m + a.v + a.m_scale + a.v_scale + a.master, b.m + b.v + b.m_scale + b.v_scale + b.master):
        assert (x is None and y is None) or (torch.equal(x, y) and x.data_ptr() != y.data_ptr())
    with pytest.raises(ValueError):
        AdamW([p.clone() for p in ps]).load_state_dict(a.state_dict())      # 32-bit moments
    with pytest.raises(ValueError):
        AdamW([ps[0].clone()], state_bits=8).load_state_dict(a.state_dict())


def test_layer_balance_refusals():
    from combine_router_top_expert_amd.layer import MoELayer

    def layer(**kw):
        return MoELayer(1, 4, 64, 4, 1, 64, 4, "f32", 4, 0, 1, device="cpu", **kw)
    with pytest.raises(RuntimeError):
        layer().balance_loss(0.1)                        # no logits kept
    L = layer(keep_logits=True)
    with pytest.raises(RuntimeError):
        L.balance_backward()                             # no loss before it
    for bad in (dict(group_offsets=torch.tensor([0, 4])), dict(group_offsets=torch.tensor([0], dtype=torch.int32)),
                dict(token_mask=torch.ones(4)), dict(token_mask=torch.ones(3, dtype=torch.uint8)),
                dict(group_offsets=torch.zeros(0, dtype=torch.int32))):
        with pytest.raises(ValueError):
            L.balance_loss(0.1, **bad)


def test_optimizer_steps_on_a_gpu_only():
    from combine_router_top_expert_amd.optim import AdamW
    opt = AdamW([torch.zeros(8)])
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(ValueError, match="grad_scale"):
            opt.step([torch.zeros(8)], grad_scale=scale)
    with pytest.raises(ValueError, match="GPU"):
        opt.step([torch.zeros(8)])


def test_balance_misaligned_outputs_are_refused():
    """Pointers that no kernel of the call may dereference: refused before any launch."""
    cfg = mok.make_config(1, 8, 64, 8, 2, 64, 1, "f32", 0)
    bal, at = mok.make_balance(1e-2, 1e-3), 1 << 20
    ok = dict(logits=at, topk=at, counts=at, prob=at, n_tok=at, loss=at)
    for bad in ok:
        a = {**ok, bad: at + 2}
        with pytest.raises(RuntimeError):
            mok.mok_balance_fwd(cfg, 8, bal, a["logits"], a["topk"], a["counts"], a["prob"], a["n_tok"], a["loss"],
                                at, None, 0)
    for bad in (dict(counts=at + 2), dict(n_tok=at + 1)):
        a = {**ok, **bad}
        with pytest.raises(RuntimeError):
            mok.mok_balance_bwd(cfg, 8, bal, at, a["counts"], a["n_tok"], None, at, None, 0)
    with pytest.raises(RuntimeError):
        mok.mok_balance_fwd(cfg, 8, mok.make_balance(1e-2, 1e-3, 2, at + 2, None), at, at, at, at, at, at, at, None, 0)


@pytest.mark.parametrize("max_norm", [0.0, -1.0, float("nan")])
def test_optimizer_refuses_norms_that_do_not_clip(max_norm):
    from combine_router_top_expert_amd.optim import AdamW
    with pytest.raises(ValueError, match="max_norm"):
        AdamW([torch.zeros(8)], max_norm=max_norm)
