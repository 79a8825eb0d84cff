"""What the Python side of the training calls refuses and hands on, on the
CPU: nothing here reaches a kernel."""
import ctypes
import gc
import os
import re
import weakref

import numpy as np
import pytest
import torch

import combine_router_top_expert_amd as mok
import combine_router_top_expert_amd.layer as layer_mod
from combine_router_top_expert_amd.layer import MoELayer
from combine_router_top_expert_amd.optim import AdamW


def _layer(**kw):
    return MoELayer(1, 4, 64, 4, 1, 64, 4, "f32", 4, 0, 1, device="cpu", keep_logits=True, **kw)


class _Device:
    """torch.cuda.device for a machine without one: notes what is current."""
    current = None

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        self.before, _Device.current = _Device.current, self.device

    def __exit__(self, *exc):
        _Device.current = self.before


@pytest.fixture
def calls(monkeypatch):
    """The layer's ABI calls are noted, with the device current for them, instead of made."""
    seen = []
    monkeypatch.setattr(torch.cuda, "device", _Device)
    for name in ("mok_balance_fwd", "mok_balance_bwd", "mok_router_bwd"):
        monkeypatch.setattr(layer_mod, name, lambda *a, _n=name: seen.append((_n, a, _Device.current)))
    return seen


def test_balance_backward_refuses_wrong_loss_weights(calls):
    """A kernel reads d_loss as two fp32 values of its device."""
    L = _layer()
    L.xs, L.w_router, L.bias = [torch.zeros(4, 64)], torch.zeros(4, 64), None
    L.balance_loss(0.1, 0.1)
    calls.clear()
    for bad in (torch.ones(2, dtype=torch.float64), torch.ones(1), torch.ones(3), torch.ones(0), torch.ones(4)[::2],
                torch.ones(2, dtype=torch.bfloat16), torch.ones(2, device="meta")):
        with pytest.raises(ValueError, match="expected"):
            L.balance_backward(bad)
        assert not calls
    L.balance_backward(torch.ones(2))
    L.balance_backward()
    assert [c[0] for c in calls] == ["mok_balance_bwd", "mok_router_bwd"] * 2


def test_calls_run_on_the_layers_device(calls, monkeypatch):
    """The kernels are launched with the layer's device current, whichever was."""
    for name in ("mok_mx_quantize", "mok_prepare_bwd"):
        monkeypatch.setattr(layer_mod, name, lambda *a, _n=name: calls.append((_n, a, _Device.current)))
    L = _layer()
    L.xs, L.w_router, L.bias = [torch.zeros(4, 64)], torch.zeros(4, 64), None
    off = torch.tensor([0, 4], dtype=torch.int32)
    L.balance_loss(0.1, 0.1, off)
    L.balance_backward()
    for prec in ("bf16", "mxfp8"):
        L = MoELayer(1, 4, 64, 4, 1, 64, 4, prec, 4, 0, 1, device="cpu", two_streams=False)
        L.w_gate = L.w_up = L.w_down = torch.zeros(4, 64, 64)
        L.wt, L.wq = [None] * 4, [(None, None)] * 3
        L.update_weights()
    assert {c[0] for c in calls} == {"mok_balance_fwd", "mok_balance_bwd", "mok_router_bwd", "mok_mx_quantize",
                                     "mok_prepare_bwd"}
    assert all(c[2] == L.device for c in calls)


def test_version_tells_the_structures_apart():
    """mok_fwd_state grew by the logits after "mok 0.1": a caller can tell."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    header = open(os.path.join(root, "include", "mok.h")).read()
    assert mok.mok_version() == re.search(r'#define MOK_VERSION "([^"]+)"', header).group(1)
    assert mok.mok_version() != "mok 0.1 gfx950"
    assert [f for f, _ in mok.mok_fwd_state._fields_][-1] == "logits"


def test_optimizer_keeps_no_autograd_graph():
    """fp32 copies of leaves that autograd knows are values: a graph kept with
    them would hold the leaves' accumulators for as long as the optimizer."""
    ps = [torch.nn.Parameter(torch.randn(40).bfloat16()), torch.nn.Parameter(torch.randn(7))]
    opt = AdamW(ps)
    state = opt.state_dict()
    assert opt.master[0].grad_fn is None and not opt.master[0].requires_grad
    state["master"] = [ps[0].float(), None]        # another optimizer's, with its graph
    opt.load_state_dict(state)
    assert opt.master[0].grad_fn is None and not opt.master[0].requires_grad
    assert torch.equal(opt.master[0], ps[0].detach().float())


def test_optimizer_takes_loaded_parameters_over():
    """Weights written into bf16 parameters after construction reach the fp32
    copies, which the next step starts from, in place."""
    ps = [torch.randn(3, 40).bfloat16(), torch.randn(7), torch.randn(0).bfloat16()]
    opt = AdamW(ps)
    at = opt.master[0].data_ptr()
    ps[0].copy_(torch.randn(3, 40))
    opt.take_params()
    assert torch.equal(opt.master[0], ps[0].float()) and opt.master[0].data_ptr() == at
    assert opt.master[1] is None
    AdamW(ps, master=False).take_params()          # nothing is kept


def test_optimizer_state_holds_the_seed():
    """A resumed run rounds as the run would have gone on."""
    p = [torch.randn(40).bfloat16()]
    a, b = AdamW(p, state_bits=8, seed=(1 << 63) + 5), AdamW([p[0].clone()], state_bits=8)
    b.load_state_dict(a.state_dict())
    assert b.args.seed == (1 << 63) + 5
    old = a.state_dict()
    del old["seed"]
    c = AdamW([p[0].clone()], state_bits=8, seed=9)
    c.load_state_dict(old)
    assert c.args.seed == 9


def test_optimizer_refuses_parameters_that_overlap():
    """Two updates of one element would race."""
    w = torch.zeros(100)
    for bad in ([w, torch.zeros(3), w], [w[:60], w[50:]], [w.bfloat16().view(-1), w, w[99:]]):
        with pytest.raises(ValueError, match="overlap"):
            AdamW(bad)
    AdamW([w[50:], w[:50], w[50:50], torch.zeros(0), torch.zeros(0)])     # neighbours and empty ones


@pytest.mark.parametrize("max_norm, scale", [(None, float("inf")), (None, 1e39), (None, 1e-46), (1e-30, 1e20),
                                             (1e-44, 64.0), (1e-50, 1.0)])
def test_optimizer_refuses_scales_beyond_fp32(max_norm, scale):
    """A scale that is infinite or zero to the kernels, or a limit that is:
    a norm limit of zero would turn the clipping off."""
    opt = AdamW([torch.zeros(8)], max_norm=max_norm)
    with pytest.raises(ValueError, match="fp32"):
        opt.step([torch.zeros(8)], grad_scale=scale)


@pytest.mark.parametrize("max_norm, scale", [(None, 1e38), (1e-30, 1e10), (1.0, 1e-40), (float("inf"), 2.0)])
def test_optimizer_takes_scales_within_fp32(max_norm, scale):
    opt = AdamW([torch.zeros(8)], max_norm=max_norm)
    with pytest.raises(ValueError, match="GPU"):      # the next thing that is looked at
        opt.step([torch.zeros(8)], grad_scale=scale)


@pytest.mark.parametrize("bad", [dict(eps=1e-39), dict(eps=1e-50), dict(lr=1e39), dict(lr=float("inf"))], ids=str)
def test_adamw_refuses_constants_beyond_fp32(bad):
    """An eps below 2^-126 has no finite reciprocal in fp32: elements without
    gradients would become NaN."""
    q = mok.mok_param(16, 16, None, 16, 16, None, None, 8, mok.MOK_F32, mok.MOK_F32, 32, 0.0)
    with pytest.raises(mok.MokError, match="EINVAL"):
        mok.mok_adamw(mok.make_params([q]), mok.make_adamw(**{**dict(lr=1e-3, eps=1e-8), **bad}), 0)
    mok.mok_adamw(mok.make_params([]), mok.make_adamw(1e-3, eps=2.0 ** -126), 0)      # nothing to do
    mok.mok_adamw(mok.make_params([]), mok.make_adamw(1e-3, eps=0.0), 0)


def test_balance_refuses_more_groups_than_a_launch_holds():
    """Refused before the first launch, not by the second one's failure."""
    cfg = mok.make_config(1, 8, 64, 2, 1, 64, 1, "f32", 0)
    for G, ok in (((1 << 23) - 1, True), (1 << 23, False), (1 << 29, False)):
        bal = mok.mok_balance(0.1, 0.1, G, 16, None)
        assert (mok.mok_balance_ws_bytes(cfg, 8, bal) > 0) == ok
    at = 1 << 20
    for call in (mok.lib().mok_balance_fwd, mok.lib().mok_balance_bwd):
        bal = mok.mok_balance(0.1, 0.1, 1 << 23, at, None)
        assert call(ctypes.byref(cfg), 8, ctypes.byref(bal), *[at] * (len(call.argtypes) - 5), None, None) == -1


def test_router_bwd_refuses_rows_at_the_end_of_int32():
    """Row numbers run past the last row by up to a block: from 2^31 - 16 on
    they would wrap."""
    for prec in ("f32", "bf16"):
        for T, ok in (((1 << 31) - 1, False), ((1 << 31) - 4096, False), ((1 << 31) - 4097, True)):
            cfg = mok.make_config(1, T, 64, 1, 1, 64, 1, prec, 0)
            assert (mok.mok_router_bwd_ws_bytes(cfg, 1) > 0) == ok
            assert mok.mok_router_bwd_ws_bytes(cfg, 0) > 0
            if not ok:
                with pytest.raises(mok.MokError, match="EINVAL"):
                    mok.mok_router_bwd(cfg, 0, 1, torch.zeros(4), None, None, None, None, torch.zeros(1), False,
                                       torch.zeros(64), 0)


def test_optimizer_holds_the_memory_it_bound():
    """A bound step names memory by address: giving a parameter or a gradient
    other memory leaves the former one held until the next bind."""
    arrays = [np.ones(40, dtype=np.float32) for _ in range(2)]
    alive = [weakref.ref(a) for a in arrays]
    p, g = (torch.from_numpy(a) for a in arrays)
    del arrays
    opt = AdamW([p])
    opt.bind([g])
    p.data, g.data = torch.zeros(40), torch.zeros(40)
    gc.collect()
    assert all(a() is not None for a in alive)
    opt.bind([g])
    gc.collect()
    assert all(a() is None for a in alive)
    assert (opt._desc[0].p, opt._desc[0].g) == (p.data_ptr(), g.data_ptr())
