"""What the Python side of the training calls refuses and hands on, on the
CPU: nothing here reaches a kernel."""
import pytest
import torch

import combine_router_top_expert_amd.layer as layer_mod
from combine_router_top_expert_amd.layer import MoELayer


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
