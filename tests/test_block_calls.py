"""The order and the arguments of the calls that a block makes, on the CPU:
nothing here reaches a kernel."""
import pytest
import torch

import combine_router_top_expert_amd.block as block_mod
import combine_router_top_expert_amd.layer as layer_mod
from combine_router_top_expert_amd.block import MoEBlock
from combine_router_top_expert_amd.layer import MoELayer

BF, F = torch.bfloat16, torch.float32


class _Device:
    def __init__(self, device):
        pass

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


@pytest.fixture
def calls(monkeypatch):
    """The ABI calls are noted instead of made."""
    seen = []
    monkeypatch.setattr(torch.cuda, "device", _Device)
    monkeypatch.setattr(torch.cuda, "stream", _Device)
    note = lambda n: (lambda *a, **k: seen.append((n, a)))  # noqa: E731
    for m, names in ((block_mod, ("mok_norm_fwd", "mok_norm_bwd")),
                     (layer_mod, ("mok_layer_fwd", "mok_layer_bwd", "mok_balance_fwd", "mok_balance_bwd",
                                  "mok_router_bwd"))):
        for n in names:
            monkeypatch.setattr(m, n, note(n))
    return seen


def _block(own=(0, 1), S=1, T=4, d=64, E=4, **kw):
    L = MoELayer(S, T, d, E, 2, 64, E, "bf16", 8, own[0], own[1], device="cpu", two_streams=False,
                 transposed_weights=False, **kw)
    b = MoEBlock(L, torch.ones(d, dtype=BF), "f32")
    L.xs, L.w_router, L.bias, L.e2l = [n.y for n in b.norms], torch.zeros(E, d, dtype=BF), None, None
    L.weights = None
    return b


def test_block_backward_adds_the_balance_gradient_before_the_norm(calls):
    """The norm's backward reads d_x: the losses' gradient has to be in it by then."""
    b = _block(keep_logits=True)
    dout = [torch.zeros(4, 64, dtype=BF)]
    b.forward([torch.zeros(4, 64)])
    with pytest.raises(RuntimeError, match="balance_loss"):
        b.backward(dout, balance=True)
    b.layer.balance_loss(0.1, 0.1)
    calls.clear()
    with pytest.raises(ValueError, match="router_grad"):
        b.backward(dout, balance=True, router_grad=False)
    for bad in (torch.ones(3), torch.ones(2, dtype=BF)):
        with pytest.raises(ValueError, match="expected"):
            b.backward(dout, balance=True, d_loss=bad)
    assert not calls
    w = torch.ones(2)
    b.backward(dout, balance=True, d_loss=w)
    assert [n for n, _ in calls] == ["mok_layer_bwd", "mok_balance_bwd", "mok_router_bwd", "mok_norm_bwd"]
    assert any(t is w for t in calls[1][1])
    # behind the norm's backward the gradient would be lost
    with pytest.raises(RuntimeError, match="balance=True"):
        b.layer.balance_backward()
    calls.clear()
    b.layer.backward(dout)
    b.layer.balance_backward()
    assert [n for n, _ in calls] == ["mok_layer_bwd", "mok_balance_bwd", "mok_router_bwd"]


@pytest.mark.parametrize("own", [(0, 1), (0, 2)])
def test_block_refuses_rows_that_the_layer_would_not_have(calls, own):
    """The layer routes all rows of its sources: rows that the norm does not write would be an earlier call's."""
    b = _block(own, S=2)
    n = own[1]
    res, delta = [torch.zeros(4, 64) for _ in range(n)], [torch.zeros(4, 64, dtype=BF) for _ in range(n)]
    short, narrow = res[:-1] + [torch.zeros(3, 64)], res[:-1] + [torch.zeros(4, 32)]
    for args in ((short,), (short, delta[:-1] + [torch.zeros(3, 64, dtype=BF)]), (res, delta[:-1] + [torch.zeros(3, 64, dtype=BF)]),
                 (narrow,), (res[:-1],), (res + res[:1],), (res, delta[:-1]), (res, delta + delta), ([None] * n,),
                 (res[:-1] + [torch.zeros(5, 64)],), ([t.to(BF) for t in res],), (res, res)):
        with pytest.raises(ValueError):
            b.forward(*args)
    assert not calls
    b.forward(res, delta)
    b.forward([None] * n, delta)
    assert [c for c, _ in calls] == (["mok_norm_fwd"] * n + ["mok_layer_fwd"]) * 2


def test_block_backward_refuses_before_it_writes_gradients(calls):
    """Refused arguments leave the layer's gradients as they were."""
    b = _block((0, 2), S=2)
    dout, dres = [torch.zeros(4, 64, dtype=BF)] * 2, [torch.zeros(4, 64)] * 2
    with pytest.raises(RuntimeError, match="forward"):
        b.backward(dout)
    b.forward(dres)
    calls.clear()
    for bad in ((dout, dres[:1]), (dout, dres + dres), (dout, [torch.zeros(3, 64)] * 2), (dout, dout),
                (dout, [dres[0], torch.zeros(64, 4).t()])):
        with pytest.raises(ValueError):
            b.backward(*bad)
    b.norms[1].forward(torch.zeros(3, 64, dtype=BF))
    calls.clear()
    with pytest.raises(RuntimeError, match="3 rows"):
        b.backward(dout, dres)
    assert not calls
    b.forward(dres)
    b.backward(dout, [None, dres[1]])
    assert [c for c, _ in calls] == ["mok_norm_fwd", "mok_norm_fwd", "mok_layer_fwd", "mok_layer_bwd", "mok_norm_bwd", "mok_norm_bwd"]


def test_block_without_own_sources(calls):
    """A rank that holds experts and no tokens: the norm's weight has no gradient, whatever an earlier step left."""
    b = _block((0, 0), S=2)
    b.dw_norm.fill_(float("nan"))
    assert b.forward([]) == []
    assert b.backward([torch.zeros(4, 64, dtype=BF)] * 2) == []
    assert (b.dw_norm == 0).all()


def test_block_on_one_device(calls):
    """The layer reads the norms' rows: a weight of another device would put them there."""
    L = _block().layer
    with pytest.raises(ValueError, match="meta"):
        MoEBlock(L, torch.ones(64, dtype=BF, device="meta"))


def test_scratch_of_the_same_device_by_another_name(calls):
    """"cuda" and "cuda:0" (here "cpu" and "cpu:0") name one device; another one is refused."""
    make = lambda device, **kw: MoELayer(1, 4, 64, 4, 2, 64, 4, "bf16", 8, 0, 1, device=device, two_streams=False,  # noqa: E731
                                         checkpoint=True, **kw)
    a = make("cpu")
    assert make("cpu:0", scratch=a).ab is a.ab
    with pytest.raises(ValueError, match="device"):
        make("meta", scratch=a)
