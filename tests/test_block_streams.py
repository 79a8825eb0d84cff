"""How the classes around the layer order themselves over streams and hold
their memory, on the CPU with streams that note what is asked of them."""
import pytest
import torch

import combine_router_top_expert_amd as mok
import combine_router_top_expert_amd.block as block_mod
import combine_router_top_expert_amd.decode as decode_mod
import combine_router_top_expert_amd.layer as layer_mod
import combine_router_top_expert_amd.streams as streams_mod
from combine_router_top_expert_amd.block import MoEBlock, RMSNorm
from combine_router_top_expert_amd.decode import MoEDecoder
from combine_router_top_expert_amd.layer import MoELayer
from combine_router_top_expert_amd.streams import StreamUser

BF = torch.bfloat16


class _Stream:
    def __init__(self, handle, notes):
        self.cuda_stream, self.notes, self.captured = handle, notes, False

    def record_event(self):
        return f"event of {self.cuda_stream}"

    def wait_event(self, e):
        self.notes.append((self.cuda_stream, "waits for", e))


class _Buffer:
    def __init__(self, notes):
        self.notes = notes

    def record_stream(self, s):
        self.notes.append(("held for", s.cuda_stream))


@pytest.fixture
def gpu(monkeypatch):
    """Three streams, the first of them current."""
    notes = []
    streams = [_Stream(i, notes) for i in range(3)]
    now = [streams[0]]

    class Context:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            self.before = now[0]
            if isinstance(self.what, _Stream):
                now[0] = self.what

        def __exit__(self, *exc):
            now[0] = self.before
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0].captured)
    monkeypatch.setattr(streams_mod, "_stream", lambda s: (now[0] if s is None else s).cuda_stream, raising=False)
    return streams, notes, Context


def test_first_call_on_a_stream_comes_after_the_making(gpu):
    streams, notes, on = gpu

    class User(StreamUser):
        device = torch.device("cuda", 0)

        def _buffers(self):
            return [_Buffer(notes), _Buffer(notes)]
    u = User()
    u._ready()
    u._enter(None)
    u._enter(streams[0])
    assert not notes
    u._enter(streams[1])
    first = [(1, "waits for", "event of 0"), ("held for", 1), ("held for", 1)]
    assert notes == first
    u._enter(streams[1])
    with on(streams[1]):
        u._enter(None)
    assert notes == first
    # a capture waits for nothing outside it, and its stream's first eager call does
    streams[2].captured = True
    u._enter(streams[2])
    assert notes == first
    streams[2].captured = False
    with on(streams[2]):
        u._enter(None)
    assert notes[3:] == [(2, "waits for", "event of 0"), ("held for", 2), ("held for", 2)]
    # made within a capture: no event to wait for outside it
    notes.clear()
    streams[0].captured = True
    u = User()
    u._ready()
    streams[0].captured = False
    u._enter(streams[1])
    assert notes == [("held for", 1), ("held for", 1)]


@pytest.fixture
def entered(monkeypatch, gpu):
    """What enters on which stream, and the ABI calls, in their order."""
    seen = []
    monkeypatch.setattr(StreamUser, "_enter", lambda self, s: seen.append((type(self).__name__, s)), raising=False)
    monkeypatch.setattr(StreamUser, "_hold", lambda self, s, *t: None)
    for m, names in ((block_mod, ("mok_norm_fwd", "mok_norm_bwd")),
                     (decode_mod, ("mok_route", "mok_decode_ffn", "mok_mxfp4_quantize")), (mok, ("mok_mxfp4_tile",))):
        for n in names:
            monkeypatch.setattr(m, n, lambda *a, _n=n, **k: seen.append(_n))
    return seen


def test_calls_enter_on_their_stream(entered, gpu):
    s = gpu[0][1]
    n = RMSNorm(torch.ones(64, dtype=BF), 4, mx=True)
    x = torch.zeros(3, 64, dtype=BF)
    n.forward(x, stream=s)
    n.backward(x, stream=s)
    assert entered == [("RMSNorm", s), "mok_norm_fwd", ("RMSNorm", s), "mok_norm_bwd"]
    w = [torch.zeros(2, 128, 128, dtype=BF)] * 3
    d = MoEDecoder(torch.zeros(8, 128, dtype=BF), torch.zeros(8), torch.zeros(8, dtype=torch.int32), *w, 2, 4)
    entered.clear()
    d(torch.zeros(3, 128, dtype=BF), stream=s)
    assert entered == [("MoEDecoder", s), "mok_route", "mok_decode_ffn"]
    entered.clear()
    d.update_weights(*w, stream=s)
    assert entered[0] == ("MoEDecoder", s) and "mok_mxfp4_quantize" in entered


def test_buffers_are_all_that_the_calls_name(entered):
    """Every tensor that a call reads or writes beside its arguments is held."""
    n = RMSNorm(torch.ones(64, dtype=BF), 4, mx=True, res_type="f32")
    own = {id(t) for t in n._buffers()}
    assert all(id(t) in own for t in (n.weight, n.res, n.y, n.codes, n.scales, n.rstd, n.d_r, n.d_x, n.dw, n.ws))
    w = [torch.zeros(2, 128, 128, dtype=BF)] * 3
    d = MoEDecoder(torch.zeros(8, 128, dtype=BF), torch.zeros(8), torch.zeros(8, dtype=torch.int32), *w, 2, 4)
    own = {id(t) for t in d._buffers()}
    assert all(id(t) in own for t in (d.w_router, d.bias, d.e2l, d.topk_idx, d.topk_gate, d.out, d.ws, d.status,
                                      *d.weights.tensors))
    L = MoELayer(1, 4, 64, 4, 2, 64, 4, "bf16", 8, 0, 1, device="cpu", two_streams=False, transposed_weights=False)
    b = MoEBlock(L, torch.ones(64, dtype=BF))
    assert id(b.dw_norm) in {id(t) for t in b.norms[0]._buffers()}


def test_w4_on_a_stream(gpu, monkeypatch):
    """The layout runs with the weights' device current, after the current stream's work (which may still write the
    codes, or use the memory that the new tensors got), and what it reads and writes is held for its stream."""
    streams, notes, on = gpu
    seen = []

    class Tensor:
        """A tensor that calls itself one of a GPU."""
        dtype, device = torch.uint8, torch.device("cuda", 1)

        def __init__(self, *shape):
            self.shape, self.t = shape, torch.zeros(*shape, dtype=torch.uint8)

        def numel(self):
            return self.t.numel()

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return self.t.data_ptr()

        def record_stream(self, s):
            notes.append((id(self), s.cuda_stream))
    devices = []

    class Device(on):
        def __enter__(self):
            devices.append(self.what)
            super().__enter__()
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: Tensor(n))
    monkeypatch.setattr(_Stream, "wait_stream", lambda self, s: notes.append((self.cuda_stream, "waits for", s.cuda_stream)),
                        raising=False)
    monkeypatch.setattr(mok, "mok_mxfp4_tile", lambda *a: seen.append((a, list(notes), list(devices))))
    w, s = Tensor(2, 16, 64), Tensor(2, 16, 4)
    r = mok.make_w4(w, w, w, s, s, s, stream=streams[1])
    for args, before, made_on in seen:
        assert args[-1] is streams[1] and made_on == [torch.device("cuda", 1)]
        assert before[0] == (1, "waits for", 0)
        held = {i for i, h in before[1:] if h == 1}
        assert held >= {id(t) for t in (*r.tensors, w, s)}
    assert len(seen) == 3


def test_layer_enters_on_its_stream(gpu, monkeypatch):
    """The layer's zeros, 8-bit checkpoint and transposed weights are work of the current stream too."""
    seen = []
    monkeypatch.setattr(StreamUser, "_enter", lambda self, s: seen.append(s))
    monkeypatch.setattr(StreamUser, "_hold", lambda self, s, *t: None)
    for n in ("mok_layer_fwd", "mok_layer_bwd", "mok_layer_bwd_checkpoint", "mok_checkpoint_pack", "mok_prepare_bwd"):
        monkeypatch.setattr(layer_mod, n, lambda *a, _n=n, **k: seen.append(_n))
    L = MoELayer(1, 4, 64, 4, 2, 64, 4, "bf16", 8, 0, 1, device="cpu", two_streams=False, checkpoint=True)
    w = [torch.zeros(4, 64, dtype=BF), None, torch.arange(4, dtype=torch.int32)] + [torch.zeros(4, 64, 64, dtype=BF)] * 3
    before = L._streams
    L.set_inputs([torch.zeros(4, 64, dtype=BF)], *w)
    assert before is not None and L._streams is not before       # made anew on the current stream
    s = gpu[0][1]
    seen.clear()
    L.forward(s)
    L.backward([torch.zeros(4, 64, dtype=BF)], s)
    L.update_weights(s)
    assert seen == [s, "mok_layer_fwd", "mok_checkpoint_pack", s, "mok_layer_bwd_checkpoint", s, "mok_prepare_bwd"]
    own = {id(t) for t in L._buffers()}
    assert all(id(t) in own for t in (L.ck_codes, L.ck_scales, L.ab, L.h, L.ws, L.status, *L.staging, *L.out, *L.dx_stage,
                                      *L.d_x, *L.wt, L.dw_gate, L.dw_up, L.dw_down, L.dw_router, L.w_gate, L.offsets))


def test_backward_holds_the_gradients_it_is_given(gpu, monkeypatch):
    """d_out is read by work on the call's stream, though its owner lets it go."""
    streams, notes, _ = gpu
    for n in ("mok_layer_bwd",):
        monkeypatch.setattr(layer_mod, n, lambda *a, **k: notes.append("backward"))
    L = MoELayer(2, 4, 64, 4, 2, 64, 4, "bf16", 8, 0, 2, device="cpu", two_streams=False, transposed_weights=False)
    L.xs, L.w_router, L.bias, L.e2l, L.weights = [], None, None, None, None
    L.backward([_Buffer(notes), None], streams[1])
    assert notes == [("held for", 1), "backward"]
