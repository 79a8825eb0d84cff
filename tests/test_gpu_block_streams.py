"""The norm and the 4-bit experts on another stream than the one that made
them, behind work that keeps either busy: the bytes of the same calls on one
stream."""
import pytest
import torch

import combine_router_top_expert_amd as mok
from combine_router_top_expert_amd.block import RMSNorm
from combine_router_top_expert_amd.decode import MoEDecoder
from combine_router_top_expert_amd.layer import MoELayer
from test_gpu_train import DEV, _gen, _log
from test_gpu_train_streams import _busy, _same

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _norm_inputs():
    g = _gen(3)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    return (1 + 0.2 * rnd(512)).to(BF), rnd(700, 512).to(BF), rnd(700, 512), rnd(700, 512).to(BF), rnd(700, 512)


def _make_norm(w):
    return RMSNorm(w, 700, "bf16", "f32", mx=True)


def _norm_calls(n, x, res, dy, up, stream):
    y = n.forward(x, res, stream)
    d_r = n.backward(dy, up, stream=stream)
    return [y, d_r, n.dw, n.d_x, n.codes, n.scales]


def _decoder_inputs(tokens=37):
    g = _gen(4)
    E, d, I = 8, 256, 384
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV, BF)  # noqa: E731
    w = [rnd(E, d), rnd(E, I, d), rnd(E, I, d), rnd(E, d, I)]
    return w, rnd(tokens, d)


def _make_decoder(w):
    return MoEDecoder(w[0], None, torch.arange(8, dtype=torch.int32, device=DEV), *w[1:], 2, 64)


def _bytes(ts):
    torch.cuda.synchronize()
    return [t.clone().view(torch.uint8) for t in ts]


def _churn(buffers):
    """New tensors as large as these, so that memory given back too early is written over."""
    return [torch.full((t.numel() * t.element_size(),), 0xFF, dtype=torch.uint8, device=DEV) for t in buffers for _ in range(2)]


@pytest.mark.parametrize("raw", [False, True])
def test_first_call_on_another_stream(raw):
    """Made behind a busy stream, used on an idle one: after the zeros of dw and status, and the weights' layout."""
    _log("block first call", raw)
    wn, x, res, dy, up = _norm_inputs()
    w, rows = _decoder_inputs()
    want = _bytes(_norm_calls(_make_norm(wn), x, res, dy, up, None)) + _bytes([_make_decoder(w)(rows)])
    side = torch.cuda.Stream()
    arg = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream())
    n = _make_norm(wn)
    got = _norm_calls(n, x, res, dy, up, arg)
    _busy(torch.cuda.current_stream())
    dec = _make_decoder(w)
    got.append(dec(rows, stream=arg))
    _same(_bytes(got), want)
    dec.check_status()
    with torch.cuda.stream(side):              # the stream as the current one
        _busy(torch.cuda.default_stream())
    n = _make_norm(wn)
    with torch.cuda.stream(side):
        got = _norm_calls(n, x, res, dy, up, None)
    _same(_bytes(got), want[:-1])


@pytest.mark.parametrize("raw", [False, True])
def test_objects_go_before_their_calls_are_done(raw):
    """Deleted while their calls wait on a busy stream: the memory serves others only afterwards."""
    _log("block deleted", raw)
    wn, x, res, dy, up = _norm_inputs()
    w, rows = _decoder_inputs()
    want = _bytes(_norm_calls(_make_norm(wn), x, res, dy, up, None)) + _bytes([_make_decoder(w)(rows)])
    side = torch.cuda.Stream()
    arg = side.cuda_stream if raw else side
    n, dec = _make_norm(wn), _make_decoder(w)
    torch.cuda.synchronize()
    _busy(side)
    got = _norm_calls(n, x, res, dy, up, arg)
    got.append(dec(rows, stream=arg))
    sizes = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8) for t in n._buffers() + dec._buffers()]
    del n, dec
    junk = _churn(sizes)
    _same(_bytes(got), want)
    assert all(bool((t == 0xFF).all()) for t in junk)


def test_weights_of_a_busy_stream():
    """Other weights, given and let go of while a busy stream has yet to read them."""
    _log("block weights stream")
    w, rows = _decoder_inputs()
    dec = _make_decoder(w)
    dec.update_weights(2 * w[1], w[2], w[3])
    want = _bytes([dec(rows)])
    dec = _make_decoder(w)
    side = torch.cuda.Stream()
    new = [2 * w[1], w[2].clone(), w[3].clone()]
    torch.cuda.synchronize()
    _busy(side)
    dec.update_weights(*new, stream=side)
    sizes = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8) for t in new]
    del new
    junk = _churn(sizes)
    got = dec(rows, stream=side)
    _same(_bytes([got]), want)
    del junk


@pytest.mark.parametrize("raw", [False, True])
def test_w4_on_a_busy_stream(raw):
    """Codes that the current stream still writes, laid out on a busy stream and let go of at once."""
    _log("w4 stream", raw)
    g = _gen(6)
    codes = [torch.randint(0, 256, (2, 256, 128), generator=g, dtype=torch.uint8).to(DEV) for _ in range(3)]
    scales = [torch.randint(118, 123, (2, 256, 8), generator=g, dtype=torch.uint8).to(DEV) for _ in range(3)]
    want = _bytes(mok.make_w4(*codes, *scales).tensors)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(side)
    _busy(torch.cuda.current_stream())
    mine = [t.clone() for t in codes + scales]
    w = mok.make_w4(*mine, stream=side.cuda_stream if raw else side)
    sizes = [torch.empty(t.numel(), dtype=torch.uint8) for t in mine]
    del mine
    junk = _churn(sizes)
    _same(_bytes(w.tensors), want)
    del junk


@pytest.mark.parametrize("prec", ["f32", "bf16", "mxfp8"])
def test_layer_on_another_stream(prec):
    """A checkpointing layer made behind a busy stream and run at once on another, and deleted before that is done."""
    _log("layer stream", prec)
    S, T, d, E, k, I, dt = 1, 64, 128, 4, 2, 128, torch.float32 if prec == "f32" else BF
    g = _gen(3)
    rnd = lambda *s: (s[-1] ** -0.5 * torch.randn(*s, generator=g)).to(DEV, dt)  # noqa: E731
    x, dout, w = rnd(T, d), rnd(T, d), [rnd(E, d), rnd(E, I, d), rnd(E, I, d), rnd(E, d, I)]
    e2l = torch.arange(E, dtype=torch.int32, device=DEV)

    def run(side):
        torch.cuda.synchronize()
        if side is not None:
            _busy(torch.cuda.current_stream())
        L = MoELayer(S, T, d, E, k, I, E, prec, T * k, 0, 1, device=DEV, checkpoint=True, two_streams=False)
        L.set_inputs([x], w[0], None, e2l, *w[1:])
        if side is not None:
            L.forward(side)
            _busy(side)
        else:
            L.forward()
        L.backward([dout], side)
        out = [L.out[0], L.d_x[0], L.dw_gate, L.dw_router, L.ck_codes]
        if side is not None:
            keep = {t.data_ptr() for t in (*out, x, *w, e2l)}
            large = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8) for t in L._buffers() if t.data_ptr() not in keep]
            del L
            junk = _churn(large)
            del junk
        return _bytes(out)
    want = run(None)
    _same(run(torch.cuda.Stream()), want)
