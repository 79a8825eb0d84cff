"""Order of the training calls over streams: AdamW used from several streams,
each behind work that keeps it busy, gives the bytes of the same calls on one
stream."""
import pytest
import torch

from combine_router_top_expert_amd.optim import AdamW
from test_gpu_train import DEV, _balance_layer, _gen, _log

pytestmark = pytest.mark.gpu

SIZES = (70000, 333, 4096)


def _busy(stream, n=20):
    """Some milliseconds of work on the stream."""
    with torch.cuda.stream(stream):
        t = torch.ones(1 << 26, device=DEV)
        for _ in range(n):
            t.mul_(1.0)


def _make(**kw):
    gen = _gen(8)
    ps = [torch.randn(n, generator=gen).to(DEV, dt) for n, dt in zip(SIZES, (torch.float32, torch.bfloat16, torch.float32))]
    return ps, AdamW(ps, lr=1e-2, state_bits=[32, 32, 8], max_norm=0.5, seed=4, **kw)


def _grads(k):
    gen = _gen(100)
    return [[torch.randn(n, generator=gen).to(DEV) for n in SIZES] for _ in range(k)]


def _state(ps, opt):
    torch.cuda.synchronize()
    return [t.clone().view(torch.uint8) for t in (*ps, *opt.m, *opt.v, opt.norm, *(w for w in opt.master if w is not None))]


def _same(a, b):
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("capturable", [False, True])
def test_adamw_steps_on_several_streams(capturable):
    _log("adamw streams", capturable)
    gs = _grads(4)
    ps, opt = _make(capturable=capturable)
    for g in gs:
        opt.step(g)
    want = _state(ps, opt)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ps, opt = _make(capturable=capturable)
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream())
    opt.step(gs[0])                      # behind the busy stream,
    opt.step(gs[1], stream=s1)           # after it though s1 is idle,
    _busy(s1)
    opt.step(gs[2], stream=s2)           # after s1's,
    _busy(s2)
    opt.step(gs[3])                      # and after s2's
    _same(_state(ps, opt), want)


def test_adamw_set_lr_after_a_step_on_a_busy_stream():
    _log("adamw set_lr stream")
    gs = _grads(3)
    rates = (1e-2, 1e-3, 1e-1)

    def run(stream):
        ps, opt = _make(capturable=True)
        torch.cuda.synchronize()
        for g, lr in zip(gs, rates):
            opt.set_lr(lr)
            if stream is not None:
                _busy(stream)
            opt.step(g, stream=stream)
        return _state(ps, opt)
    _same(run(torch.cuda.Stream()), run(None))


def test_adamw_state_after_a_step_on_a_busy_stream():
    """state_dict and load_state_dict right behind a step on another stream,
    and a step on it right behind them."""
    _log("adamw state stream")
    gs = _grads(4)

    def run(stream):
        ps, opt = _make(capturable=True)
        other = _make(capturable=True)[1]
        other.step(gs[3])
        torch.cuda.synchronize()
        out = []
        for g in gs[:2]:
            if stream is not None:
                _busy(stream)
            opt.step(g, stream=stream)
            d = opt.state_dict()
            out.append([t.clone().view(torch.uint8) for n in ("m", "v") for t in d[n]] +
                       [torch.tensor([d["step"]], dtype=torch.uint8)])
        if stream is not None:
            _busy(stream)
        opt.step(gs[2], stream=stream)
        opt.load_state_dict(other.state_dict())
        _busy(torch.cuda.current_stream())
        opt.step(gs[3], stream=stream)
        return sum(out, []) + _state(ps, opt)
    _same(run(torch.cuda.Stream()), run(None))


def test_adamw_captured_step_on_a_second_stream():
    """A step on another stream of a capture, with set_lr around it, joins the
    capture again and replays as eager steps do."""
    _log("adamw capture stream")
    gs = _grads(4)
    eager_ps, eager = _make(capturable=True)
    ps, opt = _make(capturable=True)
    slot = [t.clone() for t in gs[0]]
    opt.bind(slot)
    opt.step()
    eager.step(gs[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.set_lr(1e-3)
        opt.step(stream=side)
        opt.set_lr(1e-1)
        opt.step(stream=side)
    for i in range(1, 4):
        for s, g in zip(slot, gs[i]):
            s.copy_(g)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for lr in (1e-3, 1e-1):
            eager.set_lr(lr)
            eager.step(gs[i])
        _same(_state(ps, opt), _state(eager_ps, eager))
    del graph


def _churn(sizes):
    """New tensors of these sizes on the current stream, all NaN, so memory
    that was given back too early is written over."""
    return [torch.full((n,), float("nan"), device=DEV) for n in sizes for _ in range(4)]


def test_adamw_keeps_gradients_of_a_busy_stream():
    """Gradients that the caller lets go of right after a step on another
    stream are read before their memory serves others."""
    _log("adamw gradients stream")
    gs = _grads(3)

    def run(stream):
        ps, opt = _make()
        torch.cuda.synchronize()
        for g in gs:
            mine = [t.clone() for t in g]
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
                _busy(stream)
            opt.step(mine, stream=stream)
            del mine
            opt.bind(gs[0])
            junk = _churn(SIZES)
            del junk
        return _state(ps, opt)
    _same(run(torch.cuda.Stream()), run(None))


def test_adamw_goes_before_its_step_is_done():
    """The optimizer is deleted while its step waits on a busy stream: its
    workspace and moments serve others only afterwards."""
    _log("adamw deleted")
    g = _grads(1)[0]

    def run(stream):
        ps, opt = _make()
        opt.bind(g)
        torch.cuda.synchronize()
        if stream is not None:
            _busy(stream)
        opt.step(stream=stream)
        del opt
        junk = _churn((*SIZES, 64, 2, 128, 3, 11))
        torch.cuda.synchronize()
        assert all(bool(torch.isnan(t).all()) for t in junk)
        return [p.clone().view(torch.uint8) for p in ps]
    _same(run(torch.cuda.Stream()), run(None))


@pytest.mark.parametrize("raw", [False, True])
def test_balance_keeps_offsets_masks_and_weights_of_a_busy_stream(raw):
    """Tensors that the caller lets go of right after a call on another stream
    (a torch stream or its handle) are read before their memory serves others."""
    _log("balance stream", raw)

    def run(stream):
        L, dout, _ = _balance_layer()
        L.forward()
        L.backward(dout)
        mask = torch.ones(300, dtype=torch.uint8)
        mask[40:70] = 0
        torch.cuda.synchronize()
        arg = stream.cuda_stream if raw and stream is not None else stream
        for off in ([0, 100, 300], [0, 50, 290]):
            o, m, w = (t.to(DEV) for t in (torch.tensor(off, dtype=torch.int32), mask, torch.tensor([2.0, 0.5])))
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
                _busy(stream)
            loss = L.balance_loss(0.5, 0.01, o, m, stream=arg)
            L.balance_backward(w, stream=arg)
            L._bal_keep = None
            del o, m, w
            junk = [torch.full((n,), 7, dtype=dt, device=DEV) for n, dt in
                    ((3, torch.int32), (300, torch.uint8), (2, torch.float32)) for _ in range(8)]
            del junk
        torch.cuda.synchronize()
        L.check_status()
        return [t.clone() for t in (loss, L.counts_all, L.d_x[0], L.dw_router)]
    _same(run(torch.cuda.Stream()), run(None))


def test_adamw_steps_from_loaded_parameters():
    """Parameters loaded before a step on a busy stream, and taken over: the
    step of an optimizer made of them."""
    _log("adamw take_params")
    gs = _grads(2)
    gen = _gen(55)
    new = [torch.randn(n, generator=gen).to(DEV) for n in SIZES]

    def run(stream):
        ps, opt = _make()
        torch.cuda.synchronize()
        if stream is not None:
            _busy(stream)
        opt.step(gs[0], stream=stream)
        torch.cuda.synchronize()
        for p, w in zip(ps, new):
            p.copy_(w)
        opt.take_params()
        _busy(torch.cuda.current_stream())
        opt.step(gs[1], stream=stream)
        return ps, opt
    ps, opt = run(torch.cuda.Stream())
    fresh = [t.to(p.dtype) for t, p in zip(new, ps)]
    other = AdamW(fresh, lr=1e-2, state_bits=[32, 32, 8], max_norm=0.5, seed=4)
    first = _make()[1]
    first.step(gs[0])
    state = first.state_dict()
    state["master"] = other.master
    other.load_state_dict(state)
    other.step(gs[1])
    _same(_state(ps, opt), _state(fresh, other))


def test_adamw_step_on_a_captured_stream_that_is_not_the_current_one():
    """The capture of the step's own stream counts: refused with a host step
    number, replayed like eager steps with one on the device."""
    _log("adamw captured other")
    gs = _grads(4)
    frozen = _make()[1]
    frozen.bind(gs[0])
    eager_ps, eager = _make(capturable=True)
    ps, opt = _make(capturable=True)
    slot = [t.clone() for t in gs[0]]
    opt.bind(slot)
    opt.step()
    eager.step(gs[0])
    torch.cuda.synchronize()
    main, cap = torch.cuda.current_stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        with torch.cuda.stream(main):
            with pytest.raises(RuntimeError, match="capturable"):
                frozen.step(stream=cap)
            opt.step(stream=cap)
    for i in range(1, 4):
        for s, g in zip(slot, gs[i]):
            s.copy_(g)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager.step(gs[i])
        _same(_state(ps, opt), _state(eager_ps, eager))
    del graph


def test_adamw_refuses_a_stream_of_another_device():
    """A stream that is no stream of the parameters' GPU cannot order the step."""
    _, opt = _make()

    class Other:
        device = torch.device("cuda", 7)
    with pytest.raises(ValueError, match="cuda:7"):
        opt.step(_grads(1)[0], stream=Other())


def test_adamw_step_writes_no_memory_that_was_given_back():
    """A parameter that gets other memory after bind: the step writes the
    memory that was bound, which nobody else has been given."""
    _log("adamw .data")
    gs = _grads(1)[0]
    ps, opt = _make()
    opt.bind(gs)
    for p in ps:
        p.data = torch.zeros_like(p)
    junk = _churn(SIZES) + [torch.full((SIZES[1],), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    opt.step()
    torch.cuda.synchronize()
    assert all(bool(torch.isnan(t).all()) for t in junk) and not any(p.any() for p in ps)
    opt.take_params()
    opt.step(gs)
    torch.cuda.synchronize()
    assert all(bool(p.any()) for p in ps)
