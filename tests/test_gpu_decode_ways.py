"""The experts of a few tokens through ways of the launch that the sizes of
test_gpu_decode do not take (on 256 compute units), against the same formula in
64 bits with the same bounds."""
import pytest
import torch

import combine_router_top_expert_amd as mok
from test_gpu_checkpoint import _pow2
from test_gpu_decode import _place, _ref, _routing, _run, _weights
from test_gpu_norm import _near
from test_gpu_train import DEV, _gen, _log

pytestmark = pytest.mark.gpu


def _rows(T, d, x8, seed=2):
    """x, its scales and the values that they stand for."""
    x = torch.randn(T, d, generator=_gen(seed)).to(DEV, torch.bfloat16)
    if not x8:
        return x, None, x.double()
    codes, xs = torch.empty(T, d, dtype=torch.uint8, device=DEV), torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    mok.mok_mx_quantize(T, d, x, codes, xs)
    torch.cuda.synchronize()
    return codes, xs, codes.view(torch.float8_e4m3fn).double() * _pow2(xs.double() - 127).repeat_interleave(32, 1)


# T, d, I, E, k, L
WAYS = {
    # one group of waves over the contraction in the first product, its columns filling the chip: slots of experts,
    # slots of items; found among up to 1024 ids, among up to 4096, and by a launch of its own
    "search, experts": (30, 256, 512, 64, 6, 64), "search, items": (10, 256, 512, 64, 6, 64),
    "long search": (200, 256, 512, 64, 6, 64), "plan": (700, 128, 128, 256, 8, 256), "plan, E 512": (600, 128, 128, 512, 8, 256),
    # two groups behind that launch, 256 columns of the second product
    "plan, two groups": (700, 1024, 128, 256, 8, 128),
    # few tokens at more than 16 columns for every compute unit: eight waves a workgroup of the second product
    "wide, one token": (1, 7168, 256, 256, 8, 8), "wide, experts": (8, 7168, 128, 256, 8, 32),
    "wide, items": (2, 4224, 128, 64, 2, 64), "wide, none local": (1, 4224, 128, 64, 1, 1),
    # few items at slots of experts, the table beyond 256
    "few, E 300": (6, 128, 256, 300, 4, 10)}


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("way", WAYS)
def test_ways(way, x8):
    T, d, I, E, k, L = WAYS[way]
    _log("decode way", way, x8)
    w, e2l = _weights(L, d, I, T + d), _place(E, L, 5)
    topk, gate = _routing(T, E, k, 9)
    if way == "wide, one token":          # some of its experts are here
        e2l.fill_(-1)
        e2l[topk[0, ::2].long()] = torch.tensor([3, 0, 7, 4], dtype=torch.int32, device=DEV)
    x, xs, val = _rows(T, d, x8)
    out, st = _run(x, xs, topk, gate, e2l, w, d, I, L)
    assert st == 0
    ref, bound = _ref(val, topk, gate, e2l, w, d, I)
    _near(out, ref, bound, "out")
    none = (e2l[topk.long()] < 0).all(1)
    assert (out[none] == 0).all()
    again, _ = _run(x, xs, topk, gate, e2l, w, d, I, L)
    assert torch.equal(out, again)


# the few-items way at slots of items and of experts, with its table in registers and beyond 256 experts, with eight
# waves in the second product; the search at slots of items, with two groups of waves and one
IDS = [(5, 128, 128, 64, 3, 64), (9, 128, 128, 64, 3, 8), (6, 128, 128, 300, 5, 200), (6, 128, 256, 300, 4, 10),
       (5, 4224, 128, 64, 2, 64), (20, 256, 128, 64, 3, 64), (10, 256, 512, 64, 6, 64)]


@pytest.mark.parametrize("T,d,I,E,k,L", IDS)
def test_bad_and_repeated_ids(T, d, I, E, k, L):
    """Ids outside the experts latch an error and add nothing; an expert listed more than once by a token counts as
    often, with its gates' sum."""
    _log("decode ids", T, d, I, E, k, L)
    w, e2l = _weights(L, d, I, 3), _place(E, L, 1)
    here = torch.nonzero(e2l >= 0)[:, 0].to(torch.int32)
    topk, gate = _routing(T, E, k, 2)
    topk[0, 0], topk[1, 1], topk[2, 0], topk[T - 1, k - 1] = here[0], E, -1, 1 << 30
    topk[3] = here[1]                          # one expert in every slot,
    topk[4, 0], topk[4, k - 1] = here[2], here[2]   # and twice
    x, _, val = _rows(T, d, False, 4)
    out, st = _run(x, None, topk, gate, e2l, w, d, I, L)
    assert st == -6
    ref, bound = _ref(val, topk, gate, e2l, w, d, I)
    assert (ref[3] != 0).any() and (ref[4] != 0).any()
    _near(out, ref, bound, "out")


@pytest.mark.parametrize("k,L", [(4, 20), (1, 64)])
def test_all_tokens_at_one_expert(k, L):
    """16 tokens whose every slot is one expert: more items than a product takes at once, in the few-items way."""
    T, d, I, E = 16, 256, 256, 64
    _log("decode one expert", k, L)
    w, e2l = _weights(L, d, I, 3), _place(E, L, 1)
    topk = torch.full((T, k), int(torch.nonzero(e2l == 7)), dtype=torch.int32, device=DEV)
    gate = torch.rand(T, k, generator=_gen(3)).to(DEV)
    x, _, val = _rows(T, d, False, 4)
    out, st = _run(x, None, topk, gate, e2l, w, d, I, L)
    assert st == 0
    ref, bound = _ref(val, topk, gate, e2l, w, d, I)
    _near(out, ref, bound, "out")


def test_no_tokens():
    """A call without tokens launches nothing and leaves its buffers."""
    d = I = 128
    cfg = mok.make_config(1, 1, d, 4, 2, I, 4, "bf16", 0)
    w = _weights(4, d, I, 3)
    out, st = torch.full((1, d), 7.0, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    e = lambda *n: torch.empty(*n, device=DEV)  # noqa: E731
    mok.mok_decode_ffn(cfg, 0, out, None, e(1, 2).int(), e(1, 2), e(4).int(),
                       mok.make_w4(*(w[p + n] for p in ("w_", "s_") for n in ("gate", "up", "down"))), out,
                       torch.empty(mok.mok_decode_ws_bytes(cfg, 0), dtype=torch.uint8, device=DEV), st)
    torch.cuda.synchronize()
    assert (out == 7).all() and int(st) == 0
