"""Python binding of the gfx950 MoE layer library (``libmok.so``).

Argument marshalling only: every function below has the name of a C entry
point declared in ``include/mok.h``, turns torch tensors into device pointers
(PyTorch provides device memory and streams) and raises ``MokError`` on a
negative status.  Every step of the layer runs in the library's HIP kernels;
there is no fallback: importing the binding works without a GPU, but calling
into it needs the built library (``build.build()``) and a gfx950 device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
# MOK_LIB: another build of the library to load instead (the host-sanitizer
# build that the CPU tests run the argument checks through)
LIB_PATH = os.environ.get("MOK_LIB") or os.path.join(HERE, "libmok.so")

MOK_F32, MOK_BF16, MOK_MXFP8 = 0, 1, 2
PREC = {"f32": MOK_F32, "bf16": MOK_BF16, "mxfp8": MOK_MXFP8}
MAX_SOURCES = 64

STATUS = {
    0: "MOK_OK", -1: "MOK_EINVAL", -2: "MOK_ESHAPE", -3: "MOK_EDEVICE", -4: "MOK_ECAPACITY",
    -5: "MOK_ETIMEOUT", -6: "MOK_EROUTE", -7: "MOK_ESCRATCH", -8: "MOK_EGROUP",
}

# every symbol include/mok.h declares
EXPORTS = ("mok_workspace_bytes", "mok_route", "mok_layout", "mok_dispatch", "mok_expert_ffn",
           "mok_combine", "mok_layer_fwd", "mok_layer_bwd", "mok_mx_quantize", "mok_tune_fwd",
           "mok_ring_layout", "mok_hbm_stream", "mok_layer_fwd_noalloc", "mok_layer_fwd_macro",
           "mok_prepare_bwd", "mok_mx_quantize_f32", "mok_mfma_probe", "mok_route_logits",
           "mok_balance_ws_bytes", "mok_balance_fwd", "mok_balance_bwd", "mok_router_bwd_ws_bytes",
           "mok_router_bwd", "mok_grad_norm_ws_bytes", "mok_grad_norm", "mok_adamw", "mok_norm_fwd",
           "mok_norm_bwd_ws_bytes", "mok_norm_bwd", "mok_checkpoint_pack", "mok_checkpoint_unpack",
           "mok_checkpoint_swiglu_bwd", "mok_layer_bwd_checkpoint", "mok_mxfp4_quantize", "mok_mxfp4_tile",
           "mok_decode_ws_bytes", "mok_decode_ffn", "mok_version")


class MokError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


class mok_config(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("T_src", ctypes.c_int32), ("d", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E_local", ctypes.c_int32), ("prec", ctypes.c_int32), ("R_cap", ctypes.c_int32),
                ("minibatch_rows", ctypes.c_int32), ("ring_bytes", ctypes.c_int64),
                ("comm_wgs", ctypes.c_int32), ("gemm_wgs", ctypes.c_int32),
                ("wait_limit_us", ctypes.c_int32), ("trace", ctypes.c_void_p),
                ("aux", ctypes.c_void_p), ("bwd_ring_bytes", ctypes.c_int64)]


class mok_trace(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)),
                ("names", ctypes.POINTER(ctypes.c_char_p)),
                ("capacity", ctypes.c_int32), ("count", ctypes.c_int32),
                ("from_", ctypes.POINTER(ctypes.c_int32)),
                ("last_stream", ctypes.c_void_p * 2), ("last_idx", ctypes.c_int32 * 2)]


class mok_aux(ctypes.Structure):
    _fields_ = [("stream", ctypes.c_void_p), ("events", ctypes.c_void_p * 3)]


def _hip_runtime():
    """The HIP runtime instance this process already uses (torch's copy when
    torch is loaded), with the event functions' signatures declared."""
    path = None
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                if "libamdhip64" in line:
                    path = line.split()[-1]
                    break
    except OSError:
        pass
    hip = ctypes.CDLL(path or "libamdhip64.so.7")
    P = ctypes.c_void_p
    hip.hipEventCreate.argtypes = [ctypes.POINTER(P)]
    hip.hipEventCreateWithFlags.argtypes = [ctypes.POINTER(P), ctypes.c_uint]
    hip.hipEventCreateWithFlags.restype = ctypes.c_int
    hip.hipEventSynchronize.argtypes = [P]
    hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), P, P]
    hip.hipEventDestroy.argtypes = [P]
    for fn in (hip.hipEventCreate, hip.hipEventSynchronize, hip.hipEventElapsedTime,
               hip.hipEventDestroy):
        fn.restype = ctypes.c_int
    return hip


class Trace:
    """Caller-owned kernel timing: `capacity` hipEvents (created through the HIP
    runtime) handed to the library through mok_config.trace."""

    def __init__(self, capacity: int):
        self.hip = _hip_runtime()
        self.capacity = capacity
        self.events = (ctypes.c_void_p * capacity)()
        for i in range(capacity):
            ev = ctypes.c_void_p()
            rc = self.hip.hipEventCreate(ctypes.byref(ev))
            if rc != 0:
                raise RuntimeError(f"hipEventCreate failed: {rc}")
            self.events[i] = ev
        self.names = (ctypes.c_char_p * capacity)()
        self.from_ = (ctypes.c_int32 * capacity)()
        self.t = mok_trace(self.events, self.names, capacity, 0, self.from_)

    def attach(self, cfg: "mok_config"):
        cfg.trace = ctypes.addressof(self.t)

    @staticmethod
    def detach(cfg: "mok_config"):
        cfg.trace = None

    def reset(self):
        self.t.count = 0
        self.t.last_stream[0] = self.t.last_stream[1] = None
        self.t.last_idx[0] = self.t.last_idx[1] = 0

    def records(self):
        """[(name, ms since the previous event on the same stream)] for every
        recorded event but the 'start' marks of each call and stream."""
        if self.t.count == 0:
            return []
        rc = self.hip.hipEventSynchronize(self.events[self.t.count - 1])
        if rc != 0:
            raise RuntimeError(f"hipEventSynchronize failed: {rc}")
        out = []
        for i in range(1, self.t.count):
            name = self.names[i].decode()
            if name == "start" or self.from_[i] < 0:
                continue
            ms = ctypes.c_float()
            rc = self.hip.hipEventElapsedTime(ctypes.byref(ms), self.events[self.from_[i]],
                                              self.events[i])
            if rc != 0:
                raise RuntimeError(f"hipEventElapsedTime failed: {rc}")
            out.append((name, float(ms.value)))
        return out

    def __del__(self):
        try:
            for i in range(self.capacity):
                self.hip.hipEventDestroy(self.events[i])
        except Exception:
            pass


class AuxStream:
    """A second stream for the backward pass (a torch stream of default
    priority) and the three events mok_aux asks for; attach() points a
    mok_config at it."""

    def __init__(self, device):
        import torch
        self.hip = _hip_runtime()
        self.stream = torch.cuda.Stream(device=device)
        evs = []
        for _ in range(3):
            ev = ctypes.c_void_p()
            rc = self.hip.hipEventCreateWithFlags(ctypes.byref(ev), 2)  # hipEventDisableTiming
            if rc != 0:
                raise RuntimeError(f"hipEventCreateWithFlags failed: {rc}")
            evs.append(ev.value)
        self.a = mok_aux(self.stream.cuda_stream, (ctypes.c_void_p * 3)(*evs))

    def attach(self, cfg: "mok_config"):
        cfg.aux = ctypes.addressof(self.a)

    def __del__(self):
        try:
            for i in range(3):
                self.hip.hipEventDestroy(self.a.events[i])
        except Exception:
            pass


class mok_expert_weights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("wt_down", ctypes.c_void_p), ("st_down", ctypes.c_void_p),
                ("wt_gu", ctypes.c_void_p), ("st_gu", ctypes.c_void_p)]


class mok_fwd_state(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_gate", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("row_src", ctypes.c_void_p), ("dest_row", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("ab", ctypes.c_void_p), ("h_scale", ctypes.c_void_p),
                ("logits", ctypes.c_void_p)]


class mok_layer_call(ctypes.Structure):
    _fields_ = [("own_lo", ctypes.c_int32), ("own_n", ctypes.c_int32),
                ("src_x", ctypes.c_void_p), ("st", ctypes.POINTER(mok_fwd_state)),
                ("staging", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class mok_balance(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("G", ctypes.c_int32),
                ("group_offsets", ctypes.c_void_p), ("token_mask", ctypes.c_void_p)]


class mok_param(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("p_type", ctypes.c_int32),
                ("g_type", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("weight_decay", ctypes.c_float)]


class mok_adamw_args(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("grad_scale", ctypes.c_float), ("random_params", ctypes.c_int32),
                ("dev_scale", ctypes.c_void_p), ("dev_lr", ctypes.c_void_p),
                ("dev_step", ctypes.c_void_p)]


class mok_w4(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]


MAX_CALLS = 8

_lib = None


def lib():
    """Load libmok.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -m combine_router_top_expert_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        cfgp = ctypes.POINTER(mok_config)
        L.mok_workspace_bytes.argtypes = [cfgp]
        L.mok_workspace_bytes.restype = ctypes.c_size_t
        L.mok_route.argtypes = [cfgp, I32, P, P, P, P, P, P]
        L.mok_layout.argtypes = [cfgp, P, P, P, P, P, P, P, P, P]
        L.mok_dispatch.argtypes = [cfgp, P, P, P, P, P, P, P]
        L.mok_expert_ffn.argtypes = [cfgp, P, P, P, ctypes.POINTER(mok_expert_weights), P, P, P, P,
                                     P, P]
        L.mok_combine.argtypes = [cfgp, P, P, P, P, I32, I32, P, P, P]
        L.mok_layer_fwd.argtypes = [cfgp, I32, I32, P, P, P, P,
                                    ctypes.POINTER(mok_expert_weights),
                                    ctypes.POINTER(mok_fwd_state), P, P, P, P, P]
        L.mok_layer_bwd.argtypes = [cfgp, I32, I32, P, P, P, P, ctypes.POINTER(mok_expert_weights),
                                    ctypes.POINTER(mok_fwd_state), P, P, P, P, P, P, P, P, P, P, P]
        L.mok_mx_quantize.argtypes = [I64, I64, P, P, P, P]
        L.mok_tune_fwd.argtypes = [cfgp, P, I32, P, I32, I32, ctypes.c_size_t, I32, I32, P, P, P, P,
                                   ctypes.POINTER(mok_expert_weights),
                                   ctypes.POINTER(mok_fwd_state), P, P, P, P, P, cfgp, P]
        L.mok_ring_layout.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t),
                                      ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(I32)]
        L.mok_hbm_stream.argtypes = [I32, P, P, I64, P]
        L.mok_mfma_probe.argtypes = [I32, I32, I64, I32, P, P]
        L.mok_layer_fwd_noalloc.argtypes = [cfgp, I32, I32, P, P, P, P,
                                            ctypes.POINTER(mok_expert_weights),
                                            ctypes.POINTER(mok_fwd_state), P, P, P, P]
        L.mok_layer_fwd_macro.argtypes = [cfgp, I32, ctypes.POINTER(mok_layer_call), P, P, P,
                                          ctypes.POINTER(mok_expert_weights), P, P, P]
        L.mok_prepare_bwd.argtypes = [cfgp, P, P, P, P, P, P, P, P]
        L.mok_mx_quantize_f32.argtypes = [I64, I64, P, P, P, P]
        balp, parp = ctypes.POINTER(mok_balance), ctypes.POINTER(mok_param)
        L.mok_route_logits.argtypes = [cfgp, I32, P, P, P, P, P, P, P]
        L.mok_balance_ws_bytes.argtypes = [cfgp, I32, balp]
        L.mok_balance_fwd.argtypes = [cfgp, I32, balp, P, P, P, P, P, P, P, P, P]
        L.mok_balance_bwd.argtypes = [cfgp, I32, balp, P, P, P, P, P, P, P]
        L.mok_router_bwd_ws_bytes.argtypes = [cfgp, I32]
        L.mok_router_bwd.argtypes = [cfgp, I32, I32, P, P, P, P, P, P, I32, P, P]
        L.mok_grad_norm_ws_bytes.argtypes = [I32, parp]
        L.mok_grad_norm.argtypes = [I32, parp, ctypes.c_float, P, P, P]
        L.mok_adamw.argtypes = [I32, parp, ctypes.POINTER(mok_adamw_args), P]
        L.mok_norm_fwd.argtypes = [cfgp, I32, P, P, I32, P, ctypes.c_float, P, P, P, P, P, P]
        L.mok_norm_bwd_ws_bytes.argtypes = [cfgp, I32]
        L.mok_norm_bwd.argtypes = [cfgp, I32, P, P, I32, P, P, P, P, P, P, I32, P, P]
        L.mok_checkpoint_pack.argtypes = [cfgp, P, P, P, P, P]
        L.mok_checkpoint_unpack.argtypes = [cfgp, P, P, P, P, P, P]
        L.mok_checkpoint_swiglu_bwd.argtypes = [cfgp, P, P, P, P, I64, P, P, P]
        L.mok_layer_bwd_checkpoint.argtypes = [cfgp, I32, I32, P, P, P, P,
                                               ctypes.POINTER(mok_expert_weights),
                                               ctypes.POINTER(mok_fwd_state), P, P, P, P, P, P, P,
                                               P, P, P, P, P, P]
        L.mok_mxfp4_quantize.argtypes = [I64, I64, I32, P, P, P, P]
        L.mok_mxfp4_tile.argtypes = [I64, I64, P, P, P, P, P]
        L.mok_decode_ws_bytes.argtypes = [cfgp, I32]
        L.mok_decode_ffn.argtypes = [cfgp, I32, P, P, P, P, P, ctypes.POINTER(mok_w4), P, P, P, P]
        L.mok_version.argtypes = []
        L.mok_version.restype = ctypes.c_char_p
        for name in EXPORTS[:-1]:
            getattr(L, name).restype = (ctypes.c_size_t if name.endswith("_bytes")
                                        else ctypes.c_int)
        _lib = L
    return _lib


# ------------------------------------------------------------------ marshalling helpers
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None


def _stream(stream) -> Optional[int]:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            # torch.cuda.current_stream() builds a Stream object, 3 us of every
            # call; the raw handle of the current device's stream is the same
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            dev = torch.cuda.current_device
            _raw_stream = ((lambda: raw(dev())) if raw is not None
                           else (lambda: torch.cuda.current_stream().cuda_stream))
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _table(tensors: Sequence) -> ctypes.Array:
    arr = (ctypes.c_void_p * MAX_SOURCES)()
    for i, t in enumerate(tensors):
        arr[i] = _ptr(t)
    return arr


def _check(fn: str, rc: int):
    if rc != 0:
        raise MokError(fn, rc)


def make_config(S, T_src, d, E, k, I, E_local, prec, R_cap, minibatch_rows=256, ring_bytes=0,
                comm_wgs=0, gemm_wgs=0, wait_limit_us=0, bwd_ring_bytes=0) -> mok_config:
    return mok_config(S, T_src, d, E, k, I, E_local, PREC.get(prec, prec), R_cap, minibatch_rows,
                      ring_bytes, comm_wgs, gemm_wgs, wait_limit_us, None, None, bwd_ring_bytes)


def make_weights(w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None, wt_down=None,
                 st_down=None, wt_gu=None, st_gu=None) -> mok_expert_weights:
    return mok_expert_weights(_ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up),
                              _ptr(s_down), _ptr(wt_down), _ptr(st_down), _ptr(wt_gu),
                              _ptr(st_gu))


def make_state(topk_idx, topk_gate, counts, offsets, row_src, dest_row, h, ab,
               h_scale=None, logits=None) -> mok_fwd_state:
    return mok_fwd_state(_ptr(topk_idx), _ptr(topk_gate), _ptr(counts), _ptr(offsets),
                         _ptr(row_src), _ptr(dest_row), _ptr(h), _ptr(ab), _ptr(h_scale),
                         _ptr(logits))


def make_balance(alpha, beta=0.0, groups=0, group_offsets=None, token_mask=None) -> mok_balance:
    """groups 0: all rows are one group.  The caller keeps the tensors alive."""
    return mok_balance(alpha, beta, groups, _ptr(group_offsets), _ptr(token_mask))


def _type(t) -> int:
    """MOK_F32 or MOK_BF16 of a tensor (anything else is refused)."""
    import torch
    if t is None or t.dtype == torch.float32:
        return MOK_F32
    if t.dtype == torch.bfloat16:
        return MOK_BF16
    raise TypeError(f"float32 or bfloat16 expected, got {t.dtype}")


def make_param(p=None, g=None, m=None, v=None, master=None, m_scale=None, v_scale=None,
               weight_decay=0.0) -> mok_param:
    """Descriptor of one tensor of mok_adamw / mok_grad_norm (which needs g
    only).  Tensors are contiguous; 8-bit moments are told by their scales."""
    for t in (p, g, m, v, master, m_scale, v_scale):
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors of an optimizer step must be contiguous")
    import torch
    n = (g if g is not None else p).numel()
    if any(t.numel() != n for t in (p, m, v, master) if t is not None):
        raise ValueError("tensors of one parameter differ in size")
    if (m_scale is None) != (v_scale is None):
        raise ValueError("8-bit moments need both scales")
    if any(t.numel() != (n + 31) // 32 for t in (m_scale, v_scale) if t is not None):
        raise ValueError("one scale per 32 elements")
    code = torch.float32 if m_scale is None else torch.uint8
    for t, want in ((m, code), (v, code), (master, torch.float32), (m_scale, torch.uint8),
                    (v_scale, torch.uint8)):
        if t is not None and t.dtype != want:
            raise TypeError(f"{want} expected, got {t.dtype}")
    return mok_param(_ptr(p), _ptr(g), _ptr(master), _ptr(m), _ptr(v), _ptr(m_scale),
                     _ptr(v_scale), n, _type(p), _type(g), 32 if m_scale is None else 8,
                     weight_decay)


def make_w4(w_gate, w_up, w_down, s_gate, s_up, s_down, stream=None, into=None) -> mok_w4:
    """Expert weights in 4 bits from rows of codes (``mok_mxfp4_quantize``):
    w_gate, w_up uint8 [E_local, I, d/2], w_down [E_local, d, I/2], scales
    s_* [..., K/32].  Lays them out as ``mok_decode_ffn`` reads them
    (``mok_mxfp4_tile``), in new tensors that the result holds, or in those of
    an earlier result of the same sizes (into).  On `stream` it comes after the
    current one's work, and the tensors are held for it."""
    import contextlib
    import torch
    from .streams import StreamUser
    user = StreamUser()
    user.device = w_gate.device
    rows = []
    for w, s in ((w_gate, s_gate), (w_up, s_up), (w_down, s_down)):
        K, n = 2 * w.shape[-1], w.numel() // w.shape[-1]
        for t, size in ((w, n * K // 2), (s, n * K // 32)):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != size or t.device != w_gate.device:
                raise ValueError(f"contiguous uint8 tensor of {size} on {w_gate.device} expected, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
        rows.append((n, K, w, s))
    sizes = [size for n, K, _, _ in rows for size in (n * K // 2, n * 16 * -(-K // 512))]
    if into is None:
        tensors = [torch.empty(size, dtype=torch.uint8, device=w_gate.device) for size in sizes]
    else:
        tensors = into.tensors
        if [t.numel() for t in tensors] != sizes or tensors[0].device != w_gate.device:
            raise ValueError("weights of other sizes, or on another device")
    on_gpu = w_gate.device.type == "cuda"
    with torch.cuda.device(w_gate.device) if on_gpu else contextlib.nullcontext():
        if on_gpu:
            user._after_current(stream, *tensors, *(t for _, _, w, s in rows for t in (w, s)))
        for i, (n, K, w, s) in enumerate(rows):
            mok_mxfp4_tile(n, K, w, s, tensors[2 * i], tensors[2 * i + 1], stream)
    r = mok_w4(*(t.data_ptr() for t in tensors[0::2] + tensors[1::2])) if into is None else into
    r.tensors = tensors
    return r


def make_params(params: Sequence[mok_param]) -> ctypes.Array:
    return (mok_param * len(params))(*params)


def make_adamw(lr, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0, grad_scale=1.0,
               random_params=False, dev_scale=None, dev_lr=None, dev_step=None) -> mok_adamw_args:
    """dev_scale fp32, dev_lr fp64 and dev_step int64 device tensors, or None."""
    return mok_adamw_args(lr, beta1, beta2, eps, step, seed & 0xFFFFFFFFFFFFFFFF, grad_scale,
                          int(random_params), _ptr(dev_scale), _ptr(dev_lr), _ptr(dev_step))


# ------------------------------------------------------------------ entry points
def mok_version() -> str:
    return lib().mok_version().decode()


def mok_workspace_bytes(cfg: mok_config) -> int:
    return int(lib().mok_workspace_bytes(ctypes.byref(cfg)))


def mok_route(cfg, T, x, w_router, bias, topk_idx, topk_gate, stream=None):
    _check("mok_route", lib().mok_route(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias),
                                        _ptr(topk_idx), _ptr(topk_gate), _stream(stream)))


def mok_layout(cfg, topk_idx_all, expert_to_local, counts, offsets, row_src, dest_row, ws,
               dev_status, stream=None):
    _check("mok_layout", lib().mok_layout(ctypes.byref(cfg), _ptr(topk_idx_all),
                                          _ptr(expert_to_local), _ptr(counts), _ptr(offsets),
                                          _ptr(row_src), _ptr(dest_row), _ptr(ws), _ptr(dev_status),
                                          _stream(stream)))


def mok_dispatch(cfg, src_x, row_src, offsets, x_perm, x_scale, dev_status, stream=None):
    _check("mok_dispatch", lib().mok_dispatch(ctypes.byref(cfg), _table(src_x), _ptr(row_src),
                                              _ptr(offsets), _ptr(x_perm), _ptr(x_scale),
                                              _ptr(dev_status), _stream(stream)))


def mok_expert_ffn(cfg, x_perm, x_scale, offsets, weights: mok_expert_weights, h, h_scale, ab, y,
                   dev_status, stream=None):
    _check("mok_expert_ffn", lib().mok_expert_ffn(ctypes.byref(cfg), _ptr(x_perm), _ptr(x_scale),
                                                  _ptr(offsets), ctypes.byref(weights), _ptr(h),
                                                  _ptr(h_scale), _ptr(ab), _ptr(y), _ptr(dev_status),
                                                  _stream(stream)))


def mok_combine(cfg, y, dest_row, topk_gate, staging, own_lo, own_n, out, dev_status,
                stream=None):
    _check("mok_combine", lib().mok_combine(ctypes.byref(cfg), _ptr(y), _ptr(dest_row),
                                            _ptr(topk_gate), _table(staging), own_lo, own_n,
                                            _table(out) if out is not None else None,
                                            _ptr(dev_status), _stream(stream)))


def mok_layer_fwd(cfg, own_lo, own_n, src_x, w_router, bias, expert_to_local,
                  weights: mok_expert_weights, state: mok_fwd_state, staging, out, ws, dev_status,
                  stream=None):
    _check("mok_layer_fwd", lib().mok_layer_fwd(
        ctypes.byref(cfg), own_lo, own_n, _table(src_x), _ptr(w_router), _ptr(bias),
        _ptr(expert_to_local), ctypes.byref(weights), ctypes.byref(state), _table(staging),
        _table(out) if out is not None else None, _ptr(ws), _ptr(dev_status), _stream(stream)))


def mok_layer_bwd(cfg, own_lo, own_n, d_out, src_x, w_router, expert_to_local,
                  weights: mok_expert_weights, state: mok_fwd_state, staging, d_gate, dx_stage,
                  d_x, dw_gate, dw_up, dw_down, dw_router, ws, dev_status, stream=None):
    _check("mok_layer_bwd", lib().mok_layer_bwd(
        ctypes.byref(cfg), own_lo, own_n, _table(d_out), _table(src_x), _ptr(w_router),
        _ptr(expert_to_local), ctypes.byref(weights), ctypes.byref(state), _table(staging),
        _ptr(d_gate), _table(dx_stage), _table(d_x) if d_x is not None else None, _ptr(dw_gate),
        _ptr(dw_up), _ptr(dw_down), _ptr(dw_router), _ptr(ws), _ptr(dev_status), _stream(stream)))


def mok_tune_fwd(cfg, mbs, comms, reps, ws_bytes, own_lo, own_n, src_x, w_router, bias,
                 expert_to_local, weights: mok_expert_weights, state: mok_fwd_state, staging, out,
                 ws, dev_status, stream=None):
    """Returns (best mok_config, {(minibatch_rows, comm_wgs): mean ms or None if skipped})."""
    mbs = list(mbs) if mbs is not None else [64, 128, 256, 512, 1024, 2048, 4096]
    if comms is None:
        import torch
        cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
        comms = [max(cus * q // 16, 1) for q in (1, 2, 3, 4)]
    comms = list(comms)
    mb_arr = (ctypes.c_int32 * len(mbs))(*mbs)
    cm_arr = (ctypes.c_int32 * len(comms))(*comms)
    times = (ctypes.c_float * (len(mbs) * len(comms)))()
    best = mok_config()
    _check("mok_tune_fwd", lib().mok_tune_fwd(
        ctypes.byref(cfg), ctypes.cast(mb_arr, ctypes.c_void_p), len(mbs),
        ctypes.cast(cm_arr, ctypes.c_void_p), len(comms), reps, ws_bytes, own_lo, own_n,
        _table(src_x), _ptr(w_router), _ptr(bias), _ptr(expert_to_local), ctypes.byref(weights),
        ctypes.byref(state), _table(staging), _table(out) if out is not None else None, _ptr(ws),
        _ptr(dev_status), _stream(stream), ctypes.byref(best), ctypes.cast(times, ctypes.c_void_p)))
    table = {}
    for i, mb in enumerate(mbs):
        for j, c in enumerate(comms):
            v = times[i * len(comms) + j]
            table[(mb, c)] = float(v) if v >= 0 else None
    return best, table


def mok_mx_quantize(rows, K, src, codes, scales, stream=None):
    _check("mok_mx_quantize", lib().mok_mx_quantize(rows, K, _ptr(src), _ptr(codes), _ptr(scales),
                                                    _stream(stream)))


def mok_mx_quantize_f32(rows, K, src, codes, scales, stream=None):
    _check("mok_mx_quantize_f32", lib().mok_mx_quantize_f32(rows, K, _ptr(src), _ptr(codes),
                                                            _ptr(scales), _stream(stream)))


def mok_prepare_bwd(cfg, w_gate, w_up, w_down, wt_down, st_down, wt_gu, st_gu, stream=None):
    _check("mok_prepare_bwd", lib().mok_prepare_bwd(
        ctypes.byref(cfg), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(wt_down), _ptr(st_down),
        _ptr(wt_gu), _ptr(st_gu), _stream(stream)))


def mok_ring_layout(cfg):
    """-> (offset, slot_bytes, nslot) of the fused path's ring inside the workspace."""
    off, sb, n = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int32()
    _check("mok_ring_layout", lib().mok_ring_layout(ctypes.byref(cfg), ctypes.byref(off),
                                                    ctypes.byref(sb), ctypes.byref(n)))
    return int(off.value), int(sb.value), int(n.value)


def mok_hbm_stream(mode, dst, src, nbytes, stream=None):
    """HBM streaming probe: mode 0 read src, 1 write dst, 2 copy src -> dst."""
    _check("mok_hbm_stream", lib().mok_hbm_stream(mode, _ptr(dst), _ptr(src), nbytes,
                                                  _stream(stream)))


def mok_mfma_probe(kind, constant, iters, workgroups, out, stream=None):
    """Matrix-core rate probe: kind 0 bf16, 1 E4M3; constant 0 hashed data, 1 ones."""
    _check("mok_mfma_probe", lib().mok_mfma_probe(kind, constant, iters, workgroups, _ptr(out),
                                                  _stream(stream)))


def mok_layer_fwd_noalloc(cfg, own_lo, own_n, src_x, w_router, bias, expert_to_local,
                          weights: mok_expert_weights, state: mok_fwd_state, staging, out,
                          dev_status, stream=None):
    _check("mok_layer_fwd_noalloc", lib().mok_layer_fwd_noalloc(
        ctypes.byref(cfg), own_lo, own_n, _table(src_x), _ptr(w_router), _ptr(bias),
        _ptr(expert_to_local), ctypes.byref(weights), ctypes.byref(state), _table(staging),
        _table(out) if out is not None else None, _ptr(dev_status), _stream(stream)))


def mok_layer_fwd_macro(cfg, calls, w_router, bias, expert_to_local, weights: mok_expert_weights,
                        ws, dev_status, stream=None):
    """calls: list of dicts with own_lo, own_n, src_x, state (mok_fwd_state),
    staging, out -- one per layer call (macrobatch)."""
    keep = []
    arr = (mok_layer_call * len(calls))()
    for i, c in enumerate(calls):
        src, stg = _table(c["src_x"]), _table(c["staging"])
        out = _table(c["out"]) if c["out"] is not None else None
        keep += [src, stg, out, c["state"]]
        arr[i] = mok_layer_call(c["own_lo"], c["own_n"], ctypes.cast(src, ctypes.c_void_p),
                                ctypes.pointer(c["state"]), ctypes.cast(stg, ctypes.c_void_p),
                                ctypes.cast(out, ctypes.c_void_p) if out is not None else None)
    _check("mok_layer_fwd_macro", lib().mok_layer_fwd_macro(
        ctypes.byref(cfg), len(calls), arr, _ptr(w_router), _ptr(bias), _ptr(expert_to_local),
        ctypes.byref(weights), _ptr(ws), _ptr(dev_status), _stream(stream)))


# ------------------------------------------------------------------ training
def mok_route_logits(cfg, T, x, w_router, bias, topk_idx, topk_gate, logits, stream=None):
    _check("mok_route_logits", lib().mok_route_logits(
        ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias), _ptr(topk_idx),
        _ptr(topk_gate), _ptr(logits), _stream(stream)))


def mok_balance_ws_bytes(cfg, T, bal: mok_balance) -> int:
    return int(lib().mok_balance_ws_bytes(ctypes.byref(cfg), T, ctypes.byref(bal)))


def mok_balance_fwd(cfg, T, bal: mok_balance, logits, topk_idx, counts, prob, n_tok, loss, ws,
                    dev_status, stream=None):
    _check("mok_balance_fwd", lib().mok_balance_fwd(
        ctypes.byref(cfg), T, ctypes.byref(bal), _ptr(logits), _ptr(topk_idx), _ptr(counts),
        _ptr(prob), _ptr(n_tok), _ptr(loss), _ptr(ws), _ptr(dev_status), _stream(stream)))


def mok_balance_bwd(cfg, T, bal: mok_balance, logits, counts, n_tok, d_loss, d_logits, dev_status,
                    stream=None):
    _check("mok_balance_bwd", lib().mok_balance_bwd(
        ctypes.byref(cfg), T, ctypes.byref(bal), _ptr(logits), _ptr(counts), _ptr(n_tok),
        _ptr(d_loss), _ptr(d_logits), _ptr(dev_status), _stream(stream)))


def mok_router_bwd_ws_bytes(cfg, own_n) -> int:
    return int(lib().mok_router_bwd_ws_bytes(ctypes.byref(cfg), own_n))


def mok_router_bwd(cfg, own_lo, own_n, d_logits, src_x, w_router, d_x, dw_router, d_bias,
                   accumulate, ws, stream=None):
    """src_x, d_x: one entry per source (own entries used); d_x, dw_router,
    d_bias may be None."""
    _check("mok_router_bwd", lib().mok_router_bwd(
        ctypes.byref(cfg), own_lo, own_n, _ptr(d_logits),
        _table(src_x) if src_x is not None else None, _ptr(w_router),
        _table(d_x) if d_x is not None else None, _ptr(dw_router), _ptr(d_bias), int(accumulate),
        _ptr(ws), _stream(stream)))


def mok_grad_norm_ws_bytes(params) -> int:
    return int(lib().mok_grad_norm_ws_bytes(len(params), params))


def mok_grad_norm(params, max_norm, out, ws, stream=None):
    """out [2] fp32: the norm and the clip factor."""
    _check("mok_grad_norm", lib().mok_grad_norm(len(params), params, max_norm, _ptr(out), _ptr(ws),
                                                _stream(stream)))


def mok_adamw(params, args: mok_adamw_args, stream=None):
    _check("mok_adamw", lib().mok_adamw(len(params), params, ctypes.byref(args), _stream(stream)))


# ------------------------------------------------------------------ around the layer
def mok_norm_fwd(cfg, T, x, res, weight, eps, res_out, y, codes, scales, rstd, stream=None):
    """res and res_out are float32 or bfloat16 alike; without either, the residual type is x's."""
    if res is not None and res_out is not None and res.dtype != res_out.dtype:
        raise TypeError(f"res is {res.dtype}, res_out {res_out.dtype}")
    kind = _type(res if res is not None else res_out if res_out is not None else x)
    _check("mok_norm_fwd", lib().mok_norm_fwd(
        ctypes.byref(cfg), T, _ptr(x), _ptr(res), kind, _ptr(weight), eps, _ptr(res_out), _ptr(y),
        _ptr(codes), _ptr(scales), _ptr(rstd), _stream(stream)))


def mok_norm_bwd_ws_bytes(cfg, T) -> int:
    return int(lib().mok_norm_bwd_ws_bytes(ctypes.byref(cfg), T))


def mok_norm_bwd(cfg, T, dy, res, weight, rstd, d_res, d_r, d_x, d_weight, accumulate, ws, stream=None):
    """d_res and d_r are of res's type, float32 or bfloat16; d_x is of dy's."""
    for t in (d_res, d_r):
        if t is not None and t.dtype != res.dtype:
            raise TypeError(f"res is {res.dtype}, its gradient {t.dtype}")
    _check("mok_norm_bwd", lib().mok_norm_bwd(
        ctypes.byref(cfg), T, _ptr(dy), _ptr(res), _type(res), _ptr(weight), _ptr(rstd), _ptr(d_res),
        _ptr(d_r), _ptr(d_x), _ptr(d_weight), int(accumulate), _ptr(ws), _stream(stream)))


def mok_checkpoint_pack(cfg, offsets, ab, codes, scales, stream=None):
    _check("mok_checkpoint_pack", lib().mok_checkpoint_pack(
        ctypes.byref(cfg), _ptr(offsets), _ptr(ab), _ptr(codes), _ptr(scales), _stream(stream)))


def mok_checkpoint_unpack(cfg, offsets, codes, scales, ab, h, stream=None):
    """ab or h may be None."""
    _check("mok_checkpoint_unpack", lib().mok_checkpoint_unpack(
        ctypes.byref(cfg), _ptr(offsets), _ptr(codes), _ptr(scales), _ptr(ab), _ptr(h), _stream(stream)))


def mok_checkpoint_swiglu_bwd(cfg, offsets, codes, scales, dh, ld_dh, dab, h, stream=None):
    """h may be None; dh may be dab (its rows' first halves, ld_dh = 2I)."""
    _check("mok_checkpoint_swiglu_bwd", lib().mok_checkpoint_swiglu_bwd(
        ctypes.byref(cfg), _ptr(offsets), _ptr(codes), _ptr(scales), _ptr(dh), ld_dh, _ptr(dab), _ptr(h),
        _stream(stream)))


def mok_layer_bwd_checkpoint(cfg, own_lo, own_n, d_out, src_x, w_router, expert_to_local,
                             weights: mok_expert_weights, state: mok_fwd_state, codes, scales, staging, d_gate,
                             dx_stage, d_x, dw_gate, dw_up, dw_down, dw_router, ws, dev_status, stream=None):
    """mok_layer_bwd of a bf16 layer from a checkpoint instead of the state's ab and h."""
    _check("mok_layer_bwd_checkpoint", lib().mok_layer_bwd_checkpoint(
        ctypes.byref(cfg), own_lo, own_n, _table(d_out), _table(src_x), _ptr(w_router),
        _ptr(expert_to_local), ctypes.byref(weights), ctypes.byref(state), _ptr(codes), _ptr(scales),
        _table(staging), _ptr(d_gate), _table(dx_stage), _table(d_x) if d_x is not None else None, _ptr(dw_gate),
        _ptr(dw_up), _ptr(dw_down), _ptr(dw_router), _ptr(ws), _ptr(dev_status), _stream(stream)))


def mok_mxfp4_quantize(rows, K, src, codes, scales, stream=None):
    """src float32 or bfloat16."""
    _check("mok_mxfp4_quantize", lib().mok_mxfp4_quantize(rows, K, _type(src), _ptr(src), _ptr(codes),
                                                          _ptr(scales), _stream(stream)))


def mok_mxfp4_tile(rows, K, codes, scales, codes_out, scales_out, stream=None):
    _check("mok_mxfp4_tile", lib().mok_mxfp4_tile(rows, K, _ptr(codes), _ptr(scales), _ptr(codes_out),
                                                  _ptr(scales_out), _stream(stream)))


def mok_decode_ws_bytes(cfg, T) -> int:
    return int(lib().mok_decode_ws_bytes(ctypes.byref(cfg), T))


def mok_decode_ffn(cfg, T, x, x_scale, topk_idx, topk_gate, expert_to_local, weights: mok_w4, out, ws, dev_status,
                   stream=None):
    """x bf16, or E4M3 codes with x_scale."""
    _check("mok_decode_ffn", lib().mok_decode_ffn(
        ctypes.byref(cfg), T, _ptr(x), _ptr(x_scale), _ptr(topk_idx), _ptr(topk_gate), _ptr(expert_to_local),
        ctypes.byref(weights), _ptr(out), _ptr(ws), _ptr(dev_status), _stream(stream)))
