"""Thin ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: torch tensors supply device pointers and the current
CUDA stream, the library does the work.  There is no fallback: if libmoe.so
is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .workloads import Workload

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
GATING = {"topk_softmax": 0, "softmax_topk_renorm": 1, "sigmoid_grouped": 2,
          "softmax": 3, "softmax_renorm": 4, "sigmoid": 5, "sigmoid_renorm": 6}
WS_ROUTE, WS_EXPERT_FFN, WS_LAYER, WS_EXPERT_FFN_INT8, WS_LAYER_INT8 = 0, 1, 2, 3, 4
WS_BLOCK, WS_BLOCK_INT8 = 5, 6


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {moe_status_string(status)} ({status})")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k_max", ctypes.c_int32), ("f", ctypes.c_int32), ("f_shared", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gating", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_score_topk", ctypes.c_int32),
                ("routed_scale", ctypes.c_float)]


class MoeRouteOut(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("logits", "topk_idx", "topk_w", "counts", "kept", "offsets", "slot_row",
                 "row_src", "n_dropped")]


EP_MAX_RANKS = 8


class MoeEpRanks(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("n_ranks", ctypes.c_int32),
                ("counts_all", ctypes.c_void_p),
                ("recv_rows", ctypes.c_void_p * EP_MAX_RANKS),
                ("y_back", ctypes.c_void_p * EP_MAX_RANKS)]


class MoeFp8Weights(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("W1", "W3", "W2", "s1", "s3", "s2")]


class MoeInt8Linear(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in
                ("rows", "K", "N", "G", "dtype", "out_dtype", "swiglu")]


class MoeInt8Weights(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("W1", "W3", "W2", "s1", "s3", "s2")]


class MoeNormConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_span", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("eps_post", ctypes.c_float),
                ("eps_pre", ctypes.c_float), ("residual_scale", ctypes.c_float)]


class MoeBlockNorms(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("w_pre", "w_post", "gate")]


class MoeNormIo(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("x", "y", "w_post", "gate", "w_pre", "z", "h", "hq", "h_scale", "rstd_post",
                 "rstd_pre")]


class MoeNormGradIo(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("dz", "dh", "z", "y", "w_post", "gate", "w_pre", "rstd_post", "rstd_pre", "dx",
                 "dy", "dw_post", "dgate", "dw_pre")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built by routing_dispatch_expert_sigmoid_b200/build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cfgp = ctypes.POINTER(MoeConfig)
        outp = ctypes.POINTER(MoeRouteOut)
        L.moe_workspace_size.argtypes = [cfgp, I, ctypes.POINTER(S)]
        L.moe_route.argtypes = [cfgp, P, P, P, P, P, outp, P, S, P]
        L.moe_route_static_scratch.argtypes = [cfgp, P, P, P, P, P, outp, P]
        L.moe_gate.argtypes = [cfgp, P, P, P, P, P, P]
        L.moe_gate_backward.argtypes = [cfgp, P, P, P, P, P]
        L.moe_dispatch.argtypes = [cfgp, P, P, P, P, P]
        L.moe_expert_ffn.argtypes = [cfgp, P, P, P, P, P, P, P, S, P]
        L.moe_combine.argtypes = [cfgp, P, P, P, P, P, P]
        L.moe_layer.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, P, P, outp, P, S, P]
        L.moe_layer_timed.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, P, P, outp, P, S, P,
                                      ctypes.POINTER(ctypes.c_void_p), I]
        fp8p = ctypes.POINTER(MoeFp8Weights)
        L.moe_quantize_fp8.argtypes = [P, I, I, I, P, P, P]
        L.moe_expert_ffn_fp8.argtypes = [cfgp, P, P, fp8p, P, P, S, P]
        L.moe_layer_fp8.argtypes = [cfgp, P, P, P, P, P, fp8p, fp8p, P, outp, P, S, P,
                                    ctypes.POINTER(ctypes.c_void_p), I]
        epp = ctypes.POINTER(MoeEpRanks)
        L.moe_ep_plan.argtypes = [cfgp, epp, P, P, P]
        L.moe_ep_dispatch.argtypes = [cfgp, epp, P, P, P, P, P, P]
        L.moe_ep_return.argtypes = [cfgp, epp, P, P, P]
        L.moe_ep_plan_host.argtypes = [I, I, I, P, P, P, P, P, I]
        linp, i8p = ctypes.POINTER(MoeInt8Linear), ctypes.POINTER(MoeInt8Weights)
        L.moe_quantize_int8.argtypes = [P, I, I, I, P, P, P]
        L.moe_quantize_rows_int8.argtypes = [P, I, I, I, P, P, P]
        L.moe_gemm_int8.argtypes = [linp, P, P, P, P, P, P, P, P, P]
        L.moe_int8_workspace_size.argtypes = [linp, ctypes.POINTER(S)]
        L.moe_linear_int8.argtypes = [linp, P, P, P, P, P, P, P, P, S, P]
        L.moe_expert_ffn_int8.argtypes = [cfgp, P, P, i8p, P, P, S, P]
        L.moe_layer_int8.argtypes = [cfgp, P, P, P, P, P, P, P, i8p, i8p, P, outp, P, S, P,
                                     ctypes.POINTER(ctypes.c_void_p), I]
        normp = ctypes.POINTER(MoeNormConfig)
        L.moe_norm.argtypes = [normp, ctypes.POINTER(MoeNormIo), P]
        L.moe_norm_workspace_size.argtypes = [normp, ctypes.POINTER(S)]
        L.moe_norm_backward.argtypes = [normp, ctypes.POINTER(MoeNormGradIo), P, S, P]
        bnp = ctypes.POINTER(MoeBlockNorms)
        L.moe_block.argtypes = [cfgp, normp, bnp, P, P, P, P, P, P, P, P, P, P, P, P, outp, P, S, P]
        L.moe_block_int8.argtypes = [cfgp, normp, bnp, P, P, P, P, P, i8p, i8p, P, outp, P, S, P]
        L.moe_check_errors.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        for fn in ("moe_workspace_size", "moe_route", "moe_route_static_scratch", "moe_dispatch",
                   "moe_expert_ffn",
                   "moe_combine", "moe_layer", "moe_layer_timed", "moe_check_errors",
                   "moe_quantize_fp8", "moe_expert_ffn_fp8", "moe_layer_fp8", "moe_ep_plan",
                   "moe_ep_dispatch", "moe_ep_return", "moe_ep_plan_host", "moe_gate",
                   "moe_gate_backward", "moe_norm", "moe_norm_workspace_size",
                   "moe_norm_backward", "moe_quantize_int8", "moe_quantize_rows_int8",
                   "moe_gemm_int8", "moe_int8_workspace_size", "moe_linear_int8",
                   "moe_expert_ffn_int8", "moe_layer_int8", "moe_block", "moe_block_int8"):
            getattr(L, fn).restype = I
        _lib = L
    return _lib


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MoeError(status, what)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current device's index (-2 without a CUDA build: host tensors have -1) and a
# device's current stream as a number: a tenth of the time of the calls that wrap
# them in objects.
_device = getattr(torch._C, "_cuda_getDevice", lambda: -2)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        device = torch.cuda.current_device()  # initialises CUDA where nothing has yet
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(device))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _current() -> int:
    """The current CUDA device, for _arg; -2 where there is none."""
    try:
        return _device()
    except RuntimeError:
        return -2


def _arg(what, device, name, t, dtype, numel, optional=False, at_least=False):
    """The device pointer of an argument, checked: a contiguous tensor of this
    type and size on the current CUDA device (or None where it may be left out).
    The library sees pointers alone and cannot tell a strided view, a tensor of
    another type or one on another device from the right one."""
    if t is None:
        if optional:
            return None
        raise MoeError(-1, f"{what}: {name} is missing")
    n = t.numel()
    if (t.dtype is dtype and (n == numel or (at_least and n > numel)) and t.is_contiguous()
            and t.get_device() == device):
        return t.data_ptr()
    if not t.is_cuda:
        raise MoeError(-1, f"{what}: {name} is on {t.device}, not on a CUDA device")
    if t.get_device() != device:
        raise MoeError(-1, f"{what}: {name} is on cuda:{t.get_device()}, the current device is "
                           f"cuda:{device}")
    raise MoeError(-1, f"{what}: {name} has to be a contiguous {dtype} tensor of "
                       f"{'at least ' if at_least else ''}{numel} elements, got {t.dtype} "
                       f"{tuple(t.shape)} with strides {t.stride()}")


def config(w: Workload, T: int | None = None) -> MoeConfig:
    """The moe_config of a workload (optionally with another token count)."""
    return MoeConfig(T=w.T if T is None else T, d=w.d, E=w.E, k_max=w.k_max, f=w.f,
                     f_shared=w.f_shared, dtype=MOE_F32 if w.dtype == "f32" else MOE_BF16,
                     gating=GATING[w.gating], capacity_factor=w.capacity_factor,
                     n_groups=w.n_groups, topk_groups=w.topk_groups,
                     group_score_topk=w.group_score_topk, routed_scale=w.routed_scale)


def moe_workspace_size(cfg: MoeConfig, kind: int = WS_LAYER) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(cfg), kind, ctypes.byref(n)),
           "moe_workspace_size")
    return int(n.value)


def workspace(cfg: MoeConfig, kind: int = WS_LAYER, device="cuda") -> torch.Tensor:
    """A caller-owned workspace of the size moe_workspace_size asks for."""
    return torch.empty(max(moe_workspace_size(cfg, kind), 1), dtype=torch.uint8, device=device)


def route_buffers(cfg: MoeConfig, device="cuda") -> dict:
    """Caller-owned routing output tensors for moe_route / moe_layer."""
    T, E, k = cfg.T, cfg.E, cfg.k_max
    i32 = dict(dtype=torch.int32, device=device)
    return dict(logits=torch.empty((T, E), dtype=torch.float32, device=device),
                topk_idx=torch.empty((T, k), **i32), topk_w=torch.empty((T, k), dtype=torch.float32,
                                                                        device=device),
                counts=torch.empty(E, **i32), kept=torch.empty(E, **i32),
                offsets=torch.empty(E + 1, **i32), slot_row=torch.empty((T, k), **i32),
                row_src=torch.empty(max(T * k, 1), **i32), n_dropped=torch.empty(1, **i32))


def _route_struct(b: dict) -> MoeRouteOut:
    return MoeRouteOut(*[b[name].data_ptr() for name, _ in MoeRouteOut._fields_])


def moe_route(cfg, x, Wr, logit_bias, sel_bias, k_per_token, out: dict, ws, stream=None):
    r = _route_struct(out)
    _check(lib().moe_route(ctypes.byref(cfg), _p(x), _p(Wr), _p(logit_bias), _p(sel_bias),
                           _p(k_per_token), ctypes.byref(r), _p(ws),
                           0 if ws is None else ws.numel(), _stream(stream)), "moe_route")


def moe_route_static_scratch(cfg, x, Wr, logit_bias, sel_bias, k_per_token, out: dict,
                             stream=None):
    """moe_route for callers that cannot provide a workspace: the library's
    fixed device scratch is used instead (see include/moe.h)."""
    r = _route_struct(out)
    _check(lib().moe_route_static_scratch(ctypes.byref(cfg), _p(x), _p(Wr), _p(logit_bias),
                                          _p(sel_bias), _p(k_per_token), ctypes.byref(r),
                                          _stream(stream)), "moe_route_static_scratch")


# ---- gating alone -----------------------------------------------------------
def gate_config(T: int, E: int, k_max: int, gating: str = "softmax", n_groups: int = 1,
                topk_groups: int = 1, group_score_topk: int = 1,
                routed_scale: float = 1.0) -> MoeConfig:
    """The moe_config of a gating step on its own (moe_gate, moe_gate_backward)."""
    return MoeConfig(T=T, d=8, E=E, k_max=k_max, f=8, f_shared=0, dtype=MOE_BF16,
                     gating=GATING[gating], capacity_factor=0.0, n_groups=n_groups,
                     topk_groups=topk_groups, group_score_topk=group_score_topk,
                     routed_scale=routed_scale)


def moe_gate(cfg, logits, sel_bias, k_per_token, topk_idx, topk_w, stream=None):
    """logits [T, E] fp32 -> topk_idx int32, topk_w fp32 [T, k_max] (step 2 of the layer)."""
    dev = _current()
    T, E, k, w = cfg.T, cfg.E, cfg.k_max, "moe_gate"
    _check(lib().moe_gate(
        ctypes.byref(cfg), _arg(w, dev, "logits", logits, torch.float32, T * E),
        _arg(w, dev, "sel_bias", sel_bias, torch.float32, E, True),
        _arg(w, dev, "k_per_token", k_per_token, torch.int32, T, True),
        _arg(w, dev, "topk_idx", topk_idx, torch.int32, T * k),
        _arg(w, dev, "topk_w", topk_w, torch.float32, T * k), _stream(stream)), w)


def moe_gate_backward(cfg, logits, topk_idx, dtopk_w, dlogits, stream=None):
    """dtopk_w [T, k_max] -> dlogits [T, E], for the indices of a forward pass."""
    dev = _current()
    T, E, k, w = cfg.T, cfg.E, cfg.k_max, "moe_gate_backward"
    _check(lib().moe_gate_backward(
        ctypes.byref(cfg), _arg(w, dev, "logits", logits, torch.float32, T * E),
        _arg(w, dev, "topk_idx", topk_idx, torch.int32, T * k),
        _arg(w, dev, "dtopk_w", dtopk_w, torch.float32, T * k),
        _arg(w, dev, "dlogits", dlogits, torch.float32, T * E), _stream(stream)), w)


def moe_dispatch(cfg, x, offsets, row_src, x_perm, stream=None):
    _check(lib().moe_dispatch(ctypes.byref(cfg), _p(x), _p(offsets), _p(row_src), _p(x_perm),
                              _stream(stream)), "moe_dispatch")


def moe_expert_ffn(cfg, x_perm, offsets, W1, W3, W2, y_perm, ws, stream=None):
    _check(lib().moe_expert_ffn(ctypes.byref(cfg), _p(x_perm), _p(offsets), _p(W1), _p(W3),
                                _p(W2), _p(y_perm), _p(ws), 0 if ws is None else ws.numel(),
                                _stream(stream)), "moe_expert_ffn")


def moe_combine(cfg, y_perm, slot_row, topk_w, shared_y, out, stream=None):
    _check(lib().moe_combine(ctypes.byref(cfg), _p(y_perm), _p(slot_row), _p(topk_w),
                             _p(shared_y), _p(out), _stream(stream)), "moe_combine")


def moe_layer(cfg, x, Wr, logit_bias, sel_bias, k_per_token, W1, W3, W2, Ws1, Ws3, Ws2, out,
              route_out: dict | None, ws, stream=None):
    r = None if route_out is None else ctypes.byref(_route_struct(route_out))
    _check(lib().moe_layer(ctypes.byref(cfg), _p(x), _p(Wr), _p(logit_bias), _p(sel_bias),
                           _p(k_per_token), _p(W1), _p(W3), _p(W2), _p(Ws1), _p(Ws3), _p(Ws2),
                           _p(out), r, _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "moe_layer")


STAGES = ("start", "route", "dispatch", "up_swiglu", "down", "shared", "combine")


def moe_layer_timed(cfg, x, Wr, logit_bias, sel_bias, k_per_token, W1, W3, W2, Ws1, Ws3, Ws2,
                    out, route_out: dict | None, ws, events, stream=None):
    """moe_layer that records events[i] (torch.cuda.Event, len(STAGES)) at stage boundary i."""
    r = None if route_out is None else ctypes.byref(_route_struct(route_out))
    handles = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_layer_timed(ctypes.byref(cfg), _p(x), _p(Wr), _p(logit_bias), _p(sel_bias),
                                 _p(k_per_token), _p(W1), _p(W3), _p(W2), _p(Ws1), _p(Ws3),
                                 _p(Ws2), _p(out), r, _p(ws), 0 if ws is None else ws.numel(),
                                 _stream(stream), handles, len(events)), "moe_layer_timed")


def moe_check_errors(stream=None) -> int:
    """Synchronise the stream and return the device error flags (raises if any)."""
    flags = ctypes.c_uint32(0)
    st = lib().moe_check_errors(_stream(stream), ctypes.byref(flags))
    if st not in (0, -6):
        _check(st, "moe_check_errors")
    if flags.value:
        raise MoeError(st, f"moe_check_errors: device flags {flags.value:#x}")
    return 0


# ---- fp8 expert weights -----------------------------------------------------
def moe_quantize_fp8(W: torch.Tensor, stream=None):
    """W [G, K, N] (or [K, N]) bf16 -> (codes uint8 [G, N, K] (or [N, K]),
    scales fp32 [G, N] (or [N])), computed by the library."""
    Wg = W if W.dim() == 3 else W.unsqueeze(0)
    G, K, N = Wg.shape
    q = torch.empty((G, N, K), dtype=torch.uint8, device=W.device)
    sc = torch.empty((G, N), dtype=torch.float32, device=W.device)
    _check(lib().moe_quantize_fp8(_p(Wg), G, K, N, _p(q), _p(sc), _stream(stream)),
           "moe_quantize_fp8")
    if W.dim() == 2:
        return q[0], sc[0]
    return q, sc


def fp8_weight_set(W1, W3, W2, stream=None) -> dict:
    """Quantise one set of expert matrices (routed [E, ...] or shared [d, f])."""
    out = {}
    for name, W in (("W1", W1), ("W3", W3), ("W2", W2)):
        q, sc = moe_quantize_fp8(W, stream)
        out[name], out["s" + name[1]] = q, sc
    return out


def _fp8_struct(ws: dict | None):
    if ws is None:
        return None
    return MoeFp8Weights(*[ws[k].data_ptr() for k in ("W1", "W3", "W2", "s1", "s3", "s2")])


def moe_expert_ffn_fp8(cfg, x_perm, offsets, weights: dict, y_perm, ws, stream=None):
    wq = _fp8_struct(weights)
    _check(lib().moe_expert_ffn_fp8(ctypes.byref(cfg), _p(x_perm), _p(offsets), ctypes.byref(wq),
                                    _p(y_perm), _p(ws), 0 if ws is None else ws.numel(),
                                    _stream(stream)), "moe_expert_ffn_fp8")


def moe_layer_fp8(cfg, x, Wr, logit_bias, sel_bias, k_per_token, experts: dict,
                  shared: dict | None, out, route_out: dict | None, ws, events=None,
                  stream=None):
    """moe_layer with fp8 expert weights (dicts from fp8_weight_set); events as
    in moe_layer_timed, or None."""
    r = None if route_out is None else ctypes.byref(_route_struct(route_out))
    we, wsh = _fp8_struct(experts), _fp8_struct(shared)
    n = 0 if events is None else len(events)
    handles = None if events is None else (ctypes.c_void_p * n)(
        *[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_layer_fp8(ctypes.byref(cfg), _p(x), _p(Wr), _p(logit_bias), _p(sel_bias),
                               _p(k_per_token), ctypes.byref(we),
                               None if wsh is None else ctypes.byref(wsh), _p(out), r, _p(ws),
                               0 if ws is None else ws.numel(), _stream(stream), handles, n),
           "moe_layer_fp8")


# ---- expert parallelism -----------------------------------------------------
def ep_ranks(rank: int, n_ranks: int, counts_all, recv_rows, y_back) -> MoeEpRanks:
    """The moe_ep_ranks of one rank: counts_all [n_ranks, E] int32 on its
    device, and every rank's receive and return buffers (device tensors)."""
    ep = MoeEpRanks()
    ep.rank, ep.n_ranks = rank, n_ranks
    ep.counts_all = counts_all.data_ptr()
    for r in range(n_ranks):
        ep.recv_rows[r] = recv_rows[r].data_ptr()
        ep.y_back[r] = y_back[r].data_ptr()
    return ep


def moe_ep_plan(cfg, ep: MoeEpRanks, recv_offsets, send_base, stream=None):
    _check(lib().moe_ep_plan(ctypes.byref(cfg), ctypes.byref(ep), _p(recv_offsets),
                             _p(send_base), _stream(stream)), "moe_ep_plan")


def moe_ep_dispatch(cfg, ep: MoeEpRanks, x, offsets, row_src, topk_idx, send_base, stream=None):
    _check(lib().moe_ep_dispatch(ctypes.byref(cfg), ctypes.byref(ep), _p(x), _p(offsets),
                                 _p(row_src), _p(topk_idx), _p(send_base), _stream(stream)),
           "moe_ep_dispatch")


def moe_ep_return(cfg, ep: MoeEpRanks, y_recv, recv_offsets, stream=None):
    _check(lib().moe_ep_return(ctypes.byref(cfg), ctypes.byref(ep), _p(y_recv),
                               _p(recv_offsets), _stream(stream)), "moe_ep_return")


def moe_ep_plan_host(n_ranks: int, E: int, rank: int, counts_all, max_recv: int):
    """Host mirror of the plan: (recv_offsets, send_base, recv_src, recv_src_row)
    as int32 numpy arrays, from counts_all [n_ranks, E] (numpy)."""
    import numpy as np
    C = np.ascontiguousarray(counts_all, dtype=np.int32)
    e_loc = E // max(n_ranks, 1)
    ro = np.zeros(e_loc + 1, np.int32)
    sb = np.zeros(E, np.int32)
    rs = np.zeros(max(max_recv, 1), np.int32)
    rr = np.zeros(max(max_recv, 1), np.int32)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(lib().moe_ep_plan_host(n_ranks, E, rank, ptr(C), ptr(ro), ptr(sb), ptr(rs), ptr(rr),
                                  max_recv), "moe_ep_plan_host")
    R = int(ro[-1])
    return ro, sb, rs[:R], rr[:R]


# ---- norms around the block -------------------------------------------------
def norm_config(T: int, d: int, dtype: str = "bf16", eps_post: float = 1e-6,
                eps_pre: float = 1e-6, residual_scale: float = 1.0, gate_span: int = 0,
                post_norm: bool = True) -> MoeNormConfig:
    return MoeNormConfig(T=T, d=d, dtype=MOE_F32 if dtype == "f32" else MOE_BF16,
                         gate_span=gate_span, post_norm=int(post_norm), eps_post=eps_post,
                         eps_pre=eps_pre, residual_scale=residual_scale)


def _gate_rows(cfg: MoeNormConfig) -> int:
    return -(-cfg.T // cfg.gate_span) if cfg.gate_span > 0 else 0


def moe_norm(cfg: MoeNormConfig, x, y=None, w_post=None, gate=None, w_pre=None, z=None, h=None,
             hq=None, h_scale=None, rstd_post=None, rstd_pre=None, stream=None):
    """z = residual_scale * x + gate * (w_post * rms(y)) (gate * y without
    post_norm), h = w_pre * rms(z), and h's int8 codes; which parts there are
    follows from the tensors given (see include/moe.h)."""
    dev = _current()
    w, dt, f32 = "moe_norm", torch.float32 if cfg.dtype == MOE_F32 else torch.bfloat16, torch.float32
    n, d = cfg.T * cfg.d, cfg.d
    io = MoeNormIo(
        _arg(w, dev, "x", x, dt, n), _arg(w, dev, "y", y, dt, n, True), _arg(w, dev, "w_post", w_post, dt, d, True),
        _arg(w, dev, "gate", gate, dt, _gate_rows(cfg) * d, True), _arg(w, dev, "w_pre", w_pre, dt, d, True),
        _arg(w, dev, "z", z, dt, n, True), _arg(w, dev, "h", h, dt, n, True),
        _arg(w, dev, "hq", hq, torch.int8, n, True), _arg(w, dev, "h_scale", h_scale, f32, cfg.T, True),
        _arg(w, dev, "rstd_post", rstd_post, f32, cfg.T, True),
        _arg(w, dev, "rstd_pre", rstd_pre, f32, cfg.T, True))
    _check(lib().moe_norm(ctypes.byref(cfg), ctypes.byref(io), _stream(stream)), w)


def norm_workspace_size(cfg: MoeNormConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_norm_workspace_size")
    return int(n.value)


def norm_workspace(cfg: MoeNormConfig, device="cuda") -> torch.Tensor:
    """A caller-owned workspace for moe_norm_backward."""
    return torch.empty(max(norm_workspace_size(cfg), 1), dtype=torch.uint8, device=device)


def moe_norm_backward(cfg: MoeNormConfig, dz=None, dh=None, z=None, y=None, w_post=None,
                      gate=None, w_pre=None, rstd_post=None, rstd_pre=None, dx=None, dy=None,
                      dw_post=None, dgate=None, dw_pre=None, ws=None, stream=None):
    """The gradients of moe_norm (see include/moe.h)."""
    dev = _current()
    w, dt, f32 = "moe_norm_backward", torch.float32 if cfg.dtype == MOE_F32 else torch.bfloat16, torch.float32
    n, d, g = cfg.T * cfg.d, cfg.d, _gate_rows(cfg) * cfg.d
    io = MoeNormGradIo(
        _arg(w, dev, "dz", dz, dt, n, True), _arg(w, dev, "dh", dh, dt, n, True), _arg(w, dev, "z", z, dt, n, True),
        _arg(w, dev, "y", y, dt, n, True), _arg(w, dev, "w_post", w_post, dt, d, True),
        _arg(w, dev, "gate", gate, dt, g, True), _arg(w, dev, "w_pre", w_pre, dt, d, True),
        _arg(w, dev, "rstd_post", rstd_post, f32, cfg.T, True),
        _arg(w, dev, "rstd_pre", rstd_pre, f32, cfg.T, True), _arg(w, dev, "dx", dx, dt, n),
        _arg(w, dev, "dy", dy, dt, n, True), _arg(w, dev, "dw_post", dw_post, f32, d, True),
        _arg(w, dev, "dgate", dgate, f32, g, True), _arg(w, dev, "dw_pre", dw_pre, f32, d, True))
    _check(lib().moe_norm_backward(
        ctypes.byref(cfg), ctypes.byref(io), _arg(w, dev, "ws", ws, torch.uint8, 0, True, True),
        0 if ws is None else ws.numel(), _stream(stream)), w)


# ---- int8 products ----------------------------------------------------------
_DTYPES = {"bf16": (MOE_BF16, torch.bfloat16), "f32": (MOE_F32, torch.float32)}
_TORCH = {MOE_BF16: torch.bfloat16, MOE_F32: torch.float32}


def moe_quantize_int8(W: torch.Tensor, stream=None):
    """W [G, K, N] (or [K, N]) bf16 -> (codes int8 [G, N, K] (or [N, K]), scales
    fp32 [G, N] (or [N]))."""
    dev = _current()
    G, K, N = W.shape if W.dim() == 3 else (1, *W.shape)
    q = torch.empty((G, N, K), dtype=torch.int8, device=W.device)
    sc = torch.empty((G, N), dtype=torch.float32, device=W.device)
    w = "moe_quantize_int8"
    _check(lib().moe_quantize_int8(_arg(w, dev, "W", W, torch.bfloat16, G * K * N), G, K, N, _p(q),
                                   _p(sc), _stream(stream)), w)
    return (q, sc) if W.dim() == 3 else (q[0], sc[0])


def int8_weight_set(W1, W3, W2, stream=None) -> dict:
    """Quantise one set of expert matrices (routed [E, ...] or shared [d, f])."""
    out = {}
    for name, W in (("W1", W1), ("W3", W3), ("W2", W2)):
        out[name], out["s" + name[1]] = moe_quantize_int8(W, stream)
    return out


def moe_quantize_rows_int8(x, xq, scale, stream=None):
    """Rows x [..., K] (bf16 or fp32) -> codes xq int8 of its shape, scale fp32 [rows]."""
    dev = _current()
    w, K = "moe_quantize_rows_int8", x.shape[-1]
    rows = x.numel() // max(K, 1)
    dt = MOE_F32 if x.dtype is torch.float32 else MOE_BF16
    _check(lib().moe_quantize_rows_int8(
        _arg(w, dev, "x", x, _TORCH[dt], rows * K), dt, rows, K,
        _arg(w, dev, "xq", xq, torch.int8, rows * K), _arg(w, dev, "scale", scale, torch.float32, rows),
        _stream(stream)), w)


def int8_linear(rows: int, K: int, N: int, G: int = 1, dtype: str = "bf16",
                out_dtype: str = "bf16", swiglu: bool = False) -> MoeInt8Linear:
    return MoeInt8Linear(rows=rows, K=K, N=N, G=G, dtype=_DTYPES[dtype][0],
                         out_dtype=_DTYPES[out_dtype][0], swiglu=int(swiglu))


def int8_workspace_size(lin: MoeInt8Linear) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_int8_workspace_size(ctypes.byref(lin), ctypes.byref(n)),
           "moe_int8_workspace_size")
    return int(n.value)


def int8_workspace(lin: MoeInt8Linear, device="cuda") -> torch.Tensor:
    """A caller-owned workspace for moe_linear_int8."""
    return torch.empty(max(int8_workspace_size(lin), 1), dtype=torch.uint8, device=device)


def _int8_operands(w, lin, offsets, W1, s1, W3, s3, out):
    dev = _current()
    n, sc = lin.G * lin.N * lin.K, lin.G * lin.N
    return (_arg(w, dev, "offsets", offsets, torch.int32, lin.G + 1, True),
            _arg(w, dev, "W1", W1, torch.int8, n), _arg(w, dev, "s1", s1, torch.float32, sc),
            _arg(w, dev, "W3", W3, torch.int8, n, True), _arg(w, dev, "s3", s3, torch.float32, sc, True),
            _arg(w, dev, "out", out, _TORCH.get(lin.out_dtype), lin.rows * lin.N))


def moe_gemm_int8(lin: MoeInt8Linear, xq, x_scale, offsets, W1, s1, W3, s3, out, stream=None):
    """Codes xq [rows, K] times W1 (and W3: SwiGLU) -> out [rows, N]."""
    dev = _current()
    w = "moe_gemm_int8"
    _check(lib().moe_gemm_int8(
        ctypes.byref(lin), _arg(w, dev, "xq", xq, torch.int8, lin.rows * lin.K),
        _arg(w, dev, "x_scale", x_scale, torch.float32, lin.rows),
        *_int8_operands(w, lin, offsets, W1, s1, W3, s3, out), _stream(stream)), w)


def moe_linear_int8(lin: MoeInt8Linear, x, offsets, W1, s1, W3, s3, out, ws, stream=None):
    """Rows x [rows, K], quantised per row, times W1 (and W3: SwiGLU) -> out [rows, N]."""
    dev = _current()
    w = "moe_linear_int8"
    _check(lib().moe_linear_int8(
        ctypes.byref(lin), _arg(w, dev, "x", x, _TORCH.get(lin.dtype), lin.rows * lin.K),
        *_int8_operands(w, lin, offsets, W1, s1, W3, s3, out),
        _arg(w, dev, "ws", ws, torch.uint8, 0, True, True), 0 if ws is None else ws.numel(),
        _stream(stream)), w)


def _int8_struct(w, ws: dict | None, G: int, d: int, f: int):
    dev = _current()
    if ws is None:
        return None
    n = dict(W1=G * d * f, W3=G * d * f, W2=G * d * f, s1=G * f, s3=G * f, s2=G * d)
    return MoeInt8Weights(*[_arg(w, dev, k, ws[k], torch.int8 if k[0] == "W" else torch.float32, n[k])
                            for k in ("W1", "W3", "W2", "s1", "s3", "s2")])


def moe_expert_ffn_int8(cfg, x_perm, offsets, weights: dict, y_perm, ws, stream=None):
    """moe_expert_ffn with int8 expert weights (a dict from int8_weight_set)."""
    dev = _current()
    w, rows = "moe_expert_ffn_int8", cfg.T * cfg.k_max
    wq = _int8_struct(w, weights, cfg.E, cfg.d, cfg.f)
    _check(lib().moe_expert_ffn_int8(
        ctypes.byref(cfg), _arg(w, dev, "x_perm", x_perm, torch.bfloat16, rows * cfg.d),
        _arg(w, dev, "offsets", offsets, torch.int32, cfg.E + 1), ctypes.byref(wq),
        _arg(w, dev, "y_perm", y_perm, torch.float32, rows * cfg.d),
        _arg(w, dev, "ws", ws, torch.uint8, 0, True, True), 0 if ws is None else ws.numel(),
        _stream(stream)), w)


def moe_layer_int8(cfg, x, Wr, logit_bias, sel_bias, k_per_token, experts: dict,
                   shared: dict | None, out, route_out: dict | None, ws, xq=None, x_scale=None,
                   events=None, stream=None):
    """moe_layer with int8 expert weights (dicts from int8_weight_set); xq and
    x_scale: the int8 form of x when there is one already; events as in
    moe_layer_timed, or None."""
    dev = _current()
    w, T, d, E, f32 = "moe_layer_int8", cfg.T, cfg.d, cfg.E, torch.float32
    r = None if route_out is None else ctypes.byref(_route_struct(route_out))
    we = _int8_struct(w, experts, E, d, cfg.f)
    wsh = _int8_struct(w, shared, 1, d, cfg.f_shared)
    n = 0 if events is None else len(events)
    handles = None if events is None else (ctypes.c_void_p * n)(
        *[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_layer_int8(
        ctypes.byref(cfg), _arg(w, dev, "x", x, torch.bfloat16, T * d),
        _arg(w, dev, "xq", xq, torch.int8, T * d, True), _arg(w, dev, "x_scale", x_scale, f32, T, True),
        _arg(w, dev, "Wr", Wr, torch.bfloat16, d * E), _arg(w, dev, "logit_bias", logit_bias, f32, E, True),
        _arg(w, dev, "sel_bias", sel_bias, f32, E, True),
        _arg(w, dev, "k_per_token", k_per_token, torch.int32, T, True), ctypes.byref(we),
        None if wsh is None else ctypes.byref(wsh), _arg(w, dev, "out", out, torch.bfloat16, T * d), r,
        _arg(w, dev, "ws", ws, torch.uint8, 0, True, True), 0 if ws is None else ws.numel(),
        _stream(stream), handles, n), w)


# ---- the block around a layer -----------------------------------------------
def _block_norms(w, norm, w_pre, w_post, gate):
    dev = _current()
    dt, d = _TORCH.get(norm.dtype), norm.d
    return MoeBlockNorms(_arg(w, dev, "w_pre", w_pre, dt, d, True),
                         _arg(w, dev, "w_post", w_post, dt, d, True),
                         _arg(w, dev, "gate", gate, dt, _gate_rows(norm) * d, True))


def moe_block(cfg, norm: MoeNormConfig, x, w_pre, w_post, gate, Wr, logit_bias, sel_bias,
              k_per_token, W1, W3, W2, Ws1, Ws3, Ws2, out, route_out: dict | None, ws, stream=None):
    """out = residual_scale * x + gate * post-norm(moe_layer(w_pre * rms(x)))."""
    dev = _current()
    w, dt, T, d, E, f, fs, f32 = ("moe_block", _TORCH.get(cfg.dtype), cfg.T, cfg.d, cfg.E, cfg.f,
                                  cfg.f_shared, torch.float32)
    bn = _block_norms(w, norm, w_pre, w_post, gate)
    r = None if route_out is None else ctypes.byref(_route_struct(route_out))
    _check(lib().moe_block(
        ctypes.byref(cfg), ctypes.byref(norm), ctypes.byref(bn), _arg(w, dev, "x", x, dt, T * d),
        _arg(w, dev, "Wr", Wr, dt, d * E), _arg(w, dev, "logit_bias", logit_bias, f32, E, True),
        _arg(w, dev, "sel_bias", sel_bias, f32, E, True),
        _arg(w, dev, "k_per_token", k_per_token, torch.int32, T, True),
        *[_arg(w, dev, n, W, dt, E * d * f) for n, W in (("W1", W1), ("W3", W3), ("W2", W2))],
        *[_arg(w, dev, n, W, dt, d * fs, True) for n, W in (("Ws1", Ws1), ("Ws3", Ws3), ("Ws2", Ws2))],
        _arg(w, dev, "out", out, dt, T * d), r, _arg(w, dev, "ws", ws, torch.uint8, 0, True, True),
        0 if ws is None else ws.numel(), _stream(stream)), w)


def moe_block_int8(cfg, norm: MoeNormConfig, x, w_pre, w_post, gate, Wr, logit_bias, sel_bias,
                   k_per_token, experts: dict, shared: dict | None, out, route_out: dict | None,
                   ws, stream=None):
    """moe_block on int8 experts (dicts from int8_weight_set); the pre-norm hands
    the layer the codes of its output."""
    dev = _current()
    w, T, d, E, f32 = "moe_block_int8", cfg.T, cfg.d, cfg.E, torch.float32
    bn = _block_norms(w, norm, w_pre, w_post, gate)
    r = None if route_out is None else ctypes.byref(_route_struct(route_out))
    we = _int8_struct(w, experts, E, d, cfg.f)
    wsh = _int8_struct(w, shared, 1, d, cfg.f_shared)
    _check(lib().moe_block_int8(
        ctypes.byref(cfg), ctypes.byref(norm), ctypes.byref(bn),
        _arg(w, dev, "x", x, torch.bfloat16, T * d), _arg(w, dev, "Wr", Wr, torch.bfloat16, d * E),
        _arg(w, dev, "logit_bias", logit_bias, f32, E, True),
        _arg(w, dev, "sel_bias", sel_bias, f32, E, True),
        _arg(w, dev, "k_per_token", k_per_token, torch.int32, T, True), ctypes.byref(we),
        None if wsh is None else ctypes.byref(wsh), _arg(w, dev, "out", out, torch.bfloat16, T * d), r,
        _arg(w, dev, "ws", ws, torch.uint8, 0, True, True), 0 if ws is None else ws.numel(),
        _stream(stream)), w)
