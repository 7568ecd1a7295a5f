"""Python binding of the C ABI in ``include/moe_route_permute.h``.

Argument marshalling only: tensors are allocated with torch on the current CUDA
device, their data pointers and torch's current stream are handed to the
library, and every step of the path runs in the library's kernels. There is no
fallback: if the compiled library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int, c_longlong, c_size_t, c_void_p

import torch

from . import build as _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SHAPE = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_ERR_DEVICE_INDEX = 6
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "workspace too small",
                4: "CUDA error", 5: "device: bounded wait ran out", 6: "device: index out of range"}
SCORE = {"softmax": 0, "sigmoid": 1}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} (status {status})")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", c_int), ("H", c_int), ("E", c_int), ("k", c_int), ("F", c_int), ("F_shared", c_int),
                ("score", c_int), ("n_groups", c_int), ("topk_groups", c_int), ("gate_scale", c_float),
                ("aux_coeff", c_float), ("out_fp32", c_int), ("inter_fp32", c_int), ("force_balanced", c_int)]


class MoeFwdSaved(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("topk_idx", "topk_gate", "logits", "row_id_map", "counts", "offsets",
                                        "x_perm", "h13", "a", "y_perm", "aux_partials", "h13_shared",
                                        "a_shared")]


_lib = None


def library_path() -> str:
    """The library this process loads: the bounds-check build when the
    environment sets MOE_BOUNDS_CHECK=1, else the default build."""
    return _build.LIB_CHECKED if os.environ.get("MOE_BOUNDS_CHECK") == "1" else _build.LIB


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing: run route_permute_grouped_gb300.build.build()")
        L = ctypes.CDLL(path)
        vp = c_void_p
        L.moe_abi_struct_bytes.restype = c_size_t
        L.moe_abi_struct_bytes.argtypes = [c_int]
        if (L.moe_abi_struct_bytes(0) != ctypes.sizeof(MoeConfig)
                or L.moe_abi_struct_bytes(1) != ctypes.sizeof(MoeFwdSaved)):
            raise RuntimeError("moe_config / moe_fwd_saved layout of the binding differs from the library")
        L.moe_workspace_bytes.restype = c_size_t
        L.moe_workspace_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_router_topk.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
        L.moe_permute.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
        L.moe_grouped_swiglu_ffn.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
        L.moe_unpermute_combine.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, vp, vp]
        L.moe_layer_fwd.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                    POINTER(MoeFwdSaved), vp, c_size_t, vp]
        L.moe_layer_bwd.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, vp, vp, vp, vp, vp, POINTER(MoeFwdSaved),
                                    vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
        L.moe_get_device_status.argtypes = [vp, vp, POINTER(c_int)]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [c_int]
        L.moe_debug_set_wait_limit_ns.argtypes = [c_longlong]
        L.moe_debug_set_wait_limit_ns.restype = None
        L.moe_debug_set_fault.argtypes = [c_int]
        L.moe_debug_set_fault.restype = None
        for n in ("moe_router_topk", "moe_permute", "moe_grouped_swiglu_ffn", "moe_unpermute_combine",
                  "moe_layer_fwd", "moe_layer_bwd", "moe_get_device_status"):
            getattr(L, n).restype = c_int
        L.moe_profile_start.argtypes = [c_int]
        L.moe_profile_start.restype = None
        L.moe_profile_stop.argtypes = []
        L.moe_profile_stop.restype = None
        L.moe_profile_read.argtypes = [POINTER(c_int), POINTER(c_float), c_int]
        L.moe_profile_read.restype = c_int
        L.moe_debug_launch_count.argtypes = []
        L.moe_debug_launch_count.restype = ctypes.c_ulonglong
        L.moe_bounds_checked.argtypes = []
        L.moe_bounds_checked.restype = c_int
        L.moe_read_ceiling.argtypes = [vp, c_size_t, vp, vp]
        L.moe_read_ceiling.restype = c_int
        L.moe_write_ceiling.argtypes = [vp, c_size_t, ctypes.c_uint, vp]
        L.moe_write_ceiling.restype = c_int
        L.moe_debug_workspace_offset.argtypes = [POINTER(MoeConfig), c_int, c_int]
        L.moe_debug_workspace_offset.restype = c_size_t
        L.moe_mx_weight_bytes.restype = c_size_t
        L.moe_mx_weight_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_mx_workspace_bytes.restype = c_size_t
        L.moe_mx_workspace_bytes.argtypes = [POINTER(MoeConfig)]
        L.moe_mx_quantize_weights.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeMxWeights), vp]
        L.moe_mx_quantize.argtypes = [vp, c_longlong, c_int, vp, vp, vp]
        L.moe_layer_fwd_mxfp8.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, POINTER(MoeMxWeights), vp, vp, vp, vp,
                                          vp, c_size_t, vp]
        for n in ("moe_mx_quantize_weights", "moe_mx_quantize", "moe_layer_fwd_mxfp8"):
            getattr(L, n).restype = c_int
        L.moe_mx_bwd_weight_bytes.restype = c_size_t
        L.moe_mx_bwd_weight_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_mx_train_workspace_bytes.restype = c_size_t
        L.moe_mx_train_workspace_bytes.argtypes = [POINTER(MoeConfig)]
        L.moe_mx_quantize_bwd_weights.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeMxBwdWeights), vp]
        L.moe_layer_fwd_mxfp8_train.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, POINTER(MoeMxWeights), vp,
                                                POINTER(MoeFwdSaved), vp, c_size_t, vp]
        L.moe_layer_bwd_mxfp8.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeMxBwdWeights),
                                          POINTER(MoeFwdSaved), vp, vp, vp, vp, vp, vp, c_int, vp, c_size_t, vp]
        for n in ("moe_mx_quantize_bwd_weights", "moe_layer_fwd_mxfp8_train", "moe_layer_bwd_mxfp8"):
            getattr(L, n).restype = c_int
        L.moe_nv_weight_bytes.restype = c_size_t
        L.moe_nv_weight_bytes.argtypes = [c_int, c_int, c_int, c_int]
        L.moe_nv_workspace_bytes.restype = c_size_t
        L.moe_nv_workspace_bytes.argtypes = [c_int, c_longlong, c_int]
        L.moe_nv_quantize_weights.argtypes = [c_int, c_int, c_int, vp, vp, vp, vp, vp]
        L.moe_nv_quantize.argtypes = [vp, c_longlong, c_int, vp, vp, vp, vp]
        L.moe_nv_grouped_gemm.argtypes = [c_int, c_longlong, c_int, c_int, vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
        for n in ("moe_nv_quantize_weights", "moe_nv_quantize", "moe_nv_grouped_gemm"):
            getattr(L, n).restype = c_int
        L.moe_nv_layer_weight_bytes.restype = c_size_t
        L.moe_nv_layer_weight_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_nv_workspace_bytes_layer.restype = c_size_t
        L.moe_nv_workspace_bytes_layer.argtypes = [POINTER(MoeConfig)]
        L.moe_nv_quantize_layer_weights.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeNvWeights), vp]
        L.moe_layer_fwd_nvfp4.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, POINTER(MoeNvWeights), vp, vp,
                                          c_size_t, vp]
        for n in ("moe_nv_quantize_layer_weights", "moe_layer_fwd_nvfp4"):
            getattr(L, n).restype = c_int
        L.moe_nv_bwd_weight_bytes.restype = c_size_t
        L.moe_nv_bwd_weight_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_nv_train_workspace_bytes.restype = c_size_t
        L.moe_nv_train_workspace_bytes.argtypes = [POINTER(MoeConfig)]
        L.moe_nv_quantize_bwd_weights.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeNvBwdWeights), vp]
        L.moe_nv_quantize_train_weights.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeNvWeights),
                                                    POINTER(MoeNvBwdWeights), vp]
        L.moe_layer_fwd_nvfp4_train.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, POINTER(MoeNvWeights), vp,
                                                POINTER(MoeFwdSaved), vp, c_size_t, vp]
        L.moe_layer_bwd_nvfp4.argtypes = [POINTER(MoeConfig), vp, vp, vp, POINTER(MoeNvBwdWeights),
                                          POINTER(MoeFwdSaved), vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
        for n in ("moe_nv_quantize_bwd_weights", "moe_nv_quantize_train_weights", "moe_layer_fwd_nvfp4_train",
                  "moe_layer_bwd_nvfp4"):
            getattr(L, n).restype = c_int
        for n in ("moe_balance_workspace_bytes", "moe_balance_stats_floats"):
            getattr(L, n).restype = c_size_t
            getattr(L, n).argtypes = [POINTER(MoeBalanceConfig)]
        L.moe_balance_loss_fwd.argtypes = [POINTER(MoeBalanceConfig)] + [vp] * 8 + [c_size_t, vp]
        L.moe_layer_bwd_dlogits.argtypes = [POINTER(MoeConfig)] + [vp] * 10 + [POINTER(MoeFwdSaved)] + [vp] * 10 + [
            c_size_t, vp]
        L.moe_layer_bwd_mxfp8_dlogits.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, POINTER(MoeMxBwdWeights),
                                                  POINTER(MoeFwdSaved)] + [vp] * 6 + [c_int, vp, c_size_t, vp]
        L.moe_layer_bwd_nvfp4_dlogits.argtypes = [POINTER(MoeConfig), vp, vp, vp, vp, POINTER(MoeNvBwdWeights),
                                                  POINTER(MoeFwdSaved)] + [vp] * 7 + [c_size_t, vp]
        L.moe_balance_loss_bwd.argtypes = [POINTER(MoeBalanceConfig)] + [vp] * 7
        for n in ("moe_adapter_plan_bytes", "moe_adapter_saved_bytes"):
            getattr(L, n).restype = c_size_t
            getattr(L, n).argtypes = [POINTER(MoeAdapterConfig)]
        L.moe_adapter_workspace_bytes.restype = c_size_t
        L.moe_adapter_workspace_bytes.argtypes = [POINTER(MoeAdapterConfig), c_int]
        L.moe_adapter_plan.argtypes = [POINTER(MoeAdapterConfig), vp, vp, c_size_t, vp]
        L.moe_adapter_fwd.argtypes = [POINTER(MoeAdapterConfig)] + [vp] * 9 + [c_size_t, vp]
        L.moe_adapter_bwd.argtypes = [POINTER(MoeAdapterConfig)] + [vp] * 12 + [c_size_t, vp]
        L.moe_tensor_list_bytes.restype = c_size_t
        L.moe_tensor_list_bytes.argtypes = [c_int]
        L.moe_tensor_list_build.argtypes = [POINTER(MoeTensor), c_int, vp, c_size_t]
        L.moe_grad_norm_workspace_bytes.restype = c_size_t
        L.moe_grad_norm_workspace_bytes.argtypes = []
        L.moe_grad_norm.argtypes = [vp, c_int, vp, vp, c_size_t, vp]
        L.moe_clip_grad_norm.argtypes = [vp, c_int, c_float, vp, vp, c_size_t, vp]
        for n in ("moe_layer_bwd_dlogits", "moe_layer_bwd_mxfp8_dlogits", "moe_layer_bwd_nvfp4_dlogits",
                  "moe_balance_loss_fwd", "moe_balance_loss_bwd", "moe_adapter_plan", "moe_adapter_fwd",
                  "moe_adapter_bwd", "moe_tensor_list_build", "moe_grad_norm", "moe_clip_grad_norm"):
            getattr(L, n).restype = c_int
        L.moe_mx4_weight_bytes.restype = c_size_t
        L.moe_mx4_weight_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_mx4_quantize.argtypes = [vp, c_longlong, c_int, vp, vp, vp]
        L.moe_mx4_dequantize.argtypes = [vp, vp, c_longlong, c_int, vp, vp]
        L.moe_mx4_quantize_weights.argtypes = [POINTER(MoeConfig)] + [vp] * 6 + [POINTER(MoeMx4Weights), vp]
        L.moe_mx4_dequantize_weights.argtypes = [POINTER(MoeConfig), POINTER(MoeMx4Weights)] + [vp] * 7
        L.moe_few_workspace_bytes.restype = c_size_t
        L.moe_few_workspace_bytes.argtypes = [POINTER(MoeConfig), c_int]
        L.moe_layer_few_fwd.argtypes = [POINTER(MoeConfig)] + [vp] * 14 + [c_size_t, vp]
        L.moe_layer_few_fwd_mxfp4.argtypes = [POINTER(MoeConfig)] + [vp] * 4 + [POINTER(MoeMx4Weights)] + [vp] * 4 + [
            c_size_t, vp]
        L.moe_norm_workspace_bytes.restype = c_size_t
        L.moe_norm_workspace_bytes.argtypes = [POINTER(MoeNormConfig)]
        L.moe_block_norm_fwd.argtypes = [POINTER(MoeNormConfig)] + [vp] * 9
        L.moe_block_norm_bwd.argtypes = [POINTER(MoeNormConfig)] + [vp] * 14 + [c_size_t, vp]
        for n in ("moe_mx4_quantize", "moe_mx4_dequantize", "moe_mx4_quantize_weights", "moe_mx4_dequantize_weights",
                  "moe_layer_few_fwd", "moe_layer_few_fwd_mxfp4", "moe_block_norm_fwd", "moe_block_norm_bwd"):
            getattr(L, n).restype = c_int
        _lib = L
    return _lib


STAGE_NAMES = {20: "nv_quantize", 21: "nv_gemm", 22: "mx_quantize_tokens", 24: "mx_dgrad_down_swiglu",
               25: "mx_dgrad_gate_up", 26: "shared_dgrad_down_swiglu", 27: "shared_wgrad_down",
               28: "shared_dgrad_gate_up", 29: "shared_wgrad_gate_up", 1: "router", 2: "permute", 3: "ffn1_gate_up", 4: "ffn2_down", 5: "shared_gate_up",
               6: "shared_down", 7: "combine", 10: "combine_bwd", 11: "router_bwd_elem", 12: "dgrad_down_swiglu",
               13: "wgrad_down", 14: "dgrad_gate_up", 15: "wgrad_gate_up", 16: "router_dgrad",
               17: "permute_bwd", 18: "router_wgrad", 19: "aux_loss", 30: "read_ceiling",
               31: "write_ceiling", 40: "grad_norm", 41: "grad_clip", 43: "balance_loss",
               44: "balance_loss_bwd", 45: "adapter_plan", 46: "adapter_shrink", 47: "adapter_expand",
               48: "adapter_wgrad", 50: "layer_few", 51: "mx4_quantize", 52: "mx4_dequantize",
               53: "block_norm", 54: "block_norm_bwd", 55: "block_norm_sums", 32: "nv_dgrad_down", 33: "nv_swiglu_bwd", 34: "nv_dgrad_gate_up"}


def profile_start(capacity: int) -> None:
    lib().moe_profile_start(int(capacity))


def profile_stop() -> None:
    lib().moe_profile_stop()


def profile_read(max_events: int):
    """[(stage name, ms)] for every recorded stage, in order."""
    tags = (c_int * max_events)()
    ms = (c_float * max_events)()
    n = lib().moe_profile_read(tags, ms, max_events)
    if n < 0:
        raise MoeError(4, "moe_profile_read")
    return [(STAGE_NAMES.get(tags[i], str(tags[i])), float(ms[i])) for i in range(n) if tags[i] != 0]


def read_ceiling(buf: torch.Tensor, sink: torch.Tensor) -> None:
    """moe_read_ceiling over the bytes of a contiguous CUDA tensor (a
    measurement helper: one read-only pass; time it with events)."""
    assert buf.is_cuda and buf.is_contiguous() and sink.is_cuda
    nbytes = buf.numel() * buf.element_size() // 16 * 16
    _check(lib().moe_read_ceiling(_p(buf), nbytes, _p(sink), _stream()), "moe_read_ceiling")


def write_ceiling(buf: torch.Tensor, word: int = 0) -> None:
    """moe_write_ceiling over the bytes of a contiguous CUDA tensor (a
    measurement helper: one write-only pass; time it with events)."""
    assert buf.is_cuda and buf.is_contiguous()
    nbytes = buf.numel() * buf.element_size() // 16 * 16
    _check(lib().moe_write_ceiling(_p(buf), nbytes, int(word) & 0xFFFFFFFF, _stream()), "moe_write_ceiling")


def launch_count() -> int:
    return int(lib().moe_debug_launch_count())


WS_TENSORS = {"dy_perm": 0, "dh13": 1, "a": 2, "dx_perm": 3}


def workspace_tensor(ws, cfg, training, name):
    """Test hook: a view of an intermediate the layer keeps in the workspace
    (bf16 dy_perm [R,H], dh13 [R,2F], a [R,F]; dx_perm [R,H], fp32 with
    inter_fp32)."""
    off = int(lib().moe_debug_workspace_offset(ctypes.byref(cfg), int(training), WS_TENSORS[name]))
    if off == ctypes.c_size_t(-1).value:
        raise MoeError(1, "moe_debug_workspace_offset")
    R = cfg.T * cfg.k
    cols = {"dy_perm": cfg.H, "dh13": 2 * cfg.F, "a": cfg.F, "dx_perm": cfg.H}[name]
    dt = torch.float32 if (name == "dx_perm" and cfg.inter_fp32) else torch.bfloat16
    nb = R * cols * (4 if dt == torch.float32 else 2)
    return ws[off:off + nb].view(dt).view(R, cols)


def _p(t):
    if t is None:
        return None
    assert t.is_contiguous(), "tensors must be contiguous"
    return c_void_p(t.data_ptr())


# The current device and its current stream as a raw handle: building a torch.cuda.Stream
# costs microseconds. A torch without these two (one built without CUDA, where the
# configurations and the host's checks still work) has the public calls.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(dev=None, _raw=_current_raw_stream, _device=_current_device):
    """The current stream of the current device (dev, where the caller knows it),
    as the library takes it."""
    return _raw(_device() if dev is None else dev)


def _check(st, where):
    if st != MOE_OK:
        raise MoeError(st, where)


def make_config(T, H, E, k, F, F_shared=0, score="softmax", n_groups=1, topk_groups=1, gate_scale=1.0,
                aux_coeff=0.0, out_fp32=False, inter_fp32=False, force_balanced=False) -> MoeConfig:
    return MoeConfig(T, H, E, k, F, F_shared, SCORE[score] if isinstance(score, str) else score, n_groups,
                     topk_groups, gate_scale, aux_coeff, int(out_fp32), int(inter_fp32), int(force_balanced))


def config_from_shape(ls, **over) -> MoeConfig:
    d = dict(T=ls.T, H=ls.H, E=ls.E, k=ls.k, F=ls.F, F_shared=ls.F_shared, score=ls.score, n_groups=ls.n_groups,
             topk_groups=ls.topk_groups, gate_scale=ls.gate_scale, aux_coeff=ls.aux_coeff, out_fp32=ls.out_fp32,
             inter_fp32=ls.inter_fp32, force_balanced=getattr(ls, "force_balanced", False))
    d.update(over)
    return make_config(**d)


def workspace_bytes(cfg: MoeConfig, training: bool = False) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(cfg), int(training)))


def workspace(cfg: MoeConfig, training: bool = False, device="cuda") -> torch.Tensor:
    n = workspace_bytes(cfg, training)
    if n == 0:
        raise MoeError(1, "moe_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()  # device status word
    return ws


def device_status(ws: torch.Tensor) -> int:
    out = c_int(0)
    _check(lib().moe_get_device_status(_p(ws), _stream(), ctypes.byref(out)), "moe_get_device_status")
    return out.value


def set_wait_limit_ns(ns: int) -> None:
    lib().moe_debug_set_wait_limit_ns(int(ns))


def set_fault(f: int) -> None:
    lib().moe_debug_set_fault(int(f))


def _inter_dtype(cfg):
    return torch.float32 if cfg.inter_fp32 else torch.bfloat16


def _out_dtype(cfg):
    return torch.float32 if cfg.out_fp32 else torch.bfloat16


def router_topk(cfg, x, router_w, expert_bias=None, logit_bias=None, want_logits=False, want_aux=False, ws=None):
    dev = x.device
    T, E, k = cfg.T, cfg.E, cfg.k
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    gate = torch.empty((T, k), dtype=torch.float32, device=dev)
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None
    aux = torch.empty((4 * ((T + 127) // 128), E), dtype=torch.float32, device=dev) if want_aux else None
    ws = workspace(cfg, False, dev) if ws is None else ws
    st = lib().moe_router_topk(ctypes.byref(cfg), _p(x), _p(router_w), _p(expert_bias), _p(logit_bias), _p(idx),
                               _p(gate), _p(logits), _p(aux), _p(ws), ws.numel(), _stream())
    _check(st, "moe_router_topk")
    return idx, gate, logits, aux


def permute(cfg, x, topk_idx, ws=None):
    dev = x.device
    T, H, E, k = cfg.T, cfg.H, cfg.E, cfg.k
    x_perm = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev)
    rows = torch.empty((T, k), dtype=torch.int32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    ws = workspace(cfg, False, dev) if ws is None else ws
    st = lib().moe_permute(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(x_perm), _p(rows), _p(counts), _p(offsets),
                           _p(ws), ws.numel(), _stream())
    _check(st, "moe_permute")
    return x_perm, rows, counts, offsets


def grouped_swiglu_ffn(cfg, x_perm, offsets, W1, W3, W2, save=False, ws=None):
    dev = x_perm.device
    R, H, F = cfg.T * cfg.k, cfg.H, cfg.F
    y_perm = torch.empty((R, H), dtype=_inter_dtype(cfg), device=dev)
    h13 = torch.empty((R, 2 * F), dtype=torch.bfloat16, device=dev) if save else None
    a = torch.empty((R, F), dtype=torch.bfloat16, device=dev) if save else None
    ws = workspace(cfg, False, dev) if ws is None else ws
    st = lib().moe_grouped_swiglu_ffn(ctypes.byref(cfg), _p(x_perm), _p(offsets), _p(W1), _p(W3), _p(W2), _p(h13),
                                      _p(a), _p(y_perm), _p(ws), ws.numel(), _stream())
    _check(st, "moe_grouped_swiglu_ffn")
    return y_perm, h13, a


def unpermute_combine(cfg, y_perm, row_id_map, topk_gate, shared=None):
    y = torch.empty((cfg.T, cfg.H), dtype=_out_dtype(cfg), device=y_perm.device)
    st = lib().moe_unpermute_combine(ctypes.byref(cfg), _p(y_perm), _p(row_id_map), _p(topk_gate), _p(shared),
                                     _p(y), _stream())
    _check(st, "moe_unpermute_combine")
    return y


def alloc_saved(cfg, device="cuda", recompute=False):
    """Tensors the training forward keeps for the backward. ``recompute``:
    the memory-saving mode, which keeps neither ``a`` nor ``y_perm`` (the
    backward recomputes ``a`` from ``h13`` and takes the gate gradient from
    the down-projection dgrad)."""
    T, H, E, k, F = cfg.T, cfg.H, cfg.E, cfg.k, cfg.F
    R = T * k
    f32, i32, bf = torch.float32, torch.int32, torch.bfloat16
    return {
        "topk_idx": torch.empty((T, k), dtype=i32, device=device),
        "topk_gate": torch.empty((T, k), dtype=f32, device=device),
        "logits": torch.empty((T, E), dtype=f32, device=device),
        "row_id_map": torch.empty((T, k), dtype=i32, device=device),
        "counts": torch.empty(E, dtype=i32, device=device),
        "offsets": torch.empty(E + 1, dtype=i32, device=device),
        "x_perm": torch.empty((R, H), dtype=bf, device=device),
        "h13": torch.empty((R, 2 * F), dtype=bf, device=device),
        "a": None if recompute else torch.empty((R, F), dtype=bf, device=device),
        "y_perm": None if recompute else torch.empty((R, H), dtype=_inter_dtype(cfg), device=device),
        "aux_partials": torch.empty((4 * ((T + 127) // 128), E), dtype=f32, device=device) if cfg.aux_coeff else None,
        "h13_shared": torch.empty((T, 2 * cfg.F_shared), dtype=bf, device=device) if cfg.F_shared else None,
        "a_shared": torch.empty((T, cfg.F_shared), dtype=bf, device=device) if cfg.F_shared else None,
    }


def _saved_struct(saved):
    return MoeFwdSaved(*[None if saved.get(n) is None else saved[n].data_ptr() for n, _ in MoeFwdSaved._fields_])


def layer_fwd(cfg, x, router_w, W1, W3, W2, expert_bias=None, logit_bias=None, Ws=None, saved=None, ws=None, y=None):
    """Whole layer forward. ``saved`` (from alloc_saved) makes it a training
    forward that keeps the tensors the backward needs."""
    dev = x.device
    if y is None:
        y = torch.empty((cfg.T, cfg.H), dtype=_out_dtype(cfg), device=dev)
    ws = workspace(cfg, saved is not None, dev) if ws is None else ws
    Ws1, Ws3, Ws2 = Ws if Ws is not None else (None, None, None)
    sv = ctypes.byref(_saved_struct(saved)) if saved is not None else None
    st = lib().moe_layer_fwd(ctypes.byref(cfg), _p(x), _p(router_w), _p(expert_bias), _p(logit_bias), _p(W1),
                             _p(W3), _p(W2), _p(Ws1), _p(Ws3), _p(Ws2), _p(y), sv, _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_fwd")
    return y


def alloc_grads(cfg, device="cuda"):
    T, H, E, F, Fs = cfg.T, cfg.H, cfg.E, cfg.F, cfg.F_shared
    f32 = torch.float32
    g = {
        "dx": torch.empty((T, H), dtype=_out_dtype(cfg), device=device),
        "dW_r": torch.empty((E, H), dtype=f32, device=device),
        "dW1": torch.empty((E, H, F), dtype=f32, device=device),
        "dW3": torch.empty((E, H, F), dtype=f32, device=device),
        "dW2": torch.empty((E, F, H), dtype=f32, device=device),
        "aux_loss": torch.zeros(1, dtype=f32, device=device),
    }
    if Fs:  # the shared expert's weight gradients
        g["dWs1"] = torch.empty((H, Fs), dtype=f32, device=device)
        g["dWs3"] = torch.empty((H, Fs), dtype=f32, device=device)
        g["dWs2"] = torch.empty((Fs, H), dtype=f32, device=device)
    return g


def _dlogits(where, cfg, dlogits):
    return _arg(where, "dlogits", dlogits, torch.float32, (cfg.T, cfg.E), optional=True)


def layer_bwd(cfg, dO, x, router_w, W1, W3, W2, saved, ws=None, grads=None, Ws=None, dlogits=None):
    """Whole layer backward (``Ws``: the shared expert's weights when
    cfg.F_shared > 0; its gradients land in grads dWs1, dWs3, dWs2).
    ``dlogits`` [T, E] fp32 (balance_loss_bwd): a gradient of the router logits
    from outside the layer, carried into dx and dW_r with the layer's own."""
    dev = x.device
    g = alloc_grads(cfg, dev) if grads is None else grads
    ws = workspace(cfg, True, dev) if ws is None else ws
    sv = _saved_struct(saved)
    Ws1, Ws3, Ws2 = Ws if Ws is not None else (None, None, None)
    st = lib().moe_layer_bwd_dlogits(ctypes.byref(cfg), _p(dO), _dlogits("layer_bwd", cfg, dlogits), _p(x),
                                     _p(router_w), _p(W1), _p(W3), _p(W2), _p(Ws1), _p(Ws3), _p(Ws2),
                                     ctypes.byref(sv), _p(g["dx"]), _p(g["dW_r"]), _p(g["dW1"]), _p(g["dW3"]),
                                     _p(g["dW2"]), _p(g.get("dWs1")), _p(g.get("dWs3")), _p(g.get("dWs2")),
                                     _p(g["aux_loss"]), _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_bwd")
    return g


# ---------------------------------------------------------------------------
# MXFP8 expert GEMMs (forward)
# ---------------------------------------------------------------------------
class MoeMxWeights(ctypes.Structure):
    """Mirror of moe_mx_weights (four device pointers)."""
    _fields_ = [("w13", c_void_p), ("sf13", c_void_p), ("w2", c_void_p), ("sf2", c_void_p)]


MX_WEIGHT_FIELDS = ("w13", "sf13", "w2", "sf2")


def mx_quantize_weights(cfg, W1, W3, W2):
    """Quantise the bf16 expert weights into new uint8 device tensors (dict
    with keys w13 [E,2,F,H], sf13, w2 [E,H,F], sf2)."""
    dev = W1.device
    out = {}
    for i, n in enumerate(MX_WEIGHT_FIELDS):
        nb = int(lib().moe_mx_weight_bytes(ctypes.byref(cfg), i))
        if nb == 0:
            raise MoeError(2, "moe_mx_weight_bytes")
        out[n] = torch.empty(nb, dtype=torch.uint8, device=dev)
    out["w13"] = out["w13"].view(cfg.E, 2, cfg.F, cfg.H)
    out["w2"] = out["w2"].view(cfg.E, cfg.H, cfg.F)
    st = lib().moe_mx_quantize_weights(ctypes.byref(cfg), _p(W1), _p(W3), _p(W2), ctypes.byref(_mx_struct(out)),
                                       _stream())
    _check(st, "moe_mx_quantize_weights")
    return out


def _mx_struct(w):
    return MoeMxWeights(*[w[n].data_ptr() for n in MX_WEIGHT_FIELDS])


def mx_quantize(x):
    """Row-major MXFP8 quantisation of a bf16 [M, K] tensor: (codes uint8
    [M, K], scales uint8 [M, K/32])."""
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    _check(lib().moe_mx_quantize(_p(x), M, K, _p(q), _p(s), _stream()), "moe_mx_quantize")
    return q, s


def mx_workspace(cfg, device="cuda"):
    n = int(lib().moe_mx_workspace_bytes(ctypes.byref(cfg)))
    if n == 0:
        raise MoeError(2, "moe_mx_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def layer_fwd_mxfp8(cfg, x, router_w, mxw, expert_bias=None, logit_bias=None, Ws=None, ws=None, y=None):
    """Whole layer forward with MXFP8 expert GEMMs (``mxw`` from
    mx_quantize_weights)."""
    dev = x.device
    if y is None:
        y = torch.empty((cfg.T, cfg.H), dtype=_out_dtype(cfg), device=dev)
    ws = mx_workspace(cfg, dev) if ws is None else ws
    Ws1, Ws3, Ws2 = Ws if Ws is not None else (None, None, None)
    st = lib().moe_layer_fwd_mxfp8(ctypes.byref(cfg), _p(x), _p(router_w), _p(expert_bias), _p(logit_bias),
                                   ctypes.byref(_mx_struct(mxw)), _p(Ws1), _p(Ws3), _p(Ws2), _p(y), _p(ws),
                                   ws.numel(), _stream())
    _check(st, "moe_layer_fwd_mxfp8")
    return y


# ---------------------------------------------------------------------------
# MXFP8 training step (forward saving, backward with MXFP8 data gradients)
# ---------------------------------------------------------------------------
class MoeMxBwdWeights(ctypes.Structure):
    """Mirror of moe_mx_bwd_weights (four device pointers)."""
    _fields_ = [("w2h", c_void_p), ("sf2h", c_void_p), ("w13f", c_void_p), ("sf13f", c_void_p)]


MX_BWD_WEIGHT_FIELDS = ("w2h", "sf2h", "w13f", "sf13f")


def mx_quantize_bwd_weights(cfg, W1, W3, W2):
    """Weights of the MXFP8 data-gradient GEMMs as new uint8 device tensors:
    w2h [E,F,H] (W2 along H), w13f [E,H,2F] (W1 | W3 along F), sf2h, sf13f."""
    dev = W1.device
    out = {}
    for i, n in enumerate(MX_BWD_WEIGHT_FIELDS):
        nb = int(lib().moe_mx_bwd_weight_bytes(ctypes.byref(cfg), i))
        if nb == 0:
            raise MoeError(2, "moe_mx_bwd_weight_bytes")
        out[n] = torch.empty(nb, dtype=torch.uint8, device=dev)
    out["w2h"] = out["w2h"].view(cfg.E, cfg.F, cfg.H)
    out["w13f"] = out["w13f"].view(cfg.E, cfg.H, 2 * cfg.F)
    w = MoeMxBwdWeights(*[out[n].data_ptr() for n in MX_BWD_WEIGHT_FIELDS])
    _check(lib().moe_mx_quantize_bwd_weights(ctypes.byref(cfg), _p(W1), _p(W3), _p(W2), ctypes.byref(w), _stream()),
           "moe_mx_quantize_bwd_weights")
    return out


def mx_train_workspace(cfg, device="cuda"):
    n = int(lib().moe_mx_train_workspace_bytes(ctypes.byref(cfg)))
    if n == 0:
        raise MoeError(2, "moe_mx_train_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def alloc_saved_mxfp8(cfg, device="cuda"):
    """Saved tensors of the MXFP8 training forward (``a`` is not kept: the
    backward recomputes it from ``h13``)."""
    sv = alloc_saved(cfg, device)
    sv["a"] = None
    return sv


def layer_fwd_mxfp8_train(cfg, x, router_w, mxw, saved, expert_bias=None, logit_bias=None, ws=None, y=None):
    """Training forward of the MXFP8 layer (``saved`` from alloc_saved_mxfp8)."""
    dev = x.device
    if y is None:
        y = torch.empty((cfg.T, cfg.H), dtype=_out_dtype(cfg), device=dev)
    ws = mx_train_workspace(cfg, dev) if ws is None else ws
    st = lib().moe_layer_fwd_mxfp8_train(ctypes.byref(cfg), _p(x), _p(router_w), _p(expert_bias), _p(logit_bias),
                                         ctypes.byref(_mx_struct(mxw)), _p(y), ctypes.byref(_saved_struct(saved)),
                                         _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_fwd_mxfp8_train")
    return y


def layer_bwd_mxfp8(cfg, dO, x, router_w, mxbw, saved, ws=None, grads=None, mx_wgrad=False, dlogits=None):
    """Backward of the MXFP8 training step (``mxbw`` from
    mx_quantize_bwd_weights); gradients and ``dlogits`` as layer_bwd. ``mx_wgrad``: the weight
    gradients in MXFP8 too (operands quantised along each expert's tokens)."""
    dev = x.device
    g = alloc_grads(cfg, dev) if grads is None else grads
    ws = mx_train_workspace(cfg, dev) if ws is None else ws
    w = MoeMxBwdWeights(*[mxbw[n].data_ptr() for n in MX_BWD_WEIGHT_FIELDS])
    st = lib().moe_layer_bwd_mxfp8_dlogits(ctypes.byref(cfg), _p(dO), _dlogits("layer_bwd_mxfp8", cfg, dlogits),
                                           _p(x), _p(router_w), ctypes.byref(w), ctypes.byref(_saved_struct(saved)),
                                           _p(g["dx"]), _p(g["dW_r"]), _p(g["dW1"]), _p(g["dW3"]), _p(g["dW2"]),
                                           _p(g["aux_loss"]), int(bool(mx_wgrad)), _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_bwd_mxfp8")
    return g


# ---------------------------------------------------------------------------
# NVFP4 grouped expert GEMM
# ---------------------------------------------------------------------------
def nv_quantize_weights(W):
    """Quantise expert weights W [E, K, N] bf16: dict with wq [E, N, K/2]
    (codes, two per byte), sf (tile-ready E4M3 scales), g [E] fp32."""
    E, K, N = W.shape
    nb = [int(lib().moe_nv_weight_bytes(E, K, N, i)) for i in range(3)]
    if 0 in nb:
        raise MoeError(2, "moe_nv_weight_bytes")
    wq = torch.empty((E, N, K // 2), dtype=torch.uint8, device=W.device)
    sf = torch.empty(nb[1], dtype=torch.uint8, device=W.device)
    g = torch.empty(E, dtype=torch.float32, device=W.device)
    _check(lib().moe_nv_quantize_weights(E, K, N, _p(W), _p(wq), _p(sf), _p(g), _stream()), "moe_nv_quantize_weights")
    return {"wq": wq, "sf": sf, "g": g, "E": E, "K": K, "N": N}


def nv_quantize(x):
    """Row-major NVFP4 quantisation of x [M, K] bf16 as one tensor: (codes
    [M, K/2], scales [M, K/16], tensor scale [1])."""
    M, K = x.shape
    q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, K // 16), dtype=torch.uint8, device=x.device)
    g = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().moe_nv_quantize(_p(x), M, K, _p(q), _p(s), _p(g), _stream()), "moe_nv_quantize")
    return q, s, g


def nv_workspace(E, R, K, device="cuda"):
    n = int(lib().moe_nv_workspace_bytes(E, R, K))
    if n == 0:
        raise MoeError(2, "moe_nv_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def nv_grouped_gemm(x, offsets, w, ws=None, y=None):
    """y [R, N] bf16 = grouped NVFP4 GEMM of x [R, K] (rows grouped by
    ``offsets``, [E+1] int32 on the device) with quantised weights ``w``."""
    R, K = x.shape
    E, N = w["E"], w["N"]
    if y is None:
        y = torch.empty((R, N), dtype=torch.bfloat16, device=x.device)
    ws = nv_workspace(E, R, K, x.device) if ws is None else ws
    st = lib().moe_nv_grouped_gemm(E, R, K, N, _p(x), _p(offsets), _p(w["wq"]), _p(w["sf"]), _p(w["g"]), _p(y),
                                   _p(ws), ws.numel(), _stream())
    _check(st, "moe_nv_grouped_gemm")
    return y


class MoeNvWeights(ctypes.Structure):
    """Mirror of moe_nv_weights (six device pointers)."""
    _fields_ = [(n, c_void_p) for n in ("w13", "sf13", "g13", "w2", "sf2", "g2")]


def nv_quantize_layer_weights(cfg, W1, W3, W2):
    """NVFP4 weights of the layer (dict of uint8 / fp32 device tensors)."""
    out = {}
    for i, n in enumerate(MoeNvWeights._fields_):
        nb = int(lib().moe_nv_layer_weight_bytes(ctypes.byref(cfg), i))
        if nb == 0:
            raise MoeError(2, "moe_nv_layer_weight_bytes")
        dt = torch.float32 if n[0].startswith("g") else torch.uint8
        out[n[0]] = torch.empty(nb // (4 if dt == torch.float32 else 1), dtype=dt, device=W1.device)
    st = lib().moe_nv_quantize_layer_weights(ctypes.byref(cfg), _p(W1), _p(W3), _p(W2), ctypes.byref(_nv_struct(out)),
                                             _stream())
    _check(st, "moe_nv_quantize_layer_weights")
    return out


def _nv_struct(w):
    return MoeNvWeights(*[w[n[0]].data_ptr() for n in MoeNvWeights._fields_])


def layer_fwd_nvfp4(cfg, x, router_w, nvw, expert_bias=None, logit_bias=None, ws=None, y=None):
    """Whole layer forward with NVFP4 expert GEMMs (``nvw`` from
    nv_quantize_layer_weights)."""
    dev = x.device
    if y is None:
        y = torch.empty((cfg.T, cfg.H), dtype=_out_dtype(cfg), device=dev)
    if ws is None:
        n = int(lib().moe_nv_workspace_bytes_layer(ctypes.byref(cfg)))
        if n == 0:
            raise MoeError(2, "moe_nv_workspace_bytes_layer")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        ws[:256].zero_()
    st = lib().moe_layer_fwd_nvfp4(ctypes.byref(cfg), _p(x), _p(router_w), _p(expert_bias), _p(logit_bias),
                                   ctypes.byref(_nv_struct(nvw)), _p(y), _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_fwd_nvfp4")
    return y


# ---------------------------------------------------------------------------
# NVFP4 training step (forward saving, backward with NVFP4 data gradients)
# ---------------------------------------------------------------------------
class MoeNvBwdWeights(ctypes.Structure):
    """Mirror of moe_nv_bwd_weights (six device pointers)."""
    _fields_ = [(n, c_void_p) for n in ("w2h", "sf2h", "g2h", "w13f", "sf13f", "g13f")]


def nv_quantize_bwd_weights(cfg, W1, W3, W2):
    """Weights of the NVFP4 data-gradient GEMMs as new device tensors: w2h
    [E,F,H/2] (W2 along H), w13f [E,H,F] (W1 | W3 along 2F; codes two per
    byte), their tile-ready scales sf2h, sf13f and tensor scales g2h, g13f [E]."""
    out = {}
    for i, (n, _) in enumerate(MoeNvBwdWeights._fields_):
        nb = int(lib().moe_nv_bwd_weight_bytes(ctypes.byref(cfg), i))
        if nb == 0:
            raise MoeError(2, "moe_nv_bwd_weight_bytes")
        dt = torch.float32 if n.startswith("g") else torch.uint8
        out[n] = torch.empty(nb // (4 if dt == torch.float32 else 1), dtype=dt, device=W1.device)
    out["w2h"] = out["w2h"].view(cfg.E, cfg.F, cfg.H // 2)
    out["w13f"] = out["w13f"].view(cfg.E, cfg.H, cfg.F)
    w = MoeNvBwdWeights(*[out[n].data_ptr() for n, _ in MoeNvBwdWeights._fields_])
    _check(lib().moe_nv_quantize_bwd_weights(ctypes.byref(cfg), _p(W1), _p(W3), _p(W2), ctypes.byref(w), _stream()),
           "moe_nv_quantize_bwd_weights")
    return out


def _nv_alloc(cfg, size_fn, fields, device):
    out = {}
    for i, (n, _) in enumerate(fields):
        nb = int(size_fn(ctypes.byref(cfg), i))
        if nb == 0:
            raise MoeError(2, size_fn.__name__)
        dt = torch.float32 if n.startswith("g") else torch.uint8
        out[n] = torch.empty(nb // (4 if dt == torch.float32 else 1), dtype=dt, device=device)
    return out


def nv_quantize_train_weights(cfg, W1, W3, W2):
    """Both weight copies of the NVFP4 training step in one call (the maxima
    taken once): the dicts nv_quantize_layer_weights and
    nv_quantize_bwd_weights return."""
    fw = _nv_alloc(cfg, lib().moe_nv_layer_weight_bytes, MoeNvWeights._fields_, W1.device)
    bw = _nv_alloc(cfg, lib().moe_nv_bwd_weight_bytes, MoeNvBwdWeights._fields_, W1.device)
    bw["w2h"] = bw["w2h"].view(cfg.E, cfg.F, cfg.H // 2)
    bw["w13f"] = bw["w13f"].view(cfg.E, cfg.H, cfg.F)
    b = MoeNvBwdWeights(*[bw[n].data_ptr() for n, _ in MoeNvBwdWeights._fields_])
    _check(lib().moe_nv_quantize_train_weights(ctypes.byref(cfg), _p(W1), _p(W3), _p(W2),
                                               ctypes.byref(_nv_struct(fw)), ctypes.byref(b), _stream()),
           "moe_nv_quantize_train_weights")
    return fw, bw


def nv_train_workspace(cfg, device="cuda"):
    n = int(lib().moe_nv_train_workspace_bytes(ctypes.byref(cfg)))
    if n == 0:
        raise MoeError(2, "moe_nv_train_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def layer_fwd_nvfp4_train(cfg, x, router_w, nvw, saved, expert_bias=None, logit_bias=None, ws=None, y=None):
    """Training forward of the NVFP4 layer (``nvw`` from
    nv_quantize_layer_weights, ``saved`` from alloc_saved)."""
    dev = x.device
    if y is None:
        y = torch.empty((cfg.T, cfg.H), dtype=_out_dtype(cfg), device=dev)
    ws = nv_train_workspace(cfg, dev) if ws is None else ws
    st = lib().moe_layer_fwd_nvfp4_train(ctypes.byref(cfg), _p(x), _p(router_w), _p(expert_bias), _p(logit_bias),
                                         ctypes.byref(_nv_struct(nvw)), _p(y), ctypes.byref(_saved_struct(saved)),
                                         _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_fwd_nvfp4_train")
    return y


def layer_bwd_nvfp4(cfg, dO, x, router_w, nvbw, saved, ws=None, grads=None, dlogits=None):
    """Backward of the NVFP4 training step (``nvbw`` from
    nv_quantize_bwd_weights); gradients and ``dlogits`` as layer_bwd."""
    dev = x.device
    g = alloc_grads(cfg, dev) if grads is None else grads
    ws = nv_train_workspace(cfg, dev) if ws is None else ws
    w = MoeNvBwdWeights(*[nvbw[n].data_ptr() for n, _ in MoeNvBwdWeights._fields_])
    st = lib().moe_layer_bwd_nvfp4_dlogits(ctypes.byref(cfg), _p(dO), _dlogits("layer_bwd_nvfp4", cfg, dlogits),
                                           _p(x), _p(router_w), ctypes.byref(w), ctypes.byref(_saved_struct(saved)),
                                           _p(g["dx"]), _p(g["dW_r"]), _p(g["dW1"]), _p(g["dW3"]), _p(g["dW2"]),
                                           _p(g["aux_loss"]), _p(ws), ws.numel(), _stream())
    _check(st, "moe_layer_bwd_nvfp4")
    return g


# ---------------------------------------------------------------------------
# Router losses with gradients
# ---------------------------------------------------------------------------
def _arg(where, name, t, dtype, shape, dev=None, optional=False, _device=_current_device):
    """A tensor argument of the calls below: on the current CUDA device (dev, from
    a call's second argument on), contiguous, of the given type (or one of them)
    and shape; its address. What a call spends here is most of its time on the
    host, so the usual case comes first and asks as little as it can."""
    if t is None and optional:
        return None
    try:
        if (t.dtype is dtype or (dtype.__class__ is tuple and t.dtype in dtype)) and t.shape == shape and t.is_contiguous():
            d = t.get_device()  # -1: not on a GPU
            if d == dev or (dev is None and d >= 0 and d == _device()):
                return t.data_ptr()
    except AttributeError:
        pass
    raise _arg_error(where, name, t, dtype if type(dtype) is tuple else (dtype,), shape)


def _arg_error(where, name, t, dtypes, shape):
    if t is None:
        why = "is missing"
    elif not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape:
        got = f"{t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__
        why = f"must be {' or '.join(str(d) for d in dtypes)} {tuple(shape)}, not {got}"
    elif not t.is_cuda or t.get_device() != torch.cuda.current_device():
        why = f"must be on the current CUDA device, not {t.device}"
    else:
        why = "must be contiguous"
    return MoeError(MOE_ERR_INVALID_ARG, f"{where}: {name} {why}")


def _ws_arg(where, ws, nbytes, dev):
    try:
        if ws.dtype is torch.uint8 and ws.numel() >= nbytes and ws.is_contiguous() and ws.get_device() == dev:
            return ws.data_ptr()
    except AttributeError:
        pass
    if not isinstance(ws, torch.Tensor):
        raise MoeError(MOE_ERR_INVALID_ARG, f"{where}: the workspace must be a uint8 tensor")
    if ws.numel() < nbytes:
        raise MoeError(MOE_ERR_WORKSPACE_TOO_SMALL, where)
    return _arg(where, "the workspace", ws, torch.uint8, ws.shape, dev)


_size_cache = {}


def _device_key():
    """The current device, by which sizes are kept: some go by its number of SMs (-1 where there is none)."""
    try:
        return _current_device()
    except (RuntimeError, AssertionError):  # no driver; a torch built without CUDA
        return -1


def _size(name, cfg, *more):
    """A size the library gives for a config, asked once for each config's
    values and device; raises for a config it refuses."""
    key = (name, bytes(cfg), more, _device_key())
    n = _size_cache.get(key)
    if n is None:
        n = int(getattr(lib(), name)(ctypes.byref(cfg), *more))
        if n == 0:
            raise MoeError(MOE_ERR_INVALID_ARG, name)
        if len(_size_cache) >= 4096:
            _size_cache.clear()
        _size_cache[key] = n
    return n


def _scratch(nbytes, device):
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()  # device status word
    return ws


class MoeBalanceConfig(ctypes.Structure):
    _fields_ = [("T", c_int), ("E", c_int), ("k", c_int), ("n_seqs", c_int), ("score", c_int),
                ("balance_coeff", c_float), ("z_coeff", c_float)]


def make_balance_config(T, E, k, n_seqs=1, score="softmax", balance_coeff=1e-2, z_coeff=0.0) -> MoeBalanceConfig:
    return MoeBalanceConfig(T, E, k, n_seqs, SCORE[score] if isinstance(score, str) else score, balance_coeff, z_coeff)


def _balance_sizes(cfg):
    return _size("moe_balance_workspace_bytes", cfg), _size("moe_balance_stats_floats", cfg)


def balance_workspace(cfg, device="cuda"):
    return _scratch(_balance_sizes(cfg)[0], device)


def balance_loss_fwd(cfg, logits, topk_idx, seq_offsets=None, token_mask=None, ws=None):
    """The router's balance loss and z-loss (cfg from make_balance_config):
    (losses [2] fp32, counts [n_seqs, E] int32, stats for the backward).
    logits [T, E] fp32, topk_idx [T, k] int32, seq_offsets [n_seqs + 1] int32
    (None with one sequence: all rows), token_mask [T] bool or uint8."""
    w = "balance_loss_fwd"
    n_ws, n_stats = _balance_sizes(cfg)
    lp = _arg(w, "logits", logits, torch.float32, (cfg.T, cfg.E))
    d = logits.get_device()
    args = [lp, _arg(w, "topk_idx", topk_idx, torch.int32, (cfg.T, cfg.k), d),
            _arg(w, "seq_offsets", seq_offsets, torch.int32, (cfg.n_seqs + 1,), d, optional=True),
            _arg(w, "token_mask", token_mask, (torch.bool, torch.uint8), (cfg.T,), d, optional=True)]
    dev = logits.device
    losses = torch.empty(2, dtype=torch.float32, device=dev)
    counts = torch.empty((cfg.n_seqs, cfg.E), dtype=torch.int32, device=dev)
    stats = torch.empty(n_stats, dtype=torch.float32, device=dev)
    ws = _scratch(n_ws, dev) if ws is None else ws
    st = lib().moe_balance_loss_fwd(ctypes.byref(cfg), *args, losses.data_ptr(), counts.data_ptr(), stats.data_ptr(),
                                    _ws_arg(w, ws, n_ws, d), ws.numel(), _stream(d))
    _check(st, "moe_balance_loss_fwd")
    return losses, counts, stats


def balance_loss_bwd(cfg, logits, stats, dlosses=None, seq_offsets=None, token_mask=None, dlogits=None):
    """Gradient of <dlosses, losses> for the logits, [T, E] fp32 (dlosses [2]
    fp32; None: 1 and 1). ``layer_bwd(..., dlogits=...)`` adds it to the layer's
    own router gradient."""
    w = "balance_loss_bwd"
    n_stats = _balance_sizes(cfg)[1]
    lp = _arg(w, "logits", logits, torch.float32, (cfg.T, cfg.E))
    d = logits.get_device()
    args = [lp, _arg(w, "stats", stats, torch.float32, (n_stats,), d),
            _arg(w, "dlosses", dlosses, torch.float32, (2,), d, optional=True),
            _arg(w, "seq_offsets", seq_offsets, torch.int32, (cfg.n_seqs + 1,), d, optional=True),
            _arg(w, "token_mask", token_mask, (torch.bool, torch.uint8), (cfg.T,), d, optional=True)]
    if dlogits is None:
        dlogits = torch.empty_like(logits)
        dp = dlogits.data_ptr()
    else:
        dp = _arg(w, "dlogits", dlogits, torch.float32, (cfg.T, cfg.E), d)
    st = lib().moe_balance_loss_bwd(ctypes.byref(cfg), *args, dp, _stream(d))
    _check(st, "moe_balance_loss_bwd")
    return dlogits


# ---------------------------------------------------------------------------
# Low-rank adapters of many requests beside a shared projection
# ---------------------------------------------------------------------------
class MoeAdapterConfig(ctypes.Structure):
    _fields_ = [("T", c_int), ("K", c_int), ("N", c_int), ("L", c_int), ("r", c_int), ("out_fp32", c_int)]


def make_adapter_config(T, K, N, L, r, out_fp32=False) -> MoeAdapterConfig:
    """T rows, a projection of K inputs and N outputs, L adapters of rank r."""
    return MoeAdapterConfig(T, K, N, L, r, int(out_fp32))


def adapter_workspace(cfg, training=False, device="cuda"):
    return _scratch(_size("moe_adapter_workspace_bytes", cfg, int(training)), device)


def alloc_adapter_saved(cfg, device="cuda"):
    """What the training forward keeps for the backward (an opaque buffer)."""
    return torch.empty(_size("moe_adapter_saved_bytes", cfg), dtype=torch.uint8, device=device)


def adapter_plan(cfg, adapter_idx, plan=None):
    """The plan of a batch (a uint8 tensor): its rows ordered by adapter.
    adapter_idx [T] int32, negative for a row without an adapter. One plan
    serves every projection of the batch, forward and backward, whose config
    has the same T and L. device_status(plan) tells of an index >= L."""
    w = "adapter_plan"
    n = _size("moe_adapter_plan_bytes", cfg)
    idx = _arg(w, "adapter_idx", adapter_idx, torch.int32, (cfg.T,))
    d = adapter_idx.get_device()
    if plan is None:
        plan = torch.empty(n, dtype=torch.uint8, device=adapter_idx.device)
        pp = plan.data_ptr()
    else:
        pp = _ws_arg(w, plan, n, d)
    _check(lib().moe_adapter_plan(ctypes.byref(cfg), idx, pp, plan.numel(), _stream(d)), "moe_adapter_plan")
    return plan


def _adapter_args(w, cfg, A, B, scale, plan, d):
    return (_arg(w, "A", A, torch.bfloat16, (cfg.L, cfg.K, cfg.r), d),
            _arg(w, "B", B, torch.bfloat16, (cfg.L, cfg.r, cfg.N), d),
            _arg(w, "scale", scale, torch.float32, (cfg.L,), d),
            _ws_arg(w, plan, _size("moe_adapter_plan_bytes", cfg), d))


def adapter_fwd(cfg, x, A, B, scale, plan, base=None, y=None, u=None, ws=None):
    """y [T, N] = base + scale (x A) B with each row's own adapter (plan from
    adapter_plan). x [T, K], A [L, K, r], B [L, r, N] bf16, scale [L] fp32;
    base and y bf16 (fp32 with cfg.out_fp32). base None: zeros; y may be base.
    u (alloc_adapter_saved): keep what adapter_bwd needs."""
    w = "adapter_fwd"
    xp = _arg(w, "x", x, torch.bfloat16, (cfg.T, cfg.K))
    d = x.get_device()
    weights = _adapter_args(w, cfg, A, B, scale, plan, d)
    out = _out_dtype(cfg)
    bp = _arg(w, "base", base, out, (cfg.T, cfg.N), d, optional=True)
    up = None if u is None else _ws_arg(w, u, _size("moe_adapter_saved_bytes", cfg), d)
    ws = adapter_workspace(cfg, False, x.device) if ws is None else ws
    wp = _ws_arg(w, ws, _size("moe_adapter_workspace_bytes", cfg, 0), d)
    if y is None:
        y = torch.empty_like(base) if base is not None else torch.empty((cfg.T, cfg.N), dtype=out, device=x.device)
        yp = y.data_ptr()
    else:
        yp = _arg(w, "y", y, out, (cfg.T, cfg.N), d)
    st = lib().moe_adapter_fwd(ctypes.byref(cfg), xp, *weights, bp, yp, up, wp, ws.numel(), _stream(d))
    _check(st, "moe_adapter_fwd")
    return y


def alloc_adapter_grads(cfg, device="cuda"):
    return {"dx": torch.empty((cfg.T, cfg.K), dtype=_out_dtype(cfg), device=device),
            "dA": torch.empty((cfg.L, cfg.K, cfg.r), dtype=torch.float32, device=device),
            "dB": torch.empty((cfg.L, cfg.r, cfg.N), dtype=torch.float32, device=device)}


def adapter_bwd(cfg, dy, x, A, B, scale, plan, u, dx_base=None, grads=None, ws=None):
    """Gradients of adapter_fwd: dict with dx [T, K] = dx_base + the adapters'
    part (bf16, fp32 with cfg.out_fp32), dA [L, K, r] and dB [L, r, N] fp32.
    dy [T, N] bf16; the gradient of base is dy itself."""
    w = "adapter_bwd"
    dyp = _arg(w, "dy", dy, torch.bfloat16, (cfg.T, cfg.N))
    d = dy.get_device()
    xp = _arg(w, "x", x, torch.bfloat16, (cfg.T, cfg.K), d)
    weights = _adapter_args(w, cfg, A, B, scale, plan, d)
    up = _ws_arg(w, u, _size("moe_adapter_saved_bytes", cfg), d)
    bp = _arg(w, "dx_base", dx_base, _out_dtype(cfg), (cfg.T, cfg.K), d, optional=True)
    ws = adapter_workspace(cfg, True, x.device) if ws is None else ws
    wp = _ws_arg(w, ws, _size("moe_adapter_workspace_bytes", cfg, 1), d)
    g = alloc_adapter_grads(cfg, x.device) if grads is None else grads
    st = lib().moe_adapter_bwd(ctypes.byref(cfg), dyp, xp, *weights, up, bp,
                               _arg(w, "dx", g["dx"], _out_dtype(cfg), (cfg.T, cfg.K), d),
                               _arg(w, "dA", g["dA"], torch.float32, (cfg.L, cfg.K, cfg.r), d),
                               _arg(w, "dB", g["dB"], torch.float32, (cfg.L, cfg.r, cfg.N), d),
                               wp, ws.numel(), _stream(d))
    _check(st, "moe_adapter_bwd")
    return g


# ---------------------------------------------------------------------------
# Global gradient norm and clipping
# ---------------------------------------------------------------------------
class MoeTensor(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("out", c_void_p), ("n", c_longlong), ("dtype", c_int), ("reserved", c_int)]


GRAD_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
NORM_KIND = {"l2": 0, "max": 1}


class TensorList:
    """The tensors of tensor_list, kept alive, and the library's list of them."""

    def __init__(self, tensors, out):
        self.tensors, self.out = tensors, out
        n = len(tensors)
        size = int(lib().moe_tensor_list_bytes(n))
        if size == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_tensor_list_bytes")
        self.device = tensors[0].get_device() if n else torch.cuda.current_device()
        items = (MoeTensor * max(n, 1))()
        for i, t in enumerate(tensors):
            o = None if out is None else out[i]
            for what, v in (("tensor", t), ("out", o)):
                if v is None and what == "out":
                    continue
                if not isinstance(v, torch.Tensor) or v.dtype not in GRAD_DTYPE or not v.is_contiguous():
                    raise MoeError(MOE_ERR_INVALID_ARG,
                                   f"tensor_list: {what} {i} must be a contiguous fp32, bf16 or fp16 tensor")
                if not v.is_cuda or v.get_device() != self.device:
                    raise MoeError(MOE_ERR_INVALID_ARG, f"tensor_list: {what} {i} must be on one CUDA device with the rest")
            if o is not None and (o.dtype != t.dtype or o.numel() != t.numel()):
                raise MoeError(MOE_ERR_INVALID_ARG, f"tensor_list: out {i} must have its tensor's type and size")
            items[i] = MoeTensor(t.data_ptr(), None if o is None else o.data_ptr(), t.numel(), GRAD_DTYPE[t.dtype], 0)
        self._list = (ctypes.c_uint64 * ((size + 7) // 8))()
        _check(lib().moe_tensor_list_build(items, n, self._list, size), "moe_tensor_list_build")
        self.ptr = ctypes.cast(self._list, c_void_p)


def tensor_list(tensors, out=None):
    """A list of gradients (contiguous fp32, bf16 or fp16 CUDA tensors, views at
    any offset) for grad_norm and clip_grad_norm, built once for buffers that
    stay where they are: building takes the host 1 us a tensor in place and 1.5
    with an out (384 tensors 0.40 and 0.59 ms, where norm and clipping take
    0.02), and calls that are given the tensors themselves build it each time.
    out: where the clipped values go (None: in place)."""
    tensors = list(tensors)
    out = None if out is None else list(out)
    if out is not None and len(out) != len(tensors):
        raise MoeError(MOE_ERR_INVALID_ARG, "tensor_list: out must have one tensor for each")
    return TensorList(tensors, out)


def grad_norm_workspace(device="cuda"):
    return _scratch(int(lib().moe_grad_norm_workspace_bytes()), device)


def _norm_call(where, tensors, kind, ws, call):
    tl = tensors if isinstance(tensors, TensorList) else tensor_list(tensors)
    if kind not in NORM_KIND:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{where}: kind must be one of {sorted(NORM_KIND)}")
    if tl.device != torch.cuda.current_device():
        raise MoeError(MOE_ERR_INVALID_ARG, f"{where}: the tensors must be on the current CUDA device")
    n = int(lib().moe_grad_norm_workspace_bytes())
    ws = _scratch(n, torch.device("cuda", tl.device)) if ws is None else ws
    wp = _ws_arg(where, ws, n, tl.device)
    norm = torch.empty(1, dtype=torch.float32, device=ws.device)
    _check(call(tl.ptr, NORM_KIND[kind], _p(norm), wp, ws.numel()), where)
    return norm


def grad_norm(tensors, kind="l2", ws=None):
    """The global norm ([1] fp32) of a list of gradients (a tensor_list or the
    tensors): "l2" or "max"."""
    return _norm_call("moe_grad_norm", tensors, kind, ws,
                      lambda p, k, norm, w, nb: lib().moe_grad_norm(p, k, norm, w, nb, _stream()))


def clip_grad_norm(tensors, max_norm, kind="l2", ws=None):
    """Scale the gradients by min(1, max_norm / (norm + 1e-6)), in place or into
    the tensor_list's out (max_norm infinite: by 1); returns the norm before
    ([1] fp32)."""
    return _norm_call("moe_clip_grad_norm", tensors, kind, ws,
                      lambda p, k, norm, w, nb: lib().moe_clip_grad_norm(p, k, float(max_norm), norm, w, nb,
                                                                         _stream()))


# ---------------------------------------------------------------------------
# MXFP4: rows and the layer's weights
# ---------------------------------------------------------------------------
class MoeMx4Weights(ctypes.Structure):
    """Mirror of moe_mx4_weights (four device pointers)."""
    _fields_ = [(n, c_void_p) for n in ("w13", "w2", "w13s", "w2s")]


def _mx4_rows(where, name, t, per):
    """(M, K) of a matrix with `per` elements a value, refused where its rows hold no blocks of 32."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{where}: {name} must be a matrix")
    M, K = t.shape
    K *= per
    if K < 1 or K % 32 or K >= 1 << 31:  # (the library takes K as an int)
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, f"{where}: rows must hold blocks of 32, fewer than 2^31 elements")
    if M < 1:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{where}: there must be rows")
    return M, K


def mx4_quantize(x):
    """MXFP4 of the rows of x [M, K] bf16 (K a multiple of 32): (codes [M, K/2]
    uint8, element 2j in the low nibble, scales [M, K/32] uint8, E8M0)."""
    M, K = _mx4_rows("mx4_quantize", "x", x, 1)
    xp = _arg("mx4_quantize", "x", x, torch.bfloat16, (M, K))
    dev, u8 = x.device, torch.uint8
    codes, scales = torch.empty((M, K // 2), dtype=u8, device=dev), torch.empty((M, K // 32), dtype=u8, device=dev)
    st = lib().moe_mx4_quantize(xp, M, K, codes.data_ptr(), scales.data_ptr(), _stream(dev.index))
    if st:
        _check(st, "moe_mx4_quantize")
    return codes, scales


def mx4_dequantize(codes, scales):
    """The values [M, K] bf16 that mx4_quantize's codes and scales stand for, exactly."""
    w = "mx4_dequantize"
    M, K = _mx4_rows(w, "codes", codes, 2)
    cp = _arg(w, "codes", codes, torch.uint8, (M, K // 2))
    dev = codes.device
    sp = _arg(w, "scales", scales, torch.uint8, (M, K // 32), dev.index)
    x = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    st = lib().moe_mx4_dequantize(cp, sp, M, K, x.data_ptr(), _stream(dev.index))
    if st:
        _check(st, "moe_mx4_dequantize")
    return x


def _layer_weights(w, cfg, W1, W3, W2, Ws, d=None):
    """The addresses of the layer's six bf16 weights, the shared expert's None without one."""
    bf, Fs = torch.bfloat16, cfg.F_shared
    p = [_arg(w, "W1", W1, bf, (cfg.E, cfg.H, cfg.F), d)]
    d = W1.get_device()
    p += [_arg(w, "W3", W3, bf, (cfg.E, cfg.H, cfg.F), d), _arg(w, "W2", W2, bf, (cfg.E, cfg.F, cfg.H), d)]
    if not Fs:
        return p + [None] * 3
    if Ws is None or len(Ws) != 3:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{w}: Ws must be the shared expert's three weights")
    return p + [_arg(w, "Ws1", Ws[0], bf, (cfg.H, Fs), d), _arg(w, "Ws3", Ws[1], bf, (cfg.H, Fs), d),
                _arg(w, "Ws2", Ws[2], bf, (Fs, cfg.H), d)]


def _mx4_sizes(cfg):
    fields = [n for n, _ in MoeMx4Weights._fields_]
    used = fields if cfg.F_shared else fields[:2]
    return [(n, _size("moe_mx4_weight_bytes", cfg, i)) for i, n in enumerate(used)]


def _mx4_struct(w, cfg, q, d=None):
    got = {}
    if not isinstance(q, dict):
        raise MoeError(MOE_ERR_INVALID_ARG, f"{w}: the weights must be mx4_quantize_weights' dict")
    for n, size in _mx4_sizes(cfg):
        if q.get(n) is None:
            raise MoeError(MOE_ERR_INVALID_ARG, f"{w}: the weights lack {n}")
        got[n] = _arg(w, n, q[n], torch.uint8, (size,), d)
    return MoeMx4Weights(*[got.get(n) for n, _ in MoeMx4Weights._fields_])


def mx4_quantize_weights(cfg, W1, W3, W2, Ws=None):
    """MXFP4 weights of the layer, the shared expert's included (cfg.F_shared, Ws), for
    layer_few_fwd_mxfp4: a dict of uint8 tensors."""
    w = "mx4_quantize_weights"
    p = _layer_weights(w, cfg, W1, W3, W2, Ws)
    q = {n: torch.empty(size, dtype=torch.uint8, device=W1.device) for n, size in _mx4_sizes(cfg)}
    d = W1.get_device()
    _check(lib().moe_mx4_quantize_weights(ctypes.byref(cfg), *p, ctypes.byref(_mx4_struct(w, cfg, q, d)), _stream(d)),
           "moe_mx4_quantize_weights")
    return q


def mx4_dequantize_weights(cfg, q):
    """(W1, W3, W2, Ws) bf16 that mx4_quantize_weights' dict stands for, exactly (Ws:
    the shared expert's three, None without one)."""
    w = "mx4_dequantize_weights"
    st = _mx4_struct(w, cfg, q)
    dev = q["w13"].device
    new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=dev)
    E, H, F, Fs = cfg.E, cfg.H, cfg.F, cfg.F_shared
    W = [new(E, H, F), new(E, H, F), new(E, F, H)]
    Ws = [new(H, Fs), new(H, Fs), new(Fs, H)] if Fs else None
    p = [t.data_ptr() for t in W] + ([t.data_ptr() for t in Ws] if Fs else [None] * 3)
    _check(lib().moe_mx4_dequantize_weights(ctypes.byref(cfg), ctypes.byref(st), *p, _stream(dev.index)),
           "moe_mx4_dequantize_weights")
    return W[0], W[1], W[2], None if Ws is None else tuple(Ws)


# ---------------------------------------------------------------------------
# The whole layer for a few tokens
# ---------------------------------------------------------------------------
FEW_MAX_T = 64


def few_workspace(cfg, mxfp4=False, device="cuda"):
    """Workspace of layer_few_fwd (mxfp4: of layer_few_fwd_mxfp4). Two calls in flight
    need two."""
    return _scratch(_size("moe_few_workspace_bytes", cfg, int(mxfp4)), device)


def _few_args(w, cfg, x, router_w, expert_bias, logit_bias, ws, y, mxfp4):
    n = _size("moe_few_workspace_bytes", cfg, int(mxfp4))
    xp = _arg(w, "x", x, torch.bfloat16, (cfg.T, cfg.H))
    d, dev = x.get_device(), x.device
    head = (xp, _arg(w, "router_w", router_w, torch.bfloat16, (cfg.E, cfg.H), d),
            _arg(w, "expert_bias", expert_bias, torch.float32, (cfg.E,), d, optional=True),
            _arg(w, "logit_bias", logit_bias, torch.float32, (cfg.E,), d, optional=True))
    idx = torch.empty((cfg.T, cfg.k), dtype=torch.int32, device=dev)
    gate = torch.empty((cfg.T, cfg.k), dtype=torch.float32, device=dev)
    out = _out_dtype(cfg)
    if y is None:
        y = torch.empty((cfg.T, cfg.H), dtype=out, device=dev)
        yp = y.data_ptr()
    else:
        yp = _arg(w, "y", y, out, (cfg.T, cfg.H), d)
    ws = _scratch(n, dev) if ws is None else ws
    tail = (idx.data_ptr(), gate.data_ptr(), yp, _ws_arg(w, ws, n, d), ws.numel(), _stream(d))
    return head, tail, (y, idx, gate), d


def layer_few_fwd(cfg, x, router_w, W1, W3, W2, expert_bias=None, logit_bias=None, Ws=None, ws=None, y=None):
    """layer_fwd at inference for at most FEW_MAX_T tokens, in one kernel: (y [T, H],
    topk_idx [T, k], topk_gate [T, k]). ws from few_workspace; y may be x."""
    w = "layer_few_fwd"
    head, tail, out, d = _few_args(w, cfg, x, router_w, expert_bias, logit_bias, ws, y, False)
    _check(lib().moe_layer_few_fwd(ctypes.byref(cfg), *head, *_layer_weights(w, cfg, W1, W3, W2, Ws, d), *tail),
           "moe_layer_few_fwd")
    return out


def layer_few_fwd_mxfp4(cfg, x, router_w, q, expert_bias=None, logit_bias=None, ws=None, y=None):
    """layer_few_fwd with MXFP4 weights (q from mx4_quantize_weights). An element of x, or
    of the activation, counts with an error of at most 2^-13 of the largest of its 32 (with
    cfg.out_fp32 2^-22). ws from few_workspace(cfg, mxfp4=True)."""
    w = "layer_few_fwd_mxfp4"
    head, tail, out, d = _few_args(w, cfg, x, router_w, expert_bias, logit_bias, ws, y, True)
    _check(lib().moe_layer_few_fwd_mxfp4(ctypes.byref(cfg), *head, ctypes.byref(_mx4_struct(w, cfg, q, d)), *tail),
           "moe_layer_few_fwd_mxfp4")
    return out


# ---------------------------------------------------------------------------
# Norms before and after a block, its gate and the scaled residual
# ---------------------------------------------------------------------------
class MoeNormConfig(ctypes.Structure):
    _fields_ = [("T", c_int), ("H", c_int), ("eps", c_float), ("residual", c_int), ("residual_scale", c_float),
                ("gate", c_int), ("post", c_int), ("pre", c_int), ("residual_fp32", c_int), ("out_fp32", c_int)]


GATE = {"none": 0, "channel": 1, "token": 2}


def make_norm_config(T, H, eps=1e-6, residual=True, residual_scale=1.0, gate="none", post=False, pre=True,
                     residual_fp32=False, out_fp32=False) -> MoeNormConfig:
    """h = residual_scale residual + gate u, u = the norm of y (post) or y; n = the norm
    of h (pre). out_fp32: y and n's gradient fp32, as the layer's y and dx."""
    return MoeNormConfig(T, H, eps, int(residual), residual_scale, GATE[gate] if isinstance(gate, str) else gate,
                         int(post), int(pre), int(residual_fp32), int(out_fp32))


def norm_workspace(cfg, device="cuda"):
    return _scratch(_size("moe_norm_workspace_bytes", cfg), device)


class _NormPlan:
    """What a norm config says, read from the struct once: shapes, types, flags."""

    def __init__(self, cfg):
        self.nbytes = _size("moe_norm_workspace_bytes", cfg)
        self.T, self.H = cfg.T, cfg.H
        self.full, self.vec, self.stats = (cfg.T, cfg.H), (cfg.H,), (cfg.T, 2)
        self.stream = torch.float32 if cfg.residual_fp32 else torch.bfloat16
        self.io = _out_dtype(cfg)
        self.residual, self.post, self.pre = bool(cfg.residual), bool(cfg.post), bool(cfg.pre)
        self.gate = (None, (cfg.H,), (cfg.T,))[cfg.gate]


_norm_plans = {}


def _norm_plan(cfg):
    key = bytes(cfg), _device_key()
    plan = _norm_plans.get(key)
    if plan is None:
        plan = _NormPlan(cfg)
        if len(_norm_plans) >= 4096:
            _norm_plans.clear()
        _norm_plans[key] = plan
    return plan


def _norm_args(w, q, y, residual, post_weight, gate, pre_weight):
    f32 = torch.float32
    yp = _arg(w, "y", y, q.io, q.full)
    d = y.get_device()
    return d, (yp, _arg(w, "residual", residual, q.stream, q.full, d) if q.residual else None,
               _arg(w, "post_weight", post_weight, f32, q.vec, d) if q.post else None,
               _arg(w, "gate", gate, f32, q.gate, d) if q.gate else None,
               _arg(w, "pre_weight", pre_weight, f32, q.vec, d) if q.pre else None)


def block_norm_fwd(cfg, y, residual=None, post_weight=None, gate=None, pre_weight=None, h=None, n=None):
    """(h [T, H], n [T, H] bf16 or None, stats [T, 2] for the backward) of the block's
    output y (cfg from make_norm_config). residual and h bf16 (fp32 with
    cfg.residual_fp32), weights [H] and gate [H] or [T] fp32. h may be residual."""
    w = "block_norm_fwd"
    q = _norm_plan(cfg)
    d, p = _norm_args(w, q, y, residual, post_weight, gate, pre_weight)
    dev = y.device
    if h is None:
        h = torch.empty(q.full, dtype=q.stream, device=dev)
        hp = h.data_ptr()
    else:
        hp = _arg(w, "h", h, q.stream, q.full, d)
    if not q.pre:
        n = np_ = None
    elif n is None:
        n = torch.empty(q.full, dtype=torch.bfloat16, device=dev)
        np_ = n.data_ptr()
    else:
        np_ = _arg(w, "n", n, torch.bfloat16, q.full, d)
    stats = torch.empty(q.stats, dtype=torch.float32, device=dev)
    st = lib().moe_block_norm_fwd(ctypes.byref(cfg), *p, hp, np_, stats.data_ptr(), _stream(d))
    if st:
        _check(st, "moe_block_norm_fwd")
    return h, n, stats


def alloc_norm_grads(cfg, device="cuda"):
    q, f32 = _norm_plan(cfg), torch.float32
    g = {"dy": torch.empty(q.full, dtype=torch.bfloat16, device=device)}
    if q.residual:
        g["dresidual"] = torch.empty(q.full, dtype=q.stream, device=device)
    if q.post:
        g["dpost"] = torch.empty(q.vec, dtype=f32, device=device)
    if q.gate:
        g["dgate"] = torch.empty(q.gate, dtype=f32, device=device)
    if q.pre:
        g["dpre"] = torch.empty(q.vec, dtype=f32, device=device)
    return g


def block_norm_bwd(cfg, dn, y, stats, dh=None, residual=None, post_weight=None, gate=None, pre_weight=None, ws=None,
                   grads=None):
    """Gradients of block_norm_fwd from those of n (dn [T, H], bf16, fp32 with
    cfg.out_fp32; None without pre) and of h (dh as residual; None: zeros): dict with
    dy [T, H] bf16 and, where cfg has them, dresidual, dpost, dgate, dpre."""
    w = "block_norm_bwd"
    q = _norm_plan(cfg)
    f32 = torch.float32
    d, p = _norm_args(w, q, y, residual, post_weight, gate, pre_weight)
    dhp = _arg(w, "dh", dh, q.stream, q.full, d, optional=True)
    dnp = _arg(w, "dn", dn, q.io, q.full, d) if q.pre else None
    sp = _arg(w, "stats", stats, f32, q.stats, d)
    ws = _scratch(q.nbytes, y.device) if ws is None else ws
    wp = _ws_arg(w, ws, q.nbytes, d)
    if grads is None:
        g = alloc_norm_grads(cfg, y.device)
        out = lambda name, on, dt, shape: g[name].data_ptr() if on else None
    else:
        g = grads
        out = lambda name, on, dt, shape: _arg(w, name, g.get(name), dt, shape, d) if on else None
    st = lib().moe_block_norm_bwd(ctypes.byref(cfg), dhp, dnp, *p, sp, out("dy", True, torch.bfloat16, q.full),
                                  out("dresidual", q.residual, q.stream, q.full), out("dpost", q.post, f32, q.vec),
                                  out("dgate", q.gate, f32, q.gate), out("dpre", q.pre, f32, q.vec), wp, ws.numel(),
                                  _stream(d))
    _check(st, "moe_block_norm_bwd")
    return g
