"""Thin Python binding of libmoe (include/moe.h).

Argument marshalling only: torch CUDA tensors are checked for device, dtype
and contiguity and passed as plain pointers together with the current CUDA
stream. Every step of the layer runs in the library's kernels; there is no
fallback path. The library is loaded on first use and must exist (build it
with ``mixture_experts_ffn_fp32_gb300.build.build()``).
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from dataclasses import dataclass

import torch

from . import build as _build

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, \
    MOE_ERR_TIMEOUT, MOE_ERR_DEVICE_INDEX = range(7)
MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
GATES = {"softmax_topk": 0, "softmax_all_renorm": 1, "sigmoid": 2}

HEADER = os.path.join(_build.ROOT, "include", "moe.h")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class Config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("E", ctypes.c_int32), ("K", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("shared_d_ff", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("routed_scale", ctypes.c_float),
                ("out_dtype", ctypes.c_int32), ("save_gate_up", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("W_router", "bias", "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down",
                 "W_down_latent", "W_up_latent")]


GRAD_NAMES = ("dx", "dW_router", "dW_gate", "dW_up", "dW_down", "dWs_gate", "dWs_up",
              "dWs_down", "dW_down_latent", "dW_up_latent")


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in GRAD_NAMES]


class Views(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "margin", "top_scores", "scores", "counts", "offsets",
                 "sorted_token", "sorted_w", "inv")]


class GroupRouteConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "E", "K", "n_groups", "topk_groups", "group_rank", "score", "renormalize")] + \
        [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class Int8Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "Ma", "K", "N", "E", "swiglu", "out_dtype")]


class BlockNormConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "d", "dtype", "kind", "post", "gate")] + \
        [("alpha", ctypes.c_float), ("eps", ctypes.c_float)]


class AdapterConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "N", "r", "E", "dtype", "out_dtype")]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe. Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"libmoe.so is not built ({path}); run "
                               "mixture_experts_ffn_fp32_gb300.build.build() first")
        L = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        cfgp = ctypes.POINTER(Config)
        sigs = {
            "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "moe_version": (ctypes.c_char_p, []),
            "moe_workspace_size": (ctypes.c_int, [cfgp, ctypes.POINTER(sz)]),
            "moe_get_workspace_views": (ctypes.c_int, [cfgp, vp, ctypes.POINTER(Views)]),
            "moe_route": (ctypes.c_int, [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_dispatch": (ctypes.c_int, [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_dispatch_noalloc": (ctypes.c_int, [cfgp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "moe_forward": (ctypes.c_int, [cfgp, vp, ctypes.POINTER(Weights), vp, vp, sz, vp]),
            "moe_forward_host": (ctypes.c_int, [cfgp, vp, ctypes.POINTER(Weights), vp, vp, sz, vp]),
            "moe_quantile_bias_update": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, sz, vp]),
            "moe_quantile_workspace_size": (sz, [i32, i32]),
            "moe_sign_bias_update": (ctypes.c_int, [i32, i32, i32, vp, vp, ctypes.c_float, vp]),
            "moe_routing_stats": (ctypes.c_int, [cfgp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_workspace_status": (ctypes.c_int, [vp, vp]),
            "moe_backward_workspace_size": (ctypes.c_int, [cfgp, ctypes.POINTER(sz)]),
            "moe_backward": (ctypes.c_int, [cfgp, vp, ctypes.POINTER(Weights), vp,
                                            ctypes.POINTER(Grads), vp, sz, vp, sz, vp]),
            "moe_layer_norm": (ctypes.c_int, [i32, i32, i32, vp, i64, vp, vp, ctypes.c_float, vp, i64,
                                              vp, vp, vp]),
            "moe_layer_norm_backward_workspace_size": (ctypes.c_int, [i32, i32, ctypes.POINTER(sz)]),
            "moe_layer_norm_backward": (ctypes.c_int, [i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, vp,
                                                       i64, vp, vp, vp, sz, vp]),
            "moe_group_route": (ctypes.c_int, [ctypes.POINTER(GroupRouteConfig), vp, i64, vp, vp, vp,
                                               vp]),
            "moe_group_route_backward": (ctypes.c_int, [ctypes.POINTER(GroupRouteConfig), vp, i64, vp,
                                                        vp, vp, vp]),
            "moe_quantize_rows": (ctypes.c_int, [i32, i32, i32, vp, i64, vp, vp, vp]),
            "moe_matmul_int8_workspace_size": (ctypes.c_int, [ctypes.POINTER(Int8Config),
                                                              ctypes.POINTER(sz)]),
            "moe_matmul_int8": (ctypes.c_int, [ctypes.POINTER(Int8Config), vp, i64, vp, vp, vp, vp, vp,
                                               vp, vp, sz, vp]),
            "moe_block_norm": (ctypes.c_int, [ctypes.POINTER(BlockNormConfig), vp, i64, vp, i64, vp, i64, vp, vp,
                                              vp, vp, vp, vp, vp, vp]),
            "moe_block_norm_backward_workspace_size": (ctypes.c_int, [ctypes.POINTER(BlockNormConfig),
                                                                      ctypes.POINTER(sz)]),
            "moe_block_norm_backward": (ctypes.c_int, [ctypes.POINTER(BlockNormConfig), vp, i64, vp, i64, vp, i64,
                                                       vp, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp,
                                                       vp, vp, sz, vp]),
            "moe_adapter_add_workspace_size": (ctypes.c_int, [ctypes.POINTER(AdapterConfig),
                                                              ctypes.POINTER(sz)]),
            "moe_adapter_add": (ctypes.c_int, [ctypes.POINTER(AdapterConfig), vp, i64, vp, vp, vp, vp, vp, vp,
                                               i64, vp, i64, vp, sz, vp]),
            "moe_timing_begin": (ctypes.c_int, [i32, ctypes.c_uint32]),
            "moe_timing_end": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), i32,
                                              ctypes.POINTER(i32), ctypes.POINTER(i32)]),
            "moe_stage_name": (ctypes.c_char_p, [i32]),
            "moe_launch_count": (ctypes.c_uint64, []),
            "moe_set_wait_timeout_ms": (ctypes.c_int, [i32]),
            "moe_selftest_wait_timeout": (ctypes.c_int, [i32, vp, vp]),
        }
        for name, (res, args) in sigs.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/moe.h declares."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\**\s*(moe_[a-z0-9_]+)\s*\(",
                                 src, flags=re.M)))


def status_string(s: int) -> str:
    return lib().moe_status_string(int(s)).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


@dataclass(frozen=True)
class LayerSpec:
    T: int
    d: int
    d_ff: int
    E: int
    K: int
    n_shared: int = 0
    shared_d_ff: int = 0
    latent_dim: int = 0
    dtype: str = "bf16"
    gate: str = "softmax_topk"
    renormalize: bool = False
    routed_scale: float = 1.0
    out_dtype: str = "f32"
    save_gate_up: bool = False  # forward keeps the gate/up products for the backward

    @staticmethod
    def of(w, out_dtype: str = "f32", save_gate_up: bool = False) -> "LayerSpec":
        """From any object with the Workload attribute names."""
        return LayerSpec(w.T, w.d, w.d_ff, w.E, w.K, w.n_shared, w.shared_d_ff, w.latent_dim,
                         w.dtype, w.gate, bool(w.renormalize), float(w.routed_scale), out_dtype,
                         bool(save_gate_up))

    def config(self) -> Config:
        return Config(self.T, self.d, self.d_ff, self.E, self.K, self.n_shared,
                      self.shared_d_ff if self.n_shared else 0, self.latent_dim,
                      MOE_F32 if self.dtype == "f32" else MOE_BF16, GATES[self.gate],
                      int(self.renormalize), float(self.routed_scale),
                      MOE_F32 if self.out_dtype == "f32" else MOE_BF16, int(self.save_gate_up))

    @property
    def torch_dtype(self):
        return torch.float32 if self.dtype == "f32" else torch.bfloat16

    @property
    def torch_out_dtype(self):
        return torch.float32 if self.out_dtype == "f32" else torch.bfloat16


def workspace_size(spec: LayerSpec) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(spec.config()), ctypes.byref(n)),
           "moe_workspace_size")
    return n.value


def alloc_workspace(spec: LayerSpec, device="cuda") -> torch.Tensor:
    return torch.empty(workspace_size(spec), dtype=torch.uint8, device=device)


def _dev(t, dtype, name, shape=None, here=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if here is not None:
        _at(t, name, here)
    elif not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def weights_struct(spec: LayerSpec, p: dict) -> Weights:
    dt = spec.torch_dtype
    de = spec.latent_dim or spec.d
    S, Fs = spec.n_shared, spec.shared_d_ff
    w = Weights()
    w.W_router = _dev(p["W_router"], torch.float32, "W_router", (spec.d, spec.E)).data_ptr()
    b = p.get("bias")
    w.bias = None if b is None else _dev(b, torch.float32, "bias", (spec.E,)).data_ptr()
    w.W_gate = _dev(p["W_gate"], dt, "W_gate", (spec.E, de, spec.d_ff)).data_ptr()
    w.W_up = _dev(p["W_up"], dt, "W_up", (spec.E, de, spec.d_ff)).data_ptr()
    w.W_down = _dev(p["W_down"], dt, "W_down", (spec.E, spec.d_ff, de)).data_ptr()
    if S:
        w.Ws_gate = _dev(p["Ws_gate"], dt, "Ws_gate", (S, spec.d, Fs)).data_ptr()
        w.Ws_up = _dev(p["Ws_up"], dt, "Ws_up", (S, spec.d, Fs)).data_ptr()
        w.Ws_down = _dev(p["Ws_down"], dt, "Ws_down", (S, Fs, spec.d)).data_ptr()
    if spec.latent_dim:
        w.W_down_latent = _dev(p["W_down_latent"], dt, "W_down_latent",
                               (spec.d, spec.latent_dim)).data_ptr()
        w.W_up_latent = _dev(p["W_up_latent"], dt, "W_up_latent",
                             (spec.latent_dim, spec.d)).data_ptr()
    return w


def route(spec: LayerSpec, x: torch.Tensor, W_router: torch.Tensor, bias=None, stream=None,
          ws: torch.Tensor | None = None):
    """moe_route: returns dict idx [T,K] int32, w [T,K], margin [T] (+ top_scores
    [T,K+1] and scores [T,E] in sigmoid mode). With a workspace the tensor-core
    router is used where the layer allows it (as in forward)."""
    dev = x.device
    _dev(x, spec.torch_dtype, "x", (spec.T, spec.d))
    _dev(W_router, torch.float32, "W_router", (spec.d, spec.E))
    if bias is not None:
        _dev(bias, torch.float32, "bias", (spec.E,))
    out = {
        "idx": torch.empty((spec.T, spec.K), dtype=torch.int32, device=dev),
        "w": torch.empty((spec.T, spec.K), dtype=torch.float32, device=dev),
        "margin": torch.empty((spec.T,), dtype=torch.float32, device=dev),
    }
    sig = spec.gate == "sigmoid"
    if sig:
        out["top_scores"] = torch.empty((spec.T, spec.K + 1), dtype=torch.float32, device=dev)
        out["scores"] = torch.empty((spec.T, spec.E), dtype=torch.float32, device=dev)
    _check(lib().moe_route(ctypes.byref(spec.config()), x.data_ptr(), W_router.data_ptr(),
                           _ptr(bias), out["idx"].data_ptr(), out["w"].data_ptr(),
                           out["margin"].data_ptr(), _ptr(out.get("top_scores")),
                           _ptr(out.get("scores")), _ptr(ws), 0 if ws is None else ws.numel(),
                           _stream(stream)), "moe_route")
    return out


def dispatch(spec: LayerSpec, idx: torch.Tensor, w: torch.Tensor, ws: torch.Tensor | None = None,
             stream=None):
    """moe_dispatch: returns dict counts, offsets, sorted_token, sorted_w, inv."""
    dev = idx.device
    _dev(idx, torch.int32, "topk_idx", (spec.T, spec.K))
    _dev(w, torch.float32, "topk_w", (spec.T, spec.K))
    ws = alloc_workspace(spec, dev) if ws is None else ws
    TK = spec.T * spec.K
    out = {
        "counts": torch.empty((spec.E,), dtype=torch.int32, device=dev),
        "offsets": torch.empty((spec.E + 1,), dtype=torch.int32, device=dev),
        "sorted_token": torch.empty((TK,), dtype=torch.int32, device=dev),
        "sorted_w": torch.empty((TK,), dtype=torch.float32, device=dev),
        "inv": torch.empty((spec.T, spec.K), dtype=torch.int32, device=dev),
    }
    _check(lib().moe_dispatch(ctypes.byref(spec.config()), idx.data_ptr(), w.data_ptr(),
                              out["counts"].data_ptr(), out["offsets"].data_ptr(),
                              out["sorted_token"].data_ptr(), out["sorted_w"].data_ptr(),
                              out["inv"].data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
           "moe_dispatch")
    out["ws"] = ws
    return out


def dispatch_noalloc(spec: LayerSpec, idx: torch.Tensor, w: torch.Tensor, out: dict | None = None,
                     stream=None):
    """moe_dispatch_noalloc: moe_dispatch without a workspace, for callers that
    cannot allocate device memory (the library keeps the scratch in a fixed
    device array; T*K <= 65536, E <= 256). ``out`` may hold preallocated
    counts, offsets, sorted_token, sorted_w and inv tensors."""
    dev = idx.device
    _dev(idx, torch.int32, "topk_idx", (spec.T, spec.K))
    _dev(w, torch.float32, "topk_w", (spec.T, spec.K))
    TK = spec.T * spec.K
    if out is None:
        out = {
            "counts": torch.empty((spec.E,), dtype=torch.int32, device=dev),
            "offsets": torch.empty((spec.E + 1,), dtype=torch.int32, device=dev),
            "sorted_token": torch.empty((TK,), dtype=torch.int32, device=dev),
            "sorted_w": torch.empty((TK,), dtype=torch.float32, device=dev),
            "inv": torch.empty((spec.T, spec.K), dtype=torch.int32, device=dev),
        }
    _check(lib().moe_dispatch_noalloc(ctypes.byref(spec.config()), idx.data_ptr(), w.data_ptr(),
                                      out["counts"].data_ptr(), out["offsets"].data_ptr(),
                                      out["sorted_token"].data_ptr(), out["sorted_w"].data_ptr(),
                                      out["inv"].data_ptr(), _stream(stream)),
           "moe_dispatch_noalloc")
    return out


def forward(spec: LayerSpec, x: torch.Tensor, params: dict, out: torch.Tensor | None = None,
            ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """moe_forward: the whole layer on device tensors."""
    _dev(x, spec.torch_dtype, "x", (spec.T, spec.d))
    ws = alloc_workspace(spec, x.device) if ws is None else ws
    if out is None:
        out = torch.empty((spec.T, spec.d), dtype=spec.torch_out_dtype, device=x.device)
    _dev(out, spec.torch_out_dtype, "out", (spec.T, spec.d))
    w = weights_struct(spec, params)
    _check(lib().moe_forward(ctypes.byref(spec.config()), x.data_ptr(), ctypes.byref(w),
                             out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
           "moe_forward")
    return out


def backward_workspace_size(spec: LayerSpec) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_backward_workspace_size(ctypes.byref(spec.config()), ctypes.byref(n)),
           "moe_backward_workspace_size")
    return int(n.value)


def grad_shapes(spec: LayerSpec) -> dict:
    de = spec.latent_dim or spec.d
    S, Fs, L = spec.n_shared, spec.shared_d_ff, spec.latent_dim
    sh = {"dx": (spec.T, spec.d), "dW_router": (spec.d, spec.E),
          "dW_gate": (spec.E, de, spec.d_ff), "dW_up": (spec.E, de, spec.d_ff),
          "dW_down": (spec.E, spec.d_ff, de)}
    if S:
        sh.update(dWs_gate=(S, spec.d, Fs), dWs_up=(S, spec.d, Fs), dWs_down=(S, Fs, spec.d))
    if L:
        sh.update(dW_down_latent=(spec.d, L), dW_up_latent=(L, spec.d))
    return sh


def backward(spec: LayerSpec, x: torch.Tensor, params: dict, dout: torch.Tensor, ws: torch.Tensor,
             grads: dict | None = None, bws: torch.Tensor | None = None, stream=None) -> dict:
    """moe_backward after a moe_forward on ws: FP32 gradients of sum(dout * out).
    ``grads`` maps names of GRAD_NAMES to preallocated FP32 tensors (absent
    names are allocated, zero-filled: an expert slice that gets no gradient
    stays as given); a name mapped to None is not computed."""
    _dev(x, spec.torch_dtype, "x", (spec.T, spec.d))
    _dev(dout, torch.float32, "dout", (spec.T, spec.d))
    shapes = grad_shapes(spec)
    out = {}
    given = grads or {}
    for n, shp in shapes.items():
        if n in given:
            if given[n] is not None:
                out[n] = _dev(given[n], torch.float32, n, shp)
        else:
            out[n] = torch.zeros(shp, dtype=torch.float32, device=x.device)
    if "dx" not in out:
        raise ValueError("dx is required")
    g = Grads()
    for n in GRAD_NAMES:
        setattr(g, n, out[n].data_ptr() if n in out else None)
    if bws is None:
        bws = torch.empty(backward_workspace_size(spec), dtype=torch.uint8, device=x.device)
    w = weights_struct(spec, params)
    _check(lib().moe_backward(ctypes.byref(spec.config()), x.data_ptr(), ctypes.byref(w),
                              dout.data_ptr(), ctypes.byref(g), ws.data_ptr(), ws.numel(),
                              bws.data_ptr(), bws.numel(), _stream(stream)),
           "moe_backward")
    return out


def forward_host(spec: LayerSpec, x_host: torch.Tensor, params: dict, out_host: torch.Tensor,
                 ws: torch.Tensor, stream=None) -> torch.Tensor:
    """moe_forward_host: host x / out (pinned for asynchronous DMA); synchronises."""
    for n, t, dt in (("x_host", x_host, spec.torch_dtype), ("out_host", out_host, spec.torch_out_dtype)):
        if t.is_cuda or not t.is_contiguous() or t.dtype != dt or t.numel() != spec.T * spec.d:
            raise ValueError(f"{n} must be a contiguous host tensor of {dt} with T*d elements")
    w = weights_struct(spec, params)
    _check(lib().moe_forward_host(ctypes.byref(spec.config()), x_host.data_ptr(), ctypes.byref(w),
                                  out_host.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
           "moe_forward_host")
    return out_host


def workspace_views(spec: LayerSpec, ws: torch.Tensor) -> dict:
    """Torch views of the routing/dispatch results a forward left in ws."""
    v = Views()
    _check(lib().moe_get_workspace_views(ctypes.byref(spec.config()), ws.data_ptr(), ctypes.byref(v)),
           "moe_get_workspace_views")
    base = ws.data_ptr()
    T, K, E = spec.T, spec.K, spec.E

    def view(ptr, n, dtype, shape):
        if ptr is None:
            return None
        off = ptr - base
        esz = torch.tensor([], dtype=dtype).element_size()
        return ws[off: off + n * esz].view(dtype).view(*shape)

    i32, f32 = torch.int32, torch.float32
    return {
        "idx": view(v.topk_idx, T * K, i32, (T, K)),
        "w": view(v.topk_w, T * K, f32, (T, K)),
        "margin": view(v.margin, T, f32, (T,)),
        "top_scores": view(v.top_scores, T * (K + 1), f32, (T, K + 1)),
        "scores": view(v.scores, T * E, f32, (T, E)),
        "counts": view(v.counts, E, i32, (E,)),
        "offsets": view(v.offsets, E + 1, i32, (E + 1,)),
        "sorted_token": view(v.sorted_token, T * K, i32, (T * K,)),
        "sorted_w": view(v.sorted_w, T * K, f32, (T * K,)),
        "inv": view(v.inv, T * K, i32, (T, K)),
    }


def quantile_bias_update(top_scores: torch.Tensor, scores: torch.Tensor, K: int, bias: torch.Tensor,
                         ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """moe_quantile_bias_update: replaces bias [E] in place and returns it."""
    T, E = scores.shape
    _dev(top_scores, torch.float32, "top_scores", (T, K + 1))
    _dev(scores, torch.float32, "scores", (T, E))
    _dev(bias, torch.float32, "bias", (E,))
    n = lib().moe_quantile_workspace_size(T, E)
    ws = torch.empty(n, dtype=torch.uint8, device=scores.device) if ws is None else ws
    _check(lib().moe_quantile_bias_update(T, E, K, top_scores.data_ptr(), scores.data_ptr(),
                                          bias.data_ptr(), ws.data_ptr(), ws.numel(),
                                          _stream(stream)), "moe_quantile_bias_update")
    return bias


def routing_stats(spec: LayerSpec, x: torch.Tensor, W_router: torch.Tensor, bias=None,
                  ws: torch.Tensor | None = None, stream=None, read: bool = True) -> dict:
    """Switch load-balancing loss (before alpha), router z-loss (before its
    weight) and mean router probabilities of one batch (moe_routing_stats).
    Returns dict(out [2+E] device tensor, ws) and, with read=True (waits for
    the stream), aux, z and P [E] on the host."""
    ws = alloc_workspace(spec, x.device) if ws is None else ws
    out = torch.empty(2 + spec.E, dtype=torch.float32, device=x.device)
    _check(lib().moe_routing_stats(ctypes.byref(spec.config()), _ptr(x), _ptr(W_router),
                                   _ptr(bias), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_routing_stats")
    res = {"out": out, "ws": ws}
    if read:
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()
        vals = out.cpu()
        res.update(aux=float(vals[0]), z=float(vals[1]), P=vals[2:])
    return res


def sign_bias_update(counts: torch.Tensor, N: int, K: int, bias: torch.Tensor, alpha: float,
                     stream=None) -> torch.Tensor:
    E = counts.shape[0]
    _dev(counts, torch.int32, "counts", (E,))
    _dev(bias, torch.float32, "bias", (E,))
    _check(lib().moe_sign_bias_update(E, N, K, counts.data_ptr(), bias.data_ptr(), float(alpha),
                                      _stream(stream)), "moe_sign_bias_update")
    return bias


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises and returns (and clears) the workspace's device error status."""
    return lib().moe_workspace_status(ws.data_ptr(), _stream(stream))


# ---------------------------------------------------------------------------
# Operators around the layer
# ---------------------------------------------------------------------------

_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}
_OUT_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SCORES = {"sigmoid": 0, "softmax": 1}


def _internal(path, public):
    """A binding that torch's own generated code uses, or, in a torch without it, the
    public function that does the same at more host time."""
    f = torch._C
    for name in path.split("."):
        f = getattr(f, name, None)
    return public if f is None else f


# An uninitialised CUDA tensor of the current device: a third less host time than
# torch.empty, of which a call has three. torch.cuda.current_stream() takes several
# microseconds, as long as a small kernel.
_empty_strided = _internal("_dynamo.guards._empty_strided_cuda",
                           lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype, device="cuda"))
_current_device = _internal("_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = _internal("_cuda_getCurrentRawStream",
                                lambda device: torch.cuda.current_stream(device).cuda_stream)


def _here(stream) -> int:
    """The device a call runs on: the current one, or the given stream's. Its outputs
    will be there, its kernels launch there, and its tensors have to be there."""
    return _current_device() if stream is None else stream.device_index


def _at(t, name, here):
    if t.get_device() != here:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{here}")


def _scratch(ws, here):
    """A caller's workspace: its elements are its memory, so that their number bounds it."""
    _at(ws, "ws", here)
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")


def _rows(t, name, dtype=None, shape=None):
    """A [rows, n] CUDA tensor with contiguous rows at any pitch; returns its pitch."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    have = t.shape
    if len(have) != 2 or have[1] < 1:
        raise ValueError(f"{name} must be a [rows, n] tensor with n >= 1, got {tuple(have)}")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype or 'float32, bfloat16 or float16'}, got {t.dtype}")
    if shape is not None and have != shape:
        raise ValueError(f"{name} has shape {tuple(have)}, expected {tuple(shape)}")
    R, n = have
    pitch, inner = t.stride()
    if inner != 1 and n > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if R <= 1:
        return n
    if pitch < n:
        raise ValueError(f"{name}'s rows must not overlap")
    return pitch


def _empty(dtype, n, m=None):
    return _empty_strided((n,), (1,), dtype) if m is None else _empty_strided((n, m), (max(m, 1), 1), dtype)


class _On:
    """Outputs and scratch of a call belong to the stream it runs on, and its
    inputs stay allocated until that stream is done with them, whichever
    stream they were made on."""

    def __init__(self, stream, *inputs):
        self.stream, self.inputs = stream, inputs

    def __enter__(self):
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)
        for t in self.inputs:
            if t is not None:
                t.record_stream(self.stream)


class _Here:
    """_On for the current stream: nothing to arrange."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Here()


def _on(stream, *inputs):
    return _HERE if stream is None else _On(stream, *inputs)


def _raw_stream(stream, here) -> int:
    """The stream's handle, else that of the device's current stream."""
    return _current_raw_stream(here) if stream is None else stream.cuda_stream


def layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5, stream=None) -> dict:
    """moe_layer_norm: x [R, d] (FP32, BF16 or FP16; rows at any pitch), weight and
    bias [d] FP32 or None. Returns y [R, d] in x's type and the FP32 statistics
    mean and rstd [R] that the backward takes."""
    xs = _rows(x, "x")
    here = _here(stream)
    _at(x, "x", here)
    R, d = x.shape
    if weight is not None:
        _dev(weight, torch.float32, "weight", (d,), here)
    if bias is not None:
        _dev(bias, torch.float32, "bias", (d,), here)
    with _on(stream, x, weight, bias):
        y = _empty(x.dtype, R, d)
        mean = _empty(torch.float32, R)
        rstd = _empty(torch.float32, R)
        _check(lib().moe_layer_norm(R, d, _DTYPES[x.dtype], x.data_ptr(), xs, _ptr(weight), _ptr(bias), eps,
                                    y.data_ptr(), d, mean.data_ptr(), rstd.data_ptr(), _raw_stream(stream, here)),
               "moe_layer_norm")
    return {"y": y, "mean": mean, "rstd": rstd}


@functools.lru_cache(maxsize=4096)
def layer_norm_backward_workspace_size(R: int, d: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layer_norm_backward_workspace_size(R, d, ctypes.byref(n)),
           "moe_layer_norm_backward_workspace_size")
    return n.value


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight=None, weight_grads: bool = True, ws: torch.Tensor | None = None,
                        stream=None) -> dict:
    """moe_layer_norm_backward: dx [R, d] in x's type and, with weight_grads,
    dweight and dbias [d] FP32, given layer_norm's mean and rstd. ws: uint8 of
    layer_norm_backward_workspace_size(R, d) bytes (allocated when None)."""
    xs = _rows(x, "x")
    here = _here(stream)
    _at(x, "x", here)
    R, d = x.shape
    dys = _rows(dy, "dy", x.dtype, x.shape)
    _at(dy, "dy", here)
    _dev(mean, torch.float32, "mean", (R,), here)
    _dev(rstd, torch.float32, "rstd", (R,), here)
    if weight is not None:
        _dev(weight, torch.float32, "weight", (d,), here)
    if ws is not None:
        _scratch(ws, here)
    with _on(stream, dy, x, mean, rstd, weight, ws):
        out = {"dx": _empty(x.dtype, R, d)}
        if weight_grads:
            out["dweight"] = _empty(torch.float32, d)
            out["dbias"] = _empty(torch.float32, d)
            if ws is None:
                ws = _empty(torch.uint8, layer_norm_backward_workspace_size(R, d))
        _check(lib().moe_layer_norm_backward(R, d, _DTYPES[x.dtype], dy.data_ptr(), dys, x.data_ptr(), xs,
                                             mean.data_ptr(), rstd.data_ptr(), _ptr(weight),
                                             out["dx"].data_ptr(), d, _ptr(out.get("dweight")),
                                             _ptr(out.get("dbias")), _ptr(ws), 0 if ws is None else ws.numel(),
                                             _raw_stream(stream, here)), "moe_layer_norm_backward")
    return out


@functools.lru_cache(maxsize=4096)
def _struct(kind, *fields):
    """A reference to a config that the library only reads (building one takes as
    long as a small kernel)."""
    return ctypes.byref(kind(*fields))


def _group_config(logits, K, n_groups, topk_groups, group_rank, score, renormalize, scale):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    T, E = logits.shape
    return _struct(GroupRouteConfig, T, E, K, n_groups, topk_groups, group_rank, SCORES[score],
                   1 if renormalize else 0, float(scale), _DTYPES[logits.dtype])


def group_route(logits: torch.Tensor, K: int, n_groups: int = 1, topk_groups: int = 1, bias=None,
                score: str = "sigmoid", group_rank: int = 2, renormalize: bool = True, scale: float = 1.0,
                stream=None) -> dict:
    """moe_group_route: group-limited top-K routing of logits [T, E] (FP32, BF16 or
    FP16; rows at any pitch). bias [E] FP32 enters the choice, not the weights;
    group_rank 1 ranks groups by their best choice, 2 by the sum of their two
    best. Experts whose logit is -inf are never taken; slots that stay empty
    hold id -1, weight 0. Returns idx [T, K] int32 and w [T, K] FP32."""
    ls = _rows(logits, "logits")
    here = _here(stream)
    _at(logits, "logits", here)
    T, E = logits.shape
    if bias is not None:
        _dev(bias, torch.float32, "bias", (E,), here)
    cfg = _group_config(logits, K, n_groups, topk_groups, group_rank, score, renormalize, scale)
    with _on(stream, logits, bias):
        out = {"idx": _empty(torch.int32, T, max(K, 0)),
               "w": _empty(torch.float32, T, max(K, 0))}
        _check(lib().moe_group_route(cfg, logits.data_ptr(), ls, _ptr(bias), out["idx"].data_ptr(),
                                     out["w"].data_ptr(), _raw_stream(stream, here)), "moe_group_route")
    return out


def group_route_backward(dw: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, score: str = "sigmoid",
                         renormalize: bool = True, scale: float = 1.0, stream=None) -> torch.Tensor:
    """moe_group_route_backward: the gradient with respect to the logits (their
    type) of sum(dw * w), the selection idx held fixed."""
    ls = _rows(logits, "logits")
    here = _here(stream)
    _at(logits, "logits", here)
    T, E = logits.shape
    if idx.dim() != 2:
        raise ValueError(f"idx must be [T, K], got {tuple(idx.shape)}")
    K = idx.size(1)
    _dev(idx, torch.int32, "idx", (T, K), here)
    _dev(dw, torch.float32, "dw", (T, K), here)
    cfg = _group_config(logits, K, 1, 1, 1, score, renormalize, scale)
    with _on(stream, dw, idx, logits):
        out = _empty(logits.dtype, T, E)
        _check(lib().moe_group_route_backward(cfg, logits.data_ptr(), ls, idx.data_ptr(),
                                              dw.data_ptr(), out.data_ptr(), _raw_stream(stream, here)),
               "moe_group_route_backward")
    return out


def quantize_rows(x: torch.Tensor, stream=None) -> dict:
    """moe_quantize_rows: x [R, K] (FP32, BF16 or FP16; rows at any pitch) to q
    [R, K] int8 and scale [R] FP32 with x ~ q * scale. Weights [E, K, N] are laid
    out for matmul_int8 by quantising the rows of their transpose:
    ``quantize_rows(W.transpose(1, 2).reshape(E * N, K))``."""
    xs = _rows(x, "x")
    here = _here(stream)
    _at(x, "x", here)
    R, K = x.shape
    with _on(stream, x):
        out = {"q": _empty(torch.int8, R, K),
               "scale": _empty(torch.float32, R)}
        _check(lib().moe_quantize_rows(R, K, _DTYPES[x.dtype], x.data_ptr(), xs, out["q"].data_ptr(),
                                       out["scale"].data_ptr(), _raw_stream(stream, here)), "moe_quantize_rows")
    return out


def _int8_config(M, Ma, K, N, E, swiglu, out_dtype) -> tuple:
    """The fields of an Int8Config."""
    if out_dtype not in _OUT_DTYPES:
        raise ValueError(f"out_dtype must be one of {sorted(_OUT_DTYPES)}, got {out_dtype!r}")
    return M, Ma, K, N, E, 1 if swiglu else 0, _DTYPES[_OUT_DTYPES[out_dtype]]


@functools.lru_cache(maxsize=4096)
def _int8_ws(*shape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_matmul_int8_workspace_size(_struct(Int8Config, *shape), ctypes.byref(n)),
           "moe_matmul_int8_workspace_size")
    return n.value


def alloc_int8_workspace(M: int, K: int, N: int, E: int = 1, swiglu: bool = False,
                         device="cuda") -> torch.Tensor:
    """A workspace for matmul_int8 calls of up to M product rows (its error word
    zeroed; workspace_status reads and clears it)."""
    n = _int8_ws(*_int8_config(M, M, K, N, E, swiglu, "f32"))
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def matmul_int8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, offsets=None,
                rows=None, swiglu: bool = False, out_dtype: str = "bf16", ws: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """moe_matmul_int8: 8-bit products grouped by expert. a [Ma, K] int8 and a_scale
    [Ma] (quantize_rows), b [E, N, K] int8 and b_scale [E, N]; offsets [E + 1]
    and rows [M] int32 as dispatch's offsets and sorted_token (None: one expert
    takes every row; rows of a in order). With swiglu the channels of an
    expert are its gates, then its ups, and the output is SiLU(gate) * up.
    Returns out [M, N] ([M, N / 2] with swiglu). ws: see alloc_int8_workspace. When
    None one is allocated for the call and its error word is not read: a bad row
    index, or a device wait that ran out, then shows by the NaNs it leaves alone."""
    if a.dim() != 2 or b.dim() != 3 or not a.is_cuda or a.dtype != torch.int8:
        raise ValueError("a must be a [Ma, K] int8 CUDA tensor and b [E, N, K]")
    E, N, K = b.shape
    Ma = a.size(0)
    if a.size(1) != K or (K > 1 and a.stride(1) != 1):
        raise ValueError(f"a must have contiguous rows of {K} elements, got {tuple(a.shape)}")
    here = _here(stream)
    _at(a, "a", here)
    _dev(b, torch.int8, "b", None, here)
    _dev(a_scale, torch.float32, "a_scale", (Ma,), here)
    _dev(b_scale, torch.float32, "b_scale", (E, N), here)
    if offsets is not None:
        _dev(offsets, torch.int32, "offsets", (E + 1,), here)
    M = Ma
    if rows is not None:
        if rows.dim() != 1:
            raise ValueError(f"rows must be [M], got {tuple(rows.shape)}")
        _dev(rows, torch.int32, "rows", None, here)
        M = rows.size(0)
    cfg = _int8_config(M, Ma, K, N, E, swiglu, out_dtype)
    if ws is not None:
        _scratch(ws, here)
    with _on(stream, a, a_scale, b, b_scale, offsets, rows, ws):
        if ws is None:
            ws = _empty(torch.uint8, _int8_ws(*cfg))
        out = _empty(_OUT_DTYPES[out_dtype], M, N // 2 if swiglu else N)
        _check(lib().moe_matmul_int8(_struct(Int8Config, *cfg), a.data_ptr(), a.stride(0) if Ma > 1 else K,
                                     a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), _ptr(offsets),
                                     _ptr(rows), out.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
                                     _raw_stream(stream, here)), "moe_matmul_int8")
    return out


NORMS = {"layer": 0, "rms": 1}
_GATE_NONE, _GATE_CHANNEL, _GATE_ELEMENT = range(3)


def _vector(t, name, shape, here):
    """_dev of an FP32 parameter, in one expression where it fits (a call has up to five)."""
    if not (t.get_device() == here and t.dtype is torch.float32 and t.shape == shape and t.is_contiguous()):
        _dev(t, torch.float32, name, shape, here)
    return t.data_ptr()


def _like(t, name, dtype, shape, here):
    """_rows and _at of a tensor of x's type and shape; returns its address and pitch."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == here:
        pitch, inner = t.stride()
        if inner == 1 and pitch >= shape[1]:
            return t.data_ptr(), pitch
    pitch = _rows(t, name, dtype, shape)
    _at(t, name, here)
    return t.data_ptr(), pitch


def _block_norm_args(x, y, gate, post_weight, post_bias, kind, post, here):
    """What both directions check alike. Returns the number of post (0 or 1), the gate's
    shape, and the addresses and pitches of x, y, gate, post_weight and post_bias."""
    if kind not in NORMS:
        raise ValueError(f"kind must be one of {sorted(NORMS)}, got {kind!r}")
    xs = _rows(x, "x")
    _at(x, "x", here)
    shape, dtype = x.shape, x.dtype
    col = (shape[1],)
    yp = gp = pw = pb = None
    ys = gs = 0
    form = _GATE_NONE
    if y is None:
        if gate is not None:
            raise ValueError("a gate needs y")
        post = False
    else:
        yp, ys = _like(y, "y", dtype, shape, here)
        if gate is not None:
            if gate.dim() == 1:
                form = _GATE_CHANNEL
                gp = _vector(gate, "gate", col, here)
            else:
                form = _GATE_ELEMENT
                gp, gs = _like(gate, "gate", dtype, shape, here)
    if post_weight is not None:
        if not post:
            raise ValueError("post_weight and post_bias need a norm of y")
        pw = _vector(post_weight, "post_weight", col, here)
    if post_bias is not None:
        if not post:
            raise ValueError("post_weight and post_bias need a norm of y")
        if kind == "rms":
            raise ValueError("an RMS norm has no bias")
        pb = _vector(post_bias, "post_bias", col, here)
    return 1 if post else 0, form, (x.data_ptr(), xs, yp, ys, gp, gs, pw, pb)


def block_norm(x: torch.Tensor, y=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None,
               alpha: float = 1.0, kind: str = "rms", post: bool = True, norm: bool = True, eps: float = 1e-5,
               stats: bool = True, stream=None) -> dict:
    """moe_block_norm: the norms on both sides of a block, fused with its gate and
    the residual. x [R, d] the residual stream, y [R, d] the block's output (FP32,
    BF16 or FP16; rows at any pitch):

        z = Norm(y; post_weight, post_bias) (y itself with post=False)
        x' = alpha x + gate z,   n = Norm(x'; weight, bias)

    kind "rms" or "layer" (which alone takes biases); gate None, [d] FP32 or [R, d]
    in x's type; vectors [d] FP32 or None. Returns x (x'), n and, with stats, the
    FP32 statistics that the backward takes. y None: n = Norm(x) alone, no x.
    norm=False: no norm follows, no n."""
    here = _here(stream)
    post, form, args = _block_norm_args(x, y, gate, post_weight, post_bias, kind, post, here)
    R, d = x.shape
    dtype = x.dtype
    wp = bp = None
    if not norm:
        if y is None:
            raise ValueError("norm=False needs y")
        if weight is not None or bias is not None:
            raise ValueError("weight and bias need a norm")
    if weight is not None:
        wp = _vector(weight, "weight", (d,), here)
    if bias is not None:
        if kind == "rms":
            raise ValueError("an RMS norm has no bias")
        bp = _vector(bias, "bias", (d,), here)
    cfg = _struct(BlockNormConfig, R, d, _DTYPES[dtype], NORMS[kind], post, form, float(alpha), float(eps))
    out = {}
    xo = no = so = None
    with _on(stream, x, y, weight, bias, post_weight, post_bias, gate):
        if y is not None:
            out["x"] = t = _empty(dtype, R, d)
            xo = t.data_ptr()
        if norm:
            out["n"] = t = _empty(dtype, R, d)
            no = t.data_ptr()
        if stats:
            out["stats"] = t = _empty(torch.float32, 2 if kind == "rms" else 4, R)
            so = t.data_ptr()
        _check(lib().moe_block_norm(cfg, *args, wp, bp, xo, no, so, _raw_stream(stream, here)), "moe_block_norm")
    return out


@functools.lru_cache(maxsize=4096)
def block_norm_backward_workspace_size(R: int, d: int, kind: str = "rms") -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_block_norm_backward_workspace_size(
        _struct(BlockNormConfig, R, d, MOE_F32, NORMS[kind], 0, 0, 1.0, 0.0), ctypes.byref(n)),
        "moe_block_norm_backward_workspace_size")
    return n.value


def block_norm_backward(x: torch.Tensor, stats: torch.Tensor, y=None, dn=None, dx=None, weight=None,
                        post_weight=None, post_bias=None, gate=None, alpha: float = 1.0, kind: str = "rms",
                        post: bool = True, weight_grads: bool = True, ws: torch.Tensor | None = None,
                        stream=None) -> dict:
    """moe_block_norm_backward: gradients of sum(dn * n) + sum(dx * x'), either of dn
    and dx (rows at any pitch) None for none. x: the forward's result x' (its input x
    where y is None); stats, y, the gate and the vectors as in the forward. Returns dx
    and, with y, dy in x's type; of an element-wise gate dgate too; with weight_grads,
    FP32, dgate of a gate [d], dpost_weight where y is normalised, dweight with dn,
    and for layer norms dpost_bias and dbias. ws: uint8 of
    block_norm_backward_workspace_size(R, d, kind) bytes (allocated when None)."""
    here = _here(stream)
    post, form, args = _block_norm_args(x, y, gate, post_weight, post_bias, kind, post, here)
    shape, dtype = x.shape, x.dtype
    R, d = shape
    layer = kind == "layer"
    if dn is None and dx is None:
        raise ValueError("dn or dx is required")
    dnp = dxp = wp = None
    dns = dxs = 0
    if dn is not None:
        dnp, dns = _like(dn, "dn", dtype, shape, here)
    elif weight is not None:
        raise ValueError("weight needs dn")
    if dx is not None:
        dxp, dxs = _like(dx, "dx", dtype, shape, here)
    if stats is None:
        raise ValueError("stats is required")
    sp = _vector(stats, "stats", (4 if layer else 2, R), here)
    if weight is not None:
        wp = _vector(weight, "weight", (d,), here)
    if ws is not None:
        _scratch(ws, here)
    cfg = _struct(BlockNormConfig, R, d, _DTYPES[dtype], NORMS[kind], post, form, float(alpha), 0.0)
    yo = go = None
    vectors = [None] * 5  # addresses of dgate, dpost_weight, dpost_bias, dweight, dbias
    with _on(stream, x, stats, y, dn, dx, weight, post_weight, post_bias, gate, ws):
        t = _empty(dtype, R, d)
        out, xo = {"dx": t}, t.data_ptr()
        if y is not None:
            out["dy"] = t = _empty(dtype, R, d)
            yo = t.data_ptr()
        if form == _GATE_ELEMENT:
            out["dgate"] = t = _empty(dtype, R, d)
            go = t.data_ptr()
        if weight_grads:
            for i, (there, name) in enumerate(((form == _GATE_CHANNEL, "dgate"), (post, "dpost_weight"),
                                               (post and layer, "dpost_bias"), (dn is not None, "dweight"),
                                               (dn is not None and layer, "dbias"))):
                if there:
                    out[name] = t = _empty_strided((d,), (1,), torch.float32)
                    vectors[i] = t.data_ptr()
            if ws is None and any(vectors):
                ws = _empty(torch.uint8, block_norm_backward_workspace_size(R, d, kind))
        _check(lib().moe_block_norm_backward(
            cfg, *args, wp, sp, dnp, dns, dxp, dxs, xo, yo, go if go is not None else vectors[0], *vectors[1:],
            _ptr(ws), 0 if ws is None else ws.numel(), _raw_stream(stream, here)), "moe_block_norm_backward")
    return out


@functools.lru_cache(maxsize=4096)
def _adapter_ws(*shape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_adapter_add_workspace_size(_struct(AdapterConfig, *shape), ctypes.byref(n)),
           "moe_adapter_add_workspace_size")
    return n.value


def alloc_adapter_workspace(T: int, d: int, N: int, r: int, E: int, dtype=torch.bfloat16, device="cuda") -> torch.Tensor:
    """A workspace for adapter_add calls of up to T rows with these sizes (its error
    word zeroed; workspace_status reads and clears it)."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    ws = torch.empty(max(_adapter_ws(T, d, N, r, E, _DTYPES[dtype], MOE_F32), 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def adapter_add(base, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, rows=None,
                scale=None, out=None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """moe_adapter_add: low-rank adapters of many requests beside a shared projection,
    whose result is base [T, N] (None: zeros):

        out[t] = base[t] + scale[e] (x[t] a[e].T) b[e].T,   e the adapter of row t

    x [T, d], a [E, r, d], b [E, N, r] of one type (FP32, BF16, FP16; smaller ranks
    padded with zeros), scale [E] FP32 or None; base in x's type or FP32. Rows are
    grouped by adapter: rows [T] int32 names each row once (None: in order), those of
    adapter e at positions offsets[e] to offsets[e + 1] (int32 [E + 1]); rows from
    offsets[E] on have no adapter. ``dispatch`` of the rows' adapter ids with K = 1 and
    E + 1 experts, the last for rows without one, gives both (its offsets without the
    last entry, its sorted_token). Rows on 16 bytes, widths and ranks that are multiples
    of 8 serve best (see the header). out: [T, N] to write, or base itself for an update in
    place (allocated when None). ws: see alloc_adapter_workspace. When None one is
    allocated for the call and its error word is not read."""
    here = _here(stream)
    xs = _rows(x, "x")
    _at(x, "x", here)
    T, d = x.shape
    dtype = x.dtype
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError(f"a must be [E, r, d] and b [E, N, r], got {tuple(a.shape)} and {tuple(b.shape)}")
    E, N, r = b.shape
    _dev(a, dtype, "a", (E, r, d), here)
    _dev(b, dtype, "b", None, here)
    _dev(offsets, torch.int32, "offsets", (E + 1,), here)
    if rows is not None:
        _dev(rows, torch.int32, "rows", (T,), here)
    sp = bp = None
    if scale is not None:
        sp = _vector(scale, "scale", (E,), here)
    like = base if base is not None else out if out is not None else x
    otype = like.dtype
    if otype is not dtype and otype is not torch.float32:
        raise ValueError(f"base and out must be {dtype} or float32, got {otype}")
    bs, os_ = 0, N
    if base is not None:
        bp, bs = _like(base, "base", otype, (T, N), here)
    if out is not None:
        _, os_ = _like(out, "out", otype, (T, N), here)
    if ws is not None:
        _scratch(ws, here)
    cfg = (T, d, N, r, E, _DTYPES[dtype], _DTYPES[otype])
    with _on(stream, base, x, a, b, offsets, rows, scale, out, ws):
        if ws is None:
            ws = _empty(torch.uint8, _adapter_ws(*cfg))
        if out is None:
            out = _empty(otype, T, N)
        _check(lib().moe_adapter_add(_struct(AdapterConfig, *cfg), x.data_ptr(), xs, a.data_ptr(), b.data_ptr(), sp,
                                     offsets.data_ptr(), _ptr(rows), bp, bs, out.data_ptr(), os_, ws.data_ptr(),
                                     ws.numel(), _raw_stream(stream, here)), "moe_adapter_add")
    return out


def launch_count() -> int:
    return int(lib().moe_launch_count())


def set_wait_timeout_ms(ms: int):
    _check(lib().moe_set_wait_timeout_ms(int(ms)), "moe_set_wait_timeout_ms")


def selftest_wait_timeout(ms: int, ws: torch.Tensor, stream=None) -> int:
    return lib().moe_selftest_wait_timeout(int(ms), ws.data_ptr(), _stream(stream))


STAGES = ["router", "latent_down", "dispatch", "gather", "gate_up", "down", "combine", "latent_up",
          "decode_fused", "route_dispatch_gather"]


class StageTimer:
    """Per-stage CUDA-event timing of moe_forward calls (library-owned events).
    stages: names to time (None = all)."""

    def __init__(self, max_calls: int, stages=None):
        mask = 0xFFFFFFFF if stages is None else sum(1 << STAGES.index(n) for n in stages)
        _check(lib().moe_timing_begin(int(max_calls), mask), "moe_timing_begin")

    def finish(self) -> tuple[dict, int]:
        arr = (ctypes.c_float * 32)()
        ns, nc = ctypes.c_int32(0), ctypes.c_int32(0)
        _check(lib().moe_timing_end(arr, 32, ctypes.byref(ns), ctypes.byref(nc)), "moe_timing_end")
        names = [lib().moe_stage_name(i).decode() for i in range(ns.value)]
        return {n: arr[i] for i, n in enumerate(names)}, nc.value
