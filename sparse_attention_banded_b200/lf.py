"""ctypes binding of liblf.so (argument marshalling only).

Each function mirrors the C entry point of the same name in ``include/lf.h``:
it takes torch CUDA tensors, passes their device pointers, sizes and the
current CUDA stream to the library, and raises :class:`LFError` on a non-zero
status.  All computation happens in the library's CUDA kernels; if the
library is missing this module raises instead of falling back to anything.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblf.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "lf.h")

LF_F32, LF_F16, LF_BF16 = 0, 1, 2
DTYPE_CODE = {torch.float32: LF_F32, torch.float16: LF_F16, torch.bfloat16: LF_BF16}

_lib = None

LAYER_FIELDS = ("W_qkv_kgvg", "b_qkv_kgvg", "W_qg", "b_qg", "W_o", "b_o", "ln1_gamma", "ln1_beta",
                "W_1", "b_1", "W_2", "b_2", "ln2_gamma", "ln2_beta")


class LayerWeights(ctypes.Structure):
    """lf_layer_weights of include/lf.h."""
    _fields_ = [("ffn_dim", ctypes.c_int)] + [(n, ctypes.c_void_p) for n in LAYER_FIELDS]


class Heads(ctypes.Structure):
    """lf_heads of include/lf.h: a view of per-head rows of 64 elements."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong)]


class LFError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


def lib():
    """Load liblf.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("liblf.so is not built; run `python -m sparse_attention_banded_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
        L.lf_status_string.argtypes = [i]
        L.lf_status_string.restype = ctypes.c_char_p
        L.lf_version.restype = i
        L.lf_device_status.argtypes = [vp, i]
        L.lf_device_status.restype = st
        L.lf_init_global_idx.argtypes = [vp, i, i, i, vp, vp, ctypes.POINTER(ctypes.c_int), vp]
        L.lf_init_global_idx.restype = st
        L.lf_attention_forward.argtypes = [vp] * 8 + [i, i, i, i, i, vp, vp]
        L.lf_attention_forward_idx.argtypes = [vp] * 8 + [i, i, i, i, i, vp, vp, vp, vp]
        L.lf_attention_forward_idx.restype = st
        L.lf_attention_forward.restype = st
        L.lf_attention_scratch_bytes.argtypes = [i, i, i, i, i]
        L.lf_attention_scratch_bytes.restype = ctypes.c_size_t
        L.lf_attention_forward_any_globals.argtypes = [vp] * 8 + [i, i, i, i, i, vp, vp]
        L.lf_attention_forward_any_globals.restype = st
        L.lf_attention_any_globals_scratch_bytes.argtypes = [i, i, i, i, i]
        L.lf_attention_any_globals_scratch_bytes.restype = ctypes.c_size_t
        L.lf_release_scratch.restype = st
        L.lf_attention_forward_noalloc.argtypes = [vp] * 8 + [i, i, i, i, i, vp, vp]
        L.lf_attention_forward_noalloc.restype = st
        L.lf_noalloc_device_status.argtypes = [vp, i]
        L.lf_noalloc_device_status.restype = st
        L.lf_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, vp]
        L.lf_selftest_bounded_wait.restype = st
        L.lf_encoder_layer_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.lf_encoder_layer_workspace_bytes.restype = ctypes.c_size_t
        L.lf_encoder_layer_forward.argtypes = [vp, vp, vp, ctypes.POINTER(LayerWeights), i, i, i, i,
                                               ctypes.c_float, ctypes.c_float, i, vp, ctypes.c_size_t, vp, vp]
        L.lf_encoder_layer_forward.restype = st
        L.lf_encoder_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        L.lf_encoder_workspace_bytes.restype = ctypes.c_size_t
        L.lf_encoder_forward.argtypes = [vp, vp, vp, ctypes.POINTER(LayerWeights), i, i, i, i, i,
                                         ctypes.c_float, ctypes.c_float, i, vp, ctypes.c_size_t, vp, vp]
        L.lf_encoder_layer_any_globals_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.lf_encoder_layer_any_globals_workspace_bytes.restype = ctypes.c_size_t
        L.lf_encoder_layer_forward_any_globals.argtypes = L.lf_encoder_layer_forward.argtypes
        L.lf_encoder_layer_forward_any_globals.restype = st
        L.lf_encoder_any_globals_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        L.lf_encoder_any_globals_workspace_bytes.restype = ctypes.c_size_t
        L.lf_encoder_forward_any_globals.argtypes = L.lf_encoder_forward.argtypes
        L.lf_encoder_forward_any_globals.restype = st
        L.lf_encoder_forward.restype = st
        L.lf_gelu_ffn_workspace_bytes.argtypes = [i, i, i, i, i]
        L.lf_gelu_ffn_workspace_bytes.restype = ctypes.c_size_t
        L.lf_gelu_ffn_forward.argtypes = [vp] * 5 + [i, i, i, i, i, vp, ctypes.c_size_t, vp, vp]
        L.lf_gelu_ffn_forward.restype = st
        L.lf_set_ffn_path.argtypes = [i]
        L.lf_set_ffn_path.restype = st
        L.lf_get_ffn_path.argtypes = []
        L.lf_get_ffn_path.restype = i
        f, ll, sz, hp = ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t, ctypes.POINTER(Heads)
        L.lf_window_attention_forward.argtypes = [hp] * 3 + [vp, vp] + [i] * 6 + [f, i, vp, vp, vp]
        L.lf_window_attention_forward.restype = st
        L.lf_window_attention_backward_workspace_bytes.argtypes = [i] * 7
        L.lf_window_attention_backward_workspace_bytes.restype = sz
        L.lf_window_attention_backward.argtypes = ([hp] * 3 + [vp] * 5 + [i] * 6 + [f, i, vp, sz, vp] + [hp] * 3)
        L.lf_window_attention_backward.restype = st
        L.lf_paged_cache_append.argtypes = [hp] * 4 + [vp] * 3 + [i] * 7 + [vp]
        L.lf_paged_cache_append.restype = st
        L.lf_paged_attention_workspace_bytes.argtypes = [i] * 9
        L.lf_paged_attention_workspace_bytes.restype = sz
        L.lf_paged_attention_forward.argtypes = [hp] * 3 + [vp] * 3 + [i] * 10 + [f, i, vp, sz, vp, vp]
        L.lf_paged_attention_forward.restype = st
        L.lf_layer_norm_forward.argtypes = [vp, ll, vp, vp, i, i, f, i, vp, vp, vp, vp]
        L.lf_layer_norm_forward.restype = st
        L.lf_layer_norm_backward_workspace_bytes.argtypes = [i, i]
        L.lf_layer_norm_backward_workspace_bytes.restype = sz
        L.lf_layer_norm_backward.argtypes = [vp, ll, vp, ll, vp, vp, vp, i, i, i, vp, sz, vp, vp, vp, vp]
        L.lf_layer_norm_backward.restype = st
        _lib = L
    return _lib


def declared_functions():
    """Names of the functions include/lf.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\*\s]+?\b(lf_\w+)\s*\(", text, re.M)))


def status_string(status: int) -> str:
    return lib().lf_status_string(int(status)).decode()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _check(status, where):
    if status != 0:
        raise LFError(status, where)


def lf_device_status(reset: bool = False, stream=None) -> int:
    """Synchronise and return the device status word (see lf.h)."""
    return lib().lf_device_status(_stream(stream), 1 if reset else 0)


def lf_init_global_idx(global_mask, w: int, global_idx=None, global_token_nums=None, sync: bool = True,
                       stream=None):
    """Global-token partition.  Returns (global_idx, global_token_nums,
    max_g); max_g is None when sync is False (then content errors go to the
    device status word)."""
    B, L = global_mask.shape
    if global_idx is None:
        global_idx = torch.empty(B, L, dtype=torch.int32, device=global_mask.device)
    if global_token_nums is None:
        global_token_nums = torch.empty(B, dtype=torch.int32, device=global_mask.device)
    mx = ctypes.c_int(-1)
    st = lib().lf_init_global_idx(_ptr(global_mask), B, L, w, _ptr(global_idx), _ptr(global_token_nums),
                                  ctypes.byref(mx) if sync else None, _stream(stream))
    _check(st, "lf_init_global_idx")
    return global_idx, global_token_nums, (mx.value if sync else None)


def lf_attention_forward(q, k, v, qg, kg, vg, local_mask, global_mask, w: int, out=None, stream=None):
    """Longformer attention; q..vg [B, H, L, 64], masks [B, L] float32.
    Returns out [B, L, H*64] in the input dtype."""
    B, H, L, _ = q.shape
    if out is None:
        out = torch.empty(B, L, H * 64, dtype=q.dtype, device=q.device)
    code = DTYPE_CODE.get(q.dtype, 99)
    st = lib().lf_attention_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(qg), _ptr(kg), _ptr(vg),
                                    _ptr(local_mask), _ptr(global_mask), B, H, L, w, code,
                                    _stream(stream), _ptr(out))
    _check(st, "lf_attention_forward")
    return out


def lf_attention_forward_idx(q, k, v, qg, kg, vg, local_mask, global_mask, w: int, out=None, global_idx=None,
                             global_token_nums=None, stream=None):
    """The partition of lf_init_global_idx and the attention in one call
    (one kernel launch for fp16 / bf16).  Returns (out, global_idx,
    global_token_nums)."""
    B, H, L, _ = q.shape
    if out is None:
        out = torch.empty(B, L, H * 64, dtype=q.dtype, device=q.device)
    if global_idx is None:
        global_idx = torch.empty(B, L, dtype=torch.int32, device=q.device)
    if global_token_nums is None:
        global_token_nums = torch.empty(B, dtype=torch.int32, device=q.device)
    code = DTYPE_CODE.get(q.dtype, 99)
    st = lib().lf_attention_forward_idx(_ptr(q), _ptr(k), _ptr(v), _ptr(qg), _ptr(kg), _ptr(vg),
                                        _ptr(local_mask), _ptr(global_mask), B, H, L, w, code,
                                        _stream(stream), _ptr(out), _ptr(global_idx), _ptr(global_token_nums))
    _check(st, "lf_attention_forward_idx")
    return out, global_idx, global_token_nums


def lf_attention_scratch_bytes(B: int, H: int, L: int, w: int, dtype) -> int:
    return lib().lf_attention_scratch_bytes(B, H, L, w, DTYPE_CODE[dtype])


def lf_attention_forward_any_globals(q, k, v, qg, kg, vg, local_mask, global_mask, w: int, out=None,
                                     stream=None):
    """Same as :func:`lf_attention_forward` with the global tokens
    (global_mask == 0.0) at any positions of the sequence."""
    B, H, L, _ = q.shape
    if out is None:
        out = torch.empty(B, L, H * 64, dtype=q.dtype, device=q.device)
    code = DTYPE_CODE.get(q.dtype, 99)
    st = lib().lf_attention_forward_any_globals(_ptr(q), _ptr(k), _ptr(v), _ptr(qg), _ptr(kg), _ptr(vg),
                                                _ptr(local_mask), _ptr(global_mask), B, H, L, w, code,
                                                _stream(stream), _ptr(out))
    _check(st, "lf_attention_forward_any_globals")
    return out


def lf_attention_any_globals_scratch_bytes(B: int, H: int, L: int, w: int, dtype) -> int:
    return lib().lf_attention_any_globals_scratch_bytes(B, H, L, w, DTYPE_CODE[dtype])


def lf_release_scratch():
    _check(lib().lf_release_scratch(), "lf_release_scratch")


def lf_attention_forward_noalloc(q, k, v, qg, kg, vg, local_mask, global_mask, w: int, out=None, stream=None):
    """Same as :func:`lf_attention_forward` through the entry point that
    allocates no device memory (fp16/bf16; scratch limited to 32 MiB)."""
    B, H, L, _ = q.shape
    if out is None:
        out = torch.empty(B, L, H * 64, dtype=q.dtype, device=q.device)
    code = DTYPE_CODE.get(q.dtype, 99)
    st = lib().lf_attention_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(qg), _ptr(kg), _ptr(vg),
                                            _ptr(local_mask), _ptr(global_mask), B, H, L, w, code,
                                            _stream(stream), _ptr(out))
    _check(st, "lf_attention_forward_noalloc")
    return out


def lf_noalloc_device_status(reset: bool = False, stream=None) -> int:
    """Synchronise and return the status word of the no-allocation entry
    point (see lf.h)."""
    return lib().lf_noalloc_device_status(_stream(stream), 1 if reset else 0)


def lf_selftest_bounded_wait(limit_ns: int, stream=None):
    """Launch the one-CTA kernel whose bounded wait runs out after limit_ns
    (see lf.h); the result is read with :func:`lf_device_status`."""
    _check(lib().lf_selftest_bounded_wait(int(limit_ns), _stream(stream)), "lf_selftest_bounded_wait")


FFN_PATH = {"auto": 0, "unfused": 1, "fused": 2}


def lf_gelu_ffn_workspace_bytes(rows: int, d_model: int, ffn_dim: int, dtype, path: str = "auto") -> int:
    return lib().lf_gelu_ffn_workspace_bytes(rows, d_model, ffn_dim, DTYPE_CODE[dtype], FFN_PATH[path])


def lf_gelu_ffn_forward(h, W_1, b_1, W_2, b_2, path: str = "auto", out=None, workspace=None, stream=None):
    """z = h + b_2 + GELU(h W_1^T + b_1) W_2^T (fp32) for h [rows, D];
    path "unfused" (two GEMMs), "fused" (one kernel, the intermediate kept
    on chip) or "auto" (see lf.h)."""
    rows, D = h.shape
    F = W_1.shape[0]
    if out is None:
        out = torch.empty(rows, D, dtype=torch.float32, device=h.device)
    need = lf_gelu_ffn_workspace_bytes(rows, D, F, h.dtype, path) if h.dtype in DTYPE_CODE else 0
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=h.device)
    st = lib().lf_gelu_ffn_forward(_ptr(h), _ptr(W_1), _ptr(b_1), _ptr(W_2), _ptr(b_2), rows, D, F,
                                   DTYPE_CODE.get(h.dtype, 99), FFN_PATH[path], _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _stream(stream), _ptr(out))
    _check(st, "lf_gelu_ffn_forward")
    return out


def lf_set_ffn_path(path: str):
    """The FFN path of the layer and encoder calls in this process."""
    _check(lib().lf_set_ffn_path(FFN_PATH[path]), "lf_set_ffn_path")


def lf_get_ffn_path() -> str:
    code = lib().lf_get_ffn_path()
    return {v: k for k, v in FFN_PATH.items()}[code]


def lf_encoder_layer_workspace_bytes(B: int, H: int, L: int, w: int, ffn_dim: int, dtype) -> int:
    return lib().lf_encoder_layer_workspace_bytes(B, H, L, w, ffn_dim, DTYPE_CODE[dtype])


def _layer(name, size_fn, x, local_mask, global_mask, weights, H, w, attn_scale, ln_eps, out, workspace, stream):
    B, L, D = x.shape
    ffn = weights["W_1"].shape[0]
    wt = LayerWeights(ffn, *[weights[n].data_ptr() for n in LAYER_FIELDS])
    for n in LAYER_FIELDS:
        _ptr(weights[n])
    if out is None:
        out = torch.empty_like(x)
    need = size_fn(B, H, L, w, ffn, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    st = getattr(lib(), name)(_ptr(x), _ptr(local_mask), _ptr(global_mask), ctypes.byref(wt), B, H, L,
                              w, attn_scale, ln_eps, DTYPE_CODE.get(x.dtype, 99), _ptr(workspace),
                              workspace.numel(), _stream(stream), _ptr(out))
    _check(st, name)
    return out


def lf_encoder_layer_forward(x, local_mask, global_mask, weights: dict, H: int, w: int, attn_scale: float = 0.125,
                             ln_eps: float = 1e-5, out=None, workspace=None, stream=None):
    """One encoder layer; x [B, L, H*64]; weights: tensors named as the
    fields of lf_layer_weights (nn.Linear layout [out, in]), LayerNorm
    parameters fp32.  Returns out [B, L, H*64]."""
    return _layer("lf_encoder_layer_forward", lf_encoder_layer_workspace_bytes, x, local_mask, global_mask,
                  weights, H, w, attn_scale, ln_eps, out, workspace, stream)


def lf_encoder_layer_any_globals_workspace_bytes(B: int, H: int, L: int, w: int, ffn_dim: int, dtype) -> int:
    return lib().lf_encoder_layer_any_globals_workspace_bytes(B, H, L, w, ffn_dim, DTYPE_CODE[dtype])


def lf_encoder_layer_forward_any_globals(x, local_mask, global_mask, weights: dict, H: int, w: int,
                                         attn_scale: float = 0.125, ln_eps: float = 1e-5, out=None, workspace=None,
                                         stream=None):
    """Same as :func:`lf_encoder_layer_forward` with the global tokens
    (global_mask == 0.0) at any positions."""
    return _layer("lf_encoder_layer_forward_any_globals", lf_encoder_layer_any_globals_workspace_bytes, x,
                  local_mask, global_mask, weights, H, w, attn_scale, ln_eps, out, workspace, stream)


def lf_encoder_workspace_bytes(n_layers: int, B: int, H: int, L: int, w: int, ffn_dim: int, dtype) -> int:
    return lib().lf_encoder_workspace_bytes(n_layers, B, H, L, w, ffn_dim, DTYPE_CODE[dtype])


def lf_encoder_forward(x, local_mask, global_mask, layers: list, H: int, w: int, attn_scale: float = 0.125,
                       ln_eps: float = 1e-5, out=None, workspace=None, stream=None):
    """The encoder: the layers in `layers` (each a weight dict as for
    lf_encoder_layer_forward, same FFN width) applied in turn to x
    [B, L, H*64].  Returns out [B, L, H*64]."""
    return _encoder("lf_encoder_forward", lf_encoder_workspace_bytes, x, local_mask, global_mask, layers, H, w,
                    attn_scale, ln_eps, out, workspace, stream)


def lf_encoder_any_globals_workspace_bytes(n_layers: int, B: int, H: int, L: int, w: int, ffn_dim: int,
                                           dtype) -> int:
    return lib().lf_encoder_any_globals_workspace_bytes(n_layers, B, H, L, w, ffn_dim, DTYPE_CODE[dtype])


def lf_encoder_forward_any_globals(x, local_mask, global_mask, layers: list, H: int, w: int,
                                   attn_scale: float = 0.125, ln_eps: float = 1e-5, out=None, workspace=None,
                                   stream=None):
    """Same as :func:`lf_encoder_forward` with the global tokens
    (global_mask == 0.0) at any positions."""
    return _encoder("lf_encoder_forward_any_globals", lf_encoder_any_globals_workspace_bytes, x, local_mask,
                    global_mask, layers, H, w, attn_scale, ln_eps, out, workspace, stream)


def _encoder(fn_name, size_fn, x, local_mask, global_mask, layers, H, w, attn_scale, ln_eps, out, workspace, stream):
    B, L, D = x.shape
    n = len(layers)
    ffn = layers[0]["W_1"].shape[0] if n else 0
    arr = (LayerWeights * max(n, 1))()
    for j, weights in enumerate(layers):
        for name in LAYER_FIELDS:
            _ptr(weights[name])
        arr[j] = LayerWeights(weights["W_1"].shape[0], *[weights[name].data_ptr() for name in LAYER_FIELDS])
    if out is None:
        out = torch.empty_like(x)
    need = size_fn(n, B, H, L, w, ffn, x.dtype) if n else 0
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    st = getattr(lib(), fn_name)(_ptr(x), _ptr(local_mask), _ptr(global_mask), arr, n, B, H, L, w, attn_scale,
                                 ln_eps, DTYPE_CODE.get(x.dtype, 99), _ptr(workspace), workspace.numel(),
                                 _stream(stream), _ptr(out))
    _check(st, fn_name)
    return out


# --------------------------------------------------------------------------
# windowed causal attention with sinks, its paged form, layer norm
# --------------------------------------------------------------------------
# stream: the torch.cuda.Stream to launch on (default: the current one).  New
# outputs belong to it: a caller that uses them on another stream orders the
# two and calls their record_stream.  The calls are no autograd functions:
# gradients are the _backward calls' to compute.
_HERE_ALREADY = contextlib.nullcontext()


def _on(first, stream, *tensors):
    """A context in which the device of `first` is current and `stream` (if
    given) the stream that outputs and workspaces are allocated on.  Where it
    is not the current stream, the tensors are marked as used on it, so that
    their memory waits for it when the caller lets go of them."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors on different devices: %s and %s" % (first.device, t.device))
    if stream is not None:
        if stream.device != first.device:
            raise ValueError("the stream belongs to %s, the tensors to %s" % (stream.device, first.device))
        if stream != torch.cuda.current_stream(dev):
            for t in (first, *tensors):
                if t is not None:
                    t.record_stream(stream)
        return torch.cuda.stream(stream)  # makes its device current too
    return _HERE_ALREADY if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _raw_stream(stream, tensor):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(tensor.get_device())


def _dense(t):
    """The address of a contiguous tensor (its device has been checked)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _want(name, t, dtype=None, shape=None):
    if dtype is not None and t.dtype is not dtype:
        raise ValueError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _new(t, like, dtype, shape, name):
    """`t` checked, or a new tensor on the device of `like`."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    return _want(name, t, dtype, shape)


def _like(t):
    """A new contiguous tensor of t's shape and dtype (0.5 us less than
    new_empty, of a call's 15)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _workspace(t, like, need):
    """(tensor, address, bytes) of the caller's workspace or a new one."""
    if t is None:
        if not need:
            return None, None, 0
        t = like.new_empty(need, dtype=torch.uint8)
        return t, t.data_ptr(), need
    return t, _dense(t), t.numel() * t.element_size()


def _int32(**values):
    """The values as Python ints; any type that stands for a whole number will
    do (NumPy's, a one-element integer tensor)."""
    ints = []
    for name, x in values.items():
        x = operator.index(x)
        if not -(1 << 31) <= x < 1 << 31:
            raise ValueError("%s: %d is not an int32" % (name, x))
        ints.append(x)
    return ints


def _too_wide(*sizes):
    """Sizes that the C interface's int would cut off are refused."""
    raise ValueError("a size of %s is not an int32" % (sizes,))


def _heads(name, t, shape=None, dtype=None):
    """lf_heads of [B, H, T, 64], or of packed [T, H, 64]."""
    if dtype is not None:
        _want(name, t, dtype, shape)
    strides = t.stride()
    if t.shape[-1] != 64 or strides[-1] != 1 and t.numel():
        raise ValueError("%s: expected rows of 64 contiguous elements, got %s" % (name, tuple(t.shape)))
    if len(strides) == 3:
        return Heads(t.data_ptr(), 0, strides[1], strides[0])
    return Heads(t.data_ptr(), strides[0], strides[1], strides[2])


def _window_shape(q, k, v, cu_seqlens, seq_lens):
    """(n_seqs, Hq, Hkv, L, shape of out, shape of lse)"""
    shape, dtype = q.shape, q.dtype
    packed = cu_seqlens is not None
    if len(shape) != (3 if packed else 4) or shape[-1] != 64:
        raise ValueError("q: expected %s, got %s" % ("packed [T, H, 64]" if packed else "[B, H, L, 64]", tuple(shape)))
    kv = k.shape
    if k.dtype is not dtype or v.dtype is not dtype or v.shape != kv or len(kv) != len(shape):
        raise ValueError("k, v: expected two [.., Hkv, .., 64] of %s like q, got %s and %s" % (dtype, tuple(kv), tuple(v.shape)))
    if (shape[0] | shape[1] | shape[-2] | kv[1]) >> 31:
        _too_wide(shape, kv)
    if packed:
        L, Hq, _ = shape
        Hkv = kv[1]
        if kv != (L, Hkv, 64):
            raise ValueError("k: expected (%d, Hkv, 64), got %s" % (L, tuple(kv)))
        if seq_lens is not None:
            raise ValueError("give cu_seqlens or seq_lens, not both")
        _want("cu_seqlens", cu_seqlens, torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens: expected [n_seqs + 1]")
        return cu_seqlens.numel() - 1, Hq, Hkv, L, (L, Hq * 64), (1, Hq, L)
    B, Hq, L, _ = shape
    Hkv = kv[1]
    if kv != (B, Hkv, L, 64):
        raise ValueError("k: expected (%d, Hkv, %d, 64), got %s" % (B, L, tuple(kv)))
    if seq_lens is not None:
        _want("seq_lens", seq_lens, torch.int32, (B,))
    return B, Hq, Hkv, L, (B, L, Hq * 64), (B, Hq, L)


def lf_window_attention_forward(q, k, v, w: int, sinks: int = 0, scale: float = 0.125, cu_seqlens=None,
                                seq_lens=None, out=None, lse=None, stream=None):
    """Causal attention in which the query at position i sees the keys j <= i
    with i - j <= w or j < sinks.  q [B, Hq, L, 64], k, v [B, Hkv, L, 64] (any
    strides, last dimension contiguous), with seq_lens [B] int32 tokens per
    row when padded; or packed q [T, Hq, 64], k, v [T, Hkv, 64] with
    cu_seqlens [n + 1] int32.  Returns (out [B, L, Hq*64] or [T, Hq*64], lse
    [B, Hq, L] or [1, Hq, T] float32, for the backward pass).  Not an autograd
    function: :func:`lf_window_attention_backward` computes the gradients."""
    w, sinks = _int32(w=w, sinks=sinks)
    n, Hq, Hkv, L, o_shape, l_shape = _window_shape(q, k, v, cu_seqlens, seq_lens)
    with _on(q, stream, k, v, cu_seqlens, seq_lens, out, lse):
        out = _new(out, q, q.dtype, o_shape, "out")
        lse = _new(lse, q, torch.float32, l_shape, "lse")
        st = lib().lf_window_attention_forward(
            _heads("q", q), _heads("k", k), _heads("v", v), _dense(cu_seqlens), _dense(seq_lens), n, Hq, Hkv, L, w,
            sinks, scale, DTYPE_CODE.get(q.dtype, 99), _raw_stream(stream, q), _dense(out), _dense(lse))
    _check(st, "lf_window_attention_forward")
    return out, lse


def lf_window_attention_backward_workspace_bytes(packed: bool, n_seqs: int, Hq: int, Hkv: int, L: int, w: int,
                                                 sinks: int) -> int:
    return lib().lf_window_attention_backward_workspace_bytes(
        int(packed), *_int32(n_seqs=n_seqs, Hq=Hq, Hkv=Hkv, L=L, w=w, sinks=sinks))


def lf_window_attention_backward(q, k, v, out, lse, dout, w: int, sinks: int = 0, scale: float = 0.125,
                                 cu_seqlens=None, seq_lens=None, dq=None, dk=None, dv=None, workspace=None,
                                 stream=None):
    """Gradients of :func:`lf_window_attention_forward`: out and lse as it
    returned them, dout like out (contiguous).  dq, dk, dv may be strided
    views (of one gradient of a fused projection, say); without them they are
    allocated like q, k, v, contiguous.  Returns (dq, dk, dv)."""
    w, sinks = _int32(w=w, sinks=sinks)
    n, Hq, Hkv, L, o_shape, l_shape = _window_shape(q, k, v, cu_seqlens, seq_lens)
    dtype = q.dtype
    _want("out", out, dtype, o_shape)
    _want("dout", dout, dtype, o_shape)
    _want("lse", lse, torch.float32, l_shape)
    with _on(q, stream, k, v, out, lse, dout, cu_seqlens, seq_lens, dq, dk, dv, workspace):
        dq = _like(q) if dq is None else dq
        dk = _like(k) if dk is None else dk
        dv = _like(v) if dv is None else dv
        need = 0
        if workspace is None:
            need = max(256, lib().lf_window_attention_backward_workspace_bytes(
                int(cu_seqlens is not None), n, Hq, Hkv, L, w, sinks))
        workspace, ws, ws_bytes = _workspace(workspace, q, need)
        st = lib().lf_window_attention_backward(
            _heads("q", q), _heads("k", k), _heads("v", v), _dense(out), _dense(lse), _dense(dout),
            _dense(cu_seqlens), _dense(seq_lens), n, Hq, Hkv, L, w, sinks, scale, DTYPE_CODE.get(dtype, 99), ws,
            ws_bytes, _raw_stream(stream, q), _heads("dq", dq, q.shape, dtype), _heads("dk", dk, k.shape, dtype),
            _heads("dv", dv, k.shape, dtype))
    _check(st, "lf_window_attention_backward")
    return dq, dk, dv


def _paged_shape(new, k_cache, v_cache, block_table, cu_seqlens, kv_lens):
    """(n_seqs, T, Hkv, max_pages, num_pages, page_size)"""
    cache, dtype, i32 = k_cache.shape, new.dtype, torch.int32
    if new.dim() != 3 or new.shape[2] != 64:
        raise ValueError("expected packed [T, H, 64], got %s" % (tuple(new.shape),))
    if len(cache) != 4 or cache[3] != 64 or v_cache.shape != cache:
        raise ValueError("k_cache, v_cache: expected two [num_pages, Hkv, page_size, 64], got %s and %s"
                         % (tuple(cache), tuple(v_cache.shape)))
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
        raise ValueError("k_cache, v_cache: expected %s, got %s and %s" % (dtype, k_cache.dtype, v_cache.dtype))
    if block_table.dim() != 2 or block_table.dtype is not i32:
        raise ValueError("block_table: expected [n_seqs, max_pages] int32")
    n, max_pages = block_table.shape
    T, heads, _ = new.shape
    num_pages, Hkv, page_size, _ = cache
    if (n | max_pages | T | heads | num_pages | Hkv | page_size) >> 31:
        _too_wide((n, max_pages), new.shape, cache)
    _want("cu_seqlens", cu_seqlens, i32, (n + 1,))
    _want("kv_lens", kv_lens, i32, (n,))
    return n, T, Hkv, max_pages, num_pages, page_size


def lf_paged_cache_append(k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, stream=None):
    """Copy new tokens' k, v [T, Hkv, 64] (packed by cu_seqlens [n + 1]) to
    the last positions of their sequences (kv_lens [n] positions in all) in
    the paged cache k_cache, v_cache [num_pages, Hkv, page_size, 64] (any
    strides) through block_table [n, max_pages] int32."""
    n, T, Hkv, max_pages, num_pages, page_size = _paged_shape(k, k_cache, v_cache, block_table, cu_seqlens, kv_lens)
    _want("k", k, k.dtype, (T, Hkv, 64))
    _want("v", v, k.dtype, (T, Hkv, 64))
    with _on(k, stream, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens):
        st = lib().lf_paged_cache_append(
            _heads("k", k), _heads("v", v), _heads("k_cache", k_cache), _heads("v_cache", v_cache),
            _dense(block_table), _dense(cu_seqlens), _dense(kv_lens), n, Hkv, T, max_pages, num_pages, page_size,
            DTYPE_CODE.get(k.dtype, 99), _raw_stream(stream, k))
    _check(st, "lf_paged_cache_append")


def lf_paged_attention_workspace_bytes(n_seqs: int, Hq: int, Hkv: int, T: int, max_q_len: int, max_pages: int,
                                       page_size: int, w: int, sinks: int) -> int:
    return lib().lf_paged_attention_workspace_bytes(
        *_int32(n_seqs=n_seqs, Hq=Hq, Hkv=Hkv, T=T, max_q_len=max_q_len, max_pages=max_pages, page_size=page_size, w=w,
                sinks=sinks))


def lf_paged_attention_forward(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_q_len: int,
                               w: int = (1 << 31) - 1, sinks: int = 0, scale: float = 0.125, out=None,
                               workspace=None, stream=None):
    """Windowed causal attention of new tokens q [T, Hq, 64] (packed by
    cu_seqlens, none of the sequences longer than max_q_len) over the paged
    cache, which holds their own keys and values already
    (:func:`lf_paged_cache_append`).  Returns out [T, Hq*64]."""
    n, T, Hkv, max_pages, num_pages, page_size = _paged_shape(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens)
    w, sinks, max_q_len = _int32(w=w, sinks=sinks, max_q_len=max_q_len)
    Hq = q.shape[1]
    with _on(q, stream, k_cache, v_cache, block_table, cu_seqlens, kv_lens, out, workspace):
        out = _new(out, q, q.dtype, (T, Hq * 64), "out")
        need = 0
        if workspace is None:
            need = lib().lf_paged_attention_workspace_bytes(n, Hq, Hkv, T, max_q_len, max_pages, page_size, w, sinks)
        workspace, ws, ws_bytes = _workspace(workspace, q, need)
        st = lib().lf_paged_attention_forward(
            _heads("q", q), _heads("k_cache", k_cache), _heads("v_cache", v_cache), _dense(block_table),
            _dense(cu_seqlens), _dense(kv_lens), n, Hq, Hkv, T, max_q_len, max_pages, num_pages, page_size, w, sinks,
            scale, DTYPE_CODE.get(q.dtype, 99), ws, ws_bytes, _raw_stream(stream, q), _dense(out))
    _check(st, "lf_paged_attention_forward")
    return out


def _rows(name, t):
    """(address, rows, N, row stride) of [..., N]: contiguous, or 2-D with a
    contiguous last dimension."""
    shape = t.shape
    if not shape:
        raise ValueError("%s: expected [..., N]" % name)
    N = shape[-1]
    rows = t.numel() // N if N else 0
    if (rows | N) >> 31:
        _too_wide(shape)
    if t.is_contiguous():
        return t.data_ptr(), rows, N, N
    if len(shape) == 2 and (t.stride(1) == 1 or N == 1):
        return t.data_ptr(), rows, N, t.stride(0)
    raise ValueError("%s: expected a contiguous tensor, or a 2-D one with a row stride" % name)


def lf_layer_norm_forward(x, gamma=None, beta=None, eps: float = 1e-5, out=None, mean=None, rstd=None, stream=None):
    """Layer norm of the rows of x [..., N]; gamma, beta [N] float32 or None.
    Returns (y, mean, rstd), mean and rstd [rows] float32 for the backward
    pass.  Not an autograd function: :func:`lf_layer_norm_backward` computes
    the gradients."""
    px, rows, N, stride = _rows("x", x)
    with _on(x, stream, gamma, beta, out, mean, rstd):
        if gamma is not None:
            _want("gamma", gamma, torch.float32, (N,))
        if beta is not None:
            _want("beta", beta, torch.float32, (N,))
        out = _like(x) if out is None else _want("out", out, x.dtype, x.shape)
        if mean is None and rstd is None:
            mean, rstd = x.new_empty((2, rows), dtype=torch.float32).unbind(0)
        else:
            mean = _new(mean, x, torch.float32, (rows,), "mean")
            rstd = _new(rstd, x, torch.float32, (rows,), "rstd")
        st = lib().lf_layer_norm_forward(px, stride, _dense(gamma), _dense(beta), rows, N, eps,
                                         DTYPE_CODE.get(x.dtype, 99), _raw_stream(stream, x), _dense(out),
                                         _dense(mean), _dense(rstd))
    _check(st, "lf_layer_norm_forward")
    return out, mean, rstd


def lf_layer_norm_backward_workspace_bytes(rows: int, N: int) -> int:
    return lib().lf_layer_norm_backward_workspace_bytes(*_int32(rows=rows, N=N))


def lf_layer_norm_backward(dy, x, gamma, mean, rstd, dx=None, dgamma=None, dbeta=None, param_grads: bool = True,
                           workspace=None, stream=None):
    """Gradients of :func:`lf_layer_norm_forward` (mean, rstd as it returned
    them).  Returns (dx, dgamma, dbeta); with param_grads False only those of
    dgamma, dbeta that were passed in are written."""
    px, rows, N, xs = _rows("x", x)
    with _on(x, stream, dy, gamma, mean, rstd, dx, dgamma, dbeta, workspace):
        pdy, _, _, dys = _rows("dy", _want("dy", dy, x.dtype, x.shape))
        if gamma is not None:
            _want("gamma", gamma, torch.float32, (N,))
        _want("mean", mean, torch.float32, (rows,))
        _want("rstd", rstd, torch.float32, (rows,))
        dx = _like(x) if dx is None else _want("dx", dx, x.dtype, x.shape)
        if param_grads or dgamma is not None:
            dgamma = _new(dgamma, x, torch.float32, (N,), "dgamma")
        if param_grads or dbeta is not None:
            dbeta = _new(dbeta, x, torch.float32, (N,), "dbeta")
        need = 0
        if workspace is None and (dgamma is not None or dbeta is not None):
            need = max(256, lib().lf_layer_norm_backward_workspace_bytes(rows, N))
        workspace, ws, ws_bytes = _workspace(workspace, x, need)
        st = lib().lf_layer_norm_backward(
            pdy, dys, px, xs, _dense(gamma), _dense(mean), _dense(rstd), rows, N, DTYPE_CODE.get(x.dtype, 99), ws,
            ws_bytes, _raw_stream(stream, x), _dense(dx), _dense(dgamma), _dense(dbeta))
    _check(st, "lf_layer_norm_backward")
    return dx, dgamma, dbeta
