"""Binding of include/moe_block.h: the operators around the layer.

Each function has the name of a C entry point, takes torch tensors on the
current GPU and the outputs and workspace to write, and enqueues on ``stream``
(the current one by default).  Types, shapes, devices and contiguity are
checked here; the library checks the rest.
"""

import ctypes

import torch

from . import _lib

_BF16, _FP32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if stream.device_index != torch.cuda.current_device():
        raise ValueError(f"stream is on cuda:{stream.device_index}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return stream.cuda_stream


def _check(first, *specs):
    """(tensor, name, dtype, shape) each: on the device of ``first``, which is
    the current one, of that type and shape, contiguous.  None is not checked."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"{specs[0][1]} must be a GPU tensor")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"{specs[0][1]} is on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    for t, name, dtype, shape in specs:
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {specs[0][1]} on {dev}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _call(name, *args):
    status = getattr(_lib.load(), name)(*args)
    if status:
        _lib.check(name, status)


def _rmsnorm_quant(name, x, weight, eps, y, residual, sum_out, q, scale, rstd, stream):
    if x.dim() != 2:
        raise ValueError(f"x must have two dimensions, got {tuple(x.shape)}")
    T, d = x.shape
    _check(x, (x, "x", _BF16, None), (weight, "weight", _BF16, (d,)), (y, "y", _BF16, (T, d)),
           (residual, "residual", _BF16, (T, d)), (sum_out, "sum_out", _BF16, (T, d)), (q, "q", _U8, (T, d)),
           (scale, "scale", _FP32, (T, d // 128)), (rstd, "rstd", _FP32, (T,)))
    _call(name, _ptr(x), _ptr(residual), _ptr(weight), T, d, eps, _ptr(sum_out), _ptr(y), _ptr(q), _ptr(scale),
          _ptr(rstd), _stream(stream))


def moe_rmsnorm_quant(x, weight, eps, y, residual=None, sum_out=None, q=None, scale=None, rstd=None, stream=None):
    """Residual addition, RMS norm and 1x128 quantisation: sum_out = x + residual, y [T, d] BF16 (or None) its
    normed rows, q [T, d] uint8 / scale [T, d/128] float32 their FP8 tiles, rstd [T] float32 for the backward.
    ``sum_out`` may be ``x`` or ``residual`` itself."""
    _rmsnorm_quant("moe_rmsnorm_quant", x, weight, eps, y, residual, sum_out, q, scale, rstd, stream)


def moe_rmsnorm_quant_pow2(x, weight, eps, y, residual=None, sum_out=None, q=None, scale=None, rstd=None,
                           stream=None):
    """moe_rmsnorm_quant with power-of-two scales."""
    _rmsnorm_quant("moe_rmsnorm_quant_pow2", x, weight, eps, y, residual, sum_out, q, scale, rstd, stream)


def moe_rmsnorm_backward_workspace_bytes(T, d):
    return int(_lib.load().moe_rmsnorm_backward_workspace_bytes(T, d))


def moe_rmsnorm_backward(dy, h, weight, rstd, dh, dweight, workspace, dres=None, stream=None):
    """Backward of the norm and the addition: dh [T, d] BF16 (the gradient of x and of the residual alike) and
    dweight [d] float32 from dy, the forward's sum ``h`` and ``rstd``; ``dres`` is the gradient that reaches the
    sum through the residual stream (dh may be its memory)."""
    if dy.dim() != 2:
        raise ValueError(f"dy must have two dimensions, got {tuple(dy.shape)}")
    T, d = dy.shape
    _check(dy, (dy, "dy", _BF16, None), (h, "h", _BF16, (T, d)), (weight, "weight", _BF16, (d,)),
           (rstd, "rstd", _FP32, (T,)), (dres, "dres", _BF16, (T, d)), (dh, "dh", _BF16, (T, d)),
           (dweight, "dweight", _FP32, (d,)), (workspace, "workspace", _U8, None))
    _call("moe_rmsnorm_backward", _ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd), _ptr(dres), T, d, _ptr(dh),
          _ptr(dweight), _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))


def moe_layer_few_workspace_bytes(T, d, f, E, k):
    return int(_lib.load().moe_layer_few_workspace_bytes(T, d, f, E, k))


def _layer_few(name, x, wg, bias, n_groups, topk_groups, topk, route_scale, w13, w13_s, w2, w2_s, idx, w, out,
               workspace, residual, stream):
    if x.dim() != 2 or wg.dim() != 2 or w2.dim() != 3:
        raise ValueError("x and wg must have two dimensions, w13 and w2 three")
    T, d = x.shape
    E, f = wg.shape[0], w2.shape[2]
    _check(x, (x, "x", _BF16, None), (wg, "wg", _BF16, (E, d)), (bias, "bias", _FP32, (E,)),
           (w13, "w13", _U8, (E + 1, 2 * f, d)), (w13_s, "w13_s", _FP32, (E + 1, 2 * f // 128, d // 128)),
           (w2, "w2", _U8, (E + 1, d, f)), (w2_s, "w2_s", _FP32, (E + 1, d // 128, f // 128)),
           (idx, "idx", _I32, (T, topk)), (w, "w", _FP32, (T, topk)), (out, "out", _BF16, (T, d)),
           (workspace, "workspace", _U8, None), (residual, "residual", _BF16, (T, d)))
    _call(name, _ptr(x), _ptr(wg), _ptr(bias), T, d, f, _lib.RouteParams(E, n_groups, topk_groups, topk, route_scale),
          _ptr(w13), _ptr(w13_s), _ptr(w2), _ptr(w2_s), _ptr(residual), _ptr(idx), _ptr(w), _ptr(out),
          _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))


def moe_layer_few(x, wg, bias, n_groups, topk_groups, topk, route_scale, w13, w13_s, w2, w2_s, idx, w, out, workspace,
                  residual=None, stream=None):
    """The whole layer for up to 16 tokens: out [T, d] BF16 (plus ``residual``, whose memory it may be), idx [T, k]
    int32 and w [T, k] float32 as moe_route writes them.  The weights are MoEWeights' arrays, the shared expert last;
    ``workspace`` is uint8 of moe_layer_few_workspace_bytes(T, d, f, E, k)."""
    _layer_few("moe_layer_few", x, wg, bias, n_groups, topk_groups, topk, route_scale, w13, w13_s, w2, w2_s, idx, w,
               out, workspace, residual, stream)


def moe_layer_few_pow2(x, wg, bias, n_groups, topk_groups, topk, route_scale, w13, w13_s, w2, w2_s, idx, w, out,
                       workspace, residual=None, stream=None):
    """moe_layer_few with power-of-two scales for x and h."""
    _layer_few("moe_layer_few_pow2", x, wg, bias, n_groups, topk_groups, topk, route_scale, w13, w13_s, w2, w2_s, idx,
               w, out, workspace, residual, stream)


# ---- gradient lists ----

_GRAD_TYPES = {_FP32: 0, _BF16: 1}


def _grad_list(grads, outs, others):
    """Host arrays of a gradient list (and its outputs), checked; ``others`` are
    (tensor, name, dtype, shape) of the call's further operands."""
    n = len(grads)
    dev = torch.cuda.current_device()
    for i, t in enumerate(grads):
        if t.device.type != "cuda" or t.device.index != dev:
            raise ValueError(f"gradient {i} is on {t.device}, the current device is cuda:{dev}")
        if t.dtype not in _GRAD_TYPES:
            raise ValueError(f"gradient {i} must be float32 or bfloat16, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"gradient {i} must be contiguous")
    if outs is not None:
        if len(outs) != n:
            raise ValueError(f"{len(outs)} outputs for {n} gradients")
        for i, (t, o) in enumerate(zip(grads, outs)):
            if o is t:
                continue
            if o.dtype != t.dtype or o.shape != t.shape or o.device != t.device or not o.is_contiguous():
                raise ValueError(f"output {i} must be a contiguous {t.dtype} tensor of shape {tuple(t.shape)} on "
                                 f"{t.device}")
    _check(others[0][0], *others)
    return ((ctypes.c_void_p * n)(*[t.data_ptr() for t in grads]),
            None if outs is None else (ctypes.c_void_p * n)(*[t.data_ptr() for t in outs]),
            (ctypes.c_int64 * n)(*[t.numel() for t in grads]),
            (ctypes.c_int * n)(*[_GRAD_TYPES[t.dtype] for t in grads]), n)


def moe_grad_norm_workspace_bytes(n_tensors):
    return int(_lib.load().moe_grad_norm_workspace_bytes(n_tensors))


def moe_grad_norm(grads, max_norm, norm, coef, workspace, stream=None):
    """norm [1] float32 = L2 norm over every element of ``grads`` (float32 and bfloat16 tensors), coef [1] float32 =
    the factor that clips them to ``max_norm`` (1 where they are within it)."""
    g, _, sizes, types, n = _grad_list(grads, None, ((norm, "norm", _FP32, (1,)), (coef, "coef", _FP32, (1,)),
                                                     (workspace, "workspace", _U8, None)))
    _call("moe_grad_norm", g, sizes, types, n, max_norm, _ptr(norm), _ptr(coef), _ptr(workspace),
          0 if workspace is None else workspace.numel(), _stream(stream))


def moe_grad_scale(grads, coef, outs=None, stream=None):
    """outs[i] = grads[i] * coef, in place without ``outs``."""
    outs = grads if outs is None else outs
    g, o, sizes, types, n = _grad_list(grads, outs, ((coef, "coef", _FP32, (1,)),))
    _call("moe_grad_scale", g, o, sizes, types, n, _ptr(coef), _stream(stream))
