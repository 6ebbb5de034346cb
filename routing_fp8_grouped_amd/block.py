"""Binding of include/moe_block.h: the operators around the layer.

Each function has the name of a C entry point, takes torch tensors on the
current GPU and the outputs and workspace to write, and enqueues on ``stream``
(the current one by default).  Types, shapes, devices and contiguity are
checked here; the library checks the rest.
"""

from array import array
from operator import attrgetter

import torch

from . import _lib

_BF16, _FP32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream    # current_stream() without building a Stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the current device is cuda:{dev}")
    return stream.cuda_stream


def _device(t, name):
    """Index of the current device, which ``t`` must be on."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _check(dev, specs):
    """(tensor, name, dtype, shape) each: on device ``dev``, of that type and
    shape, contiguous.  None is not checked."""
    for t, name, dtype, shape in specs:
        if t is None:
            continue
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _call(name, *args):
    status = getattr(_lib.load(), name)(*args)
    if status:
        _lib.check(name, status)


def _rmsnorm_quant(name, x, weight, eps, y, residual, sum_out, q, scale, rstd, stream):
    if x.dim() != 2:
        raise ValueError(f"x must have two dimensions, got {tuple(x.shape)}")
    shape = x.shape
    T, d = shape
    dev = _device(x, "x")
    _check(dev, ((x, "x", _BF16, None), (weight, "weight", _BF16, (d,)), (y, "y", _BF16, shape),
                 (residual, "residual", _BF16, shape), (sum_out, "sum_out", _BF16, shape), (q, "q", _U8, shape),
                 (scale, "scale", _FP32, (T, d // 128)), (rstd, "rstd", _FP32, (T,))))
    _call(name, _ptr(x), _ptr(residual), _ptr(weight), T, d, eps, _ptr(sum_out), _ptr(y), _ptr(q), _ptr(scale),
          _ptr(rstd), _stream(stream, dev))


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
    shape = dy.shape
    T, d = shape
    dev = _device(dy, "dy")
    _check(dev, ((dy, "dy", _BF16, None), (h, "h", _BF16, shape), (weight, "weight", _BF16, (d,)),
                 (rstd, "rstd", _FP32, (T,)), (dres, "dres", _BF16, shape), (dh, "dh", _BF16, shape),
                 (dweight, "dweight", _FP32, (d,)), (workspace, "workspace", _U8, None)))
    _call("moe_rmsnorm_backward", _ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd), _ptr(dres), T, d, _ptr(dh),
          _ptr(dweight), _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream, dev))


def moe_layer_few_workspace_bytes(T, d, f, E, k):
    return int(_lib.load().moe_layer_few_workspace_bytes(T, d, f, E, k))


def _layer_few(name, x, wg, bias, n_groups, topk_groups, topk, route_scale, w13, w13_s, w2, w2_s, idx, w, out,
               workspace, residual, stream):
    if x.dim() != 2 or wg.dim() != 2 or w2.dim() != 3:
        raise ValueError("x and wg must have two dimensions, w13 and w2 three")
    T, d = x.shape
    E, f = wg.shape[0], w2.shape[2]
    dev = _device(x, "x")
    _check(dev, ((x, "x", _BF16, None), (wg, "wg", _BF16, (E, d)), (bias, "bias", _FP32, (E,)),
                 (w13, "w13", _U8, (E + 1, 2 * f, d)), (w13_s, "w13_s", _FP32, (E + 1, 2 * f // 128, d // 128)),
                 (w2, "w2", _U8, (E + 1, d, f)), (w2_s, "w2_s", _FP32, (E + 1, d // 128, f // 128)),
                 (idx, "idx", _I32, (T, topk)), (w, "w", _FP32, (T, topk)), (out, "out", _BF16, (T, d)),
                 (workspace, "workspace", _U8, None), (residual, "residual", _BF16, (T, d))))
    _call(name, _ptr(x), _ptr(wg), _ptr(bias), T, d, f, _lib.RouteParams(E, n_groups, topk_groups, topk, route_scale),
          _ptr(w13), _ptr(w13_s), _ptr(w2), _ptr(w2_s), _ptr(residual), _ptr(idx), _ptr(w), _ptr(out),
          _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream, dev))


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


_dtype = attrgetter("dtype")
_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous


def _grad_arrays(tensors, what, dev):
    """Host arrays (pointers, sizes, types) of a list of gradients, checked.
    Over the list by map: a step's list has tens to hundreds of tensors."""
    try:
        types = array("i", [_GRAD_TYPES[t] for t in map(_dtype, tensors)])
    except KeyError:
        i, t = next((i, t) for i, t in enumerate(tensors) if t.dtype not in _GRAD_TYPES)
        raise ValueError(f"{what} {i} must be float32 or bfloat16, got {t.dtype}") from None
    if set(map(_get_device, tensors)) - {dev}:
        i, t = next((i, t) for i, t in enumerate(tensors) if t.get_device() != dev)
        raise ValueError(f"{what} {i} is on {t.device}, the current device is cuda:{dev}")
    if not all(map(_is_contiguous, tensors)):
        i = next(i for i, t in enumerate(tensors) if not t.is_contiguous())
        raise ValueError(f"{what} {i} must be contiguous")
    return array("Q", map(_data_ptr, tensors)), array("q", map(_numel, tensors)), types


def moe_grad_norm_workspace_bytes(n_tensors):
    return int(_lib.load().moe_grad_norm_workspace_bytes(n_tensors))


def moe_grad_norm(grads, max_norm, norm, coef, workspace, stream=None):
    """norm [1] float32 = L2 norm over every element of ``grads`` (float32 and bfloat16 tensors), coef [1] float32 =
    the factor that clips them to ``max_norm`` (1 where they are within it)."""
    dev = torch.cuda.current_device()
    g, sizes, types = _grad_arrays(grads, "gradient", dev)
    _check(dev, ((norm, "norm", _FP32, (1,)), (coef, "coef", _FP32, (1,)), (workspace, "workspace", _U8, None)))
    _call("moe_grad_norm", g.buffer_info()[0], sizes.buffer_info()[0], types.buffer_info()[0], len(grads), max_norm,
          _ptr(norm), _ptr(coef), _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream, dev))


def moe_grad_scale(grads, coef, outs=None, stream=None):
    """outs[i] = grads[i] * coef, in place without ``outs``."""
    dev = torch.cuda.current_device()
    o = g, sizes, types = _grad_arrays(grads, "gradient", dev)
    if outs is not None and outs is not grads:
        if len(outs) != len(grads):
            raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
        o = _grad_arrays(outs, "output", dev)
        if o[1] != sizes or o[2] != types:
            i = next(i for i in range(len(sizes)) if o[1][i] != sizes[i] or o[2][i] != types[i])
            raise ValueError(f"output {i} must be a {grads[i].dtype} tensor of {sizes[i]} elements")
    _check(dev, ((coef, "coef", _FP32, (1,)),))
    _call("moe_grad_scale", g.buffer_info()[0], o[0].buffer_info()[0], sizes.buffer_info()[0], types.buffer_info()[0],
          len(grads), _ptr(coef), _stream(stream, dev))
