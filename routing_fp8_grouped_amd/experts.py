"""Binding of include/moe_experts.h: tokens sorted by expert and back, matrix products in 16 bits, dropout.

As in ``block``: each function has the name of a C entry point, takes torch tensors on the current GPU and the outputs
and workspace to write, and enqueues on ``stream`` (the current one by default).  Types, shapes, devices and contiguity
are checked here; the library checks the rest.
"""

import torch

from . import _lib
from .block import _BF16, _FP32, _I32, _U8, _call, _check, _device, _ptr, _stream

_TYPES = {_BF16: 0, torch.float16: 1, _FP32: 2}
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}


def _type(t, name):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}") from None


def _act(act):
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"act={act!r} must be one of {', '.join(_ACTS)}") from None


def _dims(t, n, name):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {tuple(t.shape)}")


def _size(workspace):
    return 0 if workspace is None else workspace.numel()


# ---- tokens sorted by expert, and back ----

def moe_sort_workspace_bytes(T, k, E):
    return int(_lib.load().moe_sort_workspace_bytes(T, k, E))


def moe_sort(idx, n_experts, offsets, pos, row_slot, workspace=None, stream=None):
    """Stable order of the slots idx [T, k] int32 by expert (outside [0, n_experts): dropped): offsets [E + 1], pos
    [T, k] (-1 for a dropped slot) and row_slot [T * k] (-1 behind the last row), int32.  ``workspace`` is uint8 of
    moe_sort_workspace_bytes(T, k, E)."""
    _dims(idx, 2, "idx")
    T, k = idx.shape
    dev = _device(idx, "idx")
    _check(dev, ((idx, "idx", _I32, None), (offsets, "offsets", _I32, (n_experts + 1,)), (pos, "pos", _I32, (T, k)),
                 (row_slot, "row_slot", _I32, (T * k,)), (workspace, "workspace", _U8, None)))
    _call("moe_sort", _ptr(idx), T, k, n_experts, _ptr(offsets), _ptr(pos), _ptr(row_slot), _ptr(workspace),
          _size(workspace), _stream(stream, dev))


def _sizes(token, token_name, rows, rows_name, pos):
    """(T, k, d, number of rows, type, device) of a copy between the two orders."""
    if pos.dim() != 2 or token.dim() != 2 or rows.dim() != 2:
        raise ValueError(f"pos, {token_name} and {rows_name} must have two dimensions, got {tuple(pos.shape)}, "
                         f"{tuple(token.shape)} and {tuple(rows.shape)}")
    T, k = pos.shape
    n, d = rows.shape
    return T, k, d, n, token.dtype, _device(pos, "pos")


def moe_dispatch(x, pos, rows, w=None, stream=None):
    """Tokens to their rows: rows[pos[t, j]] = w[t, j] * x[t] (ones without ``w``).  x [T, d] and rows [n, d] bfloat16,
    float16 or float32, pos [T, k] int32 (negative: dropped), w [T, k] float32.  Other rows are left as they were."""
    T, k, d, n, dt, dev = _sizes(x, "x", rows, "rows", pos)
    _check(dev, ((pos, "pos", _I32, None), (x, "x", dt, (T, d)), (rows, "rows", dt, None), (w, "w", _FP32, (T, k))))
    _call("moe_dispatch", _type(x, "x"), _ptr(x), _ptr(pos), _ptr(w), T, k, d, n, _ptr(rows), _stream(stream, dev))


def moe_dispatch_backward(drows, pos, dx, w=None, x=None, dw=None, residual=None, stream=None):
    """dx[t] = sum_j w[t, j] * drows[pos[t, j]] (+ residual[t], whose memory dx may be); with the forward's ``x`` also
    dw [T, k] float32, the gradient of ``w``."""
    T, k, d, n, dt, dev = _sizes(dx, "dx", drows, "drows", pos)
    token = (T, d)
    _check(dev, ((pos, "pos", _I32, None), (dx, "dx", dt, token), (drows, "drows", dt, None), (w, "w", _FP32, (T, k)),
                 (x, "x", dt, token), (dw, "dw", _FP32, (T, k)), (residual, "residual", dt, token)))
    _call("moe_dispatch_backward", _type(dx, "dx"), _ptr(drows), _ptr(pos), _ptr(w), _ptr(x), _ptr(residual), T, k, d, n,
          _ptr(dx), _ptr(dw), _stream(stream, dev))


def moe_collect(y, pos, out, w=None, residual=None, stream=None):
    """Rows back to their tokens: out[t] = sum_j w[t, j] * y[pos[t, j]] (+ residual[t], whose memory out may be)."""
    T, k, d, n, dt, dev = _sizes(out, "out", y, "y", pos)
    token = (T, d)
    _check(dev, ((pos, "pos", _I32, None), (out, "out", dt, token), (y, "y", dt, None), (w, "w", _FP32, (T, k)),
                 (residual, "residual", dt, token)))
    _call("moe_collect", _type(out, "out"), _ptr(y), _ptr(pos), _ptr(w), _ptr(residual), T, k, d, n, _ptr(out),
          _stream(stream, dev))


def moe_collect_backward(dout, pos, dy, w=None, y=None, dw=None, stream=None):
    """dy[pos[t, j]] = w[t, j] * dout[t] (other rows are left; dy may be y's memory); with the forward's ``y`` also dw
    [T, k] float32, the gradient of ``w``."""
    T, k, d, n, dt, dev = _sizes(dout, "dout", dy, "dy", pos)
    _check(dev, ((pos, "pos", _I32, None), (dout, "dout", dt, (T, d)), (dy, "dy", dt, None), (w, "w", _FP32, (T, k)),
                 (y, "y", dt, (n, d)), (dw, "dw", _FP32, (T, k))))
    _call("moe_collect_backward", _type(dout, "dout"), _ptr(dout), _ptr(pos), _ptr(w), _ptr(y), T, k, d, n, _ptr(dy),
          _ptr(dw), _stream(stream, dev))


# ---- matrix products in 16 bits ----

def grouped_gemm16_workspace_bytes(rows, n_groups, K, N, act="none"):
    return int(_lib.load().grouped_gemm16_workspace_bytes(rows, n_groups, K, N, _act(act)))


def grouped_gemm16(a, b, out, workspace=None, offsets=None, bias=None, act="none", residual=None, pre=None,
                   stream=None):
    """out = act(a b[g]^T + bias[g]) + residual for the rows of every group g: a [rows, K], b [G, N, K], bias [G, N],
    out and residual [rows, No] (out may be residual's memory), all bfloat16 or all float16; offsets [G + 1] int32 (None: one
    group of all rows).  act: "none", "relu", "silu", "gelu" or "swiglu" (silu of the first half of the N columns times
    the second: No = N / 2, else N).  ``pre`` [rows, N] receives the activation's argument.  ``workspace`` is uint8 of
    grouped_gemm16_workspace_bytes(rows, G, K, N, act)."""
    _dims(a, 2, "a")
    _dims(b, 3, "b")
    rows, K = a.shape
    G, N, _ = b.shape
    No = N // 2 if act == "swiglu" else N
    dev, dt = _device(a, "a"), a.dtype
    _check(dev, ((a, "a", dt, None), (b, "b", dt, (G, N, K)), (out, "out", dt, (rows, No)),
                 (offsets, "offsets", _I32, (G + 1,)), (bias, "bias", dt, (G, N)),
                 (residual, "residual", dt, (rows, No)), (pre, "pre", dt, (rows, N)),
                 (workspace, "workspace", _U8, None)))
    _call("grouped_gemm16", _type(a, "a"), _ptr(a), _ptr(offsets), G, rows, K, N, _ptr(b), _ptr(bias), _act(act),
          _ptr(residual), _ptr(pre), _ptr(out), _ptr(workspace), _size(workspace), _stream(stream, dev))


def grouped_act_backward_workspace_bytes(rows, n_groups, N):
    return int(_lib.load().grouped_act_backward_workspace_bytes(rows, n_groups, N))


def grouped_act_backward(dout, pre, act, dz, offsets=None, dbias=None, workspace=None, stream=None):
    """dz [rows, N] = dout [rows, No] * act'(pre [rows, N]) (dz may be pre's memory, and dout's where No = N), and dbias
    [G, N] float32 = the sums of each group's rows; either output may be None.  ``pre`` may be None for "none".
    ``workspace``, for dbias, is uint8 of grouped_act_backward_workspace_bytes(rows, G, N)."""
    _dims(dout, 2, "dout")
    rows, No = dout.shape
    N = 2 * No if act == "swiglu" else No
    if offsets is not None:
        _dims(offsets, 1, "offsets")
    G = 1 if offsets is None else offsets.shape[0] - 1
    dev, dt = _device(dout, "dout"), dout.dtype
    _check(dev, ((dout, "dout", dt, None), (pre, "pre", dt, (rows, N)), (dz, "dz", dt, (rows, N)),
                 (offsets, "offsets", _I32, None), (dbias, "dbias", _FP32, (G, N)), (workspace, "workspace", _U8, None)))
    _call("grouped_act_backward", _type(dout, "dout"), _ptr(dout), _ptr(pre), _ptr(offsets), G, rows, N, _act(act),
          _ptr(dz), _ptr(dbias), _ptr(workspace), _size(workspace), _stream(stream, dev))


def grouped_gemm16_backward_workspace_bytes(rows, n_groups, K, N):
    return int(_lib.load().grouped_gemm16_backward_workspace_bytes(rows, n_groups, K, N))


def grouped_gemm16_dgrad(dz, b, da, workspace=None, offsets=None, residual=None, stream=None):
    """da = dz b[g] (+ residual, whose memory da may be): dz [rows, N], b [G, N, K], da [rows, K].  ``workspace`` is
    uint8 of grouped_gemm16_backward_workspace_bytes(rows, G, K, N)."""
    _dims(dz, 2, "dz")
    _dims(b, 3, "b")
    rows, N = dz.shape
    G, _, K = b.shape
    dev, dt = _device(dz, "dz"), dz.dtype
    _check(dev, ((dz, "dz", dt, None), (b, "b", dt, (G, N, K)), (da, "da", dt, (rows, K)),
                 (offsets, "offsets", _I32, (G + 1,)), (residual, "residual", dt, (rows, K)),
                 (workspace, "workspace", _U8, None)))
    _call("grouped_gemm16_dgrad", _type(dz, "dz"), _ptr(dz), _ptr(offsets), G, rows, K, N, _ptr(b), _ptr(residual),
          _ptr(da), _ptr(workspace), _size(workspace), _stream(stream, dev))


def grouped_gemm16_wgrad(dz, a, db, workspace=None, offsets=None, stream=None):
    """db [G, N, K] float32 = dz^T a over each group's rows: dz [rows, N], a [rows, K].  ``workspace`` as for
    grouped_gemm16_dgrad."""
    _dims(dz, 2, "dz")
    _dims(a, 2, "a")
    _dims(db, 3, "db")
    rows, N = dz.shape
    K, G = a.shape[1], db.shape[0]
    dev, dt = _device(dz, "dz"), dz.dtype
    _check(dev, ((dz, "dz", dt, None), (a, "a", dt, (rows, K)), (db, "db", _FP32, (G, N, K)),
                 (offsets, "offsets", _I32, (G + 1,)), (workspace, "workspace", _U8, None)))
    _call("grouped_gemm16_wgrad", _type(dz, "dz"), _ptr(dz), _ptr(a), _ptr(offsets), G, rows, K, N, _ptr(db),
          _ptr(workspace), _size(workspace), _stream(stream, dev))


# ---- dropout ----

def moe_dropout(x, p, rng, out, residual=None, stream=None):
    """out = residual + x / q where the generator keeps x, residual elsewhere (any shape; bfloat16, float16 or float32;
    out may be the memory of x or residual).  q, the probability of keeping, is 1 - p rounded to a multiple of 2^-16.
    rng [2] int64 on the device is {seed, number of the call}, read when the kernel runs."""
    dev, dt, shape = _device(x, "x"), x.dtype, x.shape
    _check(dev, ((x, "x", dt, None), (residual, "residual", dt, shape), (out, "out", dt, shape),
                 (rng, "rng", torch.int64, (2,))))
    _call("moe_dropout", _type(x, "x"), _ptr(x), _ptr(residual), x.numel(), p, _ptr(rng), _ptr(out),
          _stream(stream, dev))


def moe_dropout_backward(dout, p, rng, dx, stream=None):
    """dx = dout / q where the forward kept, 0 elsewhere, with the forward's ``p`` and ``rng``; the residual's gradient is
    dout.  dx may be dout's memory."""
    dev, dt, shape = _device(dout, "dout"), dout.dtype, dout.shape
    _check(dev, ((dout, "dout", dt, None), (dx, "dx", dt, shape), (rng, "rng", torch.int64, (2,))))
    _call("moe_dropout_backward", _type(dout, "dout"), _ptr(dout), dout.numel(), p, _ptr(rng), _ptr(dx),
          _stream(stream, dev))
