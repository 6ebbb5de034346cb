"""include/moe_block.h: every declared symbol is exported and bound, and bad
arguments are refused on the host before anything is enqueued (CPU only)."""

import ctypes
import os
import subprocess

import pytest
import torch

import routing_fp8_grouped_amd as moe
from routing_fp8_grouped_amd import _lib, build

P = ctypes.c_void_p
A, B, MIS, MIS4 = P(0x100000), P(0x900000), P(0x100004), P(0x100002)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def last(lib):
    return lib.moe_last_error().decode()


def test_exports_every_declared_symbol(lib):
    declared = _lib.header_symbols(_lib.BLOCK_HEADER)
    assert declared and not set(declared) & set(_lib.header_symbols())
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {l.split()[-1] for l in out.splitlines() if " T " in l}
    for name in declared:
        assert name in exported and name in _lib.SIGNATURES and name in moe.__all__, name


def test_header_is_c(tmp_path):
    src = tmp_path / "c.c"
    src.write_text('#include "moe_block.h"\nint main(void) { return (int)moe_rmsnorm_backward_workspace_bytes(0, 0); }\n')
    assert os.path.getsize(build.build_c_program(str(src), str(tmp_path / "c"))) > 0


@pytest.mark.parametrize("fn", ["moe_rmsnorm_quant", "moe_rmsnorm_quant_pow2"])
def test_rmsnorm_validation(lib, fn):
    f = getattr(lib, fn)

    def call(x=A, r=None, w=A, T=4, d=256, eps=1e-6, s=None, y=B, q=None, sc=None, rstd=None):
        return f(x, r, w, T, d, eps, s, y, q, sc, rstd, None)

    for kw, code, msg in [
            (dict(T=-1), 1, "T=-1"), (dict(d=100), 1, "d=100"), (dict(d=0), 1, "d=0"), (dict(d=-128), 1, "d=-128"),
            (dict(d=16512), 2, "d=16512"), (dict(eps=0.0), 1, "eps"), (dict(eps=-1.0), 1, "eps"),
            (dict(eps=float("nan")), 1, "eps"), (dict(eps=float("inf")), 1, "eps"),
            (dict(q=A), 1, "together"), (dict(sc=A), 1, "together"), (dict(y=None), 1, "no output"),
            (dict(x=None), 1, "x is NULL"), (dict(w=None), 1, "weight is NULL"), (dict(x=MIS), 1, "x is not"),
            (dict(r=MIS), 1, "residual"), (dict(s=MIS), 1, "sum"), (dict(y=MIS), 1, "y is not"),
            (dict(q=MIS, sc=A), 1, "q is not"), (dict(q=A, sc=MIS4), 1, "scale"), (dict(rstd=MIS4), 1, "rstd"),
            (dict(y=A), 1, "y must not"), (dict(r=B), 1, "y must not")]:
        assert call(**kw) == code and msg in last(lib), (kw, last(lib))
    assert f(None, None, None, 0, 256, 1e-6, None, None, None, None, None, None) == 0


def test_rmsnorm_backward_validation(lib):
    need = lib.moe_rmsnorm_backward_workspace_bytes(5, 256)
    assert need > 0 and lib.moe_rmsnorm_backward_workspace_bytes(1 << 20, 7168) <= 64 << 20
    for T, d in [(0, 256), (-1, 256), (4, 100), (4, 0), (4, 16512)]:
        assert lib.moe_rmsnorm_backward_workspace_bytes(T, d) == 0

    def call(dy=A, h=A, w=A, rstd=A, dres=None, T=5, d=256, dh=B, dw=A, ws=A, n=need):
        return lib.moe_rmsnorm_backward(dy, h, w, rstd, dres, T, d, dh, dw, ws, n, None)

    for kw, code, msg in [
            (dict(T=-1), 1, "T=-1"), (dict(d=100), 1, "d=100"), (dict(d=16512), 2, "d=16512"),
            (dict(dy=None), 1, "dy is NULL"), (dict(h=MIS), 1, "h is not"), (dict(w=None), 1, "weight"),
            (dict(rstd=None), 1, "rstd"), (dict(dres=MIS), 1, "dres"), (dict(dh=None), 1, "dh is NULL"),
            (dict(dh=A), 1, "dh must not"), (dict(dw=None), 1, "dweight"), (dict(dw=MIS4), 1, "dweight"),
            (dict(ws=None), 3, "workspace"), (dict(ws=MIS), 3, "workspace"), (dict(n=need - 1), 3, "workspace")]:
        assert call(**kw) == code and msg in last(lib), (kw, last(lib))


@pytest.mark.parametrize("fn", ["moe_layer_few", "moe_layer_few_pow2"])
def test_layer_few_validation(lib, fn):
    f = getattr(lib, fn)
    need = lib.moe_layer_few_workspace_bytes(4, 256, 128, 16, 4)
    assert need > 0
    for bad in [(0, 256, 128, 16, 4), (-1, 256, 128, 16, 4), (17, 256, 128, 16, 4), (4, 100, 128, 16, 4),
                (4, 8320, 128, 16, 4), (4, 256, 100, 16, 4), (4, 256, 128, 0, 4), (4, 256, 128, 257, 4),
                (4, 256, 128, 16, 0), (4, 256, 128, 16, 17), (4, 256, 128, 3, 4), (4, 256, 32896, 16, 4)]:
        assert lib.moe_layer_few_workspace_bytes(*bad) == 0, bad

    def call(x=A, wg=A, b=None, T=4, d=256, ff=128, p=(16, 4, 2, 4, 2.5), w13=A, s13=A, w2=A, s2=A, r=None, idx=A,
             w=A, out=B, ws=A, n=need):
        return f(x, wg, b, T, d, ff, _lib.RouteParams(*p), w13, s13, w2, s2, r, idx, w, out, ws, n, None)

    for kw, code, msg in [
            (dict(T=-1), 1, "T=-1"), (dict(T=17), 2, "T=17"), (dict(d=100), 1, "d=100"), (dict(d=0), 1, "d=0"),
            (dict(d=8320), 2, "d=8320"), (dict(ff=64), 1, "f=64"), (dict(ff=32896), 2, "f=32896"),
            (dict(p=(0, 1, 1, 1, 1.0)), 1, "n_experts"), (dict(p=(300, 4, 2, 4, 1.0)), 1, "n_experts"),
            (dict(p=(16, 3, 2, 4, 1.0)), 1, "multiple"), (dict(p=(16, 4, 5, 5, 1.0)), 1, "topk_groups"),
            (dict(p=(16, 4, 2, 3, 1.0)), 1, "multiple"), (dict(p=(64, 1, 1, 17, 1.0)), 2, "topk=17"),
            (dict(p=(16, 4, 2, 4, float("nan"))), 1, "route_scale"),
            (dict(x=None), 1, "x is NULL"), (dict(wg=MIS), 1, "wg"), (dict(b=MIS4), 1, "bias"), (dict(w13=None), 1, "w13"),
            (dict(s13=MIS4), 1, "w13_s"), (dict(w2=MIS), 1, "w2"), (dict(s2=None), 1, "w2_s"), (dict(r=MIS), 1, "residual"),
            (dict(idx=None), 1, "idx"), (dict(w=None), 1, "w is NULL"), (dict(out=MIS), 1, "out"),
            (dict(ws=None), 3, "workspace"), (dict(ws=MIS), 3, "workspace"), (dict(n=need - 1), 3, "workspace")]:
        assert call(**kw) == code and msg in last(lib), (kw, last(lib))
    assert f(None, None, None, 0, 256, 128, _lib.RouteParams(16, 4, 2, 4, 2.5), *[None] * 9, 0, None) == 0


def grads(ptrs, sizes, types):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types), n)


def test_grad_validation(lib):
    need = lib.moe_grad_norm_workspace_bytes(2)
    assert need > 0 and lib.moe_grad_norm_workspace_bytes(0) == 0 and lib.moe_grad_norm_workspace_bytes(-1) == 0
    ok = grads([0x10000, None], [10, 0], [0, 1])

    def norm(g=ok, mx=1.0, out=A, coef=A, ws=A, n=need):
        return lib.moe_grad_norm(*g, mx, out, coef, ws, n, None)

    def scale(g=ok, outs=(0x10000, None), coef=A):
        o = None if outs is None else (ctypes.c_void_p * len(outs))(*outs)
        return lib.moe_grad_scale(g[0], o, *g[1:], coef, None)

    bad_lists = [(grads([0x10000], [-1], [0]), "sizes[0]"), (grads([0x10000], [(1 << 40) + 1], [0]), "sizes[0]"),
                 (grads([0x10000], [1], [2]), "types[0]"), (grads([None], [1], [0]), "grads[0] is NULL"),
                 (grads([0x10002], [1], [0]), "aligned"), (grads([0x10001], [1], [1]), "aligned"),
                 ((None, ok[1], ok[2], 2), "grads"), ((ok[0], None, ok[2], 2), "sizes"),
                 ((ok[0], ok[1], None, 2), "types"), ((ok[0], ok[1], ok[2], -1), "n_tensors")]
    for g, msg in bad_lists:
        assert norm(g=g) == 1 and msg in last(lib), last(lib)
        assert scale(g=g) == 1 and msg in last(lib), last(lib)
    for kw, code, msg in [(dict(mx=0.0), 1, "max_norm"), (dict(mx=-1.0), 1, "max_norm"),
                          (dict(mx=float("nan")), 1, "max_norm"), (dict(out=None), 1, "norm"),
                          (dict(coef=MIS4), 1, "coef"), (dict(ws=None), 3, "workspace"),
                          (dict(ws=MIS), 3, "workspace"), (dict(n=need - 1), 3, "workspace")]:
        assert norm(**kw) == code and msg in last(lib), (kw, last(lib))
    for kw, msg in [(dict(outs=None), "outs"), (dict(outs=(None, None)), "outs[0] is NULL"),
                    (dict(outs=(0x10002, None)), "aligned"), (dict(outs=(0x10010, None)), "overlaps"),
                    (dict(outs=(0xFFF0, None)), "overlaps"), (dict(coef=None), "coef")]:
        assert scale(**kw) == 1 and msg in last(lib), (kw, last(lib))
    twice = grads([0x10000, 0x10000], [10, 10], [0, 0])
    assert scale(g=twice, outs=(0x10000, 0x10000)) == 1 and "two outputs" in last(lib)
    assert lib.moe_grad_scale(None, None, None, None, 0, A, None) == 0


def test_binding_refusals():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.zeros(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_rmsnorm_quant(x, w, 1e-6, x)
    with pytest.raises(ValueError, match="two dimensions"):
        moe.moe_rmsnorm_quant(w, w, 1e-6, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_rmsnorm_backward(x, x, w, w, x, w, w)


def test_overlapping_memory_is_refused(lib):
    """Outputs that share part of an input's or another output's memory; the same operand as a whole where the
    header allows it is tested on the GPU."""
    base, n = 0x100000, 4 * 256 * 2      # bytes of a BF16 operand
    at = lambda off: P(base + off)
    far = [P(0x1000000 * (i + 2)) for i in range(12)]

    def norm(x=at(0), r=None, w=far[0], s=far[1], y=far[2], q=far[3], sc=far[4], rstd=far[5]):
        return lib.moe_rmsnorm_quant(x, r, w, 4, 256, 1e-6, s, y, q, sc, rstd, None)

    for kw, msg in [(dict(s=at(512)), "sum must not share memory with x"), (dict(s=at(-512)), "sum"),
                    (dict(r=far[1], y=far[1]), "y must not"), (dict(r=far[6], s=P(far[6].value + n - 16)), "sum"),
                    (dict(s=far[0]), "weight"), (dict(q=at(n - 16)), "q must not"), (dict(sc=at(n - 4)), "scale must not"),
                    (dict(rstd=far[4]), "rstd must not share memory with scale"), (dict(q=P(far[2].value + 16)), "q must")]:
        assert norm(**kw) == 1 and msg in last(lib), (kw, last(lib))

    need = lib.moe_rmsnorm_backward_workspace_bytes(4, 256)

    def bwd(dy=at(0), h=far[0], dres=None, dh=far[3], dw=far[4], ws=far[5]):
        return lib.moe_rmsnorm_backward(dy, h, far[1], far[2], dres, 4, 256, dh, dw, ws, need, None)

    for kw, msg in [(dict(dh=at(16)), "dh must not"), (dict(dres=far[6], dh=P(far[6].value + 512)), "dres"),
                    (dict(dw=at(0)), "dweight"), (dict(ws=at(-16)), "workspace"), (dict(dw=far[5]), "workspace must not")]:
        assert bwd(**kw) == 1 and msg in last(lib), (kw, last(lib))

    need = lib.moe_layer_few_workspace_bytes(4, 256, 128, 16, 4)

    def few(x=at(0), r=None, idx=far[5], w=far[6], out=far[7], ws=far[8]):
        return lib.moe_layer_few(x, far[0], None, 4, 256, 128, _lib.RouteParams(16, 4, 2, 4, 2.5), far[1], far[2],
                                 far[3], far[4], r, idx, w, out, ws, need, None)

    for kw, msg in [(dict(out=at(512)), "out must not share memory with x"), (dict(r=at(n), out=at(512)), "out"),
                    (dict(idx=far[6]), "w must not share memory with idx"), (dict(ws=at(-16)), "workspace"),
                    (dict(out=far[1]), "w13"), (dict(out=P(far[8].value + need - 16)), "workspace must not")]:
        assert few(**kw) == 1 and msg in last(lib), (kw, last(lib))

    g = grads([0x10000, 0x20000], [8, 8], [0, 1])
    scale = lambda outs, coef=A: lib.moe_grad_scale(g[0], (ctypes.c_void_p * 2)(*outs), *g[1:], coef, None)
    for outs, coef, msg in [((0x20000, 0x30000), A, "grads[1]"), ((0x30000, 0x1001C), A, "grads[0]"),
                            ((0x10000, 0x30000), P(0x3000C), "coef"), ((0x10000, 0x10010), A, "two outputs"),
                            ((0x20008, 0x20000), A, "two outputs"), ((0x30000, 0x30020), P(0x30000), "coef")]:
        assert scale(outs, coef) == 1 and msg in last(lib), (outs, last(lib))
    need = lib.moe_grad_norm_workspace_bytes(2)
    assert lib.moe_grad_norm(*g, 1.0, A, A, B, need, None) == 1 and "coef must not share memory with norm" in last(lib)
    assert lib.moe_grad_norm(*g, 1.0, A, P(B.value + 64), B, need, None) == 1 and "workspace" in last(lib)


def test_workspace_sizes_leave_the_message(lib):
    """Asking for a size is no call that fails: the thread's message stays."""
    assert lib.moe_rmsnorm_quant(None, None, None, -1, 128, 1e-6, *[None] * 6) == 1
    before = last(lib)
    assert "T=-1" in before
    assert lib.moe_layer_few_workspace_bytes(99, 256, 128, 16, 4) == 0 and last(lib) == before
    assert lib.moe_layer_few_workspace_bytes(4, 256, 128, 16, 4) > 0 and last(lib) == before


def test_grad_norm_refuses_outputs_in_the_gradients(lib):
    """norm, coef and the workspace are written while gradients are read: none may share memory with one of them."""
    need = lib.moe_grad_norm_workspace_bytes(3)
    far = [P(0x1000000 * (i + 1)) for i in range(3)]
    g = grads([0x10000, None, 0x20000], [8, 0, 8], [0, 0, 1])       # 32 bytes, none, 16 bytes

    def norm(out=far[0], coef=far[1], ws=far[2], g=g, n=need):
        return lib.moe_grad_norm(*g, 1.0, out, coef, ws, n, None)

    for kw, msg in [(dict(out=P(0x10000)), "norm must not share memory with grads[0]"),
                    (dict(out=P(0x1001C)), "norm must not share memory with grads[0]"),
                    (dict(coef=P(0x2000C)), "coef must not share memory with grads[2]"),
                    (dict(ws=P(0x10018)), "workspace must not share memory with grads[0]"),
                    (dict(ws=P(0x20008)), "workspace must not share memory with grads[2]"),
                    (dict(ws=P(0x20000 + 16 - need)), "workspace must not share memory with grads"),
                    (dict(ws=P(0x10020 - need), coef=P(0x20000)), "coef must not share memory with grads[2]")]:
        assert norm(**kw) == 1 and msg in last(lib), (kw, last(lib))
    # an outer tensor whose parts the outputs are
    whole = grads([0x1000000], [1 << 24], [0])
    assert norm(g=whole, ws=P(0x100), n=1 << 16) == 1 and "norm must not share memory with grads[0]" in last(lib)
