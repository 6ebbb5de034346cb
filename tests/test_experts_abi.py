"""include/moe_experts.h: every declared symbol is exported and bound, and bad arguments are refused on the host before
anything is enqueued (CPU only)."""

import ctypes
import os
import subprocess

import pytest
import torch

import routing_fp8_grouped_amd as moe
from routing_fp8_grouped_amd import _lib, build

P = ctypes.c_void_p
A, B, C, MIS, MIS4 = P(0x1000000), P(0x9000000), P(0xF000000), P(0x1000004), P(0x1000002)
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def refused(lib, call, table):
    for kw, code, msg in table:
        got = call(**kw)
        said = lib.moe_last_error().decode()
        assert got == code and msg in said, (kw, got, said)


def test_exports_every_declared_symbol(lib):
    declared = _lib.header_symbols(_lib.EXPERTS_HEADER)
    assert len(declared) == 15
    assert not set(declared) & (set(_lib.header_symbols()) | set(_lib.header_symbols(_lib.BLOCK_HEADER)))
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {l.split()[-1] for l in out.splitlines() if " T " in l}
    for name in declared:
        assert name in exported and name in _lib.SIGNATURES and name in moe.__all__, name


def test_header_is_c(tmp_path):
    src = tmp_path / "c.c"
    src.write_text('#include "moe_experts.h"\nint main(void) { return (int)moe_sort_workspace_bytes(0, 0, 0); }\n')
    assert os.path.getsize(build.build_c_program(str(src), str(tmp_path / "c"))) > 0


def test_sort_validation(lib):
    need = lib.moe_sort_workspace_bytes(4096, 8, 64)
    assert need > 0 and lib.moe_sort_workspace_bytes(8, 8, 64) == 0
    for bad in [(0, 8, 64), (-1, 8, 64), (4, 0, 64), (4, 65, 64), (4, 8, 0), (4, 8, 1025), (1 << 30, 2, 4)]:
        assert lib.moe_sort_workspace_bytes(*bad) == 0

    def call(idx=A, T=4096, k=8, E=64, off=B, pos=C, slot=P(0xA000000), ws=P(0xB000000), n=need):
        return lib.moe_sort(idx, T, k, E, off, pos, slot, ws, n, None)

    refused(lib, call, [
        (dict(T=-1), 1, "T=-1"), (dict(k=0), 1, "k=0"), (dict(E=0), 1, "E=0"), (dict(k=65), 2, "k=65"),
        (dict(E=1025), 2, "E=1025"), (dict(T=1 << 30, k=2), 2, "T*k"), (dict(idx=None), 1, "idx is NULL"),
        (dict(off=None), 1, "offsets is NULL"), (dict(pos=MIS4), 1, "pos is not"), (dict(slot=None), 1, "row_slot"),
        (dict(ws=None), 3, "workspace"), (dict(n=need - 1), 3, "workspace"), (dict(ws=MIS4), 3, "workspace"),
        (dict(pos=A), 1, "pos must not"), (dict(off=A), 1, "offsets must not"), (dict(ws=C), 1, "workspace must not")])


@pytest.mark.parametrize("fn", ["moe_dispatch", "moe_collect_backward", "moe_collect", "moe_dispatch_backward"])
def test_copy_validation(lib, fn):
    spread = fn in ("moe_dispatch", "moe_collect_backward")
    grad = fn.endswith("backward")

    def call(type=BF16, src=A, pos=P(0x100), w=None, other=None, res=None, T=4, k=2, d=64, rows=8, out=B, dw=None):
        if fn == "moe_dispatch":
            return lib.moe_dispatch(type, src, pos, w, T, k, d, rows, out, None)
        if fn == "moe_collect_backward":
            return lib.moe_collect_backward(type, src, pos, w, other, T, k, d, rows, out, dw, None)
        if fn == "moe_collect":
            return lib.moe_collect(type, src, pos, w, res, T, k, d, rows, out, None)
        return lib.moe_dispatch_backward(type, src, pos, w, other, res, T, k, d, rows, out, dw, None)

    names = {"moe_dispatch": ("x", "out"), "moe_collect_backward": ("dout", "dy"), "moe_collect": ("y", "out"),
             "moe_dispatch_backward": ("drows", "dx")}[fn]
    refused(lib, call, [
        (dict(type=3), 1, "type=3"), (dict(type=-1), 1, "type"), (dict(T=-1), 1, "T=-1"), (dict(rows=-1), 1, "rows=-1"),
        (dict(k=0), 1, "k=0"), (dict(d=0), 1, "d=0"), (dict(k=65), 2, "k=65"),
        (dict(rows=1 << 30, d=1 << 20), 2, "2^40"), (dict(src=None), 1, names[0]), (dict(src=MIS), 1, names[0]),
        (dict(out=None), 1, names[1]), (dict(out=MIS), 1, names[1]), (dict(pos=None), 1, "pos"), (dict(pos=MIS4), 1, "pos"),
        (dict(w=MIS4), 1, "w is not"), (dict(out=A), 1, f"{names[1]} must not")])
    if grad:
        refused(lib, call, [(dict(other=C), 1, "together"), (dict(dw=C), 1, "together"),
                            (dict(other=MIS, dw=C), 1, "is not"), (dict(other=C, dw=MIS4), 1, "dw"),
                            (dict(other=C, dw=A), 1, "dw must not"), (dict(other=C, dw=B), 1, "must not")])
    if not spread:
        refused(lib, call, [(dict(res=MIS), 1, "residual")])
    assert call(T=0, src=None, out=None, pos=None) == 0


def test_gemm_validation(lib):
    def call(type=BF16, a=A, off=None, G=1, rows=4, K=64, N=64, b=B, bias=None, act=0, res=None, pre=None, out=C, ws=None,
             n=0):
        return lib.grouped_gemm16(type, a, off, G, rows, K, N, b, bias, act, res, pre, out, ws, n, None)

    refused(lib, call, [
        (dict(type=FP32), 2, "MOE_FP32"), (dict(type=5), 1, "type=5"), (dict(act=5), 1, "act=5"), (dict(act=-1), 1, "act"),
        (dict(rows=-1), 1, "rows=-1"), (dict(G=0), 1, "n_groups=0"), (dict(G=2), 1, "offsets is NULL"),
        (dict(K=0), 1, "K=0"), (dict(K=12), 1, "K=12"), (dict(N=4), 1, "N=4"), (dict(N=-8), 1, "N=-8"),
        (dict(N=24, act=4), 1, "N=24"), (dict(G=1025, off=P(0x100)), 2, "n_groups=1025"), (dict(K=(1 << 20) + 8), 2, "2^20"),
        (dict(N=(1 << 20) + 8), 2, "2^20"), (dict(a=None), 1, "a is NULL"), (dict(b=MIS), 1, "b is not"),
        (dict(out=None), 1, "out is NULL"), (dict(bias=MIS), 1, "bias"), (dict(res=MIS), 1, "residual"),
        (dict(pre=MIS), 1, "pre"), (dict(off=MIS4), 1, "offsets"), (dict(out=A), 1, "out must not"),
        (dict(pre=C), 1, "must not"), (dict(pre=B), 1, "pre must not")])
    assert call(rows=0, a=None, b=None, out=None) == 0
    size = lib.grouped_gemm16_workspace_bytes
    for bad in [(0, 1, 64, 64, 0), (-1, 1, 64, 64, 0), (4, 0, 64, 64, 0), (4, 1, 60, 64, 0), (4, 1, 64, 8, 4), (4, 1, 64, 64, 9)]:
        assert size(*bad) == 0


def test_gemm_workspace_validation(lib):
    """Few tiles over a long sum: parts of it, which need the workspace."""
    D = P(0x20000000)
    need = lib.grouped_gemm16_workspace_bytes(256, 1, 5120, 5120, 0)
    assert need >= 2 * 4 * 256 * 5120

    def call(ws=D, n=need, out=C, pre=None, res=None):
        return lib.grouped_gemm16(BF16, A, None, 1, 256, 5120, 5120, B, None, 0, res, pre, out, ws, n, None)

    refused(lib, call, [(dict(ws=None), 3, "workspace"), (dict(n=need - 1), 3, "workspace"),
                        (dict(ws=MIS4), 3, "workspace"), (dict(ws=A), 1, "must not"), (dict(ws=C), 1, "must not"),
                        (dict(pre=D), 1, "must not"), (dict(res=D), 1, "must not")])


def test_gemm_backward_validation(lib):
    def dgrad(type=BF16, dz=A, off=None, G=1, rows=4, K=64, N=64, b=B, res=None, da=C, ws=None, n=0):
        return lib.grouped_gemm16_dgrad(type, dz, off, G, rows, K, N, b, res, da, ws, n, None)

    def wgrad(type=BF16, dz=A, a=B, off=None, G=1, rows=4, K=64, N=64, db=C, ws=None, n=0):
        return lib.grouped_gemm16_wgrad(type, dz, a, off, G, rows, K, N, db, ws, n, None)

    shared = [(dict(type=FP32), 2, "MOE_FP32"), (dict(rows=-1), 1, "rows=-1"), (dict(G=0), 1, "n_groups=0"),
              (dict(G=3), 1, "offsets is NULL"), (dict(K=12), 1, "K=12"), (dict(N=4), 1, "N=4"),
              (dict(N=(1 << 20) + 8), 2, "2^20"), (dict(dz=None), 1, "dz is NULL"), (dict(dz=MIS), 1, "dz is not")]
    refused(lib, dgrad, shared + [(dict(b=None), 1, "b is NULL"), (dict(da=MIS), 1, "da is not"),
                                  (dict(res=MIS), 1, "residual"), (dict(da=B), 1, "da must not")])
    refused(lib, wgrad, shared + [(dict(a=None), 1, "a is NULL"), (dict(db=MIS), 1, "db is not"),
                                  (dict(db=None, rows=0), 1, "db is NULL"), (dict(db=A), 1, "db must not")])
    assert dgrad(rows=0, dz=None, b=None, da=None) == 0


def test_act_backward_validation(lib):
    need = lib.grouped_act_backward_workspace_bytes(100, 1, 64)
    assert need > 0 and lib.grouped_act_backward_workspace_bytes(0, 1, 64) == 0
    assert lib.grouped_act_backward_workspace_bytes(1 << 20, 64, 4096) < 1 << 30

    def call(type=BF16, dout=A, pre=B, off=None, G=1, rows=100, N=64, act=2, dz=C, dbias=None, ws=P(0xA000000), n=need):
        return lib.grouped_act_backward(type, dout, pre, off, G, rows, N, act, dz, dbias, ws, n, None)

    D = P(0xB000000)
    refused(lib, call, [
        (dict(type=FP32), 2, "MOE_FP32"), (dict(act=7), 1, "act=7"), (dict(N=12), 1, "N=12"), (dict(N=8, act=4), 1, "N=8"),
        (dict(G=2), 1, "offsets is NULL"), (dict(dz=None), 1, "no output"), (dict(dout=None), 1, "dout"),
        (dict(pre=None), 1, "pre is NULL"), (dict(dz=MIS), 1, "dz"), (dict(dbias=MIS4), 1, "dbias"),
        (dict(dbias=D, ws=None), 3, "workspace"), (dict(dbias=D, n=need - 1), 3, "workspace"),
        (dict(dbias=C), 1, "must not"), (dict(act=4, dz=A), 1, "dz must not")])


@pytest.mark.parametrize("fn", ["moe_dropout", "moe_dropout_backward"])
def test_dropout_validation(lib, fn):
    def call(type=BF16, x=A, res=None, n=100, p=0.1, rng=P(0x100), out=B):
        if fn == "moe_dropout":
            return lib.moe_dropout(type, x, res, n, p, rng, out, None)
        return lib.moe_dropout_backward(type, x, n, p, rng, out, None)

    names = ("x", "out") if fn == "moe_dropout" else ("dout", "dx")
    refused(lib, call, [
        (dict(type=3), 1, "type=3"), (dict(n=-1), 1, "n=-1"), (dict(p=-0.1), 1, "p="), (dict(p=1.5), 1, "p="),
        (dict(p=float("nan")), 1, "p="), (dict(n=(1 << 40) + 1), 2, "2^40"), (dict(x=None), 1, names[0]),
        (dict(x=MIS), 1, names[0]), (dict(out=None), 1, names[1]), (dict(rng=None), 1, "rng"), (dict(rng=MIS), 1, "rng"),
        (dict(out=P(0x1000010)), 1, f"{names[1]} must not"), (dict(rng=P(0x9000008)), 1, f"{names[1]} must not")])
    if fn == "moe_dropout":
        refused(lib, call, [(dict(res=MIS), 1, "residual")])
    assert call(n=0, x=None, out=None, rng=None) == 0


def test_binding_refuses_before_the_library():
    """Types, shapes and devices are refused with ValueError; none of these tensors is on a GPU."""
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    pos = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_dispatch(x, pos, x)
    with pytest.raises(ValueError, match="dimensions"):
        moe.moe_sort(pos[0], 4, pos, pos, pos)
    with pytest.raises(ValueError, match="dimensions"):
        moe.grouped_gemm16(x, x, x)
    with pytest.raises(ValueError, match="act="):
        moe.grouped_gemm16_workspace_bytes(1, 1, 8, 8, "tanh")
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_dropout(x, 0.1, torch.zeros(2, dtype=torch.int64), x)


def test_in_place_is_the_named_operand_only(lib):
    """An output that is the operand it may be, where another operand lies at the same address: refused, since that one
    is still read (by other rows, columns or turns) when the output is stored."""
    pos, dw = P(0x100), C

    def gemm(a=A, b=B, bias=None, res=A, out=A, act=0, N=64):
        return lib.grouped_gemm16(BF16, a, None, 1, 64, 64, N, b, bias, act, res, None, out, None, 0, None)

    refused(lib, gemm, [(dict(), 1, "out must not share memory with a"), (dict(act=4, N=128), 1, "with a"),
                        (dict(a=C, b=A), 1, "out must not share memory with b"), (dict(a=C, bias=A), 1, "with bias")])

    def dgrad(dz=A, b=B, K=64, N=64):
        return lib.grouped_gemm16_dgrad(BF16, dz, None, 1, 64, K, N, b, A, A, None, 0, None)

    refused(lib, dgrad, [(dict(), 1, "da must not share memory with dz"), (dict(K=128), 1, "with dz"),
                         (dict(dz=C, b=A), 1, "da must not share memory with b")])

    def collect(y=A, w=None, T=8, k=1):
        return lib.moe_collect(FP32, y, pos, w, A, T, k, 64, 8, A, None)

    refused(lib, collect, [(dict(), 1, "out must not share memory with y"), (dict(y=B, w=A), 1, "with w")])

    def dispatch_backward(drows=B, x=A, k=9):
        return lib.moe_dispatch_backward(BF16, drows, pos, None, x, A, 8, k, 64, 8, A, dw, None)

    refused(lib, dispatch_backward, [(dict(), 1, "dx must not share memory with x"), (dict(k=2), 1, "with x"),
                                     (dict(drows=A, x=B), 1, "dx must not share memory with drows")])

    def collect_backward(dout=A, w=None):
        return lib.moe_collect_backward(BF16, dout, pos, w, A, 8, 1, 64, 8, A, dw, None)

    refused(lib, collect_backward, [(dict(), 1, "dy must not share memory with dout"),
                                    (dict(dout=B, w=A), 1, "dy must not share memory with w")])

    def act_backward(dout=A, act=4, N=64):
        return lib.grouped_act_backward(BF16, dout, A, None, 1, 64, N, act, A, None, None, 0, None)

    refused(lib, act_backward, [(dict(), 1, "dz must not share memory with dout")])


def test_most_rows_of_a_product(lib):
    """Rows whose rounding up to a tile would leave 31 bits are refused by every product; one fewer passes this check."""
    most = (1 << 31) - 1024
    off, ws = P(0x100), P(0x10)
    calls = {
        "a is NULL": lambda rows: lib.grouped_gemm16(BF16, None, off, 1024, rows, 8, 8, None, None, 0, None, None, None, None,
                                                     0, None),
        "dz is NULL": lambda rows: lib.grouped_gemm16_dgrad(BF16, None, off, 1024, rows, 8, 8, None, None, None, None, 0, None),
        "a is NULL ": lambda rows: lib.grouped_gemm16_wgrad(BF16, A, None, off, 1024, rows, 8, 8, ws, ws, 0, None),
        "dout is NULL": lambda rows: lib.grouped_act_backward(BF16, None, None, off, 1024, rows, 8, 0, A, None, None, 0, None)}
    for msg, call in calls.items():
        for rows in (most + 1, (1 << 31) - 1):
            assert call(rows) == 2 and f"rows={rows}" in lib.moe_last_error().decode(), (msg, rows)
        assert call(most) == 1 and msg.strip() in lib.moe_last_error().decode(), msg
    for rows in (most + 1, (1 << 31) - 1):
        assert lib.grouped_gemm16_workspace_bytes(rows, 1, 8, 8, 0) == 0
        assert lib.grouped_gemm16_backward_workspace_bytes(rows, 1, 8, 8) == 0
        assert lib.grouped_act_backward_workspace_bytes(rows, 1, 8) == 0
    assert lib.grouped_gemm16_backward_workspace_bytes(most, 1, 8, 8) > 0
