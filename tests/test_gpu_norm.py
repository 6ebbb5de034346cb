"""GPU parity of the residual addition + RMS norm + FP8 output and its backward
against the float64 oracle: every forward output bit for bit, the backward
within its FP32 rounding errors."""

import os
import re

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import norm as onorm
from tests.gpu_util import DEV, to_np

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-6
FORMS = {"fp32": moe.moe_rmsnorm_quant, "pow2": moe.moe_rmsnorm_quant_pow2}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def rows(seed, T, d, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(T, d, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    return (v * (1 + 30 * (torch.rand(1, d, generator=g) > 0.99)) * scale).to(BF16)


def weight(seed, d):
    return (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed + 1000))).to(BF16)


def buffers(T, d):
    e = lambda *s, dt: torch.full(s, 7, dtype=dt, device=DEV)
    return dict(sum_out=e(T, d, dt=BF16), y=e(T, d, dt=BF16), q=e(T, d, dt=torch.uint8),
                scale=e(T, d // 128, dt=torch.float32), rstd=e(T, dt=torch.float32))


def check_forward(o, ref):
    for name, key in (("sum_out", "sum"), ("y", "y"), ("scale", "scale"), ("rstd", "rstd"), ("q", "q")):
        if o.get(name) is not None:
            assert np.array_equal(to_np(o[name]), ref[key]), name


# every split of a row: lanes of a wave in part and whole, four chunks per
# lane, workgroups from the narrowest to the widest
WIDTHS = [128, 384, 512, 640, 1152, 2048, 2176, 7168, 16384]


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("T", [1, 5, 67])
def test_forward(form, T, d):
    x, r, w = rows(T + d, T, d), rows(T * d + 3, T, d, 0.5), weight(d, d)
    for res in (r, None):
        o = buffers(T, d)
        FORMS[form](x.to(DEV), w.to(DEV), EPS, residual=None if res is None else res.to(DEV), **o)
        check_forward(o, onorm.rmsnorm(x.float().numpy(), None if res is None else res.float().numpy(),
                                       w.float().numpy(), EPS, form))


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("scale,eps", [(1e30, 1e-6), (1e-30, 1e-6), (1e-30, 1e-30), (1.0, 1e10)])
def test_extreme_magnitudes(form, scale, eps):
    T, d = 3, 256
    x, w = rows(5, T, d, scale), weight(5, d)
    x[1] = 0      # a row without energy
    o = buffers(T, d)
    FORMS[form](x.to(DEV), w.to(DEV), eps, **o)
    check_forward(o, onorm.rmsnorm(x.float().numpy(), None, w.float().numpy(), eps, form))
    assert not o["y"][1].any() and (o["scale"][1] == 1).all() and not o["q"][1].any()


@pytest.mark.parametrize("form", sorted(FORMS))
def test_tiles_with_infinities_and_nan_are_the_quantisers(form):
    """Infinities from a product beyond BF16's range, and a row with a NaN: y's tiles are what the quantiser makes of
    them all the same, and the rows beside them are untouched."""
    T, d = 4, 384
    x, w = rows(11, T, d), weight(11, d)
    w[3], w[200] = 3e38, -3e38
    x[0, 3], x[2, 200] = 50.0, 50.0
    x[3, 7] = float("nan")
    o = buffers(T, d)
    FORMS[form](x.to(DEV), w.to(DEV), EPS, **o)
    assert o["y"][0, 3] == float("inf") and o["y"][2, 200] == -float("inf") and o["y"][3].isnan().all()
    q, s = torch.empty_like(o["q"]), torch.empty_like(o["scale"])
    (moe.fp8_quant_1x128_pow2 if form == "pow2" else moe.fp8_quant_1x128)(o["y"], q, s)
    assert torch.equal(q, o["q"]) and torch.equal(s, o["scale"])
    ref = onorm.rmsnorm(x[1:2].float().numpy(), None, w.float().numpy(), EPS, form)
    assert np.array_equal(to_np(o["y"][1:2]), ref["y"])


@pytest.mark.parametrize("form", sorted(FORMS))
def test_tiles_are_the_quantisers(form):
    T, d = 33, 7168
    x, w = rows(1, T, d).to(DEV), weight(1, d).to(DEV)
    o = buffers(T, d)
    FORMS[form](x, w, EPS, **o)
    q, s = torch.empty_like(o["q"]), torch.empty_like(o["scale"])
    (moe.fp8_quant_1x128 if form == "fp32" else moe.fp8_quant_1x128_pow2)(o["y"], q, s)
    assert torch.equal(q, o["q"]) and torch.equal(s, o["scale"])


def test_each_output_alone():
    T, d = 9, 2176
    x, w, r = rows(2, T, d).to(DEV), weight(2, d).to(DEV), rows(3, T, d).to(DEV)
    full = buffers(T, d)
    moe.moe_rmsnorm_quant(x, w, EPS, residual=r, **full)
    for names in (["y"], ["q", "scale"], ["sum_out"], ["rstd"]):
        o = {n: v for n, v in buffers(T, d).items() if n in names}
        moe.moe_rmsnorm_quant(x, w, EPS, o.pop("y", None), residual=r, **o) if "y" not in names else \
            moe.moe_rmsnorm_quant(x, w, EPS, residual=r, **o)
        for n, v in o.items():
            assert torch.equal(v, full[n]), n


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("d", [256, 7168])
def test_sum_in_place(which, d):
    T = 65
    x, w, r = rows(4, T, d).to(DEV), weight(4, d).to(DEV), rows(6, T, d).to(DEV)
    full = buffers(T, d)
    moe.moe_rmsnorm_quant(x, w, EPS, residual=r, **full)
    x2, r2 = x.clone(), r.clone()
    o = buffers(T, d)
    o["sum_out"] = x2 if which == "x" else r2
    moe.moe_rmsnorm_quant(x2, w, EPS, residual=r2, **o)
    for n in full:
        assert torch.equal(o[n], full[n]), n
    assert torch.equal(x2 if which == "residual" else r2, x if which == "residual" else r)


def test_rows_beyond_are_left():
    T, d = 5, 640
    x, w = rows(7, T, d).to(DEV), weight(7, d).to(DEV)
    o = buffers(T + 2, d)
    moe.moe_rmsnorm_quant(x, w, EPS, **{n: v[:T] for n, v in o.items()})
    for v in o.values():
        assert (v[T:] == 7).all()


def backward_bound(dy, h, w, rstd, ref, adds):
    """FP32 error bound of dh before its BF16 rounding: a few roundings of each term, and c's sum of d terms, at most
    ``adds`` additions deep."""
    dy, h, w = (a.astype(np.float64) for a in (dy, h, w))
    rs = rstd.astype(np.float64)[:, None]
    xh, g = h * rs, dy * w
    c_abs = np.abs(g * xh).mean(1, keepdims=True)
    u = 2.0 ** -24
    fp32 = u * (6 * rs * (np.abs(g) + np.abs(xh) * c_abs) + (adds + 4) * rs * np.abs(xh) * c_abs + 2 * np.abs(ref))
    return fp32 + 2.0 ** -8 * (np.abs(ref) + fp32)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("T", [1, 6, 1029, 4099])
def test_backward(T, d):
    if T * d > 32 << 20:
        T = 300
    h, dy, dres, w = rows(T, T, d), rows(T + 1, T, d, 0.1), rows(T + 2, T, d, 0.1), weight(T, d)
    f = lambda t: t.float().numpy()
    rstd = onorm.rmsnorm(f(h), None, f(w), EPS)["rstd"]
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    for res in (dres, None):
        dh = torch.full((T, d), 7, dtype=BF16, device=DEV)
        dw = torch.full((d,), 7, dtype=torch.float32, device=DEV)
        moe.moe_rmsnorm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), torch.from_numpy(rstd).to(DEV), dh, dw, ws,
                                 dres=None if res is None else res.to(DEV))
        ref, refw = onorm.rmsnorm_backward(f(dy), f(h), f(w), rstd, None if res is None else f(res))
        # per thread at most 32 terms, then 6 steps over the lanes and at most 16 waves
        assert np.all(np.abs(to_np(dh) - ref) <= backward_bound(f(dy), f(h), f(w), rstd, ref, 32 + 6 + 16))
        # a thread's rows one after another (T over the partial sums), four waves joined; two roundings per term
        mag = (np.abs(f(dy).astype(np.float64)) * np.abs(f(h).astype(np.float64) * rstd[:, None])).sum(0)
        per = -(-T // (ws.numel() // (4 * d)))
        assert np.all(np.abs(to_np(dw) - refw) <= 2.0 ** -24 * ((per + 4 + 3) * mag + np.abs(refw)))


def test_backward_in_place_and_repeatable():
    T, d = 513, 7168
    h, dy, dres, w = (t.to(DEV) for t in (rows(1, T, d), rows(2, T, d), rows(3, T, d), weight(4, d)))
    rstd = torch.rand(T, device=DEV) + 0.5
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    dh, dw, dw2 = torch.empty_like(h), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    moe.moe_rmsnorm_backward(dy, h, w, rstd, dh, dw, ws, dres=dres)
    moe.moe_rmsnorm_backward(dy, h, w, rstd, dres, dw2, ws, dres=dres)
    assert torch.equal(dh, dres) and torch.equal(dw, dw2)


def test_no_rows():
    d = 256
    e = buffers(0, d)
    moe.moe_rmsnorm_quant(torch.empty(0, d, dtype=BF16, device=DEV), weight(0, d).to(DEV), EPS, **e)
    dw = torch.full((d,), 7.0, device=DEV)
    z = torch.empty(0, d, dtype=BF16, device=DEV)
    moe.moe_rmsnorm_backward(z, z, weight(0, d).to(DEV), torch.empty(0, device=DEV), z, dw,
                             torch.empty(16, dtype=torch.uint8, device=DEV))
    assert not dw.any()


def test_refusals():
    T, d = 4, 256
    x, w = rows(1, T, d).to(DEV), weight(1, d).to(DEV)
    y = torch.empty_like(x)
    wide = torch.empty(T, 2 * d, dtype=BF16, device=DEV)
    for kw, msg in [(dict(y=y.float()), "y must be"), (dict(y=y[:3]), "y must have shape"),
                    (dict(y=wide[:, :d]), "contiguous"), (dict(y=y.cpu()), "y is on cpu"),
                    (dict(y=y, residual=wide), "residual"), (dict(y=y, rstd=torch.empty(3, device=DEV)), "rstd"),
                    (dict(y=y, q=torch.empty(T, d, dtype=torch.uint8, device=DEV),
                          scale=torch.empty(T, 1, device=DEV)), "scale")]:
        with pytest.raises(ValueError, match=msg):
            moe.moe_rmsnorm_quant(x, w, EPS, **kw)
    with pytest.raises(moe.MoEError, match="eps"):
        moe.moe_rmsnorm_quant(x, w, 0.0, y)
    with pytest.raises(moe.MoEError, match="workspace"):
        moe.moe_rmsnorm_backward(y, x, w, torch.ones(T, device=DEV), torch.empty_like(y), torch.empty(d, device=DEV),
                                 torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("d", [256, 7168])
def test_replays_in_a_graph(d):
    """Forward and backward captured together; every replay, with new inputs and eager work on another stream in
    between, gives the eager result."""
    T = 130
    x, w, r = rows(1, T, d).to(DEV), weight(1, d).to(DEV), rows(2, T, d).to(DEV)
    o = buffers(T, d)
    dh, dw = torch.empty_like(x), torch.empty(d, device=DEV)
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)

    def step(o, dh, dw, ws):
        moe.moe_rmsnorm_quant(x, w, EPS, residual=r, **o)
        moe.moe_rmsnorm_backward(o["y"], o["sum_out"], w, o["rstd"], dh, dw, ws, dres=r)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(o, dh, dw, ws)
    o2, dh2, dw2, ws2 = buffers(T, d), torch.empty_like(x), torch.empty(d, device=DEV), torch.empty_like(ws)
    for rep in range(3):
        x.copy_(rows(10 + rep, T, d))
        step(o2, dh2, dw2, ws2)
        g.replay()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(o[n], o2[n]), n
        assert torch.equal(dh, dh2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,d", [(44000, 512), (9001, 2560), (3001, 7168)])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_large_batches_are_their_parts(form, T, d):
    """A call that moves more than the caches hold gives each row what a small call gives it, in place too; the
    backward's dh likewise, and its dw the sum of the parts'."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x, r = (torch.randn(T, d, generator=g, device=DEV).to(BF16) for _ in range(2))
    w = weight(d, d).to(DEV)
    o, keep = buffers(T, d), r.clone()
    o["sum_out"] = r      # in place of the residual
    FORMS[form](x, w, EPS, residual=r, **o)
    n = 1000
    dh, dw = torch.empty_like(x), torch.empty(d, device=DEV)
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    moe.moe_rmsnorm_backward(o["y"], r, w, o["rstd"], dh, dw, ws, dres=x)
    total, mag, dw1 = torch.zeros(d, dtype=torch.float64, device=DEV), torch.zeros(d, device=DEV), torch.empty(d, device=DEV)
    for a in range(0, T, n):
        b = min(T, a + n)
        p = buffers(b - a, d)
        FORMS[form](x[a:b], w, EPS, residual=keep[a:b], **p)
        for name in p:
            assert torch.equal(p[name], o[name][a:b]), name
        dh1 = torch.empty_like(p["y"])
        moe.moe_rmsnorm_backward(p["y"], p["sum_out"], w, p["rstd"], dh1, dw1, ws, dres=x[a:b])
        assert torch.equal(dh1, dh[a:b])
        total += dw1
        mag += (p["y"].float() * p["sum_out"].float() * p["rstd"][:, None]).abs().sum(0)
    # both sides: rows one after another in FP32 (at most T over the partial sums, four waves joined), two roundings a term
    per = -(-T // (ws.numel() // (4 * d)))
    assert ((dw.double() - total).abs() <= 2.0 ** -24 * (2 * (per + 4 + 3) * 1.001 * mag.double() + 2 * total.abs() + mag)).all()


# every split of a row whose data goes past the caches, forward and backward: a wave with one chunk a lane and with
# four, a workgroup of up to 512 threads and beyond
@pytest.mark.parametrize("T,d", [(44000, 512), (20000, 1152), (12500, 2048), (3200, 7168), (1400, 16384)])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_past_the_caches(form, T, d):
    src = open(os.path.join(os.path.dirname(moe.__file__), "csrc", "norm.hip")).read()
    forward, backward = (int(re.search(rf"{name} = size_t\((\d+)\) << 20;", src)[1]) << 20
                         for name in ("kForwardCached", "kBackwardCached"))
    assert 9 * T * d > forward and 8 * T * d > backward
    assert 9 * 1000 * d < forward     # the parts' go through them
    test_large_batches_are_their_parts(form, T, d)
