"""The block around the layer, run as a user runs it: norm, layer and residual
in one training step with its backward and clipping; and the decode step, norm
and few-token layer.  Each is the composition of its calls bit for bit, and the
whole agrees with float64."""

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import layer as olayer, norm as onorm
from routing_fp8_grouped_amd import configs, inputs
from tests.gpu_util import DEV, OracleExperts, device_weights, layer_allowance, log, to_np

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def setup(T, scales="fp32", dispatch=False):
    cfg = configs.with_tokens(configs.get("tiny"), T)
    x, wg, b = (t.to(DEV) for t in inputs.host_inputs(cfg))
    g = torch.Generator(device=DEV).manual_seed(T)
    res = torch.randn(T, cfg.d, generator=g, device=DEV).to(BF16)
    wn = (1 + 0.2 * torch.randn(cfg.d, generator=g, device=DEV)).to(BF16)
    W = device_weights(cfg, pow2=scales == "pow2")
    L = moe.MoELayer(T, cfg.d, cfg.E, cfg.G, cfg.M, cfg.k, cfg.f, cfg.route_scale, dispatch=dispatch, scales=scales)
    return cfg, x, wg, b, res, wn, W, L


@pytest.mark.parametrize("T,scales,dispatch", [(1, "fp32", False), (37, "pow2", False), (256, "fp32", True)])
def test_forward_is_its_calls(T, scales, dispatch):
    cfg, x, wg, b, res, wn, W, L = setup(T, scales, dispatch)
    out = L.forward_normed(x, wn, EPS, wg, b, W, residual=res).clone()
    h, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_rmsnorm_quant(x, wn, EPS, y, residual=res, sum_out=h)
    assert torch.equal(L.hsum, h) and torch.equal(L.xn, y)
    R = moe.MoELayer(T, cfg.d, cfg.E, cfg.G, cfg.M, cfg.k, cfg.f, cfg.route_scale, dispatch=dispatch, scales=scales)
    R.forward(y, wg, b, W)
    want = torch.empty_like(x)
    moe.moe_combine(R.y, R.pos, R.w, T * cfg.k, want, residual=h)
    assert torch.equal(out, want) and torch.equal(L.xq, R.xq) and torch.equal(L.idx, R.idx)


def test_forward_against_float64():
    T = 64
    cfg, x, wg, b, res, wn, W, L = setup(T)
    out = to_np(L.forward_normed(x, wn, EPS, wg, b, W, residual=res)).astype(np.float64)
    f = lambda t: t.float().cpu().numpy()
    ref = onorm.rmsnorm(f(x), f(res), f(wn), EPS)
    oe = OracleExperts(cfg)
    oe.prepare(range(cfg.E + 1))
    r = olayer.moe_layer(ref["y"], f(wg), f(b), oe, cfg.G, cfg.M, cfg.k, cfg.route_scale)
    ok = ~r["route"]["near_tie"]
    pos = np.asarray(r["pos"], np.int64)
    routed = np.einsum("tk,tkd->td", r["route"]["w"].astype(np.float64), r["y"][pos].astype(np.float64))
    want = routed + r["y"][T * cfg.k:] + ref["sum"].astype(np.float64)
    allow, _, _ = layer_allowance(r, oe, T, cfg.k, cfg.E)
    # the expert outputs' BF16 rounding on either side of a midpoint, and that of the output
    slack = 2.0 ** -7 * (np.einsum("tk,tkd->td", np.abs(r["route"]["w"]), np.abs(r["y"][pos])) + np.abs(r["y"][T * cfg.k:]))
    assert ok.all() and np.all(np.abs(out - want) <= allow + slack + 2.0 ** -8 * np.abs(want))


def test_training_step():
    """Forward, backward and clipping: each gradient is that of the calls, the clipped ones have the norm asked for."""
    T = 200
    cfg, x, wg, b, res, wn, W, L = setup(T)
    Wt = W.transposed()
    g = torch.Generator(device=DEV).manual_seed(1)
    dout = torch.randn(T, cfg.d, generator=g, device=DEV).to(BF16)
    L.forward_normed(x, wn, EPS, wg, b, W, residual=res, train=True)
    ds, dnorm, dw13, dw2, dgate = (t.clone() for t in L.backward_normed(dout, wn, Wt))

    R = moe.MoELayer(T, cfg.d, cfg.E, cfg.G, cfg.M, cfg.k, cfg.f, cfg.route_scale)
    R.forward(L.xn, wg, b, W, train=True)
    dx, r13, r2, rgate = R.backward(dout, Wt)
    assert torch.equal(dw13, r13) and torch.equal(dw2, r2) and torch.equal(dgate, rgate)
    f = lambda t: t.float().cpu().numpy()
    want, wantw = onorm.rmsnorm_backward(f(dx), f(L.hsum), f(wn), f(L.rstd), f(dout))
    err = np.abs(f(ds) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * np.abs(want).max())
    assert np.allclose(f(dnorm), wantw, rtol=0, atol=2.0 ** -17 * np.abs(wantw).max())

    n, c = onorm.grad_norm([f(dw13), f(dw2), f(dnorm)], 1.0)
    norm = L.clip_grads(1.0, extra=[L.dnorm])
    assert abs(float(norm) - n) <= 2.0 ** -23 * n and c < 1
    for got, raw in ((L.dw13, dw13), (L.dw2, dw2), (L.dnorm, dnorm)):
        assert torch.equal(got, raw * L.grad_coef)
    assert abs(float(L.clip_grads(2.0, extra=[L.dnorm])) - 1.0) <= 2.0 ** -20 and float(L.grad_coef) == 1


@pytest.mark.parametrize("scales", ["fp32", "pow2"])
def test_decode_step(scales):
    """Norm, then the few-token layer with the norm's sum as residual: the prefill path's result on the same tokens up
    to the roundings in which the two differ (the expert outputs' and h's)."""
    T = 7
    cfg, x, wg, b, res, wn, W, L = setup(T, scales)
    want = L.forward_normed(x, wn, EPS, wg, b, W, residual=res).float()
    norm = moe.moe_rmsnorm_quant_pow2 if scales == "pow2" else moe.moe_rmsnorm_quant
    norm(x, wn, EPS, L.xn, residual=res, sum_out=res)     # the residual stream, in place
    idx, w = L.idx.clone(), L.w.clone()
    out = L.forward_few(L.xn, wg, b, W, residual=res)
    assert torch.equal(idx, L.idx) and torch.allclose(w, L.w, rtol=2.0 ** -22, atol=0)
    rel = float((out.float() - want).norm() / want.norm())
    log(f"decode step {scales}: rel {rel:.1e}")
    assert rel < 4e-3       # two BF16 roundings of the sum, half a step of 2^-8 each


def test_decode_step_in_a_graph():
    T = 5
    cfg, x, wg, b, res, wn, W, L = setup(T)
    L.forward_few(x, wg, b, W)     # the workspace
    h, y = torch.empty_like(x), torch.empty_like(x)

    def step():
        moe.moe_rmsnorm_quant(x, wn, EPS, y, residual=res, sum_out=h)
        return L.forward_few(y, wg, b, W, residual=h)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for rep in range(3):
        x.copy_(torch.randn(T, cfg.d, generator=torch.Generator(device=DEV).manual_seed(rep), device=DEV))
        want = step().clone()
        L.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.out, want)


def test_captured_clipping_keeps_its_workspace():
    """A graph that clips goes on using the workspace of its own list's size after an eager call with a longer list
    has needed a larger one."""
    T = 33
    cfg, x, wg, b, res, wn, W, L = setup(T)
    L.dw13 = torch.randn(cfg.E + 1, 2 * cfg.f, cfg.d, device=DEV)
    L.dw2 = torch.randn(cfg.E + 1, cfg.d, cfg.f, device=DEV)
    fresh = [t.clone() for t in (L.dw13, L.dw2)]
    L.clip_grads(1e30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        L.clip_grads(1.0)
    held = {n: t.data_ptr() for n, t in L.grad_ws.items()}
    extra = [torch.randn(50 + i, device=DEV) for i in range(130)]
    for rep in range(3):
        L.clip_grads(1.0, extra=extra)
        assert all(L.grad_ws[n].data_ptr() == p for n, p in held.items()) and len(L.grad_ws) == 2
        other = torch.full((max(held),), 7, dtype=torch.uint8, device=DEV)
        for t, f in zip((L.dw13, L.dw2), fresh):
            t.copy_(f).mul_(rep + 1)
        g.replay()
        torch.cuda.synchronize()
        assert (other == 7).all()
        n, c = onorm.grad_norm([(f.cpu() * (rep + 1)).numpy() for f in fresh], 1.0)
        assert abs(float(L.grad_norm) - n) <= 2.0 ** -23 * n
        assert torch.equal(L.dw13, fresh[0] * (rep + 1) * L.grad_coef)


def test_backward_after_a_decode_step():
    """A few-token pass between a training forward and its backward leaves the gradients as they were."""
    T = 16
    cfg, x, wg, b, res, wn, W, L = setup(T)
    Wt = W.transposed()
    dout = torch.randn(T, cfg.d, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(BF16)
    L.forward_normed(x, wn, EPS, wg, b, W, residual=res, train=True)
    idx, w = L.idx.clone(), L.w.clone()
    want = [t.clone() for t in L.backward_normed(dout, wn, Wt)]
    other = L.forward_few(x.flip(0).contiguous(), wg, b, W).clone()
    assert not torch.equal(L.idx, idx)
    for got, ref in zip(L.backward_normed(dout, wn, Wt), want):
        assert torch.equal(got, ref)
    L.forward(x, wg, b, W)
    assert not torch.equal(L.idx, idx) and torch.equal(L.forward_few(x.flip(0).contiguous(), wg, b, W), other)
    L.forward_normed(x, wn, EPS, wg, b, W, residual=res)
    assert torch.equal(L.idx, idx) and torch.equal(L.w, w)


def test_first_calls_on_a_busy_devices_other_stream():
    """A training step on a stream of its own while the current stream still works on memory that it has let go: the
    buffers that the step makes are none of that memory."""
    T = 200
    cfg, x, wg, b, res, wn, W, L = setup(T)
    Wt = W.transposed()
    dout = torch.randn(T, cfg.d, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(BF16)

    def step(L, stream=None):
        out = L.forward_normed(x, wn, EPS, wg, b, W, residual=res, train=True, stream=stream)
        return [out, *L.backward_normed(dout, wn, Wt, stream=stream), L.clip_grads(1.0, extra=[L.dnorm], stream=stream)]

    want = [t.clone() for t in step(L)]
    L2 = moe.MoELayer(T, cfg.d, cfg.E, cfg.G, cfg.M, cfg.k, cfg.f, cfg.route_scale)
    sizes = [t.numel() * t.element_size() for t in vars(L).values() if isinstance(t, torch.Tensor)]
    big, side = torch.zeros(1 << 26, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(100):
        big.add_(1)
    for n in sizes:
        let_go = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(4)]
        del let_go
    got = step(L2, side)
    side.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_backward_after_a_replayed_forward():
    """The training forward in a graph, other passes of the layer between its replays, the backward eager."""
    T = 96
    cfg, x, wg, b, res, wn, W, L = setup(T)
    Wt = W.transposed()
    dout = torch.randn(T, cfg.d, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(BF16)
    other = x.flip(0).contiguous()
    L.forward_normed(x, wn, EPS, wg, b, W, residual=res, train=True)
    want = [t.clone() for t in L.backward_normed(dout, wn, Wt)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        L.forward_normed(x, wn, EPS, wg, b, W, residual=res, train=True)
    bias = b.clone()
    for _ in range(3):
        L.forward(other, wg, b, W)
        g.replay()
        for got, ref in zip(L.backward_normed(dout, wn, Wt), want):
            assert torch.equal(got, ref)
        L.update_bias(bias, 1e-3)
    torch.cuda.synchronize()
