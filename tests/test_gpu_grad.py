"""GPU parity of the global gradient norm and the scaling against float64."""

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import norm as onorm
from tests.gpu_util import DEV, to_np

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def tensors(sizes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(BF16 if i % 3 == 1 else FP32).to(DEV)
            for i, n in enumerate(sizes)]


def norm_of(ts, max_norm, ws=None):
    if ws is None:
        ws = torch.empty(moe.moe_grad_norm_workspace_bytes(len(ts)), dtype=torch.uint8, device=DEV)
    norm, coef = torch.full((1,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    moe.moe_grad_norm(ts, max_norm, norm, coef, ws)
    return norm, coef


def check_norm(ts, max_norm):
    norm, coef = norm_of(ts, max_norm)
    n, c = onorm.grad_norm([to_np(t) for t in ts], max_norm)
    # one rounding to FP32 each (half a step), and 2^-40 for the order of 64-bit sums
    assert abs(float(norm) - n) <= (2.0 ** -24 + 2.0 ** -40) * n
    assert abs(float(coef) - c) <= (2.0 ** -24 + 2.0 ** -40) * c and (c != 1.0 or float(coef) == 1.0)
    return norm, coef


SETS = {"one": [1], "single_empty": [0], "small": [3, 0, 7, 1, 128], "chunk_edges": [8191, 8192, 8193, 16384, 16385],
        "odd": [1000003, 5, 70001, 0, 4097], "many": [(i * 7919) % 5000 for i in range(200)],
        "batch_edge": [17] * 64, "batch_over": [17] * 65, "empties": [0] * 130}


@pytest.mark.parametrize("name", sorted(SETS))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_norm_and_scale(name, max_norm):
    ts = tensors(SETS[name], seed=len(name))
    norm, coef = check_norm(ts, max_norm)
    outs = [torch.full_like(t, 7) for t in ts]
    moe.moe_grad_scale(ts, coef, outs)
    want = [(t.float() * coef).to(t.dtype) for t in ts]
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    moe.moe_grad_scale(ts, coef)
    for t, w in zip(ts, want):
        assert torch.equal(t, w)
    again = norm_of(outs, max_norm)[0]
    assert float(again) <= max(max_norm, 0) * 1.01 or name in ("single_empty", "empties")


def test_empty_list():
    norm, coef = norm_of([], 1.0, torch.empty(0, dtype=torch.uint8, device=DEV))
    assert float(norm) == 0 and float(coef) == 1
    moe.moe_grad_scale([], coef)


@pytest.mark.parametrize("dt", [FP32, BF16])
@pytest.mark.parametrize("shift", [(0, 1), (1, 1), (3, 2), (2, 3)])
def test_views_at_any_element(dt, shift):
    """Tensors that start between two 16-byte boundaries, source and output at different ones, with guards around."""
    n = 9001
    a = torch.randn(n + 16, device=DEV).to(dt)
    b = torch.full((n + 16,), 7.0, device=DEV).to(dt)
    src, out = a[shift[0]:shift[0] + n], b[shift[1]:shift[1] + n]
    norm, coef = check_norm([src], 3.0)
    moe.moe_grad_scale([src], coef, [out])
    assert torch.equal(out, (src.float() * coef).to(dt))
    assert (b[:shift[1]] == 7).all() and (b[shift[1] + n:] == 7).all()


@pytest.mark.parametrize("scale", [1e-30, 1e25])
def test_squares_beyond_fp32(scale):
    check_norm(tensors([5000, 300], scale=scale), 1.0)


def test_infinities_and_nan():
    for bad, n_ok, c_ok in ((float("inf"), lambda v: v == float("inf"), lambda v: v == 0),
                            (float("nan"), lambda v: v != v, lambda v: v != v)):
        ts = tensors([1000, 10])
        ts[0][17] = bad
        norm, coef = norm_of(ts, 1.0)
        assert n_ok(float(norm)) and c_ok(float(coef))
        moe.moe_grad_scale(ts, coef)
        assert torch.isnan(ts[0][17])
        assert torch.isnan(ts[1]).all() if bad != bad else not ts[1].any()


def test_below_the_limit_nothing_is_written():
    ts = tensors([4096, 3, 999], scale=1e-4)
    was = [t.clone() for t in ts]
    coef = norm_of(ts, 1.0)[1]
    assert float(coef) == 1
    moe.moe_grad_scale(ts, coef)
    for t, w in zip(ts, was):
        assert torch.equal(t, w)


def test_more_elements_than_32_bits():
    """One tensor of 2^32 + 5 BF16 elements: its last ones count and are scaled."""
    n = (1 << 32) + 5
    t = torch.zeros(n, dtype=BF16, device=DEV)
    t[0], t[-1], t[1 << 31] = 3.0, 4.0, 12.0
    norm, coef = norm_of([t], 6.5)
    assert float(norm) == 13.0 and float(coef) == 0.5
    moe.moe_grad_scale([t], coef)
    assert float(t[0]) == 1.5 and float(t[-1]) == 2.0 and float(t[1 << 31]) == 6.0
    assert int(torch.count_nonzero(t[-1000:])) == 1


def test_repeatable_and_in_a_graph():
    ts = tensors([300001, 77, 8192 * 5, 0], seed=3)
    outs = [torch.empty_like(t) for t in ts]
    ws = torch.empty(moe.moe_grad_norm_workspace_bytes(len(ts)), dtype=torch.uint8, device=DEV)
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        moe.moe_grad_norm(ts, 1.0, norm, coef, ws)
        moe.moe_grad_scale(ts, coef, outs)
    for rep in range(3):
        for t in ts:
            t.mul_(0.5).add_(0.01)
        n2, c2 = norm_of(ts, 1.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, n2) and torch.equal(coef, c2)
        for t, o in zip(ts, outs):
            assert torch.equal(o, (t.float() * c2).to(t.dtype))


def test_refusals():
    ts = tensors([10, 10])
    coef = torch.ones(1, device=DEV)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="gradient 0"):
        moe.moe_grad_norm([ts[0].half()], 1.0, coef, coef.clone(), ws)
    with pytest.raises(ValueError, match="gradient 1"):
        moe.moe_grad_norm([ts[0], ts[1].cpu()], 1.0, coef, coef.clone(), ws)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_grad_norm([ts[0][::2]], 1.0, coef, coef.clone(), ws)
    with pytest.raises(ValueError, match="norm must"):
        moe.moe_grad_norm(ts, 1.0, coef.double(), coef, ws)
    with pytest.raises(moe.MoEError, match="max_norm"):
        moe.moe_grad_norm(ts, 0.0, coef, coef.clone(), ws)
    with pytest.raises(moe.MoEError, match="workspace"):
        moe.moe_grad_norm(ts, 1.0, coef, coef.clone(), ws[:8])
    with pytest.raises(ValueError, match="outputs for"):
        moe.moe_grad_scale(ts, coef, ts[:1])
    with pytest.raises(ValueError, match="output 0"):
        moe.moe_grad_scale(ts, coef, [ts[0].double(), ts[1]])
    with pytest.raises(moe.MoEError, match="two outputs"):
        moe.moe_grad_scale([ts[0], ts[0]], coef)
    with pytest.raises(moe.MoEError, match="in part"):
        a = torch.zeros(20, device=DEV)
        moe.moe_grad_scale([a[:10]], coef, [a[4:14]])


def test_a_list_past_the_caches():
    """More than 256 MB of both types, tensors that start between 16-byte boundaries among them: the norm in 64 bits,
    the scaling out of place and in place."""
    g = torch.Generator(device=DEV).manual_seed(5)
    ts = [torch.randn(n + 3, generator=g, device=DEV)[o:o + n].to(dt) for n, o, dt in
          ((60_000_001, 0, FP32), (9, 1, FP32), (30_000_000, 0, BF16))]
    whole = torch.randn(10_000_008, generator=g, device=DEV)
    ts.append(whole[1:10_000_002])
    assert sum(t.numel() * t.element_size() for t in ts) > 1 << 28 and ts[-1].data_ptr() % 16 == 4
    n = float(torch.stack([t.double().square().sum() for t in ts]).sum().sqrt())
    norm, coef = norm_of(ts, 2.5)
    # one rounding to FP32 each (half a step), and 2^-40 for the order of 64-bit sums
    assert abs(float(norm) - n) <= (2.0 ** -24 + 2.0 ** -40) * n
    assert abs(float(coef) - 2.5 / n) <= (2.0 ** -24 + 2.0 ** -40) * 2.5 / n
    want = [(t.float() * coef).to(t.dtype) for t in ts]
    ends = whole[0].clone(), whole[10_000_002:].clone()
    outs = [torch.full_like(t, 7) for t in ts]
    moe.moe_grad_scale(ts, coef, outs)
    moe.moe_grad_scale(ts, coef)
    for t, o, w in zip(ts, outs, want):
        assert torch.equal(o, w) and torch.equal(t, w)
    assert torch.equal(whole[0], ends[0]) and torch.equal(whole[10_000_002:], ends[1])


def test_a_factor_of_one_writes_nothing_in_place():
    """Shown on NaNs whose bits a product with 1 would change: BF16 results have one NaN, FP32 products quiet ones."""
    b = torch.tensor([0x7FA5, -1, 0x3F80, 0x7FFF] * 3000, dtype=torch.int16, device=DEV)
    f = torch.tensor([0x7FA00001, 0x3F800000, 0x7F800001] * 3001, dtype=torch.int32, device=DEV)
    ts = [b.clone().view(BF16), f.clone().view(FP32)]
    one = torch.ones(1, device=DEV)
    moe.moe_grad_scale(ts, one)
    assert torch.equal(ts[0].view(torch.int16), b) and torch.equal(ts[1].view(torch.int32), f)
    outs = [torch.empty_like(t) for t in ts]
    moe.moe_grad_scale(ts, one, outs)
    assert not torch.equal(outs[0].view(torch.int16), b)
