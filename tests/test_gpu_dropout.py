"""GPU parity of dropout with the residual addition and of its backward: the generator's values exactly, the results
exactly as FP32 arithmetic rounded once."""

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import experts as ox
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def rng_of(seed, call):
    return torch.tensor([seed, call], dtype=torch.int64, device=DEV)


def expected(x, res, p, seed, call):
    """FP64 sum of the FP32-scaled value: one rounding to the type (the FP32 rounding before it is in the tolerance)."""
    keep, q = ox.keep(x.numel(), p, seed, call)
    v = np.where(keep, x.double().numpy().reshape(-1) * float(np.float32(1 / q if q else 0)), 0.0)
    return v + (0 if res is None else res.double().numpy().reshape(-1)), keep


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 40001])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(ty, n, p):
    dt = TYPES[ty]
    g = torch.Generator().manual_seed(n)
    x, res = torch.randn(n, generator=g).to(dt), torch.randn(n, generator=g).to(dt)
    seed, call = 0x1234567890ABCDEF + n, (n << 33) + 5
    f = torch.finfo(dt)
    for r in (None, res):
        out = torch.full((n + 5,), 7.0, dtype=dt, device=DEV)
        moe.moe_dropout(x.to(DEV), p, rng_of(seed, call), out[:n], residual=None if r is None else r.to(DEV))
        ref, keep = expected(x, r, p, seed, call)
        got = out[:n].double().cpu().numpy()
        # one FP32 rounding, one to the type
        assert np.all(np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + f.eps / 2 * np.abs(ref) * (1 + 2.0 ** -23)
                      + f.smallest_normal * f.eps)
        if r is None:
            assert np.array_equal(got == 0, ~keep | (x.double().numpy() == 0))
            dx = torch.empty(n, dtype=dt, device=DEV)
            moe.moe_dropout_backward(x.to(DEV), p, rng_of(seed, call), dx)
            assert torch.equal(dx, out[:n])
        else:
            assert np.array_equal(got[~keep], r.double().numpy()[~keep])
            for which in (0, 1):      # in place
                a, b = x.to(DEV), r.to(DEV)
                o = (a, b)[which]
                moe.moe_dropout(a, p, rng_of(seed, call), o, residual=b)
                assert torch.equal(o, out[:n])
        assert (out[n:] == 7).all()


def test_negative_seed_and_call():
    n, seed, call = 100, -3, -(1 << 40)
    x = torch.ones(n)
    out = torch.empty(n, device=DEV)
    moe.moe_dropout(x.to(DEV), 0.5, rng_of(seed, call), out)
    keep, _ = ox.keep(n, 0.5, seed & (2 ** 64 - 1), call & (2 ** 64 - 1))
    assert np.array_equal(out.cpu().numpy() != 0, keep)


def test_dropped_elements_hide_nan():
    n = 4096
    x, res = torch.full((n,), float("nan"), device=DEV, dtype=torch.float16), torch.ones(n, device=DEV, dtype=torch.float16)
    out = torch.empty_like(x)
    moe.moe_dropout(x, 0.5, rng_of(1, 2), out, residual=res)
    keep, _ = ox.keep(n, 0.5, 1, 2)
    assert np.array_equal(out.isnan().cpu().numpy(), keep) and (out[torch.from_numpy(~keep).to(DEV)] == 1).all()


def test_positions_beyond_32_bits():
    """The last elements of a tensor of more than 2^32 elements."""
    n = (1 << 32) + 19
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    moe.moe_dropout(x, 0.5, rng_of(11, 3), x)
    for first, last in ((0, 64), ((1 << 32) - 9, n)):
        keep, _ = ox.keep(last, 0.5, 11, 3, first=first)
        assert np.array_equal(x[first:last].float().cpu().numpy(), np.where(keep, 2.0, 0.0))


def test_replays_follow_the_generator():
    """A captured call drops other elements once rng was changed, the same ones while it was not."""
    n = 100000
    x, rng, out = torch.randn(n, device=DEV), rng_of(5, 0), torch.empty(n, device=DEV)
    moe.moe_dropout(x, 0.25, rng, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_dropout(x, 0.25, rng, out)
    seen = []
    for call in (0, 1, 1, 2):
        rng[1] = call
        graph.replay()
        eager = torch.empty_like(out)
        moe.moe_dropout(x, 0.25, rng_of(5, call), eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        seen.append(out.clone())
    assert torch.equal(seen[1], seen[2]) and not torch.equal(seen[0], seen[1]) and not torch.equal(seen[2], seen[3])


def test_another_stream():
    x, s = torch.randn(5001, device=DEV), torch.cuda.Stream()
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_dropout(x, 0.25, rng_of(5, 0), a)
    r = rng_of(5, 0)
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_dropout(x, 0.25, r, b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_more_threads_than_a_launch_dimension_takes():
    """2^35 elements and some (2^32 threads of eight): windows of the front, of the middle and of the end."""
    n = (1 << 35) + 19
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    moe.moe_dropout(x, 0.5, rng_of(11, 3), x)
    for first, last in ((0, 64), ((1 << 33) - 9, (1 << 33) + 9), ((1 << 34) - 9, (1 << 34) + 9), ((1 << 35) - 9, n)):
        keep, _ = ox.keep(last, 0.5, 11, 3, first=first)
        assert np.array_equal(x[first:last].float().cpu().numpy(), np.where(keep, 2.0, 0.0)), first
    # half of the elements are kept: within five deviations of a binomial count
    kept = sum(int((part != 0).sum()) for part in x.split(1 << 32))
    assert abs(kept - n / 2) < 5 * (n / 4) ** 0.5
    del x
    torch.cuda.empty_cache()
