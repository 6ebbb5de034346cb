"""GPU parity of the token sorting and the copies between token and expert order, forward and backward, against the
float64 reference: the sort and the spread rows exactly, the sums within their FP32 rounding errors."""

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import experts as ox
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
I32, F32 = torch.int32, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def np64(t):
    return t.detach().double().cpu().numpy()


def half_step(dt, v):
    """Half a step of the type at values v, subnormals included."""
    f = torch.finfo(dt)
    return np.maximum(f.eps / 2 * np.abs(v), f.smallest_normal * f.eps / 2)


def run_sort(idx, E, guard=3):
    T, k = idx.shape
    o = [torch.full((n + guard,), 77, dtype=I32, device=DEV) for n in (E + 1, T * k, T * k)]
    ws = torch.empty(moe.moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
    moe.moe_sort(torch.from_numpy(idx).to(DEV), E, o[0][:E + 1], o[1][:T * k].view(T, k), o[2][:T * k], ws)
    for t, n in zip(o, (E + 1, T * k, T * k)):
        assert (t[n:] == 77).all()
    return o[0][:E + 1], o[1][:T * k].view(T, k), o[2][:T * k]


def indices(kind, T, k, E, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)      # repeated experts among them
    if kind == "dropped":
        idx[rng.random((T, k)) < 0.3] = -1
        idx.reshape(-1)[rng.integers(0, T * k, 2)] = E      # out of range on the other side
        idx.reshape(-1)[0] = -2 ** 31
    return idx


# one workgroup up to 4096 slots, blocks of 1024 and more beyond; experts of one pass and of several
@pytest.mark.parametrize("kind", ["all", "dropped", "one", "none"])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 3, 7), (64, 8, 256), (512, 8, 33), (513, 8, 256),
                                   (1000, 7, 1024), (4097, 64, 5), (16384, 8, 256), (300001, 1, 300), (3, 2, 2), (512, 8, 1024), (64, 3, 1023)])
def test_sort(kind, T, k, E):
    idx = indices(kind, T, k, E, T + k)
    for got, ref in zip(run_sort(idx, E), ox.sort(idx, E)):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_sort_of_nothing():
    E = 5
    offsets = torch.full((E + 1,), 7, dtype=I32, device=DEV)
    e = torch.empty(0, 2, dtype=I32, device=DEV)
    moe.moe_sort(e, E, offsets, e, torch.empty(0, dtype=I32, device=DEV))
    assert (offsets == 0).all()


class Case:
    """Sorted slots of some experts, a few dropped, and three rows behind the last."""

    def __init__(self, dt, T, k, d, seed=0, drop=0.25, weights=True):
        g = torch.Generator().manual_seed(seed + T + 7 * d + 1000 * k)
        rng = np.random.default_rng(seed)
        self.dt, self.T, self.k, self.d = dt, T, k, d
        idx = rng.integers(0, 5, (T, k)).astype(np.int32)
        idx[rng.random((T, k)) < drop] = -1
        _, pos, _ = ox.sort(idx, 5)
        self.n = int((pos >= 0).sum()) + 3
        pos[(pos == -1) & (rng.random((T, k)) < 0.5)] = self.n     # dropped, past the end
        r = lambda *s: torch.randn(*s, generator=g).to(dt)
        self.pos, self.live = pos, (pos >= 0) & (pos < self.n)
        self.x, self.y, self.res = r(T, d), r(self.n, d), r(T, d)
        self.w = torch.randn(T, k, generator=g) if weights else None
        self.w_np = None if self.w is None else self.w.numpy()
        self.dev = {n: None if v is None else v.to(DEV) for n, v in
                    dict(x=self.x, y=self.y, res=self.res, w=self.w, pos=torch.from_numpy(pos)).items()}

    def expected_rows(self, tok, before):
        """Exactly: the FP32 product rounded once."""
        out = before.clone()
        for t, j, r in ox.slots(self.pos, self.n):
            out[r] = (tok[t].float() * (1.0 if self.w is None else self.w[t, j])).to(self.dt)
        return out

    def check_sum(self, got, rows, residual):
        ref, mag = ox.collect(np64(rows), self.pos, self.w_np, None if residual is None else np64(residual))
        err = (self.k + 1) * U * mag      # a fused product and addition per slot, one addition
        assert np.all(np.abs(np64(got) - ref) <= err + half_step(self.dt, np.abs(ref) + err))

    def check_dots(self, got, tok, rows):
        ref, mag = ox.dots(np64(tok), np64(rows), self.pos)
        # a thread adds at most d/16 + 8 products, then 6 steps over the lanes and at most 8 waves
        assert np.all(np.abs(np64(got) - ref) <= (self.d / 16 + 8 + 6 + 8) * U * mag + U * np.abs(ref))
        assert (got.cpu().numpy()[~self.live] == 0).all()


# every width of a team, rows that are not whole chunks, slots of every kernel and beyond
COPIES = [(1, 1, 1), (5, 2, 7), (9, 3, 8), (33, 4, 9), (3, 5, 100), (7, 8, 128), (4, 6, 257), (11, 8, 1000), (6, 9, 520),
          (5, 17, 2052), (3, 64, 72), (130, 7, 1027), (5, 8, 7168), (2, 6, 8193)]


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,k,d", COPIES)
@pytest.mark.parametrize("weights", [True, False])
def test_dispatch(ty, T, k, d, weights):
    c = Case(TYPES[ty], T, k, d, weights=weights)
    before = torch.full((c.n, d), 7.0, dtype=c.dt)
    rows = before.to(DEV)
    moe.moe_dispatch(c.dev["x"], c.dev["pos"], rows, w=c.dev["w"])
    assert torch.equal(rows.cpu(), c.expected_rows(c.x, before))


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,k,d", COPIES)
@pytest.mark.parametrize("weights", [True, False])
def test_collect_and_dispatch_backward(ty, T, k, d, weights):
    c = Case(TYPES[ty], T, k, d, seed=1, weights=weights)
    for res in (None, c.res):
        out = torch.full((T, d), 7.0, dtype=c.dt, device=DEV)
        moe.moe_collect(c.dev["y"], c.dev["pos"], out, w=c.dev["w"], residual=None if res is None else c.dev["res"])
        c.check_sum(out, c.y, res)
        dx, dw = torch.full_like(out, 7.0), torch.full((T, k), 7.0, device=DEV)
        moe.moe_dispatch_backward(c.dev["y"], c.dev["pos"], dx, w=c.dev["w"], x=c.dev["x"], dw=dw,
                                  residual=None if res is None else c.dev["res"])
        assert torch.equal(dx, out)
        c.check_dots(dw, c.x, c.y)
    inplace = c.dev["res"].clone()
    moe.moe_collect(c.dev["y"], c.dev["pos"], inplace, w=c.dev["w"], residual=inplace)
    assert torch.equal(inplace, out)


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,k,d", COPIES)
@pytest.mark.parametrize("weights", [True, False])
def test_collect_backward(ty, T, k, d, weights):
    c = Case(TYPES[ty], T, k, d, seed=2, weights=weights)
    before = torch.full((c.n, d), 7.0, dtype=c.dt)
    want = c.expected_rows(c.x, before)
    dy, dw = before.to(DEV), torch.full((T, k), 7.0, device=DEV)
    moe.moe_collect_backward(c.dev["x"], c.dev["pos"], dy, w=c.dev["w"], y=c.dev["y"], dw=dw)
    assert torch.equal(dy.cpu(), want)
    c.check_dots(dw, c.x, c.y)
    alone = before.to(DEV)
    moe.moe_collect_backward(c.dev["x"], c.dev["pos"], alone, w=c.dev["w"])
    assert torch.equal(alone, dy)
    over = c.dev["y"].clone()      # over the rows themselves
    dw2 = torch.empty_like(dw)
    moe.moe_collect_backward(c.dev["x"], c.dev["pos"], over, w=c.dev["w"], y=over, dw=dw2)
    assert torch.equal(dw2, dw) and torch.equal(over.cpu(), c.expected_rows(c.x, c.y))


@pytest.mark.parametrize("d", [24, 2056])
def test_dropped_slots_see_no_nan(d):
    """Row 0, which a dropped slot reads in its place, and dropped weights hold NaN and infinities."""
    T, k = 4, 3
    pos = torch.tensor([[0, 1, 2], [3, -1, 4], [-1, -1, -1], [5, 99, 6]], dtype=I32, device=DEV)
    y = torch.randn(8, d, device=DEV, dtype=torch.bfloat16)
    y[0] = float("nan")
    y[7] = float("inf")     # a row that no slot has
    x = torch.randn(T, d, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(T, k, device=DEV)
    w[pos < 0] = float("nan")
    w[3, 1] = float("inf")
    out, dw = torch.empty(T, d, device=DEV, dtype=torch.bfloat16), torch.empty(T, k, device=DEV)
    moe.moe_dispatch_backward(y, pos, out, w=w, x=x, dw=dw)
    assert out[0].isnan().all() and out[1:].isfinite().all() and (out[2] == 0).all()
    assert dw[0, 0].isnan() and dw[0, 1:].isfinite().all() and dw[1:].isfinite().all()
    dw2 = torch.empty(T, k, device=DEV)
    dy = torch.zeros_like(y)
    moe.moe_collect_backward(x, pos, dy, w=w, y=y, dw=dw2)
    assert torch.equal(dw2[1:], dw[1:]) and dy.isfinite().all() and (dy[7] == 0).all()


def test_without_rows():
    T, k, d = 3, 2, 40
    pos = torch.full((T, k), -1, dtype=I32, device=DEV)
    x = torch.randn(T, d, device=DEV)
    none = torch.empty(0, d, device=DEV)
    out, dw = torch.full((T, d), 7.0, device=DEV), torch.full((T, k), 7.0, device=DEV)
    moe.moe_dispatch(x, pos, none)
    moe.moe_collect(none, pos, out, residual=x)
    assert torch.equal(out, x)
    moe.moe_dispatch_backward(none, pos, out, x=x, dw=dw)
    assert (out == 0).all() and (dw == 0).all()
    dw.fill_(7)
    moe.moe_collect_backward(x, pos, none, y=none, dw=dw)
    assert (dw == 0).all()
    empty = torch.empty(0, d, device=DEV)
    e = torch.empty(0, k, dtype=I32, device=DEV)
    moe.moe_dispatch(empty, e, none)
    moe.moe_collect(none, e, empty)


def test_rows_beyond_4_gib():
    T, k, d = 300000, 2, 4096
    pos = torch.randperm(T * k, device=DEV).int().view(T, k)
    pos[-1] = -1
    x, w = torch.randn(T, d, device=DEV).half(), torch.rand(T, k, device=DEV)
    rows = torch.zeros(T * k, d, dtype=torch.float16, device=DEV)
    moe.moe_dispatch(x, pos, rows, w=w)
    at = torch.cat([torch.arange(0, T - 1, 997, device=DEV), torch.arange(T - 9, T - 1, device=DEV)])
    for j in range(k):
        assert torch.equal(rows[pos[at, j].long()], (x[at].float() * w[at, j, None]).half())
    out = torch.empty_like(x)
    moe.moe_collect(rows, pos, out)
    total = sum(rows[pos[at, j].long()].float() for j in range(k))
    assert torch.equal(out[at], total.half()) and not out[-1].any()


def test_gradients_are_differences():
    """dx and dw of out = collect(dispatch(x) * c): both are linear, so a central difference in FP32 is the gradient up to
    rounding."""
    c = Case(torch.float32, 6, 3, 40, seed=5)
    d = c.dev
    dout = torch.randn(c.T, c.d, device=DEV)

    def f(x, w):
        rows, out = torch.zeros(c.n, c.d, device=DEV), torch.empty(c.T, c.d, device=DEV)
        moe.moe_dispatch(x, d["pos"], rows, w=w)
        moe.moe_collect(rows * d["y"], d["pos"], out)
        return (out.double() * dout.double()).sum().item()

    drows, dx, dw = torch.zeros(c.n, c.d, device=DEV), torch.empty(c.T, c.d, device=DEV), torch.empty(c.T, c.k, device=DEV)
    moe.moe_collect_backward(dout, d["pos"], drows)
    moe.moe_dispatch_backward(drows * d["y"], d["pos"], dx, w=d["w"], x=d["x"], dw=dw)
    # f's terms: at most k of d products per token, each rounded a few times; the difference divides by 2 h = 1
    tol = 20 * U * c.T * c.k * c.d * 20
    for t, j in [(0, 0), (3, 1), (5, 2)]:
        w1, w2 = d["w"].clone(), d["w"].clone()
        w1[t, j] += 0.5
        w2[t, j] -= 0.5
        assert abs(f(d["x"], w1) - f(d["x"], w2) - dw[t, j].item()) < tol
        x1, x2 = d["x"].clone(), d["x"].clone()
        x1[t, j] += 0.5
        x2[t, j] -= 0.5
        assert abs(f(x1, d["w"]) - f(x2, d["w"]) - dx[t, j].item()) < tol


def test_replays_and_another_stream():
    """A captured run of the calls, replayed with new inputs between eager work; then all of it on another stream."""
    T, k, E, d = 700, 8, 64, 520
    gen = torch.Generator(device=DEV).manual_seed(3)
    idx = torch.randint(-1, E, (T, k), generator=gen, device=DEV, dtype=I32)
    x, w = torch.randn(T, d, generator=gen, device=DEV, dtype=torch.bfloat16), torch.rand(T, k, generator=gen, device=DEV)
    def buffers():
        return dict(offsets=torch.empty(E + 1, dtype=I32, device=DEV), pos=torch.empty(T, k, dtype=I32, device=DEV),
                    slot=torch.empty(T * k, dtype=I32, device=DEV), rows=torch.zeros(T * k, d, dtype=x.dtype, device=DEV),
                    out=torch.empty(T, d, dtype=x.dtype, device=DEV), dw=torch.empty(T, k, device=DEV),
                    ws=torch.empty(moe.moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV))
    def run(b, stream=None):
        moe.moe_sort(idx, E, b["offsets"], b["pos"], b["slot"], b["ws"], stream=stream)
        moe.moe_dispatch(x, b["pos"], b["rows"], stream=stream)
        moe.moe_collect(b["rows"], b["pos"], b["out"], w=w, stream=stream)
        moe.moe_collect_backward(x, b["pos"], b["rows"], w=w, y=b["rows"], dw=b["dw"], stream=stream)
    b = buffers()
    run(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b)
    for i in range(4):
        idx.copy_(torch.randint(-1, E, (T, k), generator=gen, device=DEV, dtype=I32))
        x.copy_(torch.randn(T, d, generator=gen, device=DEV, dtype=x.dtype))
        b["rows"].zero_()
        graph.replay()
        e = buffers()
        run(e)
        torch.cuda.synchronize()
        for n in ("offsets", "pos", "slot", "rows", "out", "dw"):
            assert torch.equal(b[n], e[n]), (i, n)
    s, o = torch.cuda.Stream(), buffers()
    s.wait_stream(torch.cuda.current_stream())
    run(o, s)
    s.synchronize()
    for n in ("offsets", "pos", "slot", "rows", "out", "dw"):
        assert torch.equal(o[n], e[n]), n


@pytest.mark.parametrize("T,d", [((1 << 28) + 3, 8), (22369700, 1032)])
def test_more_threads_than_a_launch_dimension_takes(T, d):
    """Teams of 16 lanes and of 192 threads, 2^32 threads and some: the tokens in reverse order and back."""
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16).random_(1 << 14)       # finite, positive
    pos = torch.arange(T - 1, -1, -1, dtype=I32, device=DEV).view(T, 1)
    rows = torch.full_like(x, 7.0)
    moe.moe_dispatch(x, pos, rows)
    step = 1 << 20
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        assert torch.equal(rows[T - hi:T - lo].flip(0), x[lo:hi]), lo
    # back, the weights' gradient along: products of a row with itself where one token in many is not zero
    at = torch.tensor([0, 1, T // 2, (1 << 22) * 16 % T, T - 1], device=DEV)
    some = x[at].clone()
    x.zero_()
    x[at] = some
    dx, dw = torch.full_like(x, 7.0), torch.full((T, 1), 7.0, device=DEV)
    moe.moe_dispatch_backward(rows, pos, dx, x=x, dw=dw)
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        assert torch.equal(rows[T - hi:T - lo].flip(0), dx[lo:hi]), lo
    ref = np64(some) ** 2
    assert np.all(np.abs(np64(dw[at, 0]) - ref.sum(1)) <= (d + 16) * U * ref.sum(1))
    dw[at] = 0
    assert not dw.any()
    del x, rows, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
def test_widest_rows(ty):
    """Two tokens of 2^31 - 1 elements, whose last chunk is cut off: there, back, and the weights' gradient."""
    T, d, dt = 2, (1 << 31) - 1, TYPES[ty]
    g = torch.Generator().manual_seed(3)
    at = torch.tensor([0, 9, d // 2, d - 400, d - 9, d - 8, d - 2, d - 1], device=DEV)
    v = torch.randn(T, len(at), generator=g).to(dt)
    x, rows = torch.zeros(T, d, dtype=dt, device=DEV), torch.full((T + 1, d), 7.0, dtype=dt, device=DEV)
    x[:, at] = v.to(DEV)
    pos = torch.tensor([[2], [0]], dtype=I32, device=DEV)
    moe.moe_dispatch(x, pos, rows)
    assert torch.equal(rows[2], x[0]) and torch.equal(rows[0], x[1]) and (rows[1] == 7).all()
    dx, dw = torch.full_like(x, 7.0), torch.full((T, 1), 7.0, device=DEV)
    moe.moe_dispatch_backward(rows, pos, dx, x=x, dw=dw)
    assert torch.equal(dx, x)
    ref = (np64(v) ** 2).sum(1, keepdims=True)
    # zeros add without rounding; eight terms, and the joins of lanes and waves
    assert np.all(np.abs(np64(dw) - ref) <= (8 + 6 + 8) * U * ref)
    del x, rows, dx
    torch.cuda.empty_cache()
