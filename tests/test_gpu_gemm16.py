"""GPU parity of the 16-bit matrix products and of their gradients against the float64 reference, within the rounding
errors of FP32 sums and of one rounding to the type."""

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import experts as ox
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]
U = 2.0 ** -24
I32, F32 = torch.int32, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def np64(t):
    return t.detach().double().cpu().numpy()


def steps(K):
    """Roundings a product passes on its way through a sum of K: 32 inside one matrix instruction, one for each of the
    K / 32 instructions, and up to 64 joins of partial sums."""
    return 32 + K / 32 + 64


def rounded(dt, ref, err):
    """Bound of a value within err of ref, rounded to the type."""
    f = torch.finfo(dt)
    return err + np.maximum(f.eps / 2 * (np.abs(ref) + err), f.smallest_normal * f.eps / 2)


def offsets_of(sizes):
    return None if sizes is None else np.cumsum([0] + list(sizes)).astype(np.int32)


def to_dev(o):
    return None if o is None else torch.from_numpy(o).to(DEV)


def act_bounds(z, ez, act):
    """(value, error) of the activation of z +- ez: its steepest slope near z, and a few roundings of each factor.  The
    slopes of silu and gelu change by at most 0.8 per unit."""
    v, slopes = ox.act(z, act)
    if act in ("none", "relu"):
        return v, ez
    if act != "swiglu":
        return v, (np.abs(slopes[0]) + 0.8 * ez) * ez + 12 * U * np.abs(v) + 2.0 ** -126
    f = z.shape[1] // 2
    eg, eu, u = ez[:, :f], ez[:, f:], np.abs(z[:, f:])
    return v, (np.abs(slopes[0]) + 0.8 * (u + eu) * eg) * eg + (np.abs(slopes[1]) + 1.1 * eg) * eu + 12 * U * np.abs(v) \
        + 2.0 ** -126


class Product:
    def __init__(self, dt, rows, K, N, sizes=None, seed=0, bias=False, residual=None):
        g = torch.Generator().manual_seed(seed + rows + 3 * K + 5 * N)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dt)
        self.dt, self.rows, self.K, self.N = dt, rows, K, N
        self.G = 1 if sizes is None else len(sizes)
        self.off = offsets_of(sizes)
        self.used = rows if sizes is None else int(self.off[-1])
        self.a, self.b, self.dz = r(rows, K), r(self.G, N, K, scale=K ** -0.5), r(rows, N)
        self.bias = r(self.G, N) if bias else None
        self.res = r(rows, residual) if residual else None
        d = lambda t: None if t is None else t.to(DEV)
        self.dev = dict(a=d(self.a), b=d(self.b), dz=d(self.dz), bias=d(self.bias), res=d(self.res), off=to_dev(self.off))

    def forward(self, act, pre=True, stream=None):
        No = self.N // 2 if act == "swiglu" else self.N
        out = torch.full((self.rows, No), 7.0, dtype=self.dt, device=DEV)
        z = torch.full((self.rows, self.N), 7.0, dtype=self.dt, device=DEV) if pre else None
        n = moe.grouped_gemm16_workspace_bytes(self.rows, self.G, self.K, self.N, act)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        moe.grouped_gemm16(self.dev["a"], self.dev["b"], out, ws, offsets=self.dev["off"], bias=self.dev["bias"], act=act,
                           residual=self.dev["res"], pre=z, stream=stream)
        return out, z

    def check_forward(self, act):
        out, z = self.forward(act)
        zr, mag = ox.gemm(np64(self.a), np64(self.b), self.off, None if self.bias is None else np64(self.bias))
        n = self.used
        zr, ez = zr[:n], (steps(self.K) * U * mag + U * np.abs(zr))[:n]
        assert np.all(np.abs(np64(z)[:n] - zr) <= rounded(self.dt, zr, ez)), "pre"
        v, e = act_bounds(zr, ez, act)
        if self.res is not None:
            v = v + np64(self.res)[:n]
            e = e + U * np.abs(v)
        assert np.all(np.abs(np64(out)[:n] - v) <= rounded(self.dt, v, e)), "out"
        assert (out[n:] == 7).all() and (z[n:] == 7).all()

    def backward(self, stream=None):
        da = torch.full((self.rows, self.K), 7.0, dtype=self.dt, device=DEV)
        db = torch.full((self.G, self.N, self.K), 7.0, device=DEV)
        n = moe.grouped_gemm16_backward_workspace_bytes(self.rows, self.G, self.K, self.N)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        moe.grouped_gemm16_dgrad(self.dev["dz"], self.dev["b"], da, ws, offsets=self.dev["off"], residual=self.dev["res"],
                                 stream=stream)
        moe.grouped_gemm16_wgrad(self.dev["dz"], self.dev["a"], db, ws, offsets=self.dev["off"], stream=stream)
        return da, db

    def check_backward(self):
        da, db = self.backward()
        ref, mag = ox.dgrad(np64(self.dz), np64(self.b), self.off)
        n = self.used
        ref, err = ref[:n], steps(self.N) * U * mag[:n]
        if self.res is not None:
            ref = ref + np64(self.res)[:n]
            err = err + U * np.abs(ref)
        assert np.all(np.abs(np64(da)[:n] - ref) <= rounded(self.dt, ref, err)), "da"
        assert (da[n:] == 7).all()
        ref, mag = ox.wgrad(np64(self.dz), np64(self.a), self.off, self.G)
        most = self.rows if self.off is None else max(np.diff(self.off), default=0)
        assert np.all(np.abs(np64(db) - ref) <= steps(most) * U * mag + U * np.abs(ref)), "db"


# one row to several tiles; K and N below, at and beside the blocks' edges
SHAPES = [(1, 8, 16), (1, 64, 128), (3, 72, 48), (16, 128, 256), (17, 1000, 1008), (64, 200, 80), (65, 136, 528),
          (127, 64, 144), (129, 520, 128), (257, 1024, 272), (300, 8, 2064), (512, 328, 1040)]


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,K,N", SHAPES)
def test_forward(ty, act, rows, K, N):
    Product(TYPES[ty], rows, K, N).check_forward(act)
    Product(TYPES[ty], rows, K, N, seed=1, bias=True, residual=N // 2 if act == "swiglu" else N).check_forward(act)


# no rows in the first, the middle or the last group; rows behind the last; one group of many; many small ones
GROUPS = [[0, 5, 0], [1, 0, 1, 130, 0, 17], [128, 128], [0, 0, 300], [129, 127, 1, 0, 256, 3], [2] * 70, [0] * 9]


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("sizes", GROUPS, ids=str)
@pytest.mark.parametrize("behind", [0, 37])
def test_forward_grouped(ty, act, sizes, behind):
    rows = sum(sizes) + behind
    if rows:
        Product(TYPES[ty], rows, 200, 304, sizes, bias=True).check_forward(act)


# few rows a group on average, but more than 8 or 16 in one of them
@pytest.mark.parametrize("sizes", [[0] * 5 + [12] + [1] * 4, [3] * 7 + [17, 0], [9] + [0] * 11, [0, 40] + [0] * 30 + [2]], ids=str)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_forward_few_uneven(sizes, act):
    Product(torch.bfloat16, sum(sizes) + 1, 520, 272, sizes, bias=True).check_forward(act)


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("rows,K,N", SHAPES)
def test_backward(ty, rows, K, N):
    Product(TYPES[ty], rows, K, N, seed=2).check_backward()
    Product(TYPES[ty], rows, K, N, seed=3, residual=K).check_backward()


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("sizes", GROUPS, ids=str)
@pytest.mark.parametrize("behind", [0, 37])
def test_backward_grouped(ty, sizes, behind):
    rows = sum(sizes) + behind
    if rows:
        Product(TYPES[ty], rows, 200, 304, sizes).check_backward()


@pytest.mark.parametrize("rows,K,N,sizes", [(4100, 2048, 1024, None), (3000, 768, 1536, [1000, 0, 1999, 1]),
                                            (1, 7168, 4096, None), (48, 7168, 512, None), (128, 512, 4096, [3, 40, 0, 85])])
def test_larger(rows, K, N, sizes):
    p = Product(torch.bfloat16, rows, K, N, sizes, bias=True)
    p.check_forward("swiglu")
    p.check_backward()


# products with enough tiles for the kernel's large ones, their rows, columns and K cut off anywhere; sums split into parts
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("rows,K,N,sizes", [(4000, 72, 4040, None), (3990, 200, 4048, [300, 0, 3500, 64, 101, 20])])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_large_tiles_forward(ty, rows, K, N, sizes, act):
    N = 2 * N if act == "swiglu" else N
    Product(TYPES[ty], rows, K, N, sizes, bias=True, residual=N // 2 if act == "swiglu" else N).check_forward(act)


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("rows,K,N,sizes", [(4000, 4040, 72, None), (3990, 4048, 136, [300, 0, 3500, 64, 101, 20]),
                                            (72, 4040, 4000, None), (1, 4096, 4088, None), (5000, 264, 520, None),
                                            (3000, 136, 2056, None), (2000, 1032, 4104, [1500, 0, 490, 10]),
                                            (300, 1496, 1504, [0, 5, 64, 65, 0, 130, 36]), (40, 5376, 5120, None),
                                            (200, 5120, 5384, None)])
def test_large_tiles_and_parts_backward(ty, rows, K, N, sizes):
    Product(TYPES[ty], rows, K, N, sizes).check_backward()


# Few and narrow tiles over a long k; the last four sum it in parts
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("rows,K,N,sizes", [(6000, 3000, 144, None), (5000, 4000, 272, [0, 1900, 0, 3000, 1, 60, 0]),
                                            (4151, 3560, 240, None), (256, 5120, 5120, None),
                                            (4151, 3560, 240, [0, 4000, 151]),
                                            (1200, 4104, 1040, [700, 0, 1, 400])])
def test_forward_long_sums(ty, act, rows, K, N, sizes):
    if (rows, K) in ((4151, 3560), (256, 5120), (1200, 4104)):
        assert moe.grouped_gemm16_workspace_bytes(rows, len(sizes or [0]), K, N, act) > 0
    Product(TYPES[ty], rows, K, N, sizes, bias=True, residual=N // 2 if act == "swiglu" else N).check_forward(act)


def test_operands_beyond_4_gib():
    """Rows on both sides of 2^32 bytes, of the operands and of the results."""
    rows, K, N = 280000, 8192, 16
    at = torch.tensor([0, 1, 262143, 262144, 262145, rows - 1], device=DEV)     # 2^32 bytes are 262144 rows
    a, b = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV), torch.randn(1, N, K, device=DEV).bfloat16()
    a[at] = torch.randn(len(at), K, device=DEV).bfloat16()
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    moe.grouped_gemm16(a, b, out)
    z, mag = ox.gemm(np64(a[at]), np64(b), None, None)
    assert np.all(np.abs(np64(out[at]) - z) <= rounded(torch.bfloat16, z, steps(K) * U * mag))
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not out[rest].any()
    ws = lambda: torch.empty(max(16, moe.grouped_gemm16_backward_workspace_bytes(rows, 1, K, N)), dtype=torch.uint8, device=DEV)
    db = torch.empty(1, N, K, device=DEV)
    dz = torch.randn(rows, N, device=DEV).bfloat16()
    moe.grouped_gemm16_wgrad(dz, a, db, ws())
    ref, mag = ox.wgrad(np64(dz[at]), np64(a[at]), None, 1)
    assert np.all(np.abs(np64(db) - ref) <= steps(rows) * U * mag + U * np.abs(ref))
    moe.grouped_gemm16_dgrad(dz, b, a, ws())
    ref, mag = ox.dgrad(np64(dz[at]), np64(b), None)
    assert np.all(np.abs(np64(a[at]) - ref) <= rounded(torch.bfloat16, ref, steps(N) * U * mag))
    before = a[at]
    moe.grouped_act_backward(a, a, "relu", a)
    assert torch.equal(a[at], before.clamp_min(0))


def test_parts_forward_replayed():
    """The forward in parts, captured, replayed with other rows and group sizes; NaN behind the last row and in one
    group; the residual's own memory as out."""
    rows, K, N, G = 1200, 4104, 1040, 4
    p = Product(torch.bfloat16, rows, K, N, [700, 0, 1, 400], bias=True, residual=N)
    ws = torch.empty(moe.grouped_gemm16_workspace_bytes(rows, G, K, N, "silu"), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    a0, res, out, pre = p.dev["a"].clone(), p.dev["res"].clone(), p.dev["res"].clone(), torch.zeros_like(p.dev["dz"])

    def run(o, z, w):
        moe.grouped_gemm16(p.dev["a"], p.dev["b"], o, w, offsets=p.dev["off"], bias=p.dev["bias"], act="silu",
                           residual=o, pre=z)

    run(out, pre, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, pre, ws)
    for i, sizes in enumerate([[700, 0, 1, 400], [0, 0, 0, 1200], [0, 0, 0, 0], [300, 300, 300, 299], [1, 1, 0, 0]]):
        off = offsets_of(sizes)
        n = int(off[-1])
        p.dev["off"].copy_(torch.from_numpy(off))
        p.dev["a"].copy_(a0.roll(i, 0))
        clean, cz = res.clone(), torch.full_like(pre, 7.0)
        run(clean, cz, torch.empty_like(ws))
        p.dev["a"][n:] = float("nan")
        if sizes[0]:
            p.dev["a"][0] = float("nan")
        out.copy_(res)
        pre.fill_(7.0)
        ws.fill_(255)     # NaN, whichever parts are not written
        graph.replay()
        torch.cuda.synchronize()
        lo = 1 if sizes[0] else 0
        assert torch.equal(out[lo:], clean[lo:]) and torch.equal(pre[lo:], cz[lo:]), i
        assert torch.equal(out[n:], res[n:]) and (pre[n:] == 7).all(), i
        assert not lo or (out[0].isnan().all() and pre[0].isnan().all()), i


@pytest.mark.parametrize("rows,sizes", [(3, [1, 1, 1]), (400, [130, 140, 130]), (40, [13, 14, 13])])
def test_nan_and_infinities_stay_in_their_rows(rows, sizes):
    """Rows, groups and memory behind the last row that hold NaN and infinities reach no other row's results."""
    p = Product(torch.bfloat16, rows + 5, 72, 144, sizes, seed=4)
    clean, _ = p.forward("silu")
    da, db = p.backward()
    lo, hi = int(p.off[1]), int(p.off[2])
    for name in ("a", "dz"):
        t = p.dev[name]
        t[hi - 1] = float("nan")
        t[p.used:] = float("inf")
    p.dev["b"][1, 3] = float("inf")
    got, _ = p.forward("silu")
    keep = torch.ones(rows + 5, dtype=torch.bool)
    keep[lo:hi] = False
    assert torch.equal(got[keep], clean[keep])
    assert got[hi - 1].isnan().all()
    if hi - lo > 1:      # b's infinite row reaches its column only
        cols = [c for c in range(144) if c != 3]
        assert torch.equal(got[lo:hi - 1][:, cols], clean[lo:hi - 1][:, cols])
        assert not got[lo:hi - 1, 3].isfinite().all()
    da2, db2 = p.backward()
    assert torch.equal(da2[keep], da[keep]) and torch.equal(db2[[0, 2]], db[[0, 2]]) and db2[1].isnan().all()


def test_zeros_do_not_hide_beyond_the_end():
    """K that is no whole block: what lies behind a row (the next one, NaN) is not multiplied by the other's zeros."""
    p = Product(torch.float16, 20, 40, 48, [20], seed=6)
    big = torch.full((20, 48), float("nan"), dtype=torch.float16, device=DEV)
    a = torch.full((21, 40), float("nan"), dtype=torch.float16, device=DEV)
    a[:20] = p.dev["a"]
    p.dev["a"] = a[:20]
    out, _ = p.forward("none")
    assert out.isfinite().all() and big.isnan().all()


@pytest.mark.parametrize("kind", ["act", "both"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,N,sizes", [(1, 16, None), (9, 48, None), (700, 1040, None), (333, 2064, [100, 0, 200, 1, 20]),
                                          (5, 64, [0, 0, 3]), (9000, 128, [4000, 0, 4999])])
@pytest.mark.parametrize("ty", TYPES)
def test_act_backward(ty, rows, N, sizes, act, kind):
    dt = TYPES[ty]
    No, off = N // 2 if act == "swiglu" else N, offsets_of(sizes)
    G, used = (1, rows) if off is None else (len(sizes), int(off[-1]))
    g = torch.Generator().manual_seed(rows + N)
    dout, z = torch.randn(rows, No, generator=g).to(dt), (2 * torch.randn(rows, N, generator=g)).to(dt)
    z[0, :8] = torch.tensor([0.0, -0.0, 20, -20, 90, -90, 1e-3, -1e-3]).to(dt)
    dz = torch.full((rows, N), 7.0, dtype=dt, device=DEV)
    db = torch.full((G, N), 7.0, device=DEV)
    ws = torch.empty(moe.grouped_act_backward_workspace_bytes(rows, G, N), dtype=torch.uint8, device=DEV)
    d, zz, o = dout.to(DEV), z.to(DEV), to_dev(off)
    moe.grouped_act_backward(d, zz, act, dz, offsets=o, dbias=db if kind == "both" else None,
                             workspace=ws if kind == "both" else None)
    _, slopes = ox.act(np64(z), act)
    # a slope's error: e (1 + z (1 - e)) and Phi(z) + z phi(z) have terms up to 1 + |z|, each a few roundings
    zn, dn = np64(z), np64(dout)
    ref = np.concatenate([s * dn for s in slopes], 1)
    zh = np.abs(zn[:, :No])
    grow = np.abs(zn[:, No:]) if act == "swiglu" else 1.0
    err = [16 * U * (1 + zh) * grow * np.abs(dn)] + ([16 * U * (1 + zh) * np.abs(dn)] if act == "swiglu" else [])
    err = np.concatenate(err, 1) + 2.0 ** -126 if act not in ("none", "relu") else np.zeros_like(ref)
    n = used
    assert np.all(np.abs(np64(dz) - ref)[:n] <= rounded(dt, ref, err)[:n])
    assert (dz[n:] == 7).all()
    if kind == "both":
        for i, (lo, hi) in enumerate(ox.ranges(off, rows)):
            # a lane adds at most 16 rows, four waves join, then the chunks (64 rows or fewer) one after another
            depth = 16 + 4 + (hi - lo) / 8 + 8
            bound = err[lo:hi].sum(0) + depth * U * (np.abs(ref[lo:hi]) + err[lo:hi]).sum(0)
            assert np.all(np.abs(np64(db)[i] - ref[lo:hi].sum(0)) <= bound)
        only = torch.full((G, N), 7.0, device=DEV)
        moe.grouped_act_backward(d, zz, act, None, offsets=o, dbias=only, workspace=ws)
        assert torch.equal(only, db)
    over = zz.clone()
    moe.grouped_act_backward(d, over, act, over, offsets=o)
    assert torch.equal(over[:n], dz[:n]) and torch.equal(over[n:], zz[n:])


def test_without_rows():
    G, N, K = 3, 32, 24
    db, dbias = torch.full((G, N, K), 7.0, device=DEV), torch.full((G, N), 7.0, device=DEV)
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(G + 1, dtype=I32, device=DEV)
    b = torch.randn(G, N, K, device=DEV).bfloat16()
    moe.grouped_gemm16(e(0, K), b, e(0, N), offsets=off)
    moe.grouped_gemm16_dgrad(e(0, N), b, e(0, K), offsets=off)
    moe.grouped_gemm16_wgrad(e(0, N), e(0, K), db, offsets=off)
    moe.grouped_act_backward(e(0, N), e(0, N), "gelu", e(0, N), offsets=off, dbias=dbias)
    assert (db == 0).all() and (dbias == 0).all()


@pytest.mark.parametrize("rows,K,N,sizes", [(5, 520, 272, None), (700, 520, 272, [300, 0, 399]), (40, 1032, 96, [7, 30, 3])])
def test_in_place_residual_and_same_bits(rows, K, N, sizes):
    p = Product(torch.bfloat16, rows, K, N, sizes, bias=True, residual=N)
    out, pre = p.forward("gelu")
    again, pre2 = p.forward("gelu")
    assert torch.equal(out, again) and torch.equal(pre, pre2)
    p.dev["res"] = p.dev["res"].clone()
    n = moe.grouped_gemm16_workspace_bytes(rows, p.G, K, N, "gelu")
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    moe.grouped_gemm16(p.dev["a"], p.dev["b"], p.dev["res"], ws, offsets=p.dev["off"], bias=p.dev["bias"], act="gelu",
                       residual=p.dev["res"])
    assert torch.equal(p.dev["res"][:p.used], out[:p.used])
    q = Product(torch.bfloat16, rows, K, N, sizes, seed=9, residual=K)
    da, db = q.backward()
    da2, db2 = q.backward()
    assert torch.equal(da, da2) and torch.equal(db, db2)
    moe.grouped_gemm16_dgrad(q.dev["dz"], q.dev["b"], q.dev["res"],
                             torch.empty(max(16, moe.grouped_gemm16_backward_workspace_bytes(rows, q.G, K, N)),
                                         dtype=torch.uint8, device=DEV), offsets=q.dev["off"], residual=q.dev["res"])
    assert torch.equal(q.dev["res"][:q.used], da[:q.used])


@pytest.mark.parametrize("rows", [6, 500])
def test_replays_and_another_stream(rows):
    """A captured forward and backward, replayed with other inputs and group sizes between eager work."""
    K, N, G = 264, 528, 4
    p = Product(torch.bfloat16, rows, K, N, [rows // 2, 0, rows - rows // 2, 0], bias=True)
    gen = torch.Generator(device=DEV).manual_seed(1)
    bufs = {}

    def run(o, stream=None):
        moe.grouped_gemm16(p.dev["a"], p.dev["b"], o["out"], o["ws"], offsets=p.dev["off"], bias=p.dev["bias"],
                           act="swiglu", pre=o["pre"], stream=stream)
        moe.grouped_act_backward(o["out"], o["pre"], "swiglu", o["dz"], offsets=p.dev["off"], dbias=o["dbias"],
                                 workspace=o["ws2"], stream=stream)
        moe.grouped_gemm16_dgrad(o["dz"], p.dev["b"], o["da"], o["ws3"], offsets=p.dev["off"], stream=stream)
        moe.grouped_gemm16_wgrad(o["dz"], p.dev["a"], o["db"], o["ws3"], offsets=p.dev["off"], stream=stream)

    def buffers():
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
        b = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        return dict(out=e(rows, N // 2), pre=e(rows, N), dz=e(rows, N), da=e(rows, K), db=e(G, N, K, dt=F32),
                    dbias=e(G, N, dt=F32), ws=b(moe.grouped_gemm16_workspace_bytes(rows, G, K, N, "swiglu")),
                    ws2=b(moe.grouped_act_backward_workspace_bytes(rows, G, N)),
                    ws3=b(moe.grouped_gemm16_backward_workspace_bytes(rows, G, K, N)))

    o = buffers()
    run(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(o)
    names = ("out", "pre", "dz", "da", "db", "dbias")
    for i, sizes in enumerate([[rows, 0, 0, 0], [0, 1, rows - 1, 0], [rows // 4] * 4, [0, 0, 0, rows]]):
        p.dev["off"].copy_(torch.from_numpy(offsets_of(sizes)))
        p.dev["a"].copy_(torch.randn(rows, K, generator=gen, device=DEV))
        for n in names:
            o[n].zero_()
        graph.replay()
        e = buffers()
        run(e)
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(o[n], e[n]), (i, n)
    s, o2 = torch.cuda.Stream(), buffers()
    s.wait_stream(torch.cuda.current_stream())
    run(o2, s)
    s.synchronize()
    for n in names:
        assert torch.equal(o2[n], e[n]), n


def test_most_rows():
    """The largest number of rows, in groups of which one has almost all: nearly all rows are zeros, so are their results."""
    rows, K, N = (1 << 31) - 1024, 8, 8
    at = torch.tensor([0, 1, 5, rows // 2, rows - 300, rows - 2, rows - 1], device=DEV)
    off = torch.tensor([0, 2, 2, rows], dtype=I32, device=DEV)
    few = Product(torch.bfloat16, len(at), K, N, [2, 0, 5], seed=11)
    a, out = (torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    a[at] = few.dev["a"]

    def check(got, ref, err, name):
        assert np.all(np.abs(np64(got[at]) - ref) <= rounded(torch.bfloat16, ref, err)), name
        got[at] = 0
        assert not got.view(torch.int64).any(), name

    ws = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device=DEV)
    moe.grouped_gemm16(a, few.dev["b"], out, ws(moe.grouped_gemm16_workspace_bytes(rows, 3, K, N)), offsets=off)
    ref, mag = ox.gemm(np64(few.a), np64(few.b), few.off, None)
    check(out, ref, steps(K) * U * mag, "out")
    w = ws(moe.grouped_gemm16_backward_workspace_bytes(rows, 3, K, N))
    db = torch.full((3, N, K), 7.0, device=DEV)
    out[at] = few.dev["dz"]
    moe.grouped_gemm16_wgrad(out, a, db, w, offsets=off)
    ref, mag = ox.wgrad(np64(few.dz), np64(few.a), few.off, 3)
    # zeros add without rounding; the others are at most five terms and their joins
    assert np.all(np.abs(np64(db) - ref) <= steps(5) * U * mag + U * np.abs(ref))
    moe.grouped_gemm16_dgrad(out, few.dev["b"], a, w, offsets=off)
    ref, mag = ox.dgrad(np64(few.dz), np64(few.b), few.off)
    check(a, ref, steps(N) * U * mag, "da")
    del a, out
    torch.cuda.empty_cache()


def test_most_rows_act_backward():
    """The largest number of rows (more chunks than a launch takes, were they of 64 rows): almost all are zeros."""
    rows, N = (1 << 31) - 1024, 8
    at = torch.tensor([0, 1, 5, rows // 2, rows - 300, rows - 2, rows - 1], device=DEV)
    off = torch.tensor([0, 2, 2, rows], dtype=I32, device=DEV)
    dout, z = torch.randn(len(at), N).bfloat16(), torch.randn(len(at), N).bfloat16()
    d, dz = (torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    d[at], dz[at] = dout.to(DEV), z.to(DEV)
    db = torch.full((3, N), 7.0, device=DEV)
    ws = torch.empty(moe.grouped_act_backward_workspace_bytes(rows, 3, N), dtype=torch.uint8, device=DEV)
    moe.grouped_act_backward(d, dz, "silu", dz, offsets=off, dbias=db, workspace=ws)
    _, slopes = ox.act(np64(z), "silu")
    ref = np64(dout) * slopes[0]
    # a slope's error as in test_act_backward; zeros add without rounding
    err = 16 * U * (1 + np.abs(np64(z))) * np.abs(np64(dout)) + 2.0 ** -126
    assert np.all(np.abs(np64(dz[at]) - ref) <= rounded(torch.bfloat16, ref, err))
    for g, part in enumerate((slice(0, 2), slice(0, 0), slice(2, 7))):
        bound = err[part].sum(0) + 8 * U * (np.abs(ref[part]) + err[part]).sum(0)
        assert np.all(np.abs(np64(db)[g] - ref[part].sum(0)) <= bound), g
    dz[at] = 0
    assert not dz.view(torch.int64).any()
    del d, dz
    torch.cuda.empty_cache()
