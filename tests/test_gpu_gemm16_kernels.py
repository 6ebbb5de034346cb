"""GPU tests of the 16-bit products kernel by kernel: every form that the forward may take, seen to be taken; NaN and
infinities beside the operands and in other groups; very many groups; a group's matrix above 2 GiB."""

import re

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import experts as ox
from tests.gpu_util import DEV
from tests.test_gpu_gemm16 import TYPES, U, Product, act_bounds, np64, rounded, steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def kernels(call):
    """Short names of the products' kernels that a call launches: slimRxC (rows and weight rows of a tile in sixteens, 8x1
    the one for eight rows), tileRxC (rows and columns), the latter with a p where it sums a part of K."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    names = [e.name for e in p.events()]
    if not any("kernel" in n for n in names):
        pytest.skip("the profiler reports no kernels here")
    found = []
    for n in names:
        s = re.search(r"slim_kernel<[^,]+, \w+, (\d+), (\d+), \d+, (\d+)>", n)
        t = re.search(r"gemm16_kernel<[^,]+, .*?(\d+), (\d+), (\d+), \d+, \d+>", n)
        if s:
            found.append("slim8x1" if s[3] == "8" else f"slim{s[1]}x{s[2]}")
        if t:
            found.append(f"tile{t[2]}x{t[3]}" + ("p" if int(t[1]) >= 4 else ""))
    return found


# rows, K and N at no multiple of a tile; dense and ragged
FORMS = [("slim8x1", 5, 520, 272, None), ("slim8x1", 8, 72, 1040, [1, 0, 5]),
         ("slim1x1", 16, 1000, 528, None), ("slim1x1", 45, 72, 1040, [40, 0, 1, 3]),
         ("slim2x1", 27, 1000, 528, None), ("slim2x1", 67, 712, 48, [33, 1, 32]),
         ("slim2x2", 100, 456, 304, None), ("slim2x2", 90, 200, 304, [5, 64, 0, 20]),
         ("slim2x4", 333, 1000, 1008, None), ("slim2x4", 813, 328, 304, None), ("slim2x4", 120, 328, 2096, None),
         ("slim2x4", 147, 344, 688, [40, 1, 0, 33, 32, 0, 7, 30]),
         ("slim4x2", 312, 968, 1632, None), ("slim4x2", 815, 1224, 592, None),
         ("slim4x2", 1290, 1272, 336, [700, 65, 500]),
         ("slim4x4", 403, 200, 1296, None), ("slim4x4", 164, 200, 1264, [64, 0, 65, 1, 3, 0, 0, 30]),
         ("tile128x128p", 1200, 4104, 1040, None), ("tile128x128p", 1200, 4104, 1040, [700, 0, 1, 400]),
         ("tile128x128", 2000, 104, 2064, None), ("tile128x128", 3000, 136, 1552, [1000, 0, 1871, 129]),
         ("tile256x256", 4000, 72, 8112, None), ("tile256x256", 3990, 200, 8112, [300, 0, 3500, 64, 101, 20])]


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("name,rows,K,N,sizes", FORMS)
def test_forward_takes_and_passes(name, rows, K, N, sizes, act):
    for ty in TYPES if name in ("slim2x4", "slim4x2") else ("bf16",):
        p = Product(TYPES[ty], rows, K, N, sizes, bias=True, residual=N // 2 if act == "swiglu" else N)
        assert kernels(lambda: p.forward(act)) == [name], ty
        p.check_forward(act)


def in_nan(t):
    """A copy of t with NaN in the memory before and behind it."""
    n, guard = t.numel(), 4096
    buf = torch.full((n + 2 * guard,), float("nan"), dtype=t.dtype, device=DEV)
    buf[guard:guard + n] = t.flatten()
    return buf[guard:guard + n].view(t.shape)


ONE_OF_EACH = [f for i, f in enumerate(FORMS) if f[4] and all(f[0] != g[0] or not g[4] for g in FORMS[:i])]


@pytest.mark.parametrize("name,rows,K,N,sizes", ONE_OF_EACH)
def test_nan_beside_the_operands(name, rows, K, N, sizes):
    """K, N and rows that are no whole blocks: what lies around an operand, and rows behind the last group, are not
    multiplied by the zeros that fill a block up."""
    p = Product(torch.bfloat16, rows, K, N, sizes, seed=6, bias=True)
    clean, pre = p.forward("none")
    da, db = p.backward()
    assert clean.isfinite().all()
    for t in ("a", "b", "dz", "bias"):
        p.dev[t] = in_nan(p.dev[t])
    for t in ("a", "dz"):
        p.dev[t][p.used:] = float("nan")
    assert kernels(lambda: p.forward("none")) == [name]
    got, pre2 = p.forward("none")
    assert torch.equal(got, clean) and torch.equal(pre2, pre)
    da2, db2 = p.backward()
    assert torch.equal(da2, da) and torch.equal(db2, db)


@pytest.mark.parametrize("name,rows,K,N,sizes", [
    ("slim2x4", 147, 344, 688, [40, 30, 0, 33, 32, 0, 7, 5]), ("slim4x2", 1290, 1272, 336, [600, 190, 500]),
    ("slim4x4", 403, 200, 1296, [130, 140, 133]), ("tile128x128", 3000, 136, 1552, [1000, 129, 1871]),
    ("tile256x256", 6000, 72, 6160, [2500, 1000, 2500]), ("tile128x128p", 1200, 4104, 1040, [500, 300, 400])])
def test_nan_and_infinities_stay_in_their_rows(name, rows, K, N, sizes):
    """A row of NaN, an infinite row of one group's matrix, and rows behind the last: no other result changes."""
    p = Product(torch.bfloat16, rows + 5, K, N, sizes, seed=4)
    clean, _ = p.forward("silu")
    da, db = p.backward()
    lo, hi = int(p.off[1]), int(p.off[2])
    for t in ("a", "dz"):
        p.dev[t][hi - 1] = float("nan")
        p.dev[t][p.used:] = float("inf")
    p.dev["b"][1, 3] = float("inf")
    assert kernels(lambda: p.forward("silu")) == [name]
    got, _ = p.forward("silu")
    keep = torch.ones(rows + 5, dtype=torch.bool)
    keep[lo:hi] = False
    assert torch.equal(got[keep], clean[keep]) and got[hi - 1].isnan().all()
    cols = [c for c in range(N) if c != 3]
    assert torch.equal(got[lo:hi - 1][:, cols], clean[lo:hi - 1][:, cols]) and not got[lo:hi - 1, 3].isfinite().all()
    da2, db2 = p.backward()
    others = [g for g in range(p.G) if g != 1]
    assert torch.equal(da2[keep], da[keep]) and torch.equal(db2[others], db[others]) and db2[1].isnan().all()


def many(groups, rows, seed, uneven):
    r = np.random.default_rng(seed)
    share = np.exp(uneven * r.standard_normal(groups)) * (r.random(groups) < 0.8)
    return r.multinomial(rows, share / share.sum()).tolist()


# few rows and many for very many groups, evenly and very unevenly
@pytest.mark.parametrize("groups,rows,uneven", [(256, 300, 0.5), (256, 2048, 2.0), (1024, 900, 1.0), (1024, 9000, 0.3),
                                                (1000, 5000, 3.0)])
def test_many_groups(groups, rows, uneven):
    K, N, sizes = 72, 112, many(groups, rows, groups + rows, uneven)
    for act in ("none", "swiglu"):
        Product(torch.bfloat16, rows + 9, K, N, sizes, bias=True, residual=N // 2 if act == "swiglu" else N).check_forward(act)
    p = Product(torch.bfloat16, rows + 9, K, N, sizes, residual=K)
    p.check_backward()
    # the activation's gradient, its sums per group
    z, dout = p.dz, p.a[:, :N // 2].contiguous()
    dz, db = torch.full_like(p.dev["dz"], 7.0), torch.full((groups, N), 7.0, device=DEV)
    ws = torch.empty(moe.grouped_act_backward_workspace_bytes(rows + 9, groups, N), dtype=torch.uint8, device=DEV)
    moe.grouped_act_backward(dout.to(DEV), p.dev["dz"], "swiglu", dz, offsets=p.dev["off"], dbias=db, workspace=ws)
    _, slopes = ox.act(np64(z), "swiglu")
    d, zn = np64(dout), np64(z)
    ref = np.concatenate([s * d for s in slopes], 1)
    # as in test_act_backward: a slope's terms are up to 1 + |z|, each a few roundings
    scale = 16 * U * (1 + np.abs(zn[:, :N // 2])) * np.abs(d)
    err = np.concatenate([scale * np.abs(zn[:, N // 2:]), scale], 1) + 2.0 ** -126
    n = p.used
    assert np.all(np.abs(np64(dz) - ref)[:n] <= rounded(torch.bfloat16, ref, err)[:n]) and (dz[n:] == 7).all()
    for g, (lo, hi) in enumerate(ox.ranges(p.off, rows)):
        bound = err[lo:hi].sum(0) + (28 + (hi - lo) / 8) * U * (np.abs(ref[lo:hi]) + err[lo:hi]).sum(0)
        assert np.all(np.abs(np64(db[g]) - ref[lo:hi].sum(0)) <= bound), g


def test_matrix_above_2_gib():
    """Few rows, which would go to slim tiles were a group's matrix not beyond one buffer's bounds."""
    rows, K, N, G, dt = 3, 8192, 131104, 2, torch.bfloat16
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=dt)
    a, b, dz = rand(rows, K), rand(G, N, K), rand(rows, N)
    out = torch.empty(rows, N, dtype=dt, device=DEV)
    n = max(moe.grouped_gemm16_workspace_bytes(rows, G, K, N), moe.grouped_gemm16_backward_workspace_bytes(rows, G, K, N))
    ws = torch.empty(max(16, n), dtype=torch.uint8, device=DEV)
    assert kernels(lambda: moe.grouped_gemm16(a, b, out, ws, offsets=off))[0].startswith("tile")
    da = torch.empty_like(a)
    moe.grouped_gemm16_dgrad(dz, b, da, ws, offsets=off)
    total, mags = torch.zeros(rows, K, dtype=torch.float64, device=DEV), torch.zeros(rows, K, dtype=torch.float64, device=DEV)
    for lo in range(0, N, 16384):
        for grp, part in ((0, slice(0, 1)), (1, slice(1, 3))):
            m = b[grp, lo:lo + 16384].double()
            ref, mag = a[part].double() @ m.T.contiguous(), a[part].double().abs() @ m.abs().T.contiguous()
            got = np64(out[part, lo:lo + 16384])
            assert np.all(np.abs(got - np64(ref)) <= rounded(dt, np64(ref), steps(K) * U * np64(mag))), (lo, grp)
            d = dz[part, lo:lo + 16384].double()
            total[part] += d @ m
            mags[part] += d.abs() @ m.abs()
    assert np.all(np.abs(np64(da) - np64(total)) <= rounded(dt, np64(total), steps(N) * U * np64(mags)))
    del b
    db = torch.full((G, N, K), 7.0, device=DEV)
    moe.grouped_gemm16_wgrad(dz, a, db, ws, offsets=off)
    for lo in range(0, N, 16384):
        for grp, part in ((0, slice(0, 1)), (1, slice(1, 3))):
            d = dz[part, lo:lo + 16384].double().T.contiguous()
            ref, mag = d @ a[part].double(), d.abs() @ a[part].double().abs()
            err = (db[grp, lo:lo + 16384].double() - ref).abs()
            assert (err <= steps(rows) * U * mag + U * ref.abs()).all(), (lo, grp)
    del db
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_far_from_zero(act):
    """Arguments up to the end of FP32's exponents: the sigmoid is 0 where it is below 2^-126, from -87.3 on, where
    silu is at most 2^-119."""
    z = torch.cat([torch.linspace(-130, -70, 121), torch.linspace(-20, 20, 100), torch.linspace(60, 300, 35)]).bfloat16()
    n = len(z)
    width = 2 * n if act == "swiglu" else n
    eye = torch.eye(n, dtype=torch.bfloat16)
    b = torch.cat([eye, eye]) if act == "swiglu" else eye
    out = torch.empty(1, n, dtype=torch.bfloat16, device=DEV)
    moe.grouped_gemm16(z.view(1, n).to(DEV), b.view(1, width, n).contiguous().to(DEV), out, act=act)
    zn = np64(z).reshape(1, n)
    full = np.concatenate([zn, zn], 1) if act == "swiglu" else zn
    with np.errstate(over="ignore"):
        ref, err = act_bounds(full, np.zeros_like(full), act)
    # silu's factor: (4 + |z|) 2^-23; gelu's: 4e-6
    err = err + ((4 + np.abs(zn)) * 2.0 ** -23 if act != "gelu" else 4e-6) * np.abs(ref)
    err = err + {"silu": 2.0 ** -119, "gelu": 0.0, "swiglu": 2.0 ** -119 * np.abs(zn)}[act]
    assert np.all(np.abs(np64(out) - ref) <= rounded(torch.bfloat16, ref, err))
