"""The operators of 16-bit experts together, as a fine-tuning step uses them: router, sort, dispatch, two products, collect
with the gates, dropout with the residual; and all the way back.  Against the same step in float64 with torch's autograd on
the CPU, on the selection the GPU made."""

import math

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import experts as ox
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
I32, F32 = torch.int32, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


class Step:
    """One layer of E experts (SwiGLU, bias on the way down) on T tokens, with every buffer of its two passes."""

    def __init__(self, dt, T, d, f, E, k, drop, p=0.1, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dt)
        self.dt, self.T, self.d, self.f, self.E, self.k, self.p, self.drop = dt, T, d, f, E, k, p, drop
        self.host = dict(x=r(T, d), res=r(T, d), w13=r(E, 2 * f, d, scale=d ** -0.5), w2=r(E, d, f, scale=f ** -0.5),
                         b2=r(E, d, scale=0.1), dout=r(T, d), wg=(torch.randn(E, d, generator=g) * d ** -0.5).bfloat16(),
                         full=torch.rand(T, k, generator=g) < drop)
        for n, t in self.host.items():
            setattr(self, n, t.to(DEV))
        self.rng = torch.tensor([77 + seed, 5], dtype=torch.int64, device=DEV)
        e = lambda *s, dt=dt: torch.zeros(*s, dtype=dt, device=DEV)
        S = self.S = T * k
        self.idx, self.w, self.pos = e(T, k, dt=I32), e(T, k, dt=F32), e(T, k, dt=I32)
        self.offsets, self.slot = e(E + 1, dt=I32), e(S, dt=I32)
        self.rows, self.z, self.h, self.y = e(S, d), e(S, 2 * f), e(S, f), e(S, d)
        self.branch, self.out = e(T, d), e(T, d)
        self.dbranch, self.dy, self.dw, self.db2 = e(T, d), e(S, d), e(T, k, dt=F32), e(E, d, dt=F32)
        self.dh, self.dz, self.drows, self.dx = e(S, f), e(S, 2 * f), e(S, d), e(T, d)
        self.dw2, self.dw13 = e(E, d, f, dt=F32), e(E, 2 * f, d, dt=F32)
        u8 = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device=DEV)
        self.ws_sort = u8(moe.moe_sort_workspace_bytes(T, k, E))
        self.ws = u8(max(moe.grouped_gemm16_workspace_bytes(S, E, d, 2 * f, "swiglu"),
                         moe.grouped_gemm16_workspace_bytes(S, E, f, d),
                         moe.grouped_gemm16_backward_workspace_bytes(S, E, d, 2 * f),
                         moe.grouped_gemm16_backward_workspace_bytes(S, E, f, d),
                         moe.grouped_act_backward_workspace_bytes(S, E, d)))

    def forward(self):
        moe.moe_route(self.x.bfloat16(), self.wg, None, 1, 1, self.k, 2.5, self.idx, self.w)
        if self.drop:
            self.idx.masked_fill_(self.full, -1)      # slots whose experts are full
        moe.moe_sort(self.idx, self.E, self.offsets, self.pos, self.slot, self.ws_sort)
        moe.moe_dispatch(self.x, self.pos, self.rows)
        moe.grouped_gemm16(self.rows, self.w13, self.h, self.ws, offsets=self.offsets, act="swiglu", pre=self.z)
        moe.grouped_gemm16(self.h, self.w2, self.y, self.ws, offsets=self.offsets, bias=self.b2)
        moe.moe_collect(self.y, self.pos, self.branch, w=self.w)
        moe.moe_dropout(self.branch, self.p, self.rng, self.out, residual=self.res)
        return self.out

    def backward(self):
        o = dict(offsets=self.offsets)
        moe.moe_dropout_backward(self.dout, self.p, self.rng, self.dbranch)
        moe.moe_collect_backward(self.dbranch, self.pos, self.dy, w=self.w, y=self.y, dw=self.dw)
        moe.grouped_act_backward(self.dy, None, "none", None, dbias=self.db2, workspace=self.ws, **o)
        moe.grouped_gemm16_dgrad(self.dy, self.w2, self.dh, self.ws, **o)
        moe.grouped_gemm16_wgrad(self.dy, self.h, self.dw2, self.ws, **o)
        moe.grouped_act_backward(self.dh, self.z, "swiglu", self.dz, **o)
        moe.grouped_gemm16_dgrad(self.dz, self.w13, self.drows, self.ws, **o)
        moe.grouped_gemm16_wgrad(self.dz, self.rows, self.dw13, self.ws, **o)
        moe.moe_dispatch_backward(self.drows, self.pos, self.dx)
        return dict(dx=self.dx, dw=self.dw, dw13=self.dw13, dw2=self.dw2, db2=self.db2)

    def reference(self):
        """Outputs and gradients in float64 by autograd, for the selection and gates in idx and w."""
        leaf = {n: self.host[n].double().requires_grad_() for n in ("x", "w13", "w2", "b2")}
        w = self.w.double().cpu().requires_grad_()
        idx, out = self.idx.cpu(), torch.zeros(self.T, self.d, dtype=torch.float64)
        for e in range(self.E):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            z = leaf["x"][t] @ leaf["w13"][e].T
            h = torch.nn.functional.silu(z[:, :self.f]) * z[:, self.f:]
            out = out.index_add(0, t, (h @ leaf["w2"][e].T + leaf["b2"][e]) * w[t, j, None])
        keep, q = ox.keep(self.T * self.d, self.p, int(self.rng[0]), int(self.rng[1]))
        mask = torch.from_numpy(keep).view(self.T, self.d).double() / q
        total = out * mask + self.host["res"].double()
        total.backward(self.host["dout"].double())
        return total.detach(), dict(dx=leaf["x"].grad, dw=w.grad, dw13=leaf["w13"].grad, dw2=leaf["w2"].grad,
                                    db2=leaf["b2"].grad)


def close(got, ref, dt, stages):
    """Root mean square of the difference against that of the reference: each of the ``stages`` tensors on the way is
    rounded by at most half a step, which is below eps / 2 of it, and the products and sums that follow add the errors
    of their terms as they add the terms; SwiGLU's slopes, at most 1.1 of each factor, let them grow by that."""
    err = (got.double().cpu() - ref).square().mean().sqrt() / ref.square().mean().sqrt()
    assert err <= stages * 1.1 ** 2 * torch.finfo(dt).eps / 2, float(err)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,d,f,E,k,drop", [(1, 128, 64, 8, 2, 0.0), (37, 128, 72, 8, 3, 0.2), (300, 256, 128, 16, 4, 0.0),
                                            (1200, 256, 200, 6, 2, 0.3)])
def test_step(dt, T, d, f, E, k, drop):
    s = Step(dt, T, d, f, E, k, drop)
    out, grads = s.forward(), s.backward()
    ref, refs = s.reference()
    close(out, ref, dt, 5)           # z is not rounded before h; rows of x are exact: h, y, branch, out, and x for fp16's router
    for n, stages in (("db2", 2), ("dw2", 4), ("dw", 4), ("dw13", 6), ("dx", 7)):
        # dbranch, dy; h and dy; y; dh, dz and z; drows and dx
        close(grads[n], refs[n], dt, stages)


def test_step_replayed():
    """Both passes in one graph, replayed with other tokens and another call number of the dropout between eager steps."""
    s, e = (Step(torch.bfloat16, 200, 128, 64, 8, 2, 0.0) for _ in range(2))
    s.forward(), s.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.forward(), s.backward()
    gen = torch.Generator(device=DEV).manual_seed(4)
    for call in range(4):
        x = torch.randn(200, 128, generator=gen, device=DEV).bfloat16()
        for t in (s, e):
            t.x.copy_(x)
            t.rng[1] = call
        graph.replay()
        e.forward()
        ge = e.backward()
        torch.cuda.synchronize()
        assert torch.equal(s.out, e.out)
        for n, t in ge.items():
            assert torch.equal(getattr(s, n), t), (call, n)


def test_gradients_are_differences():
    """Small whole numbers, of which every sum is exact in every type: the gradients of the product and of the tokens'
    ways equal the differences that a step of one makes in <gradient, output>."""
    g = torch.Generator().manual_seed(0)
    whole = lambda *s, dt=torch.bfloat16: torch.randint(-2, 3, s, generator=g).to(dt).to(DEV)
    rows, K, N, T, k, E, d = 11, 24, 16, 5, 3, 4, 16
    off = torch.tensor([0, 4, 4, 11], dtype=torch.int32, device=DEV)
    a, b, dz = whole(rows, K), whole(3, N, K), whole(rows, N)

    def product():
        z = torch.empty_like(dz)
        moe.grouped_gemm16(a, b, z, offsets=off)
        return (z.double() * dz.double()).sum().item()

    da, db = torch.empty_like(a), torch.empty(3, N, K, device=DEV)
    moe.grouped_gemm16_dgrad(dz, b, da, offsets=off)
    moe.grouped_gemm16_wgrad(dz, a, db, offsets=off)

    idx = torch.tensor([[0, 3, 1], [3, -1, 3], [2, 2, 0], [1, 5, 3], [0, 1, 2]], dtype=torch.int32, device=DEV)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    pos, slot = torch.empty_like(idx), torch.empty(T * k, dtype=torch.int32, device=DEV)
    moe.moe_sort(idx, E, offsets, pos, slot)
    x, y, w = whole(T, d), whole(T * k, d), whole(T, k, dt=torch.float32)
    drows, dout = whole(T * k, d), whole(T, d)
    drows[13:] = 0          # behind the last row of a slot

    def dispatch():
        out = torch.zeros_like(drows)
        moe.moe_dispatch(x, pos, out, w=w)
        return (out.double() * drows.double()).sum().item()

    def collect():
        out = torch.empty_like(dout)
        moe.moe_collect(y, pos, out, w=w)
        return (out.double() * dout.double()).sum().item()

    dx, dw1, dy, dw2 = torch.empty_like(x), torch.empty_like(w), torch.zeros_like(y), torch.empty_like(w)
    moe.moe_dispatch_backward(drows, pos, dx, w=w, x=x, dw=dw1)
    moe.moe_collect_backward(dout, pos, dy, w=w, y=y, dw=dw2)
    for f, t, grad in [(product, a, da), (product, b, db), (dispatch, x, dx), (dispatch, w, dw1), (collect, y, dy),
                       (collect, w, dw2)]:
        base, flat, want = f(), t.view(-1), grad.double().view(-1).tolist()
        for i in range(0, flat.numel(), 5):
            flat[i] += 1
            assert f() - base == want[i], (f.__name__, i)
            flat[i] -= 1
