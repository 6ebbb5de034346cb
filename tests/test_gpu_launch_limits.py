"""The layer's operators on batches of 2^32 threads and more, which one dimension of a launch does not take."""

import pytest
import torch

import routing_fp8_grouped_amd as moe
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def test_quant():
    """2^28 tiles and some (2^32 threads of 16 a tile): the tiles that are not zeros, and that all others are."""
    rows = (1 << 28) + 5
    at = torch.tensor([0, 1, 17, rows // 2, (1 << 28) - 1, 1 << 28, rows - 1], device=DEV)
    x = torch.zeros(rows, 128, dtype=torch.bfloat16, device=DEV)
    few = (torch.randn(len(at), 128, generator=torch.Generator().manual_seed(5)) * 3).bfloat16().to(DEV)
    x[at] = few
    q, s = torch.full((rows, 128), 7, dtype=torch.uint8, device=DEV), torch.full((rows, 1), 7.0, device=DEV)
    moe.fp8_quant_1x128(x, q, s)
    q2, s2 = torch.empty(len(at), 128, dtype=torch.uint8, device=DEV), torch.empty(len(at), 1, device=DEV)
    moe.fp8_quant_1x128(few, q2, s2)
    assert torch.equal(q[at], q2) and torch.equal(s[at], s2)
    q[at], s[at] = 0, 1.0
    assert not q.view(torch.int64).any() and (s == 1).all()
    del x, q, s
    torch.cuda.empty_cache()


def test_permute():
    """2^24 rows and some (2^32 threads of 256 a row): every row is its token's."""
    T, k, E, d = 1900000, 8, 32, 128
    idx = torch.rand(T, E, device=DEV).topk(k, dim=1).indices.int()
    xq = torch.randint(0, 256, (T, d), dtype=torch.uint8, device=DEV)
    xs = torch.rand(T, 1, device=DEV)
    rows = T * (k + 1)
    assert rows > 1 << 24
    i32 = lambda *s: torch.full(s, 7, dtype=torch.int32, device=DEV)
    offsets, pos, row_token = i32(E + 2), i32(T, k), i32(rows)
    xp, sp = torch.zeros(rows, d, dtype=torch.uint8, device=DEV), torch.zeros(rows, 1, device=DEV)
    ws = torch.empty(moe.moe_permute_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
    moe.moe_permute(idx, E, offsets, pos, row_token, ws, xq, xs, xp, sp)
    token = row_token.long()
    assert torch.equal(token[pos.long().flatten()], torch.arange(T, device=DEV).repeat_interleave(k))
    assert torch.equal(token[T * k:], torch.arange(T, device=DEV))
    assert torch.equal(xp, xq[token]) and torch.equal(sp, xs[token])
    del xp
    torch.cuda.empty_cache()


def test_combine():
    """2^24 tokens and some (2^32 threads of 256 a token), forward and backward."""
    T, d = (1 << 24) + 5, 128
    y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    y.view(torch.int16).random_(1 << 14)       # finite, positive
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV).view(T, 1)
    w = torch.full((T, 1), 0.5, device=DEV)
    out = torch.full_like(y, 7.0)
    moe.moe_combine(y, pos, w, -1, out)
    assert torch.equal(out, y.flip(0) * 0.5)
    dy, dw = torch.full_like(y, 7.0), torch.full((T, 1), 7.0, device=DEV)
    moe.moe_combine_backward(out, y, pos, w, -1, dy, dw)
    assert torch.equal(dy, out.flip(0) * 0.5)
    # dw = <out, y of the row>: positive terms, 128 of them, so each sum is within 128 roundings
    ref = torch.cat([(a.double() ** 2).sum(1) * 2 for a in out.split(1 << 20)])
    assert ((dw[:, 0].double() - ref).abs() <= 128 * 2.0 ** -24 * ref + 128 * 2.0 ** -149).all()
    del y, out, dy
    torch.cuda.empty_cache()


def test_combine_over_two_launches():
    """2^22 tokens and some, with shared rows, the residual and the backward's FP8 copy: the same as in two calls."""
    T, d = (1 << 22) + 5, 128
    y = torch.randn(2 * T, d, dtype=torch.bfloat16, device=DEV)
    res = torch.randn(T, d, dtype=torch.bfloat16, device=DEV)
    pos = torch.randperm(T, device=DEV).int().view(T, 1)
    w = torch.rand(T, 1, device=DEV)
    out = torch.full_like(res, 7.0)
    moe.moe_combine(y, pos, w, T, out, residual=res)
    grads = lambda: (torch.full_like(y, 7.0), torch.full((T, 1), 7.0, device=DEV),
                     torch.full((2 * T, d), 7, dtype=torch.uint8, device=DEV), torch.full((2 * T, 1), 7.0, device=DEV))
    dy, dw, dyq, dys = grads()
    moe.moe_combine_backward(out, y, pos, w, T, dy, dw, dyq=dyq, dys=dys)
    # two halves, the second's shared rows moved with its tokens
    half = T // 2
    out2, (dy2, dw2, dyq2, dys2) = torch.full_like(res, 7.0), grads()
    for lo, hi in ((0, half), (half, T)):
        cut = slice(lo, hi)
        moe.moe_combine(y, pos[cut], w[cut], T + lo, out2[cut], residual=res[cut])
        moe.moe_combine_backward(out[cut], y, pos[cut], w[cut], T + lo, dy2, dw2[cut], dyq=dyq2, dys=dys2)
    assert torch.equal(out, out2)
    for a, b in ((dy, dy2), (dw, dw2), (dyq, dyq2), (dys, dys2)):
        assert torch.equal(a, b)
    assert torch.equal(dy[T:], out) and not (dw == 7).any()
