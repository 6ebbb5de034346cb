"""The operators of experts and projections in 16 bits, measured: tokens sorted by expert and back with their weights
(and the gradient), grouped and dense matrix products with bias, activation and residual in the epilogue (and the
gradients), and dropout with the residual addition.

``run`` computes them in their plain form (elementary torch operations) or, with ``own``, by the library's calls.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]
# Widths of the V3 layer, as in routing_fp8_grouped_amd/configs.py.
D, F = 7168, 2048


def listed():
    return [
        # a decode step's tokens to their experts' rows and back
        dict(name="tokens_64", op="tokens", T=64, d=D, E=256, k=8, type="bf16", drop=0.0, win=False, residual=True),
        # ... a training batch's
        dict(name="tokens_16k", op="tokens", T=16384, d=D, E=256, k=8, type="bf16", drop=0.0, win=False,
             residual=False),
        # the gradient of both ways, of an odd batch whose experts are full for some slots; weights applied on both
        dict(name="tokens_bwd_4099_odd", op="tokens_bwd", T=4099, d=2052, E=60, k=6, type="fp16", drop=0.2, win=True,
             residual=False),
        # one token through the first product of a gated expert
        dict(name="gemm_1_swiglu", op="gemm", rows=1, groups=0, K=D, N=2 * F, type="bf16", act="swiglu", bias=False,
             residual=False, pre=False),
        # a small batch's rows over many experts: about two rows each, some experts without any
        dict(name="gemm_128_grouped", op="gemm", rows=128, groups=64, K=D, N=2 * F, type="bf16", act="swiglu",
             bias=False, residual=False, pre=False),
        # a training batch through a dense gated projection, its pre-activations kept for the backward
        dict(name="gemm_16k_swiglu", op="gemm", rows=16384, groups=0, K=D, N=2 * F, type="bf16", act="swiglu",
             bias=False, residual=False, pre=True),
        # ... through the second product of ragged experts
        dict(name="gemm_16k_ragged", op="gemm", rows=16384, groups=32, K=F, N=D, type="bf16", act="none", bias=True,
             residual=False, pre=False),
        # an odd batch through a projection with everything in the epilogue
        dict(name="gemm_333_odd", op="gemm", rows=333, groups=0, K=1000, N=1016, type="fp16", act="gelu", bias=True,
             residual=True, pre=True),
        # gradients of ragged experts' product with respect to rows and weights
        dict(name="gemm_bwd_8k_ragged", op="gemm_bwd", rows=8192, groups=32, K=F, N=D, type="bf16", residual=False),
        # the activation's gradient with that of the bias, ragged experts
        dict(name="act_bwd_8k_swiglu", op="act_bwd", rows=8192, groups=32, N=2 * F, type="bf16", act="swiglu"),
        # residual dropout: a small odd batch
        dict(name="dropout_333_odd", op="dropout", rows=333, cols=1001, type="fp16", p=0.1, residual=True),
        # ... a training batch
        dict(name="dropout_16k", op="dropout", rows=16384, cols=D, type="bf16", p=0.1, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "tokens_bwd", "gemm", "gemm", "gemm_bwd", "act_bwd", "dropout"])
    sixteen = rng.choice(["bf16", "fp16"])
    if op in ("tokens", "tokens_bwd"):
        E = _log(rng, 1, 512)
        return dict(op=op, T=_log(rng, 1, 8192), d=_log(rng, 8, 4096), E=E, k=rng.randint(1, min(8, E)),
                    type=rng.choice(["bf16", "fp16", "fp32"]), drop=rng.choice([0.0, 0.2]), win=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 8, 4096), type=rng.choice(["bf16", "fp16", "fp32"]),
                    p=rng.choice([0.0, 0.05, 0.1, 0.5]), residual=rng.random() < 0.7)
    rows, groups = _log(rng, 1, 16384), rng.choice([0, 0, 1, 8, 33, 64])
    K, N = 8 * _log(rng, 8, 640), 16 * _log(rng, 4, 320)
    if op == "act_bwd":
        return dict(op=op, rows=rows, groups=groups, N=N, type=sixteen, act=rng.choice(ACTS))
    if op == "gemm_bwd":
        return dict(op=op, rows=min(rows, 8192), groups=groups, K=K, N=N, type=sixteen, residual=rng.random() < 0.5)
    return dict(op=op, rows=rows, groups=groups, K=K, N=N, type=sixteen, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                residual=rng.random() < 0.5, pre=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------------------------------------

def _sizes(rows, groups, seed):
    """Rows of every group: uneven, the last of several groups always without any."""
    if groups <= 1:
        return [rows]
    r = np.random.default_rng(seed)
    share = np.exp(0.7 * r.standard_normal(groups))
    share[-1] = 0.0
    return r.multinomial(rows, share / share.sum()).tolist()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    dt = s["dt"] = TYPES[case["type"]]

    def randn(*shape, scale=1.0, dtype=dt):
        if dtype == torch.float32:
            return torch.randn(shape, generator=g, device=DEV).mul_(scale)
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(scale)

    def out(*shape, dtype=dt):
        return torch.zeros(shape, dtype=dtype, device=DEV)

    if case["op"] in ("tokens", "tokens_bwd"):
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        S = T * k
        # uneven experts, distinct for a token; some slots dropped
        logits = torch.randn(T, E, generator=g, device=DEV) + torch.randn(1, E, generator=g, device=DEV)
        score, idx = logits.topk(k, dim=1)
        dropped = torch.rand(T, k, generator=g, device=DEV) < case["drop"]
        s["idx"] = torch.where(dropped, torch.full_like(idx, -1), idx).int()
        s["w"] = (2.5 * torch.softmax(score, 1)).float()
        s["x"] = randn(T, d)
        s["res"] = randn(T, d) if case["residual"] else None
        s["y"] = randn(S, d)
        s["pos"] = out(T, k, dtype=torch.int32)
        if case["op"] == "tokens":
            s["offsets"], s["row_slot"] = out(E + 1, dtype=torch.int32), out(S, dtype=torch.int32)
            s["rows"], s["out"] = out(S, d), out(T, d)
            return s
        s["pos"].copy_(_sorted(s["idx"], E)["pos"])
        s["dout"], s["drows"] = randn(T, d, scale=1e-2), randn(S, d, scale=1e-2)
        s["dy"], s["dw_out"] = out(S, d), out(T, k, dtype=torch.float32)
        s["dx"], s["dw_in"] = out(T, d), out(T, k, dtype=torch.float32)
        return s
    if case["op"] == "dropout":
        n = (case["rows"], case["cols"])
        s["x"], s["res"] = randn(*n), (randn(*n) if case["residual"] else None)
        # the generator's key and the number of this call within the program
        s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device=DEV)
        s["out"] = out(*n)
        return s
    rows, G, N = case["rows"], max(1, case["groups"]), case["N"]
    s["sizes"] = _sizes(rows, case["groups"], seed)
    s["offsets"] = None
    if case["groups"]:
        s["offsets"] = torch.tensor([0] + np.cumsum(s["sizes"]).tolist(), dtype=torch.int32, device=DEV)
    if case["op"] == "act_bwd":
        width = N // 2 if case["act"] == "swiglu" else N
        s["dout"], s["z"] = randn(rows, width, scale=1e-2), randn(rows, N)
        s["dz"], s["dbias"] = out(rows, N), out(G, N, dtype=torch.float32)
        return s
    K = case["K"]
    s["a"] = randn(rows, K)
    s["b"] = randn(G, N, K, scale=1.0 / math.sqrt(K))
    if case["op"] == "gemm_bwd":
        s["dz"] = randn(rows, N, scale=1e-2)
        s["res"] = randn(rows, K, scale=1e-2) if case["residual"] else None
        s["da"], s["db"] = out(rows, K), out(G, N, K, dtype=torch.float32)
        return s
    width = N // 2 if case["act"] == "swiglu" else N
    s["bvec"] = randn(G, N, scale=0.1) if case["bias"] else None
    s["res"] = randn(rows, width) if case["residual"] else None
    s["z"] = out(rows, N) if case["pre"] else None
    s["out"] = out(rows, width)
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------------

def _sorted(idx, E):
    """Stable order of the assigned slots by expert."""
    flat = idx.flatten().long()
    S = flat.numel()
    key, order = torch.where(flat < 0, torch.full_like(flat, E), flat).sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=DEV))
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(S, device=DEV)
    pos = torch.where(flat < 0, torch.full_like(pos, -1), pos)
    slot = torch.where(key < E, order, torch.full_like(order, -1))
    return {"offsets": offsets.int(), "pos": pos.int().view_as(idx), "row_slot": slot.int()}


def _scatter(v, pos, w, like):
    """Rows pos[t, j] = w[t, j] * v[t] of a zeroed [S, d] tensor."""
    T, k = pos.shape
    rows = torch.zeros(like.shape, dtype=torch.float32, device=DEV)
    for j in range(k):
        keep = pos[:, j] >= 0
        part = v if w is None else v * w[:, j, None]
        rows[pos[:, j][keep].long()] = part[keep]
    return rows.to(like.dtype)


def _gather(y, pos, w, add):
    """Sums of w[t, j] * y[pos[t, j]] over j, plus ``add``."""
    total = torch.zeros(pos.shape[0], y.shape[1], device=DEV)
    for j in range(pos.shape[1]):
        part = y[pos[:, j].clamp_min(0).long()].float()
        if w is not None:
            part = part * w[:, j, None]
        total = total + torch.where((pos[:, j] >= 0)[:, None], part, torch.zeros_like(part))
    return total if add is None else total + add.float()


def _dots(v, y, pos):
    d = [(v * y[pos[:, j].clamp_min(0).long()].float()).sum(1) for j in range(pos.shape[1])]
    return torch.where(pos >= 0, torch.stack(d, 1), torch.zeros(pos.shape, device=DEV))


def _tokens(s):
    o = _sorted(s["idx"], s["E"])
    o["rows"] = _scatter(s["x"].float(), o["pos"], s["w"] if s["win"] else None, s["rows"])
    o["out"] = _gather(s["y"], o["pos"], s["w"], s["res"]).to(s["dt"])
    return o


def _tokens_bwd(s):
    pos, win = s["pos"], s["w"] if s["win"] else None
    o = {"dy": _scatter(s["dout"].float(), pos, s["w"], s["dy"]), "dw_out": _dots(s["dout"].float(), s["y"], pos),
         "dx": _gather(s["drows"], pos, win, s["res"]).to(s["dt"])}
    if win is not None:
        o["dw_in"] = _dots(s["x"].float(), s["drows"], pos)
    return o


def _groups(s):
    lo = 0
    for g, n in enumerate(s["sizes"]):
        if n:
            yield g, lo, lo + n
        lo += n


def _act(z, act):
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        return g * torch.sigmoid(g) * u
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z / math.sqrt(2.0)))
    return z.clamp_min(0.0) if act == "relu" else z


def _act_grad(dout, z, act):
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        e = torch.sigmoid(g)
        return torch.cat([dout * u * e * (1.0 + g * (1.0 - e)), dout * g * e], 1)
    if act == "silu":
        e = torch.sigmoid(z)
        return dout * e * (1.0 + z * (1.0 - e))
    if act == "gelu":
        return dout * (0.5 * (1.0 + torch.erf(z / math.sqrt(2.0))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    return torch.where(z > 0.0, dout, torch.zeros_like(dout)) if act == "relu" else dout


def _gemm(s):
    z = torch.empty(s["rows"], s["N"], device=DEV)
    for g, lo, hi in _groups(s):
        z[lo:hi] = s["a"][lo:hi].float() @ s["b"][g].float().T
        if s["bvec"] is not None:
            z[lo:hi] += s["bvec"][g].float()
    out = _act(z, s["act"])
    if s["res"] is not None:
        out = out + s["res"].float()
    return {"out": out.to(s["dt"]), "pre": z.to(s["dt"]) if s["pre"] else None}


def _gemm_bwd(s):
    da = torch.empty(s["rows"], s["K"], device=DEV)
    db = torch.zeros(s["b"].shape, device=DEV)
    for g, lo, hi in _groups(s):
        dz = s["dz"][lo:hi].float()
        da[lo:hi] = dz @ s["b"][g].float()
        db[g] = dz.T @ s["a"][lo:hi].float()
    if s["res"] is not None:
        da = da + s["res"].float()
    return {"da": da.to(s["dt"]), "db": db}


def _act_bwd(s):
    dz = _act_grad(s["dout"].float(), s["z"].float(), s["act"])
    dbias = torch.zeros(s["dbias"].shape, device=DEV)
    for g, lo, hi in _groups(s):
        dbias[g] = dz[lo:hi].sum(0)
    return {"dz": dz.to(s["dt"]), "dbias": dbias}


def _philox_words(n, rng):
    """Four 32-bit words each of Philox4x32-10 for n counters; 64-bit torch integers hold 32-bit words."""
    low = 0xFFFFFFFF
    i = torch.arange(n, device=DEV)
    seed, offset = rng[0], rng[1]
    c = [i & low, i >> 32, (offset & low).expand(n), ((offset >> 32) & low).expand(n)]
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # wraps: the bits are the product's
        c = [((q >> 32) & low) ^ c[1] ^ k0, q & low, ((p >> 32) & low) ^ c[3] ^ k1, p & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c


def _dropout(s):
    x = s["x"].float().flatten()
    n = x.numel()
    c = _philox_words((n + 7) // 8, s["rng"])
    u = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1).flatten()[:n]
    q = int(round((1.0 - s["p"]) * 65536))
    out = torch.where(u < q, x * (65536.0 / max(q, 1)), torch.zeros_like(x))
    if s["res"] is not None:
        out = out + s["res"].float().flatten()
    return {"out": out.to(s["dt"]).view_as(s["x"])}


# ---- the library's calls -------------------------------------------------------------------------------------------

def _workspace(s, size):
    """The workspace that a program keeps beside its other buffers."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(16, size()), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _run_own(s):
    import routing_fp8_grouped_amd as moe
    op = s["op"]
    if op == "tokens":
        ws = _workspace(s, lambda: moe.moe_sort_workspace_bytes(s["T"], s["k"], s["E"]))
        moe.moe_sort(s["idx"], s["E"], s["offsets"], s["pos"], s["row_slot"], ws)
        moe.moe_dispatch(s["x"], s["pos"], s["rows"], w=s["w"] if s["win"] else None)
        moe.moe_collect(s["y"], s["pos"], s["out"], w=s["w"], residual=s["res"])
        return {n: s[n] for n in ("offsets", "pos", "row_slot", "rows", "out")}
    if op == "tokens_bwd":
        moe.moe_collect_backward(s["dout"], s["pos"], s["dy"], w=s["w"], y=s["y"], dw=s["dw_out"])
        o = {"dy": s["dy"], "dw_out": s["dw_out"], "dx": s["dx"]}
        if s["win"]:
            moe.moe_dispatch_backward(s["drows"], s["pos"], s["dx"], w=s["w"], x=s["x"], dw=s["dw_in"],
                                      residual=s["res"])
            o["dw_in"] = s["dw_in"]
        else:
            moe.moe_dispatch_backward(s["drows"], s["pos"], s["dx"], residual=s["res"])
        return o
    if op == "gemm":
        ws = _workspace(s, lambda: moe.grouped_gemm16_workspace_bytes(s["rows"], s["b"].shape[0], s["K"], s["N"],
                                                                      s["act"]))
        moe.grouped_gemm16(s["a"], s["b"], s["out"], ws, offsets=s["offsets"], bias=s["bvec"], act=s["act"],
                           residual=s["res"], pre=s["z"])
        return {"out": s["out"], "pre": s["z"]}
    if op == "gemm_bwd":
        ws = _workspace(s, lambda: moe.grouped_gemm16_backward_workspace_bytes(s["rows"], s["b"].shape[0], s["K"],
                                                                               s["N"]))
        moe.grouped_gemm16_dgrad(s["dz"], s["b"], s["da"], ws, offsets=s["offsets"], residual=s["res"])
        moe.grouped_gemm16_wgrad(s["dz"], s["a"], s["db"], ws, offsets=s["offsets"])
        return {"da": s["da"], "db": s["db"]}
    if op == "act_bwd":
        ws = _workspace(s, lambda: moe.grouped_act_backward_workspace_bytes(s["rows"], s["dbias"].shape[0], s["N"]))
        moe.grouped_act_backward(s["dout"], s["z"], s["act"], s["dz"], offsets=s["offsets"], dbias=s["dbias"],
                                 workspace=ws)
        return {"dz": s["dz"], "dbias": s["dbias"]}
    moe.moe_dropout(s["x"], s["p"], s["rng"], s["out"], residual=s["res"])
    return {"out": s["out"]}


def run(state):
    if own:
        return _run_own(state)
    return {"tokens": _tokens, "tokens_bwd": _tokens_bwd, "gemm": _gemm, "gemm_bwd": _gemm_bwd, "act_bwd": _act_bwd,
            "dropout": _dropout}[state["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    op, z = case["op"], 4 if case["type"] == "fp32" else 2
    if op in ("tokens", "tokens_bwd"):
        T, d, k, E = case["T"], case["d"], case["k"], case["E"]
        S = T * k
        live = S * (1.0 - case["drop"])     # slots with a row
        if op == "tokens":
            # x, y, residual in, rows and out; idx, w in, offsets, pos, row_slot out
            return {"bytes": z * d * (T * (2 + case["residual"]) + 2 * live) + 16 * S + 4 * (E + 1),
                    "flops": (2 + case["win"]) * live * d}
        # dout, y, drows in, dy, dx out, x for the weights' gradient; pos, w in, dw out
        return {"bytes": z * d * (T * (2 + case["win"] + case["residual"]) + 3 * live) + S * (12 + 4 * case["win"]),
                "flops": (4 + 3 * case["win"]) * live * d}
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": z * n * (2 + case["residual"]) + 16, "flops": 2 * n}
    rows, G, N = case["rows"], max(1, case["groups"]), case["N"]
    # groups with rows, were all of them equally likely
    live = 1 if G == 1 else (G - 1) * (1.0 - (1.0 - 1.0 / (G - 1)) ** rows)
    if op == "act_bwd":
        width = N // 2 if case["act"] == "swiglu" else N
        return {"bytes": z * rows * (2 * N + width) + 4 * G * N, "flops": 8 * rows * N}
    K = case["K"]
    if op == "gemm_bwd":
        return {"bytes": z * (rows * (N + 2 * K + K * case["residual"]) + live * N * K) + 4 * G * N * K,
                "flops": 4 * rows * K * N}
    width = N // 2 if case["act"] == "swiglu" else N
    return {"bytes": z * (rows * (K + width * (1 + case["residual"]) + N * case["pre"]) + live * N * K
                          + live * N * case["bias"]), "flops": 2 * rows * K * N}


# ---- in 64 bits ----------------------------------------------------------------------------------------------------

def _exact_tokens(s):
    flat, T, k, E, d = s["idx"].flatten(), s["T"], s["k"], s["E"], s["d"]
    S = T * k
    lists = [torch.nonzero(flat == e).flatten() for e in range(E)]
    slots = torch.cat(lists)
    counts = [int(v.numel()) for v in lists]
    n = slots.numel()
    pos = torch.full((S,), -1, dtype=torch.int64, device=DEV)
    pos[slots] = torch.arange(n, device=DEV)
    if s["op"] == "tokens":
        row_slot = torch.full((S,), -1, dtype=torch.int32, device=DEV)
        row_slot[:n] = slots.int()
        offsets = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32)
        rows = torch.zeros(S, d, dtype=torch.float64, device=DEV)
        for part in torch.arange(n, device=DEV).split(16384):
            v = s["x"][slots[part] // k].double()
            rows[part] = v * s["w"].flatten()[slots[part]].double()[:, None] if s["win"] else v
        out = torch.zeros(T, d, dtype=torch.float64, device=DEV) if s["res"] is None else s["res"].double()
        for part in torch.arange(n, device=DEV).split(16384):
            gate = s["w"].flatten()[slots[part]].double()[:, None]
            out.index_add_(0, slots[part] // k, s["y"][part].double() * gate)
        return {"offsets": offsets, "pos": pos.int().view(T, k), "row_slot": row_slot, "rows": rows, "out": out}
    w = s["w"].flatten().double()
    dy = torch.zeros(S, d, dtype=torch.float64, device=DEV)
    dx = torch.zeros(T, d, dtype=torch.float64, device=DEV) if s["res"] is None else s["res"].double()
    dw_out, dw_in = (torch.zeros(S, dtype=torch.float64, device=DEV) for _ in range(2))
    for part in torch.arange(n, device=DEV).split(16384):
        slot = slots[part]
        token, gate = slot // k, w[slot][:, None]
        dout, drows = s["dout"][token].double(), s["drows"][part].double()
        dy[part] = dout * gate
        dw_out[slot] = torch.linalg.vecdot(dout, s["y"][part].double())
        dw_in[slot] = torch.linalg.vecdot(s["x"][token].double(), drows)
        dx.index_add_(0, token, drows * gate if s["win"] else drows)
    o = {"dy": dy, "dw_out": dw_out.view(T, k), "dx": dx}
    if s["win"]:
        o["dw_in"] = dw_in.view(T, k)
    return o


def _exact_act(z, act):
    """Activation and its derivative with respect to each half of z."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.maximum(z, torch.zeros_like(z)), (z > 0).double()
    if act == "gelu":
        cdf = torch.erfc(-z / math.sqrt(2.0)) / 2.0
        return z * cdf, cdf + z * torch.exp(-z.square() / 2.0) / math.sqrt(2.0 * math.pi)
    h = z if act == "silu" else z[:, :z.shape[1] // 2]
    e = 1.0 / (1.0 + torch.exp(-h))
    value, slope = h * e, e + h * e * (1.0 - e)
    if act == "silu":
        return value, slope
    u = z[:, z.shape[1] // 2:]
    return value * u, torch.cat([slope * u, value], 1)


def _exact_dropout(s):
    n, mask = s["x"].numel(), np.uint64(0xFFFFFFFF)
    m = (n + 7) // 8
    seed, offset = (int(v) for v in s["rng"].tolist())
    ctr = np.arange(m, dtype=np.uint64)
    c0, c1 = ctr & mask, ctr >> np.uint64(32)
    c2, c3 = np.full(m, offset & 0xFFFFFFFF, np.uint64), np.full(m, offset >> 32, np.uint64)
    for r in range(10):
        k0 = np.uint64((seed + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = np.uint64(0xD2511F53) * c0, np.uint64(0xCD9E8D57) * c2
        c0, c1, c2, c3 = (b >> np.uint64(32)) ^ c1 ^ k0, b & mask, (a >> np.uint64(32)) ^ c3 ^ k1, a & mask
    u = np.stack([c0, c1, c2, c3], 1).astype(np.uint32).view(np.uint16).reshape(-1)[:n]     # little-endian halves
    kept = round((1.0 - s["p"]) * 2 ** 16)
    keep = torch.from_numpy(u.astype(np.int32) < kept).to(DEV).view(s["x"].shape)
    v = s["x"].double() * (2.0 ** 16 / kept) * keep.double()
    return {"out": v if s["res"] is None else v + s["res"].double()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("tokens", "tokens_bwd"):
        return _exact_tokens(s)
    if case["op"] == "dropout":
        return _exact_dropout(s)
    edges = np.cumsum([0] + s["sizes"]).tolist()
    if case["op"] == "act_bwd":
        _, slope = _exact_act(s["z"].double(), case["act"])
        dout = s["dout"].double()
        dz = slope * (torch.cat([dout, dout], 1) if case["act"] == "swiglu" else dout)
        return {"dz": dz, "dbias": torch.stack([dz[a:b].sum(0) for a, b in zip(edges, edges[1:])])}
    if case["op"] == "gemm_bwd":
        da, db = [], []
        for g, (a, b) in enumerate(zip(edges, edges[1:])):
            dz = s["dz"][a:b].double()
            da.append(torch.matmul(dz, s["b"][g].double()))
            db.append(torch.matmul(dz.T.contiguous(), s["a"][a:b].double()))
        da = torch.cat(da)
        return {"da": da if s["res"] is None else da + s["res"].double(), "db": torch.stack(db)}
    outs, pres = [], []
    for g, (a, b) in enumerate(zip(edges, edges[1:])):
        if a == b:
            continue
        z = torch.matmul(s["a"][a:b].double(), s["b"][g].double().T.contiguous())
        if s["bvec"] is not None:
            z = z + s["bvec"][g].double()
        pres.append(z)
        outs.append(_exact_act(z, case["act"])[0])
    out = torch.cat(outs)
    return {"out": out if s["res"] is None else out + s["res"].double(), "pre": torch.cat(pres) if s["pre"] else None}
