"""GPU parity of the few-token layer against the float64 oracle: the selection
on every token, the gates, and the output within the noise of the FP8 MFMA, the
effect of h codes that lie on a rounding midpoint, and one BF16 rounding."""

import numpy as np
import pytest
import torch

import routing_fp8_grouped_amd as moe
from oracle import fp8 as ofp8, layer as olayer
from oracle.gemm import blocked_gemm
from tests.gpu_util import DEV, gemm_noise, log, to_np, token_allowance

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
FORMS = {"fp32": moe.moe_layer_few, "pow2": moe.moe_layer_few_pow2}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


class Case:
    """Inputs and FP8 weights of a layer, drawn as codes and scales directly."""

    def __init__(self, T, d, E, G, M, k, f, form="fp32", seed=0, rho=2.5):
        self.T, self.d, self.E, self.G, self.M, self.k, self.f, self.form, self.rho = T, d, E, G, M, k, f, form, rho
        g = torch.Generator(device=DEV).manual_seed(seed + 1)
        self.x = torch.randn(T, d, generator=g, device=DEV).to(BF16)
        self.wg = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(BF16)
        self.bias = torch.rand(E, generator=g, device=DEV) * 0.1 - 0.05
        self.res = torch.randn(T, d, generator=g, device=DEV).to(BF16)
        self.w13, self.w13_s = self.weights(E + 1, 2 * f, d, g)
        self.w2, self.w2_s = self.weights(E + 1, d, f, g)

    def weights(self, n, rows, cols, g):
        q = torch.empty(n, rows, cols, dtype=torch.uint8, device=DEV)
        for e in range(n):
            v = torch.randn(rows, cols, generator=g, device=DEV) * 105
            q[e] = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        u = torch.rand(n, rows // 128, cols // 128, generator=g, device=DEV)
        base = 1.0 / (105.0 * self.d ** 0.5)
        return q, (torch.exp2(torch.floor(torch.log2(base * (1 + u)))) if self.form == "pow2" else (0.8 + 0.4 * u) * base)

    def buffers(self, T=None):
        T = self.T if T is None else T
        return dict(idx=torch.full((T, self.k), -7, dtype=torch.int32, device=DEV),
                    w=torch.full((T, self.k), -7.0, device=DEV), out=torch.full((T, self.d), 7, dtype=BF16, device=DEV))

    def workspace(self):
        n = moe.moe_layer_few_workspace_bytes(self.T, self.d, self.f, self.E, self.k)
        return torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)

    def run(self, res=None, bias=True, ws=None, x=None, **over):
        o = self.buffers()
        o.update(over)
        FORMS[self.form](self.x if x is None else x, self.wg, self.bias if bias else None, self.G, self.M, self.k,
                         self.rho, self.w13, self.w13_s, self.w2, self.w2_s, o["idx"], o["w"], o["out"],
                         self.workspace() if ws is None else ws, residual=res)
        return o

    def experts(self, e):
        return tuple(to_np(a[e]) for a in (self.w13, self.w13_s, self.w2, self.w2_s))

    def check(self, o, res=None, bias=True):
        f32 = lambda t: t.float().cpu().numpy()
        _, r, extra = olayer.moe_layer_tokens(f32(self.x), f32(self.wg), f32(self.bias) if bias else None, self.experts,
                                              self.G, self.M, self.k, self.rho, self.form)
        assert np.array_equal(to_np(o["idx"]), r["idx"])
        assert np.all(np.abs(to_np(o["w"]) - r["w"]) <= 2.0 ** -23 * np.abs(r["w"]))   # two FP64-accurate roundings
        ref = np.zeros((self.T, self.d)) if res is None else f32(res).astype(np.float64)
        mag, noise = np.abs(ref), np.zeros((self.T, self.d))
        for t in range(self.T):
            for e, gate, inter in ([(int(r["idx"][t, j]), float(r["w"][t, j]), extra["inter_routed"][(t, j)])
                                    for j in range(self.k)] + [(self.E, 1.0, extra["inter_shared"][t])]):
                _, _, w2q, w2s = self.experts(e)
                y = blocked_gemm(inter["hq"], inter["hs"], w2q, w2s)
                ref[t] += gate * y[0]
                mag[t] += abs(gate) * np.abs(y[0])
                noise[t] += abs(gate) * gemm_noise(inter["hq"], inter["hs"], w2q, w2s, y)[0]
        # FP32: one sum over the K blocks of all experts, eight partial sums, gate times scale
        noise += 2.0 ** -24 * (self.f // 128 + 8 + 3) * (self.k + 1) * mag
        noise += token_allowance(extra, r, self.experts, self.E, self.form)
        err = np.abs(to_np(o["out"]) - ref)
        assert np.all(err <= noise + 2.0 ** -8 * (np.abs(ref) + noise)), float((err / (noise + 2.0 ** -8 * np.abs(ref))).max())
        rel = np.linalg.norm(err) / np.linalg.norm(ref)
        assert rel <= 6e-3, rel     # BF16 alone: 1.7e-3; the band above is the elementwise bound
        return rel


# one block and one expert; K blocks that fill one, two, four and eight per
# wave, in whole and in part; every token on the same experts; many groups
SHAPES = [(1, 128, 1, 1, 1, 1, 128), (5, 256, 16, 4, 2, 4, 128), (16, 384, 32, 8, 4, 8, 256),
          (3, 1152, 12, 1, 1, 3, 128), (16, 2176, 8, 2, 2, 4, 384), (7, 4224, 16, 4, 2, 2, 1152),
          (2, 8192, 4, 1, 1, 2, 128), (16, 256, 256, 64, 16, 16, 128), (4, 512, 250, 10, 5, 5, 128),
          (13, 128, 9, 3, 3, 9, 256), (9, 1024, 64, 8, 1, 8, 640)]


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_the_oracle(form, shape):
    c = Case(*shape, form=form, seed=sum(shape))
    for res, bias in ((c.res, True), (None, False)):
        rel = c.check(c.run(res, bias), res, bias)
        log(f"{form} {shape}: rel {rel:.1e}")


@pytest.mark.parametrize("T", [1, 2])
def test_v3_shape(T):
    c = Case(T, 7168, 256, 8, 4, 8, 2048, seed=T)
    log(f"V3 shape, T={T}")
    c.check(c.run(c.res), c.res)


@pytest.mark.parametrize("shape", [(2, 128, 3, 1, 1, 2, 32768), (3, 128, 5, 1, 1, 1, 32640), (1, 128, 2, 1, 1, 1, 8320)],
                         ids=lambda s: "x".join(map(str, s)))
def test_widest_intermediate(shape):
    """The largest f, where items and steps are many: their experts come from rounded-up reciprocals."""
    c = Case(*shape, seed=sum(shape))
    c.check(c.run(c.res), c.res)


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("shape", [(16, 1536, 32, 4, 2, 4, 512), (11, 2048, 24, 4, 4, 8, 1024), (2, 512, 16, 2, 2, 8, 2048),
                                   (16, 128, 40, 4, 2, 6, 896)], ids=lambda s: "x".join(map(str, s)))
def test_narrow_layers(form, shape):
    """Several items of the first product in flight; the steps of the second shared by several workgroups."""
    c = Case(*shape, form=form, seed=sum(shape))
    c.check(c.run(c.res), c.res)


def test_shared_steps_repeat():
    """Whichever workgroup comes last adds the others' sums: the bits are the same every time, eagerly, replayed, and
    beside another call on another stream."""
    c = Case(4, 512, 16, 2, 2, 8, 2048, seed=8)
    want = c.run(c.res)["out"]
    ws, o, ws2, o2 = c.workspace(), c.buffers(), c.workspace(), c.buffers()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for _ in range(4):
            c.run(c.res, ws=ws, **o)
    torch.cuda.synchronize()
    for rep in range(20):
        o["out"].zero_()
        o2["out"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            c.run(c.res, ws=ws2, **o2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o["out"], want) and torch.equal(o2["out"], want), rep


@pytest.mark.parametrize("T", range(1, 17))
def test_every_batch_size(T):
    c = Case(T, 256, 16, 4, 2, 4, 128, seed=100 + T)
    c.check(c.run(c.res), c.res)


def test_ties_go_to_the_lower_index():
    """x = 0: every affinity is 1/2 and the bias repeats, so ranks are decided by the tie rule alone."""
    c = Case(3, 256, 32, 8, 4, 8, 128)
    c.x.zero_()
    c.bias.copy_(torch.tensor([0.0, 0.25, 0.25, 0.0] * 8))
    o = c.run(c.res)
    assert to_np(o["idx"]).tolist() == [[1, 2, 5, 6, 9, 10, 13, 14]] * 3
    assert torch.equal(o["w"], torch.full_like(o["w"], 2.5 / 8)) and torch.equal(o["out"], c.res)
    o = c.run(bias=False)
    assert to_np(o["idx"]).tolist() == [[0, 1, 2, 3, 4, 5, 6, 7]] * 3
    assert not o["out"].any()


@pytest.mark.parametrize("low", [float("-inf"), -3.4028234663852886e38, -1e30])
def test_bias_that_masks_experts(low):
    """Experts masked by a bias of minus infinity or the type's lowest value: none of them is chosen while its group has
    others to give; a group without any ranks last, and ranks among masked ones go by the index."""
    c = Case(9, 256, 32, 8, 2, 4, 128, seed=12)
    c.bias[torch.arange(32, device=DEV) % 4 < 2] = low
    c.bias[8:16] = low      # two groups wholly
    o = c.run(c.res)
    idx = to_np(o["idx"])
    assert (idx % 4 >= 2).all() and not ((idx >= 8) & (idx < 16)).any()
    c.check(o, c.res)
    c.bias.fill_(low)       # nothing left to tell the experts apart
    o = c.run(c.res)
    assert to_np(o["idx"]).tolist() == [[0, 1, 2, 3]] * 9
    c.check(o, c.res)


def test_agrees_with_the_layer():
    """The same tokens through MoELayer: the same selection and gates, outputs within the BF16 rounding of the expert
    outputs that the layer makes and this form does not, and the codes on a midpoint."""
    c = Case(16, 1024, 32, 8, 4, 8, 512, seed=3)
    L = moe.MoELayer(16, 1024, 32, 8, 4, 8, 512)
    ref = L.forward(c.x, c.wg, c.bias, moe.MoEWeights(c.w13, c.w13_s, c.w2, c.w2_s))
    o = c.run()
    assert torch.equal(o["idx"], L.idx) and torch.allclose(o["w"], L.w, rtol=2.0 ** -22, atol=0)
    rel = float((o["out"].float() - ref.float()).norm() / ref.float().norm())
    assert rel < 6e-3, rel


@pytest.mark.parametrize("alias", ["x", "residual"])
def test_output_in_place(alias):
    c = Case(6, 512, 16, 4, 2, 4, 256)
    want = c.run(c.res)["out"]
    x, res = c.x.clone(), c.res.clone()
    out = x if alias == "x" else res
    c.run(res, x=x, out=out)
    assert torch.equal(out, want)


def test_repeatable_and_rows_beyond_are_left():
    c = Case(5, 1152, 16, 4, 2, 4, 640)
    a = c.run(c.res)
    wide = c.buffers(8)
    ws = torch.randint(0, 256, (c.workspace().numel() + 512,), dtype=torch.uint8, device=DEV)
    tail = ws[-512:].clone()
    c.run(c.res, ws=ws[:-512], **{n: v[:5] for n, v in wide.items()})
    for n in a:
        assert torch.equal(a[n], wide[n][:5]), n
        assert (wide[n][5:] == (7 if n == "out" else -7)).all()
    assert torch.equal(ws[-512:], tail)


def test_tokens_do_not_touch_each_other():
    """NaN weights of an expert that one token chose, or a NaN token, leave the other tokens' outputs as they were."""
    c = Case(4, 512, 32, 8, 4, 4, 256, seed=9)
    a = c.run(c.res)
    idx = to_np(a["idx"])
    e = next(int(e) for e in idx[0] if not (idx[1:] == e).any())
    w13, w2 = c.w13.clone(), c.w2.clone()
    c.w13[e], c.w2[e] = 0x7F, 0x7F
    b = c.run(c.res)
    assert torch.equal(a["out"][1:], b["out"][1:]) and torch.isnan(b["out"][0].float()).all()
    c.w13, c.w2 = w13, w2
    x = c.x.clone()
    x[2, 5] = float("nan")
    b = c.run(c.res, x=x)
    rest = [0, 1, 3]
    assert torch.equal(a["out"][rest], b["out"][rest]) and torch.equal(a["idx"][rest], b["idx"][rest])
    assert ((b["idx"] >= 0) & (b["idx"] < 32)).all()


@pytest.mark.parametrize("shape", [(1, 256, 16, 4, 2, 4, 128), (16, 1152, 32, 8, 4, 8, 384)])
def test_replays_in_a_graph(shape):
    """Captured and replayed with new inputs, eager calls between the replays; and two graphs that share a workspace."""
    c = Case(*shape, seed=5)
    ws, o, o2 = c.workspace(), c.buffers(), c.buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.run(c.res, ws=ws, **o)
    with torch.cuda.graph(g2, stream=side):
        c.run(None, ws=ws, **o2)
    for rep in range(4):
        c.x.copy_(torch.randn(c.T, c.d, generator=torch.Generator(device=DEV).manual_seed(rep), device=DEV))
        ref, ref2 = c.run(c.res), c.run(None)
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(o[n], ref[n]) and torch.equal(o2[n], ref2[n]), n


def test_two_streams_at_once():
    """Calls with a workspace each, in flight together on two streams."""
    c = Case(16, 2048, 64, 8, 4, 8, 512, seed=6)
    c2 = Case(3, 1024, 32, 4, 2, 4, 256, form="pow2", seed=7)
    want, want2 = c.run(c.res), c2.run(c2.res)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    sets = [(c.workspace(), c.buffers(), c2.workspace(), c2.buffers()) for _ in range(6)]
    torch.cuda.synchronize()
    for wa, oa, wb, ob in sets:
        with torch.cuda.stream(s1):
            c.run(c.res, ws=wa, **oa)
        with torch.cuda.stream(s2):
            c2.run(c2.res, ws=wb, **ob)
    torch.cuda.synchronize()
    for wa, oa, wb, ob in sets:
        for n in want:
            assert torch.equal(oa[n], want[n]) and torch.equal(ob[n], want2[n]), n


def test_refusals():
    c = Case(4, 256, 16, 4, 2, 4, 128)
    e = torch.empty(0, 256, dtype=BF16, device=DEV)
    moe.moe_layer_few(e, c.wg, c.bias, 4, 2, 4, 2.5, c.w13, c.w13_s, c.w2, c.w2_s,
                      torch.empty(0, 4, dtype=torch.int32, device=DEV), torch.empty(0, 4, device=DEV), e,
                      torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(moe.MoEError, match="T=17"):
        x = torch.zeros(17, 256, dtype=BF16, device=DEV)
        c.run(x=x, ws=torch.empty(1 << 22, dtype=torch.uint8, device=DEV), **c.buffers(17))
    with pytest.raises(moe.MoEError, match="workspace"):
        c.run(ws=c.workspace()[:-256])
    for over, msg in [(dict(out=torch.empty(4, 512, dtype=BF16, device=DEV)), "out must have shape"),
                      (dict(idx=torch.empty(4, 4, dtype=torch.int64, device=DEV)), "idx must be"),
                      (dict(w=torch.empty(4, 4)), "w is on cpu")]:
        with pytest.raises(ValueError, match=msg):
            c.run(**over)
    with pytest.raises(ValueError, match="w13 must have shape"):
        c.w13 = c.w13[:16]
        c.run()


@pytest.mark.parametrize("bias", [0.0, 0.01, -0.5])
def test_scores_apart_by_their_last_bits(bias):
    """Saturated affinities, logits 33 to 36: FP64 scores that differ in their last bits only.  The better expert, and
    the better group, is chosen wherever it stands."""
    c = Case(5, 256, 16, 4, 2, 4, 128)
    c.x.zero_()
    c.x[:, 0] = 1
    c.wg.zero_()
    c.bias.fill_(bias)
    for logits, want in (([33.0, 34.0, 35.0, 36.0] * 4, [2, 3, 6, 7]),                      # experts of a group
                         ([33.0] * 8 + [36.0] * 4 + [34.0] * 4, [8, 9, 10, 11]),            # groups
                         ([34.0] * 4 + [33.0] * 8 + [36.0] * 4, [12, 13, 14, 15]),
                         ([36.0, 33.0, 33.0, 36.0] + [33.0, 35.0, 35.0, 33.0] * 3, [0, 3, 5, 6])):
        c.wg[:, 0] = torch.tensor(logits, device=DEV)
        o = c.run(c.res)
        assert to_np(o["idx"]).tolist() == [want] * 5, logits
        c.check(o, c.res)


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("T,d,f", [(3, 384, 128), (2, 1024, 128), (16, 384, 768)])
def test_an_infinity_comes_through(form, T, d, f):
    """A token with an infinity, every product of which has the same sign: its output is infinite, not NaN, where waves
    have K blocks or steps past the end too; the other tokens keep theirs."""
    c = Case(T, d, 8, 2, 2, 2, f, form=form, seed=21)
    col = d - 123
    c.wg[:, col] = c.wg[:, col].abs() + 0.01    # affinities of 1
    c.w13[:, :, col] = 0xB8                     # -1: the infinity's code is -448, so G, U and h are +inf, h's codes -448
    c.w2 &= 0x7F                                # positive
    x = c.x.clone()
    x[0, col] = 1e30                            # the same selection
    a = c.run(c.res, x=x)
    x[0, col] = float("inf")
    o = c.run(c.res, x=x)
    assert (o["out"][0] == -float("inf")).all() and torch.equal(o["idx"][0], a["idx"][0])
    assert torch.equal(o["out"][1:], a["out"][1:]) and torch.equal(o["idx"][1:], a["idx"][1:])


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("T,f", [(2, 128), (16, 768)])      # h quantised in the last kernel, and by a kernel of its own
def test_codes_of_a_tile_with_an_infinity(form, T, f):
    """One h of the shared expert beyond FP32: its tile has an infinite scale, the infinity's code is -448 and the
    finite elements' are zeros, as fp8_quant_1x128 makes them, so an output is an infinity of the one weight's sign."""
    c = Case(T, 256, 8, 2, 2, 2, f, form=form)
    c.x.fill_(1)
    one = 77                                        # this h is (256e18)^2, the others of its tile 2^-18 of that
    c.w13[8, :128], c.w13[8, f:f + 128] = 0x01, 0x01        # 2^-9
    c.w13[8, one], c.w13[8, f + one] = 0x38, 0x38           # 1
    c.w13_s[8, 0], c.w13_s[8, f // 128] = 1e18, 1e18
    o = c.run(c.res)
    inf = torch.tensor(float("inf"), device=DEV)
    want = c.w2[8, :, one].view(torch.float8_e4m3fn).float() * -inf     # NaN for a weight of zero
    assert want.isinf().any() and torch.equal(o["out"].float().nan_to_num(nan=1.0), want.nan_to_num(nan=1.0).expand(T, 256))


# K blocks per wave that the shapes above leave out, four (d 3200 to 4096) and six (d 5248 to 6144), in whole and in
# part; 16 whole columns to a workgroup of the second product (d 4096), its h staged and not; 16 tokens at the widths
# of one and two fragments
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("shape", [(16, 4096, 8, 2, 2, 4, 256), (3, 4096, 8, 2, 2, 4, 128), (16, 4096, 8, 2, 2, 4, 512),
                                   (5, 3328, 8, 2, 2, 4, 128), (4, 6144, 8, 2, 2, 4, 128), (4, 5376, 8, 2, 2, 4, 128),
                                   (16, 7168, 16, 4, 2, 4, 256), (16, 7168, 16, 4, 2, 8, 384), (16, 8192, 4, 2, 1, 2, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_wide_layers(form, shape):
    c = Case(*shape, form=form, seed=sum(shape))
    for res, bias in ((c.res, True), (None, False)):
        rel = c.check(c.run(res, bias), res, bias)
        log(f"{form} {shape}: rel {rel:.1e}")
