"""What MoELayer keeps from one call to the next, and the calls it refuses (CPU
only: the calls into the library are replaced by recorders)."""

import pytest
import torch

import routing_fp8_grouped_amd as moe

T, D, E, F = 4, 128, 8, 128
BF16 = torch.bfloat16


class Recorder:
    """Stands for every call into the library; keeps the arguments of each."""

    def __init__(self, monkeypatch):
        self.calls = []
        for name in moe.__all__:
            if name.islower() and not name.endswith("_bytes") and name != "moe_wgrad_columns":
                monkeypatch.setattr(moe, name, self.stand_in(name))

    def stand_in(self, name):
        return lambda *args, **kw: self.calls.append((name, args, kw))

    def args(self, name):
        return next(a for n, a, _ in reversed(self.calls) if n == name)


@pytest.fixture
def recorder(monkeypatch):
    return Recorder(monkeypatch)


def layer():
    return moe.MoELayer(T, D, E, 2, 2, 2, F, device="cpu")


def operands():
    x, wg = torch.zeros(T, D, dtype=BF16), torch.zeros(E, D, dtype=BF16)
    W = moe.MoEWeights.empty(E + 1, D, F, device="cpu")
    return x, wg, torch.zeros(E), W, torch.ones(D, dtype=BF16)


def test_few_tokens_leave_the_training_selection(recorder):
    """backward reads the gates of the training forward, not those of a few-token pass in between."""
    L = layer()
    x, wg, b, W, wn = operands()
    L.forward(x, wg, b, W, train=True)
    idx, w = recorder.args("moe_route")[7:9]
    assert L.idx is idx and L.w is w
    L.forward_few(x, wg, b, W)
    few = recorder.args("moe_layer_few")[11:13]
    assert L.idx is few[0] and L.w is few[1] and few[0] is not idx and few[1] is not w
    L.backward(x, W)
    assert recorder.args("moe_combine_backward")[3] is w
    L.forward_normed(x, wn, 1e-6, wg, b, W)
    assert L.idx is idx and L.w is w and recorder.args("moe_route")[7] is idx


def test_bias_step_needs_the_loads_of_the_last_pass(recorder):
    """The loads are those that forward and forward_normed leave; there are none before them, and after a few-token
    pass they would be an older batch's."""
    L = layer()
    x, wg, b, W, wn = operands()
    with pytest.raises(RuntimeError, match="counted no expert loads"):
        L.update_bias(b, 1e-3)
    for forward in (lambda: L.forward(x, wg, b, W), lambda: L.forward_normed(x, wn, 1e-6, wg, b, W)):
        forward()
        L.update_bias(b, 1e-3)
        assert recorder.args("moe_bias_update")[:2] == (L.offsets, b)
        L.forward_few(x, wg, b, W)
        with pytest.raises(RuntimeError, match="counted no expert loads"):
            L.update_bias(b, 1e-3)


def test_backward_needs_the_activations_of_the_last_pass(recorder):
    """backward goes through one batch: not through a training forward's caches and a later pass' rows, nor through
    the sums and norms of an earlier forward_normed."""
    L = layer()
    x, wg, b, W, wn = operands()

    def normed(train):
        L.forward_normed(x, wn, 1e-6, wg, b, W, train=train)

    def refused(*methods):
        n = len(recorder.calls)
        for m in methods:
            with pytest.raises(RuntimeError, match=m + " follows"):
                L.backward(x, W) if m == "backward" else L.backward_normed(x, wn, W)
        assert len(recorder.calls) == n

    refused("backward", "backward_normed")
    L.forward(x, wg, b, W, train=True)
    L.backward(x, W)
    refused("backward_normed")
    normed(True)
    L.backward_normed(x, wn, W)
    L.backward_normed(x, wn, W)
    L.backward(x, W)
    L.forward_few(x, wg, b, W)
    L.backward_normed(x, wn, W)
    L.forward(x, wg, b, W, train=True)      # hsum and rstd are an older batch's
    refused("backward_normed")
    L.backward(x, W)
    for untrained in (lambda: L.forward(x, wg, b, W), lambda: normed(False)):
        normed(True)
        untrained()
        refused("backward", "backward_normed")


def test_clipping_needs_gradients(recorder):
    L = layer()
    x, wg, b, W, _ = operands()
    L.forward(x, wg, b, W)
    with pytest.raises(RuntimeError, match="clip_grads follows a backward"):
        L.clip_grads(1.0)
    assert not any(n.startswith("moe_grad") for n, _, _ in recorder.calls)
    L.forward(x, wg, b, W, train=True)
    L.backward(x, W)
    extra = torch.zeros(3)
    L.clip_grads(1.0, extra=(t for t in [extra]))
    for name in ("moe_grad_norm", "moe_grad_scale"):
        assert [id(t) for t in recorder.args(name)[0]] == [id(t) for t in (L.dw13, L.dw2, extra)]


def test_buffers_made_on_first_use_are_the_streams(recorder, monkeypatch):
    """Whatever a call allocates, it allocates on the stream that it was given."""
    L = layer()
    x, wg, b, W, wn = operands()
    current, made = [None], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *exc):
            current.pop()

    monkeypatch.setattr(torch.cuda, "stream", On)
    for name in ("empty", "empty_like", "ones"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _make=make, **kw: (made.append(current[-1]), _make(*a, **kw))[1])
    s = object()
    for call, some in ((lambda: L.forward_normed(x, wn, 1e-6, wg, b, W, stream=s), True),
                       (lambda: L.forward_normed(x, wn, 1e-6, wg, b, W, stream=s, train=True), True),
                       (lambda: L.backward_normed(x, wn, W, stream=s), True), (lambda: L.clip_grads(1.0, stream=s), True),
                       (lambda: L.clip_grads(1.0, extra=[torch.zeros(1)] * 70, stream=s), True),
                       (lambda: L.forward_few(x, wg, b, W, stream=s), False), (lambda: L.clip_grads(2.0, stream=s), False)):
        made.clear()
        call()
        assert bool(made) == some and all(m is s for m in made)


def test_replays_of_a_captured_pass_are_not_seen(recorder, monkeypatch):
    """A captured pass may have been replayed after any other: the calls that follow it are then not refused, those that
    follow another pass still are."""
    L = layer()
    x, wg, b, W, wn = operands()
    capturing = [True]
    monkeypatch.setattr(moe, "_capturing", lambda t: capturing[0])
    L.forward(x, wg, b, W, train=True)
    capturing[0] = False
    L.forward(x, wg, b, W)
    L.backward(x, W)
    L.forward_few(x, wg, b, W)
    L.update_bias(b, 1e-3)
    with pytest.raises(RuntimeError, match="backward_normed follows"):
        L.backward_normed(x, wn, W)
    capturing[0] = True
    L.forward_normed(x, wn, 1e-6, wg, b, W, train=True)
    capturing[0] = False
    L.forward(x, wg, b, W)
    L.backward_normed(x, wn, W)
