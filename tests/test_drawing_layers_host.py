"""Which numbers the layers that draw take: under activation checkpointing, in
copies, and in captured calls (no GPU needed: the mask is plain torch)."""
import copy
import pickle

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from approximate_multiplier_dnn_gb300 import layers
from test_between_layers_host import drawn  # noqa: F401  (a fixture)


class Blocks(torch.nn.Module):
    """Three blocks that share one of their two dropouts; a block may be recomputed in the backward pass."""

    def __init__(self):
        super().__init__()
        g = torch.Generator().manual_seed(0)
        self.w = torch.nn.ParameterList([torch.randn((20, 20), generator=g) * 0.3 for _ in range(3)])
        self.own = torch.nn.ModuleList([layers.Dropout(0.4, seed=10 + i) for i in range(3)])
        self.shared = layers.Dropout(0.3, seed=20)

    def block(self, x, i):
        y = self.own[i](torch.tanh(x @ self.w[i]))
        return torch.tanh(self.shared(y * y, x)) + self.shared(torch.sin(y))

    def forward(self, x, **kw):
        for i in range(3):
            x = checkpoint(self.block, x, i, **kw) if kw else self.block(x, i)
        return x


def gradients(net, steps, **kw):
    g, out = torch.Generator().manual_seed(1), []
    for _ in range(steps):
        x = torch.randn((8, 20), generator=g, requires_grad=True)
        y = net(x, **kw)
        net.zero_grad(set_to_none=True)
        y.square().sum().backward()
        out += [y.detach(), x.grad, *(p.grad for p in net.parameters())]
    return out


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpoint_draws_the_same_masks_again(drawn, reentrant):  # noqa: F811
    """Outputs and gradients of three steps are those without checkpointing."""
    want = gradients(Blocks(), 3)
    got = gradients(Blocks(), 3, use_reentrant=reentrant)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("reentrant", [False, True])
def test_two_forward_passes_before_their_backward_passes(drawn, reentrant):  # noqa: F811
    def run(**kw):
        net, g = Blocks(), torch.Generator().manual_seed(2)
        xs = [torch.randn((8, 20), generator=g, requires_grad=True) for _ in range(2)]
        ys = [net(x, **kw) for x in xs]
        for y in ys:
            y.square().sum().backward()
        return [x.grad for x in xs] + [p.grad for p in net.parameters()]
    assert all(torch.equal(a, b) for a, b in zip(run(use_reentrant=reentrant), run()))


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpoint_that_keeps_no_generator_is_refused(drawn, reentrant):  # noqa: F811
    """Nothing says then which call is made again; a number that the caller gives does."""
    layer, x = layers.Dropout(0.5, seed=1), torch.ones(50, requires_grad=True)
    kw = dict(use_reentrant=reentrant, preserve_rng_state=False)
    y = checkpoint(lambda t: layer(t * t).sin(), x, **kw)
    with pytest.raises(RuntimeError, match="call"):
        y.sum().backward()
    y = checkpoint(lambda t: layer(t * t, call=5).sin(), x, **kw)
    y.sum().backward()
    (want,) = torch.autograd.grad(layer(x * x, call=5).sin().sum(), x)
    assert torch.equal(x.grad, want)


@pytest.mark.parametrize("reentrant", [False, True])
def test_generator_that_is_seeded_anew(drawn, reentrant):  # noqa: F811
    """Before each step: as ever.  Between a forward pass and its backward pass:
    nothing says which of two calls is made again, and both are refused."""
    layer, x = layers.Dropout(0.5, seed=1), torch.ones(50, requires_grad=True)

    def one():
        torch.manual_seed(3)
        return checkpoint(lambda t: layer(t * t).sin(), x, use_reentrant=reentrant).sum()
    for _ in range(3):
        one().backward()
        assert drawn[-1] == drawn[-2]
    a, b = one(), one()
    for y in (b, a):
        with pytest.raises(RuntimeError, match="call"):
            y.backward()


def test_marks_are_bounded(drawn, monkeypatch):  # noqa: F811
    """Calls that nothing repeats leave the marks of the last ones only; a call that is no longer known is refused."""
    monkeypatch.setattr(layers._Draws, "remembered", 5)
    layer, x = layers.Dropout(0.5, seed=1), torch.ones(50, requires_grad=True)
    y = checkpoint(lambda t: layer(t * t).sin(), x, use_reentrant=False).sum()
    with torch.no_grad():
        for _ in range(7):
            layer(x)
    assert len(layer.draws.marks) == 5
    with pytest.raises(RuntimeError, match="call"):
        y.backward()


def test_calls_that_nothing_runs_again_leave_the_generator_alone(drawn):  # noqa: F811
    """A plain call takes nothing from torch's generator and is not remembered, between checkpointed ones too."""
    layer, x = layers.Dropout(0.5, seed=1), torch.ones(50, requires_grad=True)
    y = checkpoint(lambda t: layer(t * t).sin(), x, use_reentrant=False).sum()
    before = torch.get_rng_state()
    layer(x).sum().backward()
    assert torch.equal(torch.get_rng_state(), before) and len(layer.draws.marks) == 1
    y.backward()
    assert [n for _, n in drawn] == [0, 1, 1, 0, 0]


def test_numbers_go_on_after_checkpointing(drawn):  # noqa: F811
    """A call that is made again takes no number of its own."""
    layer, x = layers.Dropout(0.5, seed=1), torch.ones(50, requires_grad=True)
    checkpoint(lambda t: layer(t * t).sin(), x, use_reentrant=False).sum().backward()
    layer(x)
    assert {n for _, n in drawn} == {0, 1} and layer.draws.calls == 2


def test_deep_copies_draw_masks_of_their_own(drawn):  # noqa: F811
    """Blocks made by copying one; a saved and reloaded layer, pickled or by its state, goes on as before."""
    for layer in (layers.Dropout(0.5, seed=1), layers.AMAttention(None, dropout=0.5, seed=1)):
        layer.draws.calls = 3
        copies = [copy.deepcopy(layer), *copy.deepcopy(torch.nn.ModuleList([layer, layer]))]
        assert copies[1] is copies[2]                                     # one layer at two places stays one
        seeds = {layer.draws.seed, copies[0].draws.seed, copies[1].draws.seed, copy.deepcopy(copies[0]).draws.seed}
        assert len(seeds) == 4 and layer.draws.seed == 1
        assert all(c.draws.calls == 3 and c.draws.marks is not layer.draws.marks for c in copies)
        again = pickle.loads(pickle.dumps(layer))
        assert (again.draws.seed, again.draws.calls) == (1, 3)
        copies[0].load_state_dict(layer.state_dict())
        assert (copies[0].draws.seed, copies[0].draws.calls) == (1, 3)
    layer, x = layers.Dropout(0.5, seed=1), torch.ones(100)
    assert not torch.equal(copy.deepcopy(layer)(x), layer(x))
    off = layers.Dropout(0.5, seed=1).eval()
    assert not copy.deepcopy(off).training and not copy.deepcopy(off).draws.training
    torch.manual_seed(0)
    a = copy.deepcopy(layer).draws.seed
    torch.manual_seed(0)
    assert a == copy.deepcopy(layer).draws.seed                           # repeatable


def test_captured_calls_take_numbers_that_no_replay_repeats(drawn, monkeypatch):  # noqa: F811
    """A layer that is called twice in a graph, whose step is raised once a
    replay, and again after it: no two masks are alike."""
    layer, x, step = layers.Dropout(0.5, seed=1), torch.ones(10), torch.zeros(1, dtype=torch.int64)
    layer(x, step=step)
    first = layer.draws.calls
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError):
        layer(x)
    layer(x, step=step), layer(x, step=step)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    layer(x)
    before, *captured, after = [n for _, n in drawn]
    assert captured[0] == first == 1                                      # the next number, as an eager call's
    seen = {n + replay for n in captured for replay in range(1000)} | {before, after}
    assert len(seen) == 2002
