"""The layers between two contractions as they are used together: attention
with a bias, lengths and dropout against its own parts, Dropout and GroupNorm
through autograd, a small convolutional network with attention, and the
example."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rand(g, *shape, scale=1.0):
    import torch
    return (torch.randn(shape, generator=g) * scale).cuda()


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("s,t,causal", [(40, 40, True), (24, 71, False)])
def test_attention_is_its_parts(amd, luts, p, s, t, causal):
    """Output and every gradient, bit for bit, as the contractions, the softmax
    and its gradient make them one by one; padded keys are NaN."""
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(1)
    lut = luts("mitchell", 7)
    b, h, d = 3, 2, 16
    bias = layers.RelativeBias(h, generator=g)
    layer = layers.AMAttention(lut, bias=bias, causal=causal, dropout=p, seed=9)
    q, k, v = rand(g, b, h, s, d), rand(g, b, h, t, d), rand(g, b, h, t, d)
    n = torch.tensor([t, t // 2, 1], dtype=torch.int32, device="cuda")
    hidden = (torch.arange(t, device="cuda") >= n[:, None])[:, None, :, None]
    k0, v0 = k.masked_fill(hidden, 0), v.masked_fill(hidden, 0)
    q, k, v = (x.requires_grad_() for x in (q, k.masked_fill(hidden, float("nan")), v.masked_fill(hidden, float("nan"))))
    out = layer(q, k, v, lengths=n)
    up = rand(g, b, h, s, d)
    out.backward(up)

    def mm(tA, tB, A, B, m, n, k, alpha=1.0):
        return layers._bgemm(tA, tB, A.reshape(b * h, *A.shape[2:]), B.reshape(b * h, *B.shape[2:]), m, n, k, lut,
                             alpha).view(b, h, m, n)
    Q, scale = q.detach(), 1 / np.sqrt(d)
    S = mm("N", "T", Q, k0, s, t, d, scale)
    kw = dict(table=bias.table.detach(), buckets=bias.buckets, lengths=n, causal=causal, p=p, seed=9)
    P, stats = amd.attention_softmax(S, **kw)
    assert torch.equal(out, mm("N", "N", P, v0, s, d, t))
    way = dict(scores=S, stats=stats) if p else dict(probs=P)
    dS, dtable = amd.attention_softmax_backward(mm("N", "T", up, v0, s, t, d), **way, **kw)
    assert torch.equal(q.grad, mm("N", "N", dS, k0, s, d, t, scale))
    assert torch.equal(k.grad, mm("T", "N", dS, Q, t, d, s, scale))
    assert torch.equal(v.grad, mm("T", "N", P, up, t, d, s))
    assert torch.equal(bias.table.grad, dtable)
    assert not k.grad.masked_fill(~hidden, 0).any() and not v.grad.masked_fill(~hidden, 0).any()
    layer.eval()
    assert torch.equal(layer(q, k, v, lengths=n), layer(q, k, v, lengths=n))


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("s,t,causal", [(3, 0, False), (0, 5, True), (1, 1, True), (4, 6, False)])
def test_attention_over_nothing(amd, luts, s, t, causal, p):
    """No keys, no queries, lengths of zero: zeros out, and zero gradients for
    what has no effect."""
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(2)
    bias = layers.RelativeBias(2, generator=g)
    layer = layers.AMAttention(luts("mitchell", 7), bias=bias, causal=causal, dropout=p, seed=1)
    q, k, v = (rand(g, 2, 2, n, 8).requires_grad_() for n in (s, t, t))
    out = layer(q, k, v, lengths=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert out.shape == (2, 2, s, 8) and not out.any()
    out.sum().backward()
    for x in (q, k, v, bias.table):
        assert x.grad.shape == x.shape and not x.grad.any()


def test_single_tokens_continue_a_sequence(amd, luts):
    """A cache's next token, one query at its place, as that row of the whole
    sequence: the contractions' sums may be taken in another order (1e-5 of the
    magnitudes, the contractions' own bound)."""
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(2)
    layer = layers.AMAttention(luts("mitchell", 7), bias=layers.RelativeBias(2, bidirectional=False, generator=g),
                               causal=True)
    q, k, v = (rand(g, 3, 2, 30, 16) for _ in range(3))
    with torch.no_grad():
        whole = layer(q, k, v)
        n = torch.tensor([30, 7, 1], dtype=torch.int32, device="cuda")
        rows = torch.stack([q[i, :, int(n[i]) - 1] for i in range(3)])[:, :, None]
        token = layer(rows, k, v, lengths=n, offset=n - 1)
        for i in range(3):
            assert float((token[i, :, 0] - whole[i, :, int(n[i]) - 1]).abs().max()) <= 1e-4


def test_plain_attention_keeps_its_results(amd, luts):
    """Without a bias, lengths, mask or dropout the layer is what it was."""
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(3)
    q, k, v = (rand(g, 2, 2, 33, 16).requires_grad_() for _ in range(3))
    lut = luts("mitchell", 7)
    up = rand(g, 2, 2, 33, 16)
    out = layers.AMAttention(lut)(q, k, v)
    grads = torch.autograd.grad(out, (q, k, v), up)
    want = layers._AttentionFn.apply(q, k, v, lut, 0.25)
    assert torch.equal(out, want)
    assert all(torch.equal(x, y) for x, y in zip(grads, torch.autograd.grad(want, (q, k, v), up)))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_dropout_layer(amd, dtype):
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(4)
    layer = layers.Dropout(0.3, generator=g)
    x, r, up = (rand(g, 6, 50).to(getattr(torch, dtype)) for _ in range(3))
    x, r = x.t().requires_grad_(), r.t().requires_grad_()                 # neither contiguous
    y = layer(x, r)
    y.backward(up.t())
    seed = layer.draws.seed
    assert torch.equal(y, amd.dropout(x.detach().contiguous(), 0.3, seed=seed, residual=r.detach().contiguous()))
    assert torch.equal(x.grad, amd.dropout(up.t().contiguous(), 0.3, seed=seed)) and torch.equal(r.grad, up.t())
    assert not torch.equal(layer(x, r), y)


def test_captured_dropout_needs_a_step(amd):
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    layer, x, step = layers.Dropout(0.5, seed=1), torch.ones(4096, device="cuda"), torch.zeros(1, dtype=torch.int64,
                                                                                              device="cuda")
    layer(x, step=step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError):
            layer(x)
        y = layer(x, step=step)
    seen = []
    for i in range(3):
        step.fill_(i)
        graph.replay()
        assert torch.equal(y, amd.dropout(x, 0.5, seed=1, call=1 + i))
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("activation", ["none", "relu", "silu"])
def test_group_norm_layer(amd, activation):
    """Through autograd, x a slice of wider pixels: every gradient within 256 u
    of its size and 2e-6 of the largest (sums over 63 pixels)."""
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(5)
    layer = layers.GroupNorm(3, 24, activation=activation)
    with torch.no_grad():
        layer.weight.add_(rand(g, 24, scale=0.2))
        layer.bias.add_(rand(g, 24, scale=0.2))
    wide = rand(g, 2, 7, 9, 32).requires_grad_()
    up = rand(g, 2, 7, 9, 24)
    layer(wide[..., 4:28]).backward(up)
    W, w, b = (t.detach().double().requires_grad_() for t in (wide, layer.weight, layer.bias))
    x = W[..., 4:28].reshape(2, 63, 3, 8)
    var, mean = torch.var_mean(x, (1, 3), correction=0, keepdim=True)
    z = ((x - mean) * (var + 1e-5).rsqrt()).reshape(2, 7, 9, 24) * w + b
    y = z if activation == "none" else z.relu() if activation == "relu" else torch.nn.functional.silu(z)
    y.backward(up.double())
    for got, ref in ((wide.grad, W.grad), (layer.weight.grad, w.grad), (layer.bias.grad, b.grad)):
        assert bool(((got - ref).abs() <= 256 * U * ref.abs() + 2e-6 * ref.abs().max()).all())


class Net:
    """Two convolutions, each with its group norm, dropout, then attention with
    a relative bias over the pixels of the map, the loss a weighted sum."""

    def __init__(self, lut, seed):
        import torch
        from approximate_multiplier_dnn_gb300 import layers
        g = torch.Generator().manual_seed(seed)
        self.layers = torch.nn.ModuleDict(dict(
            c1=layers.AMConv2d(3, 16, 3, lut, padding=1, generator=g),
            n1=layers.GroupNorm(4, 16, activation="relu"),
            c2=layers.AMConv2d(16, 16, 3, lut, stride=2, padding=1, generator=g),
            n2=layers.GroupNorm(4, 16, activation="silu"),
            d2=layers.Dropout(0.2, seed=7),
            a=layers.AMAttention(lut, bias=layers.RelativeBias(2, generator=g), dropout=0.1, seed=8),
            d3=layers.Dropout(0.2, seed=9)))

    def __call__(self, x, step=None):
        m = self.layers
        y = m["n1"](m["c1"](x))
        y = m["d2"](m["n2"](m["c2"](y)), step=step)
        N, H, W, C = y.shape
        t = y.reshape(N, H * W, 2, C // 2).transpose(1, 2).contiguous()
        return m["d3"](m["a"](t, t, t, step=step), t, step=step)


def test_network(amd, luts):
    """All of them in a run: outputs and gradients are finite, repeat from the
    same state bit for bit, differ from call to call, and each GroupNorm's
    gradient is that of what reached it."""
    import torch
    g = torch.Generator().manual_seed(6)
    x, up = rand(g, 4, 12, 12, 3), rand(g, 4, 2, 36, 8)

    def run(net):
        y = net(x)
        y.backward(up)
        grads = [p.grad.clone() for p in net.layers.parameters()]
        for p in net.layers.parameters():
            p.grad = None
        return y.detach(), grads
    a, b = Net(luts("mitchell", 7), 0), Net(luts("mitchell", 7), 0)
    y1, g1 = run(a)
    y2, g2 = run(b)
    assert torch.equal(y1, y2) and all(torch.equal(p, q) for p, q in zip(g1, g2))
    assert bool(torch.isfinite(y1).all()) and all(bool(torch.isfinite(p).all()) and bool(p.any()) for p in g1)
    y3, _ = run(a)
    assert not torch.equal(y1, y3)
    seen = {}

    def hook(m, inp, out):
        seen["in"], seen["out"] = inp[0].detach(), out
        out.register_hook(lambda d: seen.__setitem__("dy", d))
        inp[0].register_hook(lambda d: seen.__setitem__("dx", d))
    h = a.layers["n2"].register_forward_hook(hook)
    run(a)
    h.remove()
    n2 = a.layers["n2"]
    _, mean, rstd = amd.group_norm(seen["in"], 4, n2.weight.detach(), n2.bias.detach(), activation="silu")
    dx, _, _ = amd.group_norm_backward(seen["dy"].contiguous(), seen["in"], n2.weight.detach(), n2.bias.detach(), mean,
                                       rstd, activation="silu")
    assert torch.equal(dx, seen["dx"])
    for m in a.layers.values():
        m.eval()
    assert torch.equal(a(x), a(x))
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


def test_captured_training_step(amd, luts):
    """Forward, backward and the optimizer in one graph: each replay draws by
    its step and leaves the weights that eager steps leave."""
    import torch
    from approximate_multiplier_dnn_gb300.optim import AdamW
    g = torch.Generator().manual_seed(7)
    x, up = rand(g, 2, 8, 8, 3), rand(g, 2, 2, 16, 8)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def one(net):
        for p in net.layers.parameters():
            p.grad = None
        net(x, step=step).backward(up)
        return [p.grad for p in net.layers.parameters()]
    eager, want = Net(luts("mitchell", 7), 1), []
    for _ in range(2):
        one(eager)
    for i in range(3):
        step.fill_(i)
        for m in ("d2", "a", "d3"):
            eager.layers[m].draws.calls = 2                               # the captured call's number
        want.append([t.clone() for t in one(eager)])
    net = Net(luts("mitchell", 7), 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            one(net)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = one(net)
    for i in range(3):
        step.fill_(i)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(grads, want[i]))
    assert not all(torch.equal(p, q) for p, q in zip(want[0], want[1]))
    AdamW(net.layers.parameters()).step()


@pytest.mark.parametrize("kw", [dict(positions="relative"), dict(dropout=0.1), dict(positions="relative", dropout=0.1)])
def test_example_runs(amd, kw):
    """Finite losses, no wait given up."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import masked_lm
    losses = masked_lm.train(steps=6, vocab=200, dim=64, heads=2, layers=1, **kw)
    assert np.all(np.isfinite(losses))
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)
