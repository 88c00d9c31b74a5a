"""The layers that draw, under activation checkpointing, in captured graphs and
in training steps whose forward and backward passes are captured."""
import copy

import pytest

from test_gpu_between_layers import Net, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpointed_block(amd, luts, reentrant):
    """Attention and two dropouts run again in the backward pass: outputs and
    gradients of two steps bit for bit those without checkpointing."""
    import torch
    from torch.utils.checkpoint import checkpoint
    from approximate_multiplier_dnn_gb300 import layers
    g = torch.Generator().manual_seed(1)
    bias = layers.RelativeBias(2, generator=g)
    first = torch.nn.ModuleDict(dict(a=layers.AMAttention(luts("mitchell", 7), bias=bias, causal=True, dropout=0.2, seed=1),
                                     d=layers.Dropout(0.3, seed=2)))
    x, up = rand(g, 2, 2, 37, 16), rand(g, 2, 2, 37, 16)

    def run(**kw):
        net, out = copied(first), []

        def block(t):
            return net["d"](torch.tanh(net["d"](net["a"](t, t, t), t)))
        for _ in range(2):
            t = x.clone().requires_grad_()
            y, net["a"].bias.table.grad = t, None                         # three parts, in the blocks' order either way
            for _ in range(3):
                y = checkpoint(block, y, **kw) if kw else block(y)
            y.backward(up)
            out += [y.detach(), t.grad, net["a"].bias.table.grad.clone()]
        return out

    def copied(m):                                                        # a deep copy alone draws other masks
        new = copy.deepcopy(m)
        new.load_state_dict(m.state_dict())
        return new
    want = run()
    assert all(torch.equal(a, b) for a, b in zip(run(use_reentrant=reentrant), want))
    assert not torch.equal(want[0], want[3])


def test_a_layer_twice_in_a_captured_graph(amd):
    """No two calls of any replays, or of an eager call after them, draw alike."""
    import torch
    from approximate_multiplier_dnn_gb300 import layers
    layer, x, step = layers.Dropout(0.5, seed=1), torch.ones(4096, device="cuda"), torch.zeros(1, dtype=torch.int64,
                                                                                              device="cuda")
    layer(x, step=step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = layer(x, step=step), layer(x, step=step)
    masks = []
    for i in range(4):
        step.fill_(i)
        graph.replay()
        masks += [y.clone(), z.clone()]
    masks.append(layer(x))
    assert all(not torch.equal(masks[i], masks[j]) for i in range(len(masks)) for j in range(i))


def test_captured_steps_leave_the_weights_of_eager_ones(amd, luts):
    """Forward and backward passes in one graph, the optimizer (whose count of
    steps is the host's) after each replay: gradients and every weight bit for
    bit those of a network that is trained without a graph."""
    import torch
    from approximate_multiplier_dnn_gb300.optim import AdamW
    g = torch.Generator().manual_seed(7)
    x, up = rand(g, 2, 8, 8, 3), rand(g, 2, 2, 16, 8)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def passes(net):
        for p in net.layers.parameters():
            p.grad = None
        net(x, step=step).backward(up)
    nets = [Net(luts("mitchell", 7), 1) for _ in range(2)]
    opts = [AdamW(net.layers.parameters(), lr=0.05) for net in nets]
    eager, net = nets
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            passes(net)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        passes(net)
    before = [p.detach().clone() for p in net.layers.parameters()]
    for i in range(4):
        step.fill_(i)
        for m in ("d2", "a", "d3"):
            eager.layers[m].draws.calls = 2                               # the captured call's number
        passes(eager)
        graph.replay()
        for a, b in zip(eager.layers.parameters(), net.layers.parameters()):
            assert torch.equal(a.grad, b.grad)
        for opt in opts:
            opt.step()
        for a, b in zip(eager.layers.parameters(), net.layers.parameters()):
            assert torch.equal(a, b)
    assert all(not torch.equal(p, q) for p, q in zip(net.layers.parameters(), before))
