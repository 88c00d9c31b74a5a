"""The exact operators as layers and optimizer: autograd through BlockNorm and
VocabHead against plain torch in 64 bits, AdamW against its formula over
steps, and the example that trains with all of them."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_block_norm_layer_gradients(amd):
    """Two norms in a chain (the first without a block output): every
    gradient within 256 u of its own size and 1e-6 of the largest (a handful
    of fp32 sums over 48 channels or 30 rows)."""
    import torch
    from approximate_multiplier_dnn_gb300.layers import BlockNorm
    g = torch.Generator().manual_seed(0)
    first, second = BlockNorm(48), BlockNorm(48, gate="channel", alpha=0.5)
    with torch.no_grad():
        for p in [*first.parameters(), *second.parameters()]:
            p.add_(0.2 * torch.randn(p.shape, generator=g).cuda())
    x = torch.randn((3, 10, 48), generator=g).cuda().requires_grad_()
    cr, cn = (torch.randn((3, 10, 48), generator=g).cuda() for _ in range(2))
    r0, n0 = first(x)
    r, n = second(r0, torch.sin(n0))
    ((r * cr).sum() + (n * cn).sum()).backward()

    X, W0, P, Q, G = (t.detach().double().requires_grad_() for t in
                      (x, first.w_pre, second.w_post, second.w_pre, second.gate))

    def rms(t):
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
    R = X + 0.5 * G[0] * rms(torch.sin(rms(X) * W0)) * P
    ((R * cr.double()).sum() + (rms(R) * Q * cn.double()).sum()).backward()
    for got, want in ((x, X), (first.w_pre, W0), (second.w_post, P), (second.w_pre, Q), (second.gate, G)):
        err = (got.grad.double() - want.grad).abs()
        assert bool((err <= 256 * U * want.grad.abs() + 1e-6 * want.grad.abs().max()).all())


def test_vocab_head_layer(amd):
    """The loss and both gradients through autograd, scaled upstream: 2^-8 for
    each of three bf16 roundings (G, the gradient, its scaling) relative to
    the largest terms."""
    import torch
    from approximate_multiplier_dnn_gb300.layers import VocabHead
    g = torch.Generator().manual_seed(1)
    head = VocabHead(40, 300, generator=g)
    h = torch.randn((4, 25, 40), generator=g).to(torch.bfloat16).cuda().requires_grad_()
    t = torch.randint(0, 300, (4, 25), generator=g).cuda()
    t[0] = -100
    loss = head(h, t)
    (3.0 * loss).backward()
    H, W = h.detach().double().requires_grad_(), head.weight.detach().double().requires_grad_()
    want = torch.nn.functional.cross_entropy((H.reshape(-1, 40) @ W.t()), t.reshape(-1))
    (3.0 * want).backward()
    assert abs(float(loss) - float(want)) <= 1e-5
    for got, ref in ((h.grad, H.grad), (head.weight.grad, W.grad)):
        assert got.dtype == torch.bfloat16
        assert float((got.double() - ref).abs().max()) <= 3 * 2.0 ** -8 * float(ref.abs().max())
    with torch.no_grad():
        assert abs(float(head(h, t)) - float(want)) <= 1e-5


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_optimizer(amd, bits):
    """fp32 and bf16 parameters over steps against the formula in 64 bits:
    with fp32 moments the parameters follow it to 2e-6 of the distance moved
    and their rounding; with 8-bit moments to a twentieth of it; bf16
    parameters are their master's rounding."""
    import torch
    from approximate_multiplier_dnn_gb300.optim import AdamW
    g = torch.Generator().manual_seed(2)
    a = torch.nn.Parameter(torch.randn((33, 70), generator=g).cuda())
    b = torch.nn.Parameter(torch.randn(501, generator=g).to(torch.bfloat16).cuda())
    c = torch.nn.Parameter(torch.randn(9, generator=g).cuda())              # never gets a gradient
    opt = AdamW([{"params": [a, c]}, {"params": [b], "weight_decay": 0.0, "lr": 2e-3}], lr=1e-3, moment_bits=bits)
    ref = [p.detach().double().cpu() for p in (a, b)]
    start = [t.clone() for t in ref]
    mom = [[torch.zeros_like(t), torch.zeros_like(t)] for t in ref]
    for step in range(1, 9):
        grads = [torch.randn(p.shape, generator=g).to(p.dtype) for p in (a, b)]
        a.grad, b.grad = (x.cuda() for x in grads)
        opt.step(grad_scale=torch.full((1,), 0.5, device="cuda"))
        for i, (x, lr, wd) in enumerate(zip(grads, (1e-3, 2e-3), (0.01, 0.0))):
            x = x.double() * 0.5
            m, v = mom[i]
            m.mul_(0.9).add_(x, alpha=0.1)
            v.mul_(0.999).add_(x * x, alpha=0.001)
            u = (m / (1 - 0.9 ** step)) / ((v / (1 - 0.999 ** step)).sqrt() + 1e-8)
            ref[i] = ref[i] * (1 - lr * wd) - lr * u
    master = opt.state[b]["master"]
    assert torch.equal(b.detach(), master.to(torch.bfloat16))
    for got, want, first, lr in ((a.detach().double().cpu(), ref[0], start[0], 1e-3),
                                 (master.double().cpu(), ref[1], start[1], 2e-3)):
        moved = 8 * lr
        tol = (2e-6 if bits == 32 else 0.05) * moved + 16 * U * want.abs()
        assert bool(((got - want).abs() <= tol).all()) and float((got - first).abs().max()) > lr
    assert not opt.state[c]
    m, v = opt.moments(a)
    scale = mom[0][0].abs().max()
    assert float((m.double().cpu() - mom[0][0]).abs().max()) <= (1e-6 if bits == 32 else 0.03) * float(scale)
    # a reloaded state goes on alike
    d = [torch.nn.Parameter(p.detach().clone()) for p in (a, c, b)]
    again = AdamW([{"params": d[:2]}, {"params": d[2:], "weight_decay": 0.0, "lr": 2e-3}], lr=1e-3, moment_bits=bits)
    again.load_state_dict(opt.state_dict())
    for p, q in ((a, d[0]), (b, d[2])):
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype).cuda()
        q.grad = p.grad.clone()
    opt.step()
    again.step()
    assert torch.equal(a, d[0]) and torch.equal(b, d[2]) and torch.equal(master, again.state[d[2]]["master"])


def test_layers_refuse(amd):
    import torch
    from approximate_multiplier_dnn_gb300.layers import BlockNorm, am_vocab_loss
    from approximate_multiplier_dnn_gb300.optim import AdamW
    with pytest.raises(ValueError):
        BlockNorm(8, gate="rows")
    with pytest.raises(ValueError):
        AdamW([torch.nn.Parameter(torch.zeros(3, device="cuda"))], moment_bits=4)
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(TypeError):                         # fp32 where bf16 is taken
        am_vocab_loss(x, x, torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        amd.block_norm(x, torch.zeros((4, 9), device="cuda"))
    with pytest.raises(ValueError):
        amd.block_norm(x, x, gate=torch.ones((3, 8), device="cuda"))
    with pytest.raises(TypeError):
        amd.block_norm(x.half())
    with pytest.raises(ValueError):
        amd.block_norm(x.t())
    with pytest.raises(amd.AmsimError) as e:
        amd.block_norm(torch.zeros((2, amd.AMSIM_BLOCK_NORM_MAX_COLS + 1), device="cuda"))
    assert e.value.status == amd.AMSIM_EUNSUPPORTED


@pytest.mark.parametrize("bits", [8, 32])
def test_example_learns(amd, bits):
    """The example's loss falls well below that of a uniform guess (log 1000 =
    6.9) and below where it began, under the approximate multiplier."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import masked_lm
    losses = masked_lm.train(steps=40, moment_bits=bits, vocab=200, dim=64, heads=2, layers=1)
    assert np.all(np.isfinite(losses))
    assert np.mean(losses[-5:]) < 0.8 * np.mean(losses[:3])
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)
