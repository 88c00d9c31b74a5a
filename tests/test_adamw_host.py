"""Host logic of optim.AdamW (no GPU needed): the step is replaced by the
formula in plain torch on the tensors whose addresses the table was given."""
import copy
import io

import pytest
import torch

from approximate_multiplier_dnn_gb300 import optim


class Entry:
    """What a table holds of a tensor: addresses, so the memory they had when it was made."""

    @classmethod
    def make(cls, p, g, m, v, m_scale=None, v_scale=None, copy=None, weight_decay=0.0, lr_scale=1.0):
        e = cls()
        e.p, e.g, e.m, e.v, e.copy = (None if t is None else t.detach().view(-1) for t in (p, g, m, v, copy))
        e.weight_decay, e.lr_scale = weight_decay, lr_scale
        return e


@pytest.fixture
def steps(monkeypatch):
    """Records (step, tensors) of each launch; moments are fp32."""
    calls = []

    def step(table, *, lr, beta1, beta2, eps, step, grad_scale=None):
        calls.append((step, len(table)))
        for e in table:
            g = e.g.float() if grad_scale is None else e.g.float() * grad_scale
            e.m.mul_(beta1).add_(g, alpha=1 - beta1)
            e.v.mul_(beta2).add_(g * g, alpha=1 - beta2)
            u = (e.m / (1 - beta1 ** step)) / ((e.v / (1 - beta2 ** step)).sqrt() + eps)
            e.p.mul_(1 - lr * e.lr_scale * e.weight_decay).sub_(lr * e.lr_scale * u)
            if e.copy is not None:
                # the kernel writes through an address: no version of the parameter changes
                e.copy.data.copy_(e.p)
    monkeypatch.setattr(optim, "AdamwTensor", Entry)
    monkeypatch.setattr(optim, "adamw_table", list)
    monkeypatch.setattr(optim, "adamw_step", step)
    return calls


def params(*sizes, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(n, generator=g).to(dtype)) for n in sizes]


def grads(ps, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype)


@pytest.mark.parametrize("dtype,name", [(torch.float32, "v"), (torch.float32, "m"), (torch.bfloat16, "master")])
def test_replaced_state_is_used(steps, dtype, name):
    """State that is replaced while the other tensors stay is what the next
    step reads and writes."""
    (p,) = params(40, dtype=dtype)
    opt = optim.AdamW([p])
    p.grad = torch.ones(40, dtype=dtype)
    opt.step()
    old = opt.state[p][name]
    kept = old.clone()
    opt.state[p][name] = old + 1.0
    new = opt.state[p][name].clone()
    opt.step()
    assert torch.equal(old, kept) and not torch.equal(opt.state[p][name], new)


def test_table_is_kept_while_nothing_moves(steps, monkeypatch):
    made = []
    monkeypatch.setattr(optim, "adamw_table", lambda entries: made.append(1) or list(entries))
    ps = params(5, 7)
    opt = optim.AdamW(ps)
    grads(ps, 0)
    for _ in range(3):
        opt.step()
    assert len(made) == 1
    p = ps[0]
    p.grad = p.grad.clone()
    opt.step()
    assert len(made) == 2
