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


def formula(p, gs, lr=1e-3, wd=0.01):
    """AdamW in 64 bits over the gradients that a parameter got (None: none in that step)."""
    p, m, v, t = p.detach().double().clone(), 0.0, 0.0, 0
    for g in gs:
        if g is None:
            continue
        t, g = t + 1, g.double()
        m, v = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
        p = p * (1 - lr * wd) - lr * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
    return p


def train(opt, ps, plan, seed=0):
    """Steps; plan[i] names the parameters that get a gradient in step i. The gradients of each parameter."""
    g = torch.Generator().manual_seed(seed)
    got = [[] for _ in ps]
    for which in plan:
        for i, p in enumerate(ps):
            p.grad = torch.randn(p.shape, generator=g) if i in which else None
            got[i].append(p.grad)
        opt.step()
    return got


def test_late_and_paused_gradients(steps):
    """Bias correction counts a parameter's own updates: parameters whose
    gradients start late, pause or never come follow the formula (fp32 rounding:
    30 steps of 1e-3 with some 10 roundings each)."""
    ps = params(50, 60, 70, 80)
    start = [p.detach().clone() for p in ps]
    opt = optim.AdamW(ps)
    plan = [{0}] * 20 + [set()] + [{0, 1}] * 5 + [{0, 2}, {0, 1, 2}, {1}, {0, 1, 2}]
    got = train(opt, ps, plan)
    for p, first, gs in zip(ps, start, got):
        assert float((p.detach().double() - formula(first, gs)).abs().max()) <= 30 * (1e-3 * 10 + 4) * 2.0 ** -24
    assert not opt.state[ps[3]]
    assert [opt.state[p]["step"] for p in ps[:3]] == [28, 8, 3]
    # one launch for each count of updates among a step's parameters, none without gradients
    assert [n for _, n in steps[:20]] == [1] * 20 and steps[20:22] == [(21, 1), (1, 1)]
    assert len(steps) == 20 + 0 + 5 * 2 + 2 + 3 + 1 + 3


def test_parameters_in_step_share_a_launch(steps):
    ps = params(*range(1, 12))
    opt = optim.AdamW(ps)
    train(opt, ps, [set(range(11))] * 3)
    assert steps == [(1, 11), (2, 11), (3, 11)]


def test_step_counts_are_saved(steps):
    """A reloaded optimizer goes on with each parameter's own count; a state
    saved with one count for a group goes on with that."""
    ps = params(9, 10)
    opt = optim.AdamW(ps)
    train(opt, ps, [{0}] * 4 + [{0, 1}] * 2)
    saved = copy.deepcopy(opt.state_dict())
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    again = optim.AdamW(qs)
    again.load_state_dict(saved)
    assert [again.state[q]["step"] for q in qs] == [6, 2]
    train(opt, ps, [{0, 1}], seed=7)
    train(again, qs, [{0, 1}], seed=7)
    assert all(torch.equal(p, q) for p, q in zip(ps, qs))
    old = copy.deepcopy(saved)
    for st in old["state"].values():
        del st["step"]
    old["param_groups"][0]["step"] = 6
    again.load_state_dict(old)
    assert [again.state[q]["step"] for q in qs] == [6, 6] and "step" not in again.param_groups[0]


@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
def test_copies_go_on(steps, how):
    """A copied optimizer (with its parameters) steps on like the original."""
    ps = params(9, 10)
    opt = optim.AdamW(ps)
    train(opt, ps, [{0, 1}] * 2)
    if how == "deepcopy":
        again = copy.deepcopy(opt)
    else:
        buf = io.BytesIO()
        torch.save(opt, buf)
        buf.seek(0)
        again = torch.load(buf, weights_only=False)
    qs = again.param_groups[0]["params"]
    assert qs[0] is not ps[0]
    train(opt, ps, [{0, 1}] * 2, seed=3)
    train(again, qs, [{0, 1}] * 2, seed=3)
    assert all(torch.equal(p, q) for p, q in zip(ps, qs)) and again.state[qs[0]]["step"] == 4


def test_loaded_weights_are_kept(steps):
    """Weights put into a bf16 parameter after its first step are what the next
    step starts from; elements that stay keep their master's low bits."""
    (p,) = params(64, dtype=torch.bfloat16)
    opt = optim.AdamW([p], lr=1e-2, weight_decay=0.0)
    grads([p], 0)
    opt.step()
    master = opt.state[p]["master"].clone()
    new = torch.linspace(-3, 3, 64).to(torch.bfloat16)
    new[32:] = p.detach()[32:]
    with torch.no_grad():
        p.copy_(new)                                           # as a module's load_state_dict does
    p.grad = torch.zeros_like(p)
    opt.param_groups[0]["lr"] = 0.0
    opt.step()
    assert torch.equal(p.detach(), new)
    assert torch.equal(opt.state[p]["master"][:32], new[:32].float())
    assert torch.equal(opt.state[p]["master"][32:], master[32:])
    # the same weights loaded again change nothing, and an optimizer's own state comes with its master
    with torch.no_grad():
        p.copy_(p.clone())
    opt.step()
    assert torch.equal(opt.state[p]["master"][32:], master[32:])
    saved = copy.deepcopy(opt.state_dict())
    with torch.no_grad():
        p.zero_()
    opt.load_state_dict(saved)
    opt.step()
    assert torch.equal(p.detach(), new)


def test_weights_in_new_memory_are_kept(steps):
    """A bf16 parameter that is given other memory (p.data = ...) goes on from
    what that holds; where it is the master's rounding its low bits stay."""
    (p,) = params(64, dtype=torch.bfloat16)
    opt = optim.AdamW([p], lr=1e-2, weight_decay=0.0)
    grads([p], 0)
    opt.step()
    master = opt.state[p]["master"].clone()
    new = p.detach().clone()
    new[:32] += 1
    p.data = new.clone()
    p.grad = torch.zeros_like(p)
    opt.param_groups[0]["lr"] = 0.0
    opt.step()
    assert torch.equal(p.detach(), new)
    assert torch.equal(opt.state[p]["master"], torch.cat([new[:32].float(), master[32:]]))


def test_state_is_whole_or_absent(steps, monkeypatch):
    """A state whose memory runs out half way is made again at the next step."""
    (p,) = params(20)
    opt = optim.AdamW([p])
    grads([p], 0)
    zeros, left = torch.zeros, [1]

    def failing(*a, **kw):
        if not left.pop():
            raise MemoryError
        left.append(0)
        return zeros(*a, **kw)
    monkeypatch.setattr(optim.torch, "zeros", failing)
    with pytest.raises(MemoryError):
        opt.step()
    monkeypatch.setattr(optim.torch, "zeros", zeros)
    opt.step()
    assert steps == [(1, 1)] and sorted(opt.state[p]) == ["m", "step", "v"]
