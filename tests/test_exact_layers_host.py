"""Host logic of the exact layers and their optimizer (no GPU needed): the
operators' calls are replaced by plain torch on the CPU, or recorded."""
import pytest
import torch

import approximate_multiplier_dnn_gb300 as am
from approximate_multiplier_dnn_gb300 import layers


@pytest.fixture
def losses(monkeypatch):
    """The vocabulary loss in plain torch; the list of calls made."""
    calls = []

    def loss(h, w, targets, *, row_weight=None, ignore_index=-100, reduction="mean"):
        calls.append("loss")
        z = h.detach().float() @ w.detach().float().t()
        row = torch.nn.functional.cross_entropy(z, targets, ignore_index=ignore_index, reduction="none")
        lse = torch.logsumexp(z, 1)
        return row.sum().reshape(1) / (targets != ignore_index).sum(), row, lse

    def grad(h, w, targets, **kw):
        out = loss(h, w, targets, **kw)
        calls[-1] = "grad"
        H, W = h.detach().float().requires_grad_(), w.detach().float().requires_grad_()
        with torch.enable_grad():
            z = torch.nn.functional.cross_entropy(H @ W.t(), targets, ignore_index=kw.get("ignore_index", -100))
        dh, dw = torch.autograd.grad(z, (H, W))
        return *out, dh.to(h.dtype), dw.to(w.dtype)
    monkeypatch.setattr(layers, "vocab_loss", loss)
    monkeypatch.setattr(layers, "vocab_loss_grad", grad)
    return calls


@pytest.fixture
def norms(monkeypatch):
    """The block norm without gate and weight gradients in plain torch; the
    list of (dr, dn) that its backward was given."""
    calls = []

    def forward(x, y=None, w_post=None, w_pre=None, *, gate=None, alpha=1.0, eps=1e-6, n_dtype=None):
        def rstd(t):
            return torch.rsqrt(t.square().mean(1) + eps)
        r = x if y is None else x + alpha * y * rstd(y)[:, None]
        return r, r * rstd(r)[:, None], None if y is None else rstd(y), rstd(r)

    def backward(dr, dn, r, y, w_post, w_pre, rstd_post, rstd_pre, *, gate=None, alpha=1.0):
        calls.append((dr, dn))
        return (torch.zeros_like(r), None if y is None else torch.zeros_like(y), None if gate is None else torch.zeros_like(gate),
                None if w_post is None else torch.zeros_like(w_post), None if w_pre is None else torch.zeros_like(w_pre))
    monkeypatch.setattr(layers, "block_norm", forward)
    monkeypatch.setattr(layers, "block_norm_backward", backward)
    return calls


def head_inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    head = layers.VocabHead(16, 50, device="cpu", generator=g)
    return head, torch.randn((3, 7, 16), generator=g).to(torch.bfloat16), torch.randint(0, 50, (3, 7), generator=g)


def test_evaluation_computes_the_loss_alone(losses):
    """No gradient is computed where none can be asked for: without grad mode,
    whatever requires one, and where nothing does."""
    head, h, t = head_inputs()
    with torch.no_grad():
        head(h, t)
        head(h.requires_grad_(), t)
    with torch.inference_mode():
        head(h, t)
    head.weight.requires_grad_(False)
    head(h.detach(), t)
    assert losses == ["loss"] * 4
    head(h, t).backward()                              # a frozen head, hidden states that are trained
    assert losses[4:] == ["grad"] and h.grad is not None and head.weight.grad is None


def test_second_derivatives_are_refused(losses, norms):
    """They would come out without the terms that pass through the kernels."""
    head, h, t = head_inputs()
    loss = head(h.requires_grad_(), t)
    (dh,) = torch.autograd.grad(loss.square(), h, create_graph=True)
    with pytest.raises(RuntimeError):
        dh.float().sum().backward()
    x = torch.ones(4, 8, requires_grad=True)
    r, n = layers.BlockNorm(8, device="cpu")(x, 2 * x)
    (dx,) = torch.autograd.grad(n.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_row_weight_that_requires_a_gradient_is_refused(losses):
    """It would silently get none."""
    head, h, t = head_inputs()
    a = torch.ones(21, requires_grad=True)
    with pytest.raises(ValueError):
        head(h, t, row_weight=a)
    with torch.no_grad():
        head(h, t, row_weight=a)
    head(h, t, row_weight=a.detach())
    assert losses == ["loss", "grad"]


@pytest.mark.parametrize("factor", [1 / 3, 1e-3, 65537.0, 1.0])
def test_upstream_factor_is_not_rounded(losses, factor):
    """Gradients are scaled by the fp32 factor and rounded once: to the bit."""
    head, h, t = head_inputs()
    loss = head(h.requires_grad_(), t)
    one = torch.autograd.grad(loss, (h, head.weight), retain_graph=True)
    got = torch.autograd.grad(loss * factor, (h, head.weight))
    for p, q in zip(got, one):
        assert p.dtype == torch.bfloat16
        assert torch.equal(p, (q.float() * torch.tensor(factor, dtype=torch.float32)).to(torch.bfloat16))


def test_unused_outputs_have_no_gradient(norms):
    """The gradient of an output that is not used is no tensor of zeros."""
    norm = layers.BlockNorm(8, device="cpu")
    x, y = torch.randn(4, 8, requires_grad=True), torch.randn(4, 8)
    norm(x, y)[1].sum().backward()
    norm(x, y)[0].sum().backward()
    sum(t.sum() for t in norm(x, y)).backward()
    assert [(dr is None, dn is None) for dr, dn in norms] == [(True, False), (False, True), (False, False)]


def dense(t):
    return t.is_contiguous() or (t.stride(1) == 1 and t.stride(0) >= t.shape[1])


def test_layers_take_any_layout(monkeypatch):
    """Transposed, expanded and strided inputs reach the operators as rows that
    they take (others are refused there)."""
    seen = []

    def norm(x, y=None, *a, **kw):
        assert dense(x) and (y is None or dense(y))
        seen.append("norm")
        return (x if y is None else x + y), x.clone(), None, x[:, 0]

    def loss(h, w, targets, *, row_weight=None, **kw):
        assert dense(h) and dense(w) and targets.is_contiguous() and row_weight.is_contiguous()
        seen.append("loss")
        return torch.zeros(1), None, None
    monkeypatch.setattr(layers, "block_norm", norm)
    monkeypatch.setattr(layers, "vocab_loss", loss)
    block = layers.BlockNorm(6, device="cpu")
    block(torch.ones(6, 9).t(), torch.ones(6).expand(9, 6))
    block(torch.ones(1, 6).expand(4, 6))
    wide = torch.ones(9, 20)[:, 3:9]
    assert block(wide)[0].data_ptr() == wide.data_ptr()                  # a stride of rows is no reason to copy
    with torch.no_grad():
        layers.am_vocab_loss(torch.ones(6, 9).t(), torch.ones(6, 5).t(), torch.zeros(18, dtype=torch.int64)[::2],
                             row_weight=torch.ones(9, 2)[:, 0])
    assert seen == ["norm"] * 3 + ["loss"]
